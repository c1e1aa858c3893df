// Chunk attention's segment kernel for requests with few query rows (up to kNarrowRows of a kv-head: single tokens
// and speculated ones), bf16 queries. As in kvq_chunk_umma.cu, with the products turned round so that the
// tensor cores' 128 rows are tokens and dims instead of mostly empty query rows; per 128 tokens, on tiles of N = 64
// rows (32 where no more are in use),
//   S^T [128 tokens x N] = K [128 x DK] . Q^T           (A, B from shared memory)
//   O^T [DV x N]         += V^T [DV x 128] . P^T         (A, B from shared memory; DV in blocks of 128)
//   l   [128 x N]        += 1 [128 x 128] . P^T          (A in tensor memory: every row the sums of the weights)
// Dequantising the packed pages bounds it (DK + DV elements a token, on the ALU pipe), not the products, which
// read their A operands once (36 cycles a K step) whatever the rows. So the softmax is laid out to stay out of
// the way: a thread has one token's logits of 32 rows, 4 warps share a step's, and nothing crosses lanes while
// no row's maximum grows by more than 2^8; the sums are a product as well, since their registers are needed.
//
// Warps: 4 + 4 softmax (rows 0-31 and 32-63), 4 + 4 that dequantise keys (the step's first and second page; they also
// fetch the queries), 4 + 4 values, 2 that issue the products. Where 227 KB hold no two stages of keys, the keys' codes
// and signs are handed over apart: the products with the codes run while the signs are made, and free the codes'
// half for the next step. Values are handed over by the page, three or four of them.
// 16 requests of 32 rows over 7000 tokens, 8 kv-heads, 2 bits and sketches: 120 us, 0.80 TB/s of packed pages, the call
// 134; of 64 rows 160 (the wide kernel: 242). 3 bits and a key sketch 112 and 128 (224), one bit 91 and 104 (196).
#include "kvq_chunk_dequant.cuh"
#include "kvq_pair.cuh"

namespace kvq {
namespace {

using namespace chunk;

constexpr int kPart = 32;                        // query rows of four softmax warps
constexpr int kStep = 2 * kPage;                 // tokens of a step, and rows of the key operand
constexpr int kAtom = kStep * 128;               // bytes of an atom of the key operand
constexpr float kLag = 8.f, kShift = 7.f;        // as in kvq_chunk_umma.cu
constexpr int kThreads = 32 * 28;
constexpr uint32_t kOnes = 0x3C003C00u;          // two ones in fp16

// N: query rows of a tile, 32 or 64.
template <bool KQ, bool VQ, int N>
struct Cfg {
  static constexpr int DK = KQ ? 256 : 128, DV = VQ ? 256 : 128;
  // stages: what 227 KB hold. Keys come in parts of 128 K-elements, codes and signs, a stage each
  static constexpr int KP = DK / 128, KS = KQ && !VQ ? 3 : 2, VS = VQ && N == 64 ? 3 : 4;
  // warps: softmax first, then keys, values, the two that issue; the others only give their registers back
  static constexpr int kWarpK = N / 8, kWarpV = kWarpK + 8, kWarpS = kWarpV + 8, kWarpO = kWarpS + 1;
  // Registers a thread, launched with 72. Nothing may spill where it recurs, since shared memory leaves the L1 too small to
  // hold local memory (instances with a value sketch spill one or two registers, 4 or 8 bytes). 8 * 88 + 16 * 72 + 4 * 40 and 4 * 104 + 16 * 72 + 8 * 56 are 28 * 72, on every quarter of the SM.
  static constexpr int kRegsSoftmax = N == 32 ? 104 : 88, kRegsDequant = 72, kRegsIssue = N == 32 ? 56 : 40;
  static constexpr int kPBytes = kStep * N * 2;  // P^T: [16 token groups][N / 8 row groups] of 8 tokens x 16 bytes
  static constexpr int kQBytes = N * DK * 2, kKStage = kStep * 256, kVPage = DV * 128;
  static constexpr int kOffP = kQBytes, kOffK = kOffP + 2 * kPBytes, kOffV = kOffK + KS * kKStage, kOffEnd = kOffV + VS * kVPage;
  // tensor memory: two S^T, O^T in blocks of 128 dims and the rows' sums behind them, a K step's ones
  static constexpr int kSums = DV / 128;
  static constexpr uint32_t kColO = 2 * N, kColOnes = kColO + (kSums + 1) * N, kTmemCols = 512;
};
// Warps short of registers keep their walk in shared memory; one thread takes its steps.
struct SharedWalk {
  Walk w;
  int more, steps;  // of the segment; 0 steps when nothing is attended to
  __device__ __forceinline__ void step(const ChunkSet& set) {
    more = w.next(set);
    if (more) steps = max(0, min(w.k1, (w.rows.limit + kStep - 1) / kStep) - w.k0);
  }
};

struct Bars {
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4], sfull[2], pready[2], pvdone[2], qfull, qempty, done[2];
  unsigned char vbad[4][8];   // tokens of the page whose value norm is not finite, a bit each
  float4 col[kNarrowRows / 2];  // of a pair of rows: query scales, minus the references
  float m[kNarrowRows];         // maxima the references belong to
  int last[kNarrowRows];        // last position a row attends to
  float part[8][kPart];
  SharedWalk walk[4];           // of the softmax's parts and of the two issuing warps
  uint32_t tmem;
  int fail;
};

// Barriers of four softmax warps (the part's).
__device__ __forceinline__ void bar128(int part) { asm volatile("barrier.sync %0, 128;\n" ::"r"(1 + part) : "memory"); }
__device__ __forceinline__ bool any128(int part, bool x) {
  uint32_t r;
  asm volatile("{\n .reg .pred q, r;\n setp.ne.u32 q, %1, 0;\n barrier.red.or.pred r, %2, 128, q;\n selp.u32 %0, 1, 0, r;\n}\n"
               : "=r"(r) : "r"((uint32_t)x), "r"(1 + part) : "memory");
  return r != 0;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ int segment_steps(const Walk& w) { return max(0, min(w.k1, (w.rows.limit + kStep - 1) / kStep) - w.k0); }

// Whether the call's narrow set runs on tiles of 32 rows (calls with a value sketch, launch() below).
__device__ __forceinline__ bool small_rows(const ChunkSet& s) { return s.head[2] <= 32; }

template <bool KQ, bool VQ, int N>
__global__ void __launch_bounds__(kThreads, 1) chunk_narrow(const __grid_constant__ ChunkParams p) {
  using C = Cfg<KQ, VQ, N>;
  constexpr int DK = C::DK, DV = C::DV;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(16) Bars bars;
  const ChunkSet& set = p.set[kNarrow];
  grid_dep_wait();
  if (set.head[1] == 0 || (VQ && small_rows(set) != (N == 32))) return;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&bars.kfull[i]), 8);
      mbar_init(smem_addr(&bars.kempty[i]), 1);
      mbar_init(smem_addr(&bars.vfull[i]), 4);
      mbar_init(smem_addr(&bars.vempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.sfull[i]), 1);
      mbar_init(smem_addr(&bars.pready[i]), N / 8);
      mbar_init(smem_addr(&bars.pvdone[i]), 1);
      mbar_init(smem_addr(&bars.done[i]), 1);
    }
    mbar_init(smem_addr(&bars.qfull), 8);
    mbar_init(smem_addr(&bars.qempty), 1);
    mbar_init_fence();
    bars.fail = 0;
  }
  if (warp == 0) tc::alloc(smem_addr(&bars.tmem), C::kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = bars.tmem;
  const uint32_t sm = smem_addr(smem);
  // a wait that gives up ends every later one at once; the loops are bounded by the plan
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    const uint32_t a = smem_addr(&bar);
    if (mbar_try(a, parity) || *(volatile int*)&bars.fail) return;
    if (!mbar_wait_spin(a, parity, p.wait_limit)) {
      bars.fail = 1;
      atomicOr(p.err, 1);
    }
  };
  if (warp < C::kWarpK) {  // ---- softmax: thread = token of the step, four warps a part of 32 rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kRegsSoftmax));
    const int lane = tid & 31, quarter = warp & 3, tok = tid & 127, part = warp >> 2, c0 = part * kPart;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t tS = tmem + lanes + c0, tO = tmem + lanes + C::kColO + c0;
    if (part == 0) {
      const uint32_t ones[8] = {kOnes, kOnes, kOnes, kOnes, kOnes, kOnes, kOnes, kOnes};
      tc::tmem_st8(tmem + lanes + C::kColOnes, ones);
      tc::wait_st();
    }
    SharedWalk& walk = bars.walk[part];
    if (tok == 0) walk.w.init(p, set, blockIdx.x);
    int n = 0;
    while (true) {
      if (tok == 0) walk.step(set);
      bar128(part);
      if (!walk.more) break;
      const int ns = walk.steps, count = min(max(walk.w.rows.count - c0, 0), kPart), pos0 = walk.w.rows.pos0;
      const int first = walk.w.k0 * kStep + tok;
      float* ref = reinterpret_cast<float*>(&bars.col[(c0 + lane) >> 1]) + 2 + (lane & 1);  // lane = row
      if (quarter == 0) {
        const Rows& r = walk.w.rows;
        const int row = c0 + lane;
        ref[-2] = lane < count ? p.qscale[(size_t)(r.start + r.first + row / p.group) * p.Hq + walk.w.hk * p.group + row % p.group] : 0.f;
        *ref = 0.f;
        bars.m[row] = -INFINITY;
        bars.last[row] = lane < count ? min(r.pos0 + row / p.group, r.ctx - 1) : 0x7fffffff;
      }
      bar128(part);
#pragma unroll 1
      for (int j = 0; j < ns; ++j, ++n) {
        const int b = n & 1;
        const int t = first + j * kStep;
        wait(bars.sfull[b], (n >> 1) & 1);
        if (count > 0) {
          tc::fence_after();
          float e[kPart];
#pragma unroll
          for (int h = 0; h < kPart; h += 16) {
            uint32_t s[16];
            tc::tmem_ld16(tS + N * b + h, s);
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 q = bars.col[c0 / 2 + h / 2 + c];
              e[h + 2 * c] = fmaf(__uint_as_float(s[2 * c]), q.x, q.z);
              e[h + 2 * c + 1] = fmaf(__uint_as_float(s[2 * c + 1]), q.y, q.w);
            }
          }
          if (t - tok + kStep - 1 > pos0) {  // some row does not attend to the whole step
#pragma unroll
            for (int c = 0; c < kPart; ++c) e[c] = t <= bars.last[c0 + c] ? e[c] : -INFINITY;
          }
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < kPart; ++c) mx = fmaxf(mx, e[c]);
          if (any128(part, j == 0 || mx > kShift + kLag)) {  // a row's maximum may have grown: new references
            float mine = 0.f;
#pragma unroll
            for (int c = 0; c < kPart; ++c) {
              const float x = warp_max(e[c]);
              mine = lane == c ? x : mine;
            }
            bars.part[warp][lane] = mine;
            bar128(part);
            const float(*const of)[kPart] = &bars.part[4 * part];
            const float m0 = bars.m[c0 + lane], ref0 = -*ref;  // the same in every warp
            const float top = fmaxf(fmaxf(of[0][lane], of[1][lane]), fmaxf(of[2][lane], of[3][lane])) + ref0;
            const bool grow = top > m0 + kLag || (m0 == -INFINITY && top > m0);
            const float m1 = grow ? top : m0, ref1 = grow ? top - kShift : ref0;
            const float alpha = grow ? ex2f(m0 - top) : 1.f, shift = ref1 - ref0;
#pragma unroll
            for (int c = 0; c < kPart; ++c) e[c] -= __shfl_sync(0xffffffffu, shift, c);
            if (j > 0) {
              wait(bars.pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1);
              tc::fence_after();
#pragma unroll 1
              for (int i = 0; i < (C::kSums + 1) * (kPart / 8); ++i) {
                const uint32_t col = tO + i / (kPart / 8) * N + 8 * (i % (kPart / 8));
                uint32_t o[8];
                tc::tmem_ld8(col, o);
                tc::wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  o[c] = __float_as_uint(__uint_as_float(o[c]) * __shfl_sync(0xffffffffu, alpha, 8 * (i % (kPart / 8)) + c));
                tc::tmem_st8(col, o);
              }
              tc::wait_st();
            }
            bar128(part);  // every warp has read the old references
            if (quarter == 0) {
              bars.m[c0 + lane] = m1;
              *ref = -ref1;
            }
            bar128(part);
          }
          if (n >= 2) wait(bars.pvdone[b], ((n >> 1) - 1) & 1);  // this P of two steps before is read
          const uint32_t at = sm + C::kOffP + b * C::kPBytes + (tok >> 3) * (N / 8 * 128) + (tok & 7) * 16 + c0 / 8 * 128;
#pragma unroll
          for (int g = 0; g < kPart / 8; ++g) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = 8 * g + 2 * i;
              const __half2 v = __floats2half2_rn(ex2f(e[c]), ex2f(e[c + 1]));
              h[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            sts16(at + g * 128, h[0], h[1], h[2], h[3]);
          }
          const int page = 2 * n + (tok >> 6), st = page % C::VS;
          wait(bars.vfull[st], (page / C::VS) & 1);
          if ((*(volatile unsigned char*)&bars.vbad[st][(tok >> 3) & 7] >> (tok & 7)) & 1) {
#pragma unroll 1
            for (int c = 0; c < count; ++c)  // NaN weights for the rows that attend to it
              if (t <= bars.last[c0 + c])
                asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(at + (c >> 3) * 128 + (c & 7) * 2), "h"((unsigned short)0x7e00) : "memory");
          }
          tc::fence_before();
        }
        arrive_rows(bars.pready[b]);
      }
      if (count > 0) {  // the segment's state
        if (ns > 0) {
          wait(bars.pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1);
          tc::fence_after();
        }
        float* so = segment_o(set, walk.w.item, blockIdx.x, DV);
        float l = 0.f;
#pragma unroll 1
        for (int i = 0; i < (C::kSums + 1) * (kPart / 8); ++i) {
          const int block = i / (kPart / 8), row0 = 8 * (i % (kPart / 8));
          uint32_t o[8];
          if (ns > 0) {
            tc::tmem_ld8(tO + block * N + row0, o);
            tc::wait_ld();
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float x = ns > 0 ? __uint_as_float(o[c]) : 0.f;
            if (block == C::kSums) l = row0 + c == lane ? x : l;
            else if (row0 + c < count) so[state_pos(kRowShift, kNarrowRows, c0 + row0 + c, block * 128 + tok)] = x;
          }
        }
        if (quarter == 0 && lane < count) {
          const float m = bars.m[c0 + lane];
          *reinterpret_cast<float2*>(segment_ml(set, walk.w.item, blockIdx.x, DV) + 2 * (c0 + lane)) =
              make_float2(m == -INFINITY ? m : -*ref, l);
        }
        tc::fence_before();
      }
      bar128(part);  // the next segment's rows replace these
    }
  } else if (warp < C::kWarpV) {  // ---- keys, and the queries of each segment
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegsDequant));
    const int all = tid - 32 * C::kWarpK, second = all >> 7;
    KeyThread<KQ> keys;
    keys.init(p, all & 127, kAtom);
    const uint2 lut = code_halves(p.k);
    int n = 0, seg = 0;  // n: parts handed over
    PageRegs regs = {};
    Walk w;
    w.init(p, set, blockIdx.x);
    while (w.next(set)) {
      const Rows r = w.rows;
      const int ns = segment_steps(w);
      if (ns == 0) continue;
      int page = 2 * w.k0 + second;
      if (page * kPage < r.limit) keys.fetch(p, regs, page_tile(p, w, page, page_entry(p, w, page)));
      int entry = page_entry(p, w, page + 2);  // of the page after the one in regs
      constexpr int kChunks = DK / 8, kOwn = kPart * kChunks / 256;
      const size_t qrow0 = (size_t)(r.start + r.first) * p.Hq + w.hk * p.group;
#pragma unroll 1
      for (int c0 = 0; c0 < r.count; c0 += kPart) {
        uint4 v[kOwn];  // the first loaded while the last segment's products still read theirs
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          const int row = c0 + (all + 256 * i) / kChunks, ch = all % kChunks;
          v[i] = make_uint4(0, 0, 0, 0);
          if (row < r.count)
            v[i] = *(reinterpret_cast<const uint4*>(static_cast<const __half*>(p.qprep) +
                                                    (qrow0 + (size_t)(row / p.group) * p.Hq + row % p.group) * DK) + ch);
        }
        if (c0 == 0) {
          if (seg > 0) wait(bars.qempty, (seg - 1) & 1);
          ++seg;
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          const int row = c0 + (all + 256 * i) / kChunks, ch = all % kChunks;
          *reinterpret_cast<uint4*>(smem + (ch >> 3) * (N * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = v[i];
        }
      }
      arrive_rows(bars.qfull);
      for (int j = 0; j < ns; ++j, page += 2) {
        const PageRegs cur = regs;
        if (j + 1 < ns && (page + 2) * kPage < r.limit) {
          keys.fetch(p, regs, page_tile(p, w, page + 2, entry));
          entry = page_entry(p, w, page + 4);
        }
#pragma unroll
        for (int part = 0; part < C::KP; ++part, ++n) {
          const int st = n % C::KS;
          const uint32_t base = sm + C::kOffK + st * C::kKStage + second * kPage * 128;
          if (n >= C::KS) wait(bars.kempty[st], (n / C::KS - 1) & 1);
          if (page * kPage < r.limit) {  // a second page behind the limit stays as it was: its logits are masked
            if (part == 0) keys.codes(p, cur, lut, base);
            else keys.signs(cur, base);
          }
          arrive_rows(bars.kfull[st]);
        }
      }
    }
  } else if (warp < C::kWarpS) {  // ---- values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegsDequant));
    const int all = tid - 32 * C::kWarpV, second = all >> 7, th = all & 127;
    ValueThread<VQ> values;
    values.init(p, th & 7, th >> 3, th >> 3);
    const uint2 lut = code_halves(p.v);
    int n = second;  // pages
    PageRegs regs = {};
    Walk w;
    w.init(p, set, blockIdx.x);
    while (w.next(set)) {
      const int ns = segment_steps(w), limit = w.rows.limit;
      if (ns == 0) continue;
      int page = 2 * w.k0 + second;
      if (page * kPage < limit) values.fetch(p, regs, page_tile(p, w, page, page_entry(p, w, page)));
      int entry = page_entry(p, w, page + 2);  // of the page after the one in regs
      for (int j = 0; j < ns; ++j, n += 2, page += 2) {
        const int st = n % C::VS;
        const PageRegs cur = regs;
        if (j + 1 < ns && (page + 2) * kPage < limit) {
          values.fetch(p, regs, page_tile(p, w, page + 2, entry));
          entry = page_entry(p, w, page + 4);
        }
        if (n >= C::VS) wait(bars.vempty[st], (n / C::VS - 1) & 1);
        // a second page behind the limit enters as zeros
        const uint32_t bad = values.store(p, cur, lut, sm + C::kOffV + st * C::kVPage, kHeadDim * 128, limit - page * kPage);
        if (th < 8) bars.vbad[st][th] = (unsigned char)bad;
        arrive_rows(bars.vfull[st]);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegsIssue));
    SharedWalk& walk = bars.walk[2 + (warp & 1)];
    const bool lead = (tid & 31) == 0;
    if (lead && warp <= C::kWarpO) walk.w.init(p, set, blockIdx.x);
    auto next = [&]() {
      __syncwarp();
      if (lead) walk.step(set);
      __syncwarp();
      return __shfl_sync(0xffffffffu, *(volatile int*)&walk.more, 0) != 0;
    };
    if (warp == C::kWarpS) {  // ---- S^T = K Q^T (the whole warp, so that control stays uniform)
      int n = 0, seg = 0;
      while (next()) {
        const int ns = __shfl_sync(0xffffffffu, *(volatile int*)&walk.steps, 0);
        if (ns == 0) continue;
        const uint32_t id = tc::idesc_f16(0, 0, 0, kStep, walk.w.rows.count > kPart ? N : kPart);
        wait(bars.qfull, seg & 1);
        ++seg;
        for (int j = 0; j < ns; ++j, ++n) {
          const int b = n & 1;
          if (n >= 2) wait(bars.pready[b], ((n >> 1) - 1) & 1);  // S of two steps before is read
#pragma unroll
          for (int part = 0; part < C::KP; ++part) {
            const int np = n * C::KP + part, st = np % C::KS;
            wait(bars.kfull[st], (np / C::KS) & 1);
            tc::fence_after();
            const uint64_t kd = desc_sw128(sm + C::kOffK + st * C::kKStage), qd = desc_sw128(sm + part * 2 * N * 128);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              tc::umma_f16_x4(tmem + b * N, kd + ((i * kAtom) >> 4), qd + ((i * N * 128) >> 4), id, part > 0 || i > 0);
            tc::commit_elected(smem_addr(&bars.kempty[st]));
          }
          tc::commit_elected(smem_addr(&bars.sfull[b]));
        }
        tc::commit_elected(smem_addr(&bars.qempty));
      }
      tc::commit_elected(smem_addr(&bars.done[0]));
      mbar_wait(smem_addr(&bars.done[0]), 0, p.wait_limit);
    } else if (warp == C::kWarpO) {  // ---- O^T += V^T P^T
      int n = 0;
      while (next()) {
        const int ns = __shfl_sync(0xffffffffu, *(volatile int*)&walk.steps, 0);
        const uint32_t id = tc::idesc_f16(0, 0, 1, 128, walk.w.rows.count > kPart ? N : kPart);
        for (int j = 0; j < ns; ++j, ++n) {
          const int b = n & 1;
          wait(bars.pready[b], (n >> 1) & 1);
          const uint64_t pd = tc::smem_desc(sm + C::kOffP + b * C::kPBytes, N / 8 * 128, 128);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int page = 2 * n + g, st = page % C::VS;
            wait(bars.vfull[st], (page / C::VS) & 1);
            tc::fence_after();
            const uint64_t vd = desc_sw128(sm + C::kOffV + st * C::kVPage), pg = pd + ((g * C::kPBytes / 2) >> 4);
#pragma unroll
            for (int i = 0; i < DV / 128; ++i)
              tc::umma_f16_x4<32, 2 * (N / 8) * 128>(tmem + C::kColO + i * N, vd + ((i * 128 * 128) >> 4), pg, id, j > 0 || g > 0);
            tc::umma_f16_ta_x4<2 * (N / 8) * 128>(tmem + C::kColO + C::kSums * N, tmem + C::kColOnes, pg, id, j > 0 || g > 0);
            tc::commit_elected(smem_addr(&bars.vempty[st]));
          }
          tc::commit_elected(smem_addr(&bars.pvdone[b]));
        }
      }
      tc::commit_elected(smem_addr(&bars.done[1]));
      mbar_wait(smem_addr(&bars.done[1]), 0, p.wait_limit);
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::dealloc(tmem, C::kTmemCols);
  }
}

template <bool KQ, bool VQ, int N>
cudaError_t launch_rows(const ChunkParams& p, cudaStream_t s) {
  constexpr int smem = Cfg<KQ, VQ, N>::kOffEnd;
  const cudaError_t e = cudaFuncSetAttribute(chunk_narrow<KQ, VQ, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_after(chunk_narrow<KQ, VQ, N>, p, p.set[kNarrow].ctas, kThreads, smem, 1, s);
}
// With a value sketch, tiles of 64 rows leave room for three pages of values instead of four; a call whose fullest tile has
// 32 rows keeps the fourth. Where the host cannot tell, both are launched, and one of them ends at once (2 us).
// 16 requests of 32 rows over 7000 tokens, 2 bits and sketches: 134 us so, 141 on tiles of 64 rows; 64 rows 160 and 159.
template <bool KQ, bool VQ>
cudaError_t launch(const ChunkParams& p, cudaStream_t s) {
  const cudaError_t e = VQ && (long long)p.n_tokens * p.group <= 32 ? cudaSuccess : launch_rows<KQ, VQ, 64>(p, s);
  if constexpr (VQ) return e != cudaSuccess ? e : launch_rows<KQ, VQ, 32>(p, s);
  return e;
}

}  // namespace

cudaError_t launch_chunk_narrow(const ChunkParams& p, cudaStream_t s) {
  if (p.k.qjl) return p.v.qjl ? launch<true, true>(p, s) : launch<true, false>(p, s);
  return p.v.qjl ? launch<false, true>(p, s) : launch<false, false>(p, s);
}

}  // namespace kvq
