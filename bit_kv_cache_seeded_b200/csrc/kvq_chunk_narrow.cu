// Chunk attention's segment kernel for requests with few query rows (up to kNarrowRows of a kv-head: single tokens
// and speculated ones), bf16 queries. As in kvq_chunk_umma.cu, with the products turned round so that the
// tensor cores' 128 rows are tokens and dims instead of mostly empty query rows; per 128 tokens
//   S^T [128 tokens x 32] = K [128 x DK] . Q^T          (A, B from shared memory)
//   O^T [DV x 32]        += V^T [DV x 128] . P^T         (A, B from shared memory; DV in blocks of 128)
// Dequantising the packed pages bounds it (DK + DV elements a token, on the ALU pipe), not the products, which
// read their A operands once (36 cycles a K step) whatever the rows. So the softmax is laid out to stay out of
// the way: a thread has one token's logits of all rows, 4 warps share a step, and nothing crosses lanes while
// no row's maximum grows by more than 2^8: sums stay with their thread until the segment's end.
//
// Warps: 4 softmax, 4 + 4 that dequantise keys (the step's first and second page; they also fetch the queries), 4 +
// 4 values, 2 that issue the products. Where 227 KB hold two stages of values, but one of keys, the keys' codes
// and signs are handed over apart: the products with the codes run while the signs are made, and free the codes'
// half for the next step. 16 requests of 4-32 rows over 7000 tokens, 8 kv-heads, 2 bits and sketches: 116 us, 0.83
// TB/s of packed pages; the wide kernel takes 223.
#include "kvq_chunk_dequant.cuh"
#include "kvq_pair.cuh"

namespace kvq {
namespace {

using namespace chunk;

constexpr int N = kNarrowRows;
constexpr int kStep = 2 * kPage;                 // tokens of a step, and rows of the key operand
constexpr int kAtom = kStep * 128;               // bytes of an atom of the key operand
constexpr int kPBytes = kStep * N * 2;           // P^T: [16 token groups][N / 8 row groups] of 8 tokens x 16 bytes
constexpr float kLag = 8.f, kShift = 7.f;        // as in kvq_chunk_umma.cu
constexpr uint32_t kColO = 2 * N, kTmemCols = 128;

template <bool KQ, bool VQ>
struct Cfg {
  static constexpr int DK = KQ ? 256 : 128, DV = VQ ? 256 : 128;
  // stages: what 227 KB hold. Keys come in parts of 128 K-elements, codes and signs, a stage each
  static constexpr int KP = DK / 128, KS = KQ && VQ ? 2 : 2 * KP, VS = 2;
  static constexpr int kQBytes = N * DK * 2, kKStage = kStep * 256, kVPage = DV * 128, kVStage = 2 * kVPage;
  static constexpr int kOffP = kQBytes, kOffK = kOffP + 2 * kPBytes, kOffV = kOffK + KS * kKStage, kOffEnd = kOffV + VS * kVStage;
};
// Registers a thread: launched with 80 (24 warps, of which two only give theirs back). The softmax keeps two sets of 32;
// nothing may spill, since shared memory leaves the L1 too small to hold local memory (232 us where 100 bytes did).
// 4 * 136 + 16 * 72 + 4 * 56 = 24 * 80, on every quarter of the SM.
constexpr int kRegsSoftmax = 136, kRegsDequant = 72, kRegsIssue = 56;
constexpr int kWarpK = 4, kWarpV = 12, kWarpS = 20, kWarpO = 21, kThreads = 32 * 24;

struct Bars {
  uint64_t kfull[4], kempty[4], vfull[2], vempty[2], sfull[2], pready[2], pvdone[2], qfull, qempty, done[2];
  unsigned char vbad[2][16];  // tokens of the step whose value norm is not finite, a bit each
  float4 col[N / 2];          // of a pair of rows: query scales, minus the references
  float m[N];                 // maxima the references belong to
  int last[N];                // last position a row attends to
  float part[4][N];
  uint32_t tmem;
  int fail;
};

__device__ __forceinline__ void bar128() { asm volatile("barrier.sync 1, 128;\n" ::: "memory"); }
__device__ __forceinline__ bool any128(bool x) {
  uint32_t r;
  asm volatile("{\n .reg .pred q, r;\n setp.ne.u32 q, %1, 0;\n barrier.red.or.pred r, 1, 128, q;\n selp.u32 %0, 1, 0, r;\n}\n"
               : "=r"(r) : "r"((uint32_t)x) : "memory");
  return r != 0;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ int segment_steps(const Walk& w) { return max(0, min(w.k1, (w.rows.limit + kStep - 1) / kStep) - w.k0); }

template <bool KQ, bool VQ>
__global__ void __launch_bounds__(kThreads, 1) chunk_narrow(const __grid_constant__ ChunkParams p) {
  using C = Cfg<KQ, VQ>;
  constexpr int DK = C::DK, DV = C::DV;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(16) Bars bars;
  const ChunkSet& set = p.set[kNarrow];
  grid_dep_wait();
  if (set.head[1] == 0) return;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&bars.kfull[i]), 8);
      mbar_init(smem_addr(&bars.kempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.vfull[i]), 8);
      mbar_init(smem_addr(&bars.vempty[i]), 1);
      mbar_init(smem_addr(&bars.sfull[i]), 1);
      mbar_init(smem_addr(&bars.pready[i]), 4);
      mbar_init(smem_addr(&bars.pvdone[i]), 1);
      mbar_init(smem_addr(&bars.done[i]), 1);
    }
    mbar_init(smem_addr(&bars.qfull), 8);
    mbar_init(smem_addr(&bars.qempty), 1);
    mbar_init_fence();
    bars.fail = 0;
  }
  if (warp == 0) tc::alloc(smem_addr(&bars.tmem), kTmemCols);
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
  Walk w;
  w.init(p, set, blockIdx.x);

  if (warp < kWarpK) {  // ---- softmax: thread = token of the step
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsSoftmax));
    const int lane = tid & 31;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const uint32_t tS = tmem + lanes, tO = tmem + lanes + kColO;
    int n = 0;
    while (w.next(set)) {
      const Rows r = w.rows;
      const int ns = segment_steps(w);
      if (tid < N) {
        const bool row = tid < r.count;
        float* col = reinterpret_cast<float*>(&bars.col[tid >> 1]);
        col[tid & 1] = row ? p.qscale[(size_t)(r.start + r.first + tid / p.group) * p.Hq + w.hk * p.group + tid % p.group] : 0.f;
        col[2 + (tid & 1)] = 0.f;
        bars.m[tid] = -INFINITY;
        bars.last[tid] = row ? min(r.pos0 + tid / p.group, r.ctx - 1) : 0x7fffffff;
      }
      bar128();
      float l[N];
#pragma unroll
      for (int c = 0; c < N; ++c) l[c] = 0.f;
#pragma unroll 1
      for (int j = 0; j < ns; ++j, ++n) {
        const int b = n & 1;
        const int t0 = (w.k0 + j) * kStep, t = t0 + tid;
        wait(bars.sfull[b], (n >> 1) & 1);
        tc::fence_after();
        float e[N];
#pragma unroll
        for (int h = 0; h < N; h += 16) {
          uint32_t s[16];
          tc::tmem_ld16(tS + N * b + h, s);
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float4 q = bars.col[h / 2 + c];
            e[h + 2 * c] = fmaf(__uint_as_float(s[2 * c]), q.x, q.z);
            e[h + 2 * c + 1] = fmaf(__uint_as_float(s[2 * c + 1]), q.y, q.w);
          }
        }
        if (t0 + kStep - 1 > r.pos0) {  // some row does not attend to the whole step
#pragma unroll
          for (int c = 0; c < N; ++c) e[c] = t <= bars.last[c] ? e[c] : -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < N; ++c) mx = fmaxf(mx, e[c]);
        if (any128(j == 0 || mx > kShift + kLag)) {  // a row's maximum may have grown: new references
          float mine = 0.f;
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const float x = warp_max(e[c]);
            mine = lane == c ? x : mine;
          }
          bars.part[warp][lane] = mine;
          bar128();
          // lane = row, the same in every warp
          const float m0 = bars.m[lane], ref0 = -reinterpret_cast<const float*>(&bars.col[lane >> 1])[2 + (lane & 1)];
          const float top =
              fmaxf(fmaxf(bars.part[0][lane], bars.part[1][lane]), fmaxf(bars.part[2][lane], bars.part[3][lane])) + ref0;
          const bool grow = top > m0 + kLag || (m0 == -INFINITY && top > m0);
          const float m1 = grow ? top : m0, ref1 = grow ? top - kShift : ref0;
          const float alpha = grow ? ex2f(m0 - top) : 1.f, shift = ref1 - ref0;
#pragma unroll
          for (int c = 0; c < N; ++c) {
            e[c] -= __shfl_sync(0xffffffffu, shift, c);
            l[c] *= __shfl_sync(0xffffffffu, alpha, c);
          }
          if (j > 0) {
            wait(bars.pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1);
            tc::fence_after();
#pragma unroll 1
            for (int i = 0; i < DV / 128 * (N / 8); ++i) {
              uint32_t o[8];
              tc::tmem_ld8(tO + 8 * i, o);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 8; ++c)
                o[c] = __float_as_uint(__uint_as_float(o[c]) * __shfl_sync(0xffffffffu, alpha, 8 * (i % (N / 8)) + c));
              tc::tmem_st8(tO + 8 * i, o);
            }
            tc::wait_st();
          }
          bar128();  // every warp has read the old references
          if (warp == 0) {
            bars.m[lane] = m1;
            reinterpret_cast<float*>(&bars.col[lane >> 1])[2 + (lane & 1)] = -ref1;
          }
          bar128();
        }
        if (n >= 2) wait(bars.pvdone[b], ((n >> 1) - 1) & 1);  // this P of two steps before is read
        const uint32_t at = sm + C::kOffP + b * kPBytes + (tid >> 3) * (N / 8 * 128) + (tid & 7) * 16;
#pragma unroll
        for (int g = 0; g < N / 8; ++g) {
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 8 * g + 2 * i;
            const float a = ex2f(e[c]), d = ex2f(e[c + 1]);
            l[c] += a;
            l[c + 1] += d;
            const __half2 v = __floats2half2_rn(a, d);
            h[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
          sts16(at + g * 128, h[0], h[1], h[2], h[3]);
        }
        wait(bars.vfull[b], (n >> 1) & 1);
        if ((*(volatile unsigned char*)&bars.vbad[b][tid >> 3] >> (tid & 7)) & 1) {
#pragma unroll
          for (int c = 0; c < N; ++c)
            if (t <= bars.last[c]) l[c] = NAN;
        }
        tc::fence_before();
        arrive_rows(bars.pready[b]);
      }
      // the segment's state
      float mine = 0.f;
#pragma unroll
      for (int c = 0; c < N; ++c) {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], x);
        mine = lane == c ? l[c] : mine;
      }
      bars.part[warp][lane] = mine;
      bar128();
      if (tid < r.count) {
        const float m = bars.m[tid], ref = -reinterpret_cast<const float*>(&bars.col[tid >> 1])[2 + (tid & 1)];
        *reinterpret_cast<float2*>(segment_ml(set, w.item, blockIdx.x, DV) + 2 * tid) =
            make_float2(m == -INFINITY ? m : ref, (bars.part[0][tid] + bars.part[1][tid]) + (bars.part[2][tid] + bars.part[3][tid]));
      }
      float* so = segment_o(set, w.item, blockIdx.x, DV) + tid;
      if (ns > 0) {
        wait(bars.pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1);
        tc::fence_after();
      }
#pragma unroll 1
      for (int i = 0; i < DV / 128 * (N / 8); ++i) {
        uint32_t o[8];
        if (ns > 0) {
          tc::tmem_ld8(tO + 8 * i, o);
          tc::wait_ld();
        }
        const int row0 = 8 * (i % (N / 8)), dim = i / (N / 8) * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (row0 + c < r.count) so[(size_t)(row0 + c) * DV + dim] = ns > 0 ? __uint_as_float(o[c]) : 0.f;
      }
      tc::fence_before();
      bar128();  // the next segment's rows replace these
    }
  } else if (warp < kWarpV) {  // ---- keys, and the queries of each segment
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsDequant));
    const int all = tid - 32 * kWarpK, second = all >> 7;
    KeyThread<KQ> keys;
    keys.init(p, all & 127, kAtom);
    const uint2 lut = code_halves(p.k);
    int n = 0, seg = 0;  // n: parts handed over
    PageRegs regs = {};
    while (w.next(set)) {
      const Rows r = w.rows;
      const int ns = segment_steps(w);
      if (ns == 0) continue;
      int page = 2 * w.k0 + second;
      if (page * kPage < r.limit) keys.fetch(p, regs, page_tile(p, w, page, page_entry(p, w, page)));
      int entry = page_entry(p, w, page + 2);  // of the page after the one in regs
      constexpr int kChunks = DK / 8, kOwn = N * kChunks / 256;
      const size_t qrow0 = (size_t)(r.start + r.first) * p.Hq + w.hk * p.group;
      uint4 v[kOwn];  // loaded while the last segment's products still read theirs
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int row = (all + 256 * i) / kChunks, ch = all % kChunks;
        v[i] = make_uint4(0, 0, 0, 0);
        if (row < r.count)
          v[i] = *(reinterpret_cast<const uint4*>(static_cast<const __half*>(p.qprep) +
                                                  (qrow0 + (size_t)(row / p.group) * p.Hq + row % p.group) * DK) + ch);
      }
      if (seg > 0) wait(bars.qempty, (seg - 1) & 1);
      ++seg;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int row = (all + 256 * i) / kChunks, ch = all % kChunks;
        *reinterpret_cast<uint4*>(smem + (ch >> 3) * (N * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = v[i];
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
  } else if (warp < kWarpS) {  // ---- values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsDequant));
    const int all = tid - 32 * kWarpV, second = all >> 7, th = all & 127;
    ValueThread<VQ> values;
    values.init(p, th & 7, th >> 3, th >> 3);
    const uint2 lut = code_halves(p.v);
    int n = 0;
    PageRegs regs = {};
    while (w.next(set)) {
      const int ns = segment_steps(w), limit = w.rows.limit;
      if (ns == 0) continue;
      int page = 2 * w.k0 + second;
      if (page * kPage < limit) values.fetch(p, regs, page_tile(p, w, page, page_entry(p, w, page)));
      int entry = page_entry(p, w, page + 2);  // of the page after the one in regs
      for (int j = 0; j < ns; ++j, ++n, page += 2) {
        const int st = n % C::VS;
        const PageRegs cur = regs;
        if (j + 1 < ns && (page + 2) * kPage < limit) {
          values.fetch(p, regs, page_tile(p, w, page + 2, entry));
          entry = page_entry(p, w, page + 4);
        }
        if (n >= C::VS) wait(bars.vempty[st], (n / C::VS - 1) & 1);
        // a second page behind the limit enters as zeros
        const uint32_t bad = values.store(p, cur, lut, sm + C::kOffV + st * C::kVStage + second * C::kVPage, kHeadDim * 128, limit - page * kPage);
        if (th < 8) bars.vbad[st][8 * second + th] = (unsigned char)bad;
        arrive_rows(bars.vfull[st]);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsIssue));
    if (warp == kWarpS) {  // ---- S^T = K Q^T (the whole warp, so that control stays uniform)
      constexpr uint32_t id = tc::idesc_f16(0, 0, 0, kStep, N);
      int n = 0, seg = 0;
      while (w.next(set)) {
        const int ns = __shfl_sync(0xffffffffu, segment_steps(w), 0);
        if (ns == 0) continue;
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
    } else if (warp == kWarpO) {  // ---- O^T += V^T P^T
      constexpr uint32_t id = tc::idesc_f16(0, 0, 1, 128, N);
      int n = 0;
      while (w.next(set)) {
        const int ns = __shfl_sync(0xffffffffu, segment_steps(w), 0);
        for (int j = 0; j < ns; ++j, ++n) {
          const int st = n % C::VS, b = n & 1;
          wait(bars.vfull[st], (n / C::VS) & 1);
          wait(bars.pready[b], (n >> 1) & 1);
          tc::fence_after();
          const uint64_t vd = desc_sw128(sm + C::kOffV + st * C::kVStage);
          const uint64_t pd = tc::smem_desc(sm + C::kOffP + b * kPBytes, N / 8 * 128, 128);
  #pragma unroll
          for (int g = 0; g < 2; ++g)
  #pragma unroll
            for (int i = 0; i < DV / 128; ++i)
              tc::umma_f16_x4<32, 2 * (N / 8) * 128>(tmem + kColO + i * N, vd + ((g * C::kVPage + i * 128 * 128) >> 4),
                                                     pd + ((g * kPBytes / 2) >> 4), id, j > 0 || g > 0);
          tc::commit_elected(smem_addr(&bars.pvdone[b]));
          tc::commit_elected(smem_addr(&bars.vempty[st]));
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
    tc::dealloc(tmem, kTmemCols);
  }
}

template <bool KQ, bool VQ>
cudaError_t launch(const ChunkParams& p, cudaStream_t s) {
  constexpr int smem = Cfg<KQ, VQ>::kOffEnd;
  const cudaError_t e = cudaFuncSetAttribute(chunk_narrow<KQ, VQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_after(chunk_narrow<KQ, VQ>, p, p.set[kNarrow].ctas, kThreads, smem, 1, s);
}

}  // namespace

cudaError_t launch_chunk_narrow(const ChunkParams& p, cudaStream_t s) {
  if (p.k.qjl) return p.v.qjl ? launch<true, true>(p, s) : launch<true, false>(p, s);
  return p.v.qjl ? launch<false, true>(p, s) : launch<false, false>(p, s);
}

}  // namespace kvq
