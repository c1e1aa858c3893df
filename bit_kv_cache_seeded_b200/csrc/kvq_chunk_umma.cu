// Chunk attention's segment kernel on 5th-generation tensor cores (tcgen05, kind::f16, fp32 sums), for bf16
// queries of requests with many rows (kvq_chunk_narrow.cu takes the others). Work plan and the states it leaves:
// kvq_chunk.cuh.
//
// A pair of CTAs (cta_group::2) walks its segments page by page (64 tokens). Per page and tile of 256 query rows
//   S [256 x 64] = Q [256 x DK] . K^T             (A, B from shared memory; DK = 128, + 128 of the key sketch)
//   O [256 x DV] += P [256 x 64] . V               (A from tensor memory; DV = 128, + 128 of the value sketch)
// with K and V dequantised from the packed page into fp16 (kvq_chunk_dequant.cuh). Each CTA holds 128 rows of a
// tile and makes half of either operand: keys, 32 of the tokens; values, 64 of the dims. NT row tiles share the
// operands: two where tensor memory holds their sums (O takes 2 x 128 columns, S 2 x 2 x 64), one with a value
// sketch (O 256). Measured on a 2048-token chunk of 64 heads over 32768 tokens (3 bits, a key sketch): 2.37 ms, 1.3
// PFLOP/s with the sketch's products. A CTA of its own, which dequantises everything for half as many rows, took
// 2.72 ms at the same stage of the work; pairs with S over 128 tokens, which leaves tensor memory for one S a tile
// and so puts S, softmax and P V of a tile in a row, 2.79. The softmax's issue bounds it, and the tensor pipe next.
//
// Warps: 4 per row tile for the softmax (thread = row), 4 or 8 that dequantise keys (and fetch the queries of
// a segment), 4 or 8 for values, and in the first CTA 2 that issue the products, S and P V. K and V are staged
// four times, S twice per tile, so that dequantisation, S, softmax and P V of neighbouring pages overlap. P
// overwrites the first half of its S. Barriers that the products wait for are the first CTA's, and the second
// arrives there; those that they complete are told to both.
//
// A row that attends to a value whose norm is not finite ends as NaN: rows attend to all of a segment's positions up
// to their own, so the first such position decides.
//
// Softmax weights are p = 2^(x - m + 7), m the row's maximum but for steps under 2^8, by which it may lag
// before O is rescaled: p stays under 2^15 in fp16, and a weight is dropped only below 2^-31 of the largest.
#include "kvq_chunk_dequant.cuh"
#include "kvq_pair.cuh"

namespace kvq {
namespace {

using namespace chunk;

constexpr int kStages = 4;
constexpr int kTileRows = 128;        // of a CTA
// Slots of segments for the first position whose value norm is not finite. The values' first group resets a slot half a
// round before its segment. It may be kStages + VG segments ahead of the softmax, where they are a page long: it stores
// page n once the products have read page n - kStages, whose rows may still have their slot to read, and then walks on,
// without a wait, to its next page, n + VG. The slot that it resets there belongs to the segment kSlots / 2 before.
constexpr int kSlots = 32;
constexpr float kLag = 8.f, kShift = 7.f;
constexpr uint32_t kColS = 256, kTmemCols = 512;

template <bool KQ, bool VQ>
struct Cfg {
  static constexpr int NT = VQ ? 1 : 2, NB = 2;  // row tiles, and S of each
  static constexpr int DK = KQ ? 256 : 128, DV = VQ ? 256 : 128;
  // groups of 2 warps that dequantise a side, page n on group n % G: twice as many where a sketch doubles the work
  static constexpr int KG = KQ ? 4 : 2, VG = VQ ? 4 : 2;
  static_assert(kSlots / 2 > kStages + VG, "a slot is reset while the softmax may still read it");
  static constexpr int kWarpK = 4 * NT, kWarpV = kWarpK + 2 * KG, kWarpS = kWarpV + 2 * VG, kWarpO = kWarpS + 1;
  // With a key sketch 22 warps, and two more that only give their registers back: 80 a thread at launch, shared out
  // so that nothing spills (shared memory leaves the L1 too small to hold local memory).
  static constexpr bool kShare = KQ;
  static constexpr int kRegsSoftmax = VQ ? 104 : 88, kRegsDequant = 80 /* as launched */, kRegsIssue = 56;
  static constexpr int kThreads = 32 * (kShare ? 24 : kWarpO + 1);
  static_assert(!kShare || 4 * NT * kRegsSoftmax + 2 * (KG + VG) * kRegsDequant + 4 * kRegsIssue <= 24 * 80, "registers");
  static constexpr int kKAtom = kTile * 128, kVAtom = DV / 2 * 128;  // operand atoms of 64 K-elements, this CTA's rows
  static constexpr int kQTile = kTileRows * DK * 2, kKStage = DK / 64 * kKAtom, kVStage = kVAtom;
  static constexpr int kOffK = NT * kQTile, kOffV = kOffK + kStages * kKStage, kOffEnd = kOffV + kStages * kVStage;
};

template <int NT, int NB>
struct Bars {
  uint64_t kfull[kStages], vfull[kStages], pready[NT][NB], qfull;                  // the first CTA's count both
  uint64_t kempty[kStages], vempty[kStages], sfull[NT][NB], pvdone[NT][NB], qempty, done[2];
  int bad[kSlots];                  // by segment: the first position whose value norm is not finite
  uint32_t tmem;
  int fail;
};

// Pairs of fp32 (one issue for two).
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^x on the FMA pipe, for x < 126: x = k + f, k the nearest integer, 2^f by a cubic fitted to |f| <= 1/2 with
// the least largest relative error (2^-13.7, under the weights' own rounding to fp16, 2^-11). Below 2^-126
// stays 2^-126; a NaN stays one. The special-function unit makes 4 powers a cycle and quarter of an SM, which
// bounds the softmax where nothing else does; a quarter of them is made here then (one-bit chunks 374 -> 368 us;
// beside the dequantisation of key sketches it costs more than it gives, 2.39 -> 2.48 ms).
__device__ __forceinline__ F2 ex2_fma(F2 x) {
  float a, b;
  x.get(a, b);
  asm("max.NaN.f32 %0, %0, %1;\n" : "+f"(a) : "f"(-126.f));
  asm("max.NaN.f32 %0, %0, %1;\n" : "+f"(b) : "f"(-126.f));
  x = F2(a, b);
  const F2 t = add(x, F2(12582912.f, 12582912.f));  // 1.5 * 2^23: k in the low bits
  const F2 f = fma(add(t, F2(-12582912.f, -12582912.f)), F2(-1.f, -1.f), x);
  F2 y = fma(f, F2(0.0551716648f, 0.0551716648f), F2(0.2426111251f, 0.2426111251f));
  y = fma(f, y, F2(0.6932609677f, 0.6932609677f));
  y = fma(f, y, F2(0.9999280572f, 0.9999280572f));
  t.get(a, b);
  return mul(y, F2(__int_as_float(__float_as_int(a) * (1 << 23) + 0x3f800000), __int_as_float(__float_as_int(b) * (1 << 23) + 0x3f800000)));
}

__device__ __forceinline__ int segment_pages(const Walk& w) { return max(0, min(w.k1, (w.rows.limit + kPage - 1) / kPage) - w.k0); }

// Of a warp whose threads have written operand rows: visible to the pair's products, one arrival at the first CTA.
__device__ __forceinline__ void arrive_first(uint64_t& bar) {
  fence_proxy_async();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive_at(smem_addr(&bar), 0);
}

template <bool SHARE, int REGS>
__device__ __forceinline__ void more_registers() {
  if (SHARE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(REGS));
}
template <bool SHARE, int REGS>
__device__ __forceinline__ void fewer_registers() {
  if (SHARE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(REGS));
}

// 32 bytes, a whole sector, at once.
__device__ __forceinline__ void store8(float* at, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}

template <bool KQ, bool VQ>
__global__ void __launch_bounds__(Cfg<KQ, VQ>::kThreads, 1) chunk_umma(const __grid_constant__ ChunkParams p) {
  using C = Cfg<KQ, VQ>;
  constexpr int NT = C::NT, NB = C::NB, DK = C::DK, DV = C::DV;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(16) Bars<NT, NB> bars;
  const ChunkSet& set = p.set[kWide];
  grid_dep_wait();
  if (set.head[1] == 0) return;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&bars.kfull[i]), 4);
      mbar_init(smem_addr(&bars.kempty[i]), 1);
      mbar_init(smem_addr(&bars.vfull[i]), 4);
      mbar_init(smem_addr(&bars.vempty[i]), 1);
    }
    for (int t = 0; t < NT; ++t)
      for (int b = 0; b < NB; ++b) {
        mbar_init(smem_addr(&bars.sfull[t][b]), 1);
        mbar_init(smem_addr(&bars.pready[t][b]), 8);
        mbar_init(smem_addr(&bars.pvdone[t][b]), 1);
      }
    mbar_init(smem_addr(&bars.qfull), 4 * C::KG);
    mbar_init(smem_addr(&bars.qempty), 1);
    mbar_init(smem_addr(&bars.done[0]), 1);
    mbar_init(smem_addr(&bars.done[1]), 1);
    mbar_init_fence();
    for (int i = 0; i < kSlots; ++i) bars.bad[i] = 0x7fffffff;
    bars.fail = 0;
  }
  if (warp == 0) tc::pair_alloc(smem_addr(&bars.tmem), kTmemCols);
  tc::fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and tensor memory are there
  tc::fence_after();
  const uint32_t tmem = bars.tmem;
  const uint32_t sm = smem_addr(smem);
  // a wait that gives up ends every later one of its CTA at once; the loops are bounded by the plan
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    const uint32_t a = smem_addr(&bar);
    if (mbar_try(a, parity) || *(volatile int*)&bars.fail) return;
    if (!mbar_wait_spin(a, parity, p.wait_limit)) {
      bars.fail = 1;
      atomicOr(p.err, 1);
    }
  };
  auto wait_both = [&](uint64_t& bar, uint32_t parity) {  // for arrivals of both CTAs
    if (*(volatile int*)&bars.fail) return;
    if (!mbar_wait_cluster(smem_addr(&bar), parity, p.wait_limit)) {
      bars.fail = 1;
      atomicOr(p.err, 1);
    }
  };
  Walk w;
  w.init(p, set, pair);

  if (warp < C::kWarpK) {  // ---- softmax: thread = row
    more_registers<C::kShare, C::kRegsSoftmax>();
    const int t = warp >> 2, row = t * 2 * kTileRows + rank * kTileRows + (tid & 127);  // of the NT * 256
    const int row0 = row & ~31;                                                    // of this warp
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tO = tmem + lanes + t * DV, tS = tmem + lanes + kColS + t * NB * kPage;
    int n = 0, seg = 0;  // pages this tile, and segments the pair, has seen
    while (w.next(set)) {
      const Rows r = w.rows;
      const int ns = segment_pages(w);
      const bool used = t * 2 * kTileRows < r.count && ns > 0;
      const bool work = row0 < r.count;
      // rows of no token count as unmasked: what they compute is not kept, and the others' mask may still be empty
      const int last = row < r.count ? min(r.pos0 + row / p.group, r.ctx - 1) : 0x7fffffff;
      float qs = 1.f;
      if (row < r.count)
        qs = p.qscale[(size_t)(r.start + r.first + row / p.group) * p.Hq + w.hk * p.group + row % p.group];
      const F2 qs2(qs, qs);
      float m = -INFINITY, ref = 0.f;
      F2 sum[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
      for (int j = 0; used && j < ns; ++j, ++n) {
        const int b = n % NB;
        wait(bars.sfull[t][b], (n / NB) & 1);
        tc::fence_after();
        if (work) {
          const int reach = last - (w.k0 + j) * kPage;  // the page's tokens 0 .. reach are attended
          const bool full = __all_sync(0xffffffffu, reach >= kPage - 1);
          // 32 columns at a time, in a rolled loop (the code of all roles has to stay in the instruction cache)
#pragma unroll 1
          for (int c = 0; c < kPage; c += 32) {
            uint32_t s[32], ph[16];
            tc::tmem_ld32(tS + kPage * b + c, s);
            tc::wait_ld();
            if (!full) {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = c + i <= reach ? s[i] : 0xff800000u;
            }
            float mx2[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 16; ++i)
              mx2[i & 1] = max3(mx2[i & 1], __uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
            const float mx = fmaxf(mx2[0], mx2[1]) * qs;
            const bool grow = mx > m + kLag || (m == -INFINITY && mx > m);
            if (__any_sync(0xffffffffu, grow)) {  // a new reference: what came before is brought to it
              const float alpha = grow ? ex2f(m - mx) : 1.f;
              if (grow) {
                m = mx;
                ref = mx - kShift;
              }
              sum[0] = mul(sum[0], F2(alpha, alpha));
              sum[1] = mul(sum[1], F2(alpha, alpha));
              if (c > 0) {  // this page's first weights
                tc::wait_st();
                tc::tmem_ld16(tS + kPage * b, ph);
                tc::wait_ld();
                const uint32_t a2 = half_bits(alpha) * 0x10001u;
#pragma unroll
                for (int i = 0; i < 16; ++i) ph[i] = mul2(ph[i], a2);
                tc::tmem_st16(tS + kPage * b, ph);
              }
              if (j > 0) {
                wait(bars.pvdone[t][(n - 1) % NB], ((n - 1) / NB) & 1);
                tc::fence_after();
#pragma unroll 1
                for (int o = 0; o < DV; o += 16) {
                  tc::tmem_ld16(tO + o, ph);
                  tc::wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i) ph[i] = __float_as_uint(__uint_as_float(ph[i]) * alpha);
                  tc::tmem_st16(tO + o, ph);
                }
              }
            }
            const F2 ref2(-ref, -ref);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              F2 x = fma(F2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), qs2, ref2);
              float a, d;
              if (!KQ && (i & 3) == 3) {
                x = ex2_fma(x);
                x.get(a, d);
              } else {
                x.get(a, d);
                a = ex2f(a);
                d = ex2f(d);
                x = F2(a, d);
              }
              sum[i & 1] = add(sum[i & 1], x);
              const __half2 h = __floats2half2_rn(a, d);
              ph[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            tc::tmem_st16(tS + kPage * b + c / 2, ph);
          }
          tc::wait_st();
        }
        tc::fence_before();
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive_at_tmem(smem_addr(&bars.pready[t][b]), 0);
      }
      // the segment's state
      if (used) {
        wait(bars.pvdone[t][(n - 1) % NB], ((n - 1) / NB) & 1);
        tc::fence_after();
      }
      if (work) {
        float la, l;
        add(sum[0], sum[1]).get(la, l);
        l += la;
        if (m == -INFINITY && l == l) l = 0.f;  // ex2_fma leaves 2^-126 of a masked position
        if (ns > 0 && *(volatile int*)&bars.bad[seg % kSlots] <= last && row < r.count) l = NAN;
        float* ml = segment_ml(set, w.item, pair, DV) + 2 * row;
        float* so = segment_o(set, w.item, pair, DV);
        if (row < r.count) *reinterpret_cast<float2*>(ml) = make_float2(m == -INFINITY ? m : ref, l);
#pragma unroll 1
        for (int c = 0; c < DV; c += 16) {
          uint32_t o[16];
          if (used) {
            tc::tmem_ld16(tO + c, o);
            tc::wait_ld();
          }
          // with a sketch each CTA's half of the columns is 64 codes, 64 signs
          const int dim = VQ ? (c & 63) + (c & 128) / 2 + (c & 64) * 2 : c;
          if (row < r.count) {
            float* to = so + state_pos(kWideShift, set.rows, row, dim);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = used ? o[i] : 0u;
            store8(to, o);
            store8(to + 8, o + 8);
          }
        }
      }
      seg += ns > 0;
      tc::fence_before();
    }
  } else if (warp < C::kWarpV) {  // ---- keys of 32 tokens of a page, and the queries of each segment
    const int all = tid - 32 * C::kWarpK, grp = all >> 6;
    KeyThread<KQ> keys;
    keys.init(p, (all & 63) + 64 * rank, C::kKAtom);
    keys.row_off -= rank * C::kKAtom;  // the page's second 32 rows come first here
    const uint2 lut = code_halves(p.k);
    int n = 0, seg = 0;
    PageRegs regs = {};
    while (w.next(set)) {
      const Rows r = w.rows;
      const int ns = segment_pages(w);
      if (ns == 0) continue;
      const int first = (grp + C::KG - n % C::KG) % C::KG;  // this group's first page of the segment
      int page = w.k0 + first;
      if (first < ns) keys.fetch(p, regs, page_tile(p, w, page, page_entry(p, w, page)));
      int entry = page_entry(p, w, page + C::KG);  // of the page after the one in regs
      if (seg > 0) wait(bars.qempty, (seg - 1) & 1);
      ++seg;
      constexpr int kChunks = DK / 8;
      const unsigned char* q0 = static_cast<const unsigned char*>(p.qprep) +
                                ((size_t)(r.start + r.first) * p.Hq + w.hk * p.group) * DK * sizeof(__half);
      const int shift = 31 - __clz(p.group);  // groups are powers of two
      // copied asynchronously: loads that wait for one another's stores took 19000 cycles a segment, registers to hold
      // them spilled
#pragma unroll 4
      for (int i = all; i < NT * kTileRows * kChunks; i += 64 * C::KG) {
        const int here = i / kChunks, ch = i % kChunks;
        const int t = here / kTileRows, rr = here & (kTileRows - 1), row = t * 2 * kTileRows + rank * kTileRows + rr;
        unsigned char* dst = smem + t * C::kQTile + (ch >> 3) * (kTileRows * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
        if (row < r.count) cp_async16(dst, q0 + (size_t)(((row >> shift) * p.Hq + (row & (p.group - 1))) * (DK * 2) + 16 * ch));
        else *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
      }
      cp_async_commit();
      cp_async_wait<0>();
      arrive_first(bars.qfull);
      for (int j = first; j < ns; j += C::KG, page += C::KG) {
        const int nj = n + j, st = nj % kStages;
        const PageRegs cur = regs;
        if (j + C::KG < ns) {
          keys.fetch(p, regs, page_tile(p, w, page + C::KG, entry));
          entry = page_entry(p, w, page + 2 * C::KG);
        }
        if (nj >= kStages) wait(bars.kempty[st], (nj / kStages - 1) & 1);
        const uint32_t base = sm + C::kOffK + st * C::kKStage;
        keys.both(p, cur, lut, base, 2 * C::kKAtom);
        arrive_first(bars.kfull[st]);
      }
      n += ns;
    }
  } else if (warp < C::kWarpS) {  // ---- dims 64 rank .. + 63 of a page's values
    const int th = (tid - 32 * C::kWarpV) & 63, grp = (tid - 32 * C::kWarpV) >> 6;
    ValueThread<VQ> values;
    values.init(p, th & 7, 8 * rank + (th >> 3), th >> 3);
    const uint2 lut = code_halves(p.v);
    int n = 0, seg = 0;
    PageRegs regs = {};
    while (w.next(set)) {
      const int ns = segment_pages(w), limit = w.rows.limit;
      if (ns == 0) continue;
      if (th == 0 && grp == 0) bars.bad[(seg + kSlots / 2) % kSlots] = 0x7fffffff;  // last read before: kSlots
      const int first = (grp + C::VG - n % C::VG) % C::VG;  // this group's first page of the segment
      int page = w.k0 + first;
      if (first < ns) values.fetch(p, regs, page_tile(p, w, page, page_entry(p, w, page)));
      int entry = page_entry(p, w, page + C::VG);  // of the page after the one in regs
      for (int j = first; j < ns; j += C::VG, page += C::VG) {
        const int nj = n + j, st = nj % kStages;
        const PageRegs cur = regs;
        if (j + C::VG < ns) {
          values.fetch(p, regs, page_tile(p, w, page + C::VG, entry));
          entry = page_entry(p, w, page + 2 * C::VG);
        }
        if (nj >= kStages) wait(bars.vempty[st], (nj / kStages - 1) & 1);
        const uint32_t bad = values.store(p, cur, lut, sm + C::kOffV + st * C::kVStage, 64 * 128, limit - page * kPage);
        if (bad != 0 && th < 8) atomicMin(&bars.bad[seg % kSlots], page * kPage + 8 * th + __ffs(bad) - 1);
        arrive_first(bars.vfull[st]);
      }
      n += ns;
      ++seg;
    }
  } else {
    fewer_registers<C::kShare, C::kRegsIssue>();
    if (rank == 0 && warp == C::kWarpS) {  // ---- S = Q K^T (the whole warp, so that control stays uniform)
      constexpr uint32_t id = tc::idesc_f16(0, 0, 0, 2 * kTileRows, kPage);
      int n = 0, seg = 0, nt[NT] = {};
      while (w.next(set)) {
        const int ns = __shfl_sync(0xffffffffu, segment_pages(w), 0), count = __shfl_sync(0xffffffffu, w.rows.count, 0);
        if (ns == 0) continue;
        wait_both(bars.qfull, seg & 1);
        ++seg;
        for (int j = 0; j < ns; ++j, ++n) {
          const int st = n % kStages;
          wait_both(bars.kfull[st], (n / kStages) & 1);
          const uint64_t kd = desc_sw128(sm + C::kOffK + st * C::kKStage);
  #pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t * 2 * kTileRows >= count) continue;
            const int b = nt[t] % NB;
            if (nt[t] >= NB) wait(bars.pvdone[t][b], (nt[t] / NB - 1) & 1);  // the P that lies there is read
            tc::fence_after();
            const uint64_t qd = desc_sw128(sm + t * C::kQTile);
  #pragma unroll
            for (int i = 0; i < DK / 64; ++i)
              tc::pair_f16_x4(tmem + kColS + (t * NB + b) * kPage, qd + ((i * kTileRows * 128) >> 4), kd + ((i * C::kKAtom) >> 4),
                              id, i > 0);
            tc::pair_commit(smem_addr(&bars.sfull[t][b]));
            ++nt[t];
          }
          tc::pair_commit(smem_addr(&bars.kempty[st]));
        }
        tc::pair_commit(smem_addr(&bars.qempty));
      }
      tc::pair_commit(smem_addr(&bars.done[0]));
      mbar_wait(smem_addr(&bars.done[0]), 0, p.wait_limit);
    } else if (rank == 0 && warp == C::kWarpO) {  // ---- O += P V
      constexpr uint32_t id = tc::idesc_f16(0, 0, 0, 2 * kTileRows, DV);
      int n = 0, nt[NT] = {};
      while (w.next(set)) {
        const int ns = __shfl_sync(0xffffffffu, segment_pages(w), 0), count = __shfl_sync(0xffffffffu, w.rows.count, 0);
        for (int j = 0; j < ns; ++j, ++n) {
          const int st = n % kStages;
          wait_both(bars.vfull[st], (n / kStages) & 1);
          const uint64_t vd = desc_sw128(sm + C::kOffV + st * C::kVStage);
  #pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t * 2 * kTileRows >= count) continue;
            const int b = nt[t] % NB;
            wait_both(bars.pready[t][b], (nt[t] / NB) & 1);
            tc::fence_after();
            tc::pair_f16_ta_x4(tmem + t * DV, tmem + kColS + (t * NB + b) * kPage, vd, id, j > 0);
            tc::pair_commit(smem_addr(&bars.pvdone[t][b]));
            ++nt[t];
          }
          tc::pair_commit(smem_addr(&bars.vempty[st]));
        }
      }
      tc::pair_commit(smem_addr(&bars.done[1]));
      mbar_wait(smem_addr(&bars.done[1]), 0, p.wait_limit);
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  cluster_sync();  // the products are done, and no arrival is on its way to a CTA that has left
  if (warp == 0) {
    tc::fence_after();
    tc::pair_dealloc(tmem, kTmemCols);
  }
}

template <bool KQ, bool VQ>
cudaError_t launch(const ChunkParams& p, cudaStream_t s) {
  constexpr int smem = Cfg<KQ, VQ>::kOffEnd;
  const cudaError_t e = cudaFuncSetAttribute(chunk_umma<KQ, VQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_after(chunk_umma<KQ, VQ>, p, 2 * p.set[kWide].ctas, Cfg<KQ, VQ>::kThreads, smem, 2, s);
}

}  // namespace

int chunk_umma_rows(bool v_qjl) { return 2 * kTileRows * (v_qjl ? Cfg<true, true>::NT : Cfg<true, false>::NT); }

cudaError_t launch_chunk_umma(const ChunkParams& p, cudaStream_t s) {
  if (p.k.qjl) return p.v.qjl ? launch<true, true>(p, s) : launch<true, false>(p, s);
  return p.v.qjl ? launch<false, true>(p, s) : launch<false, false>(p, s);
}

}  // namespace kvq
