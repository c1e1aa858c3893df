// Chunk attention's segment kernel on 5th-generation tensor cores (tcgen05, kind::f16, fp32 sums), for bf16
// queries. Work plan and the states it leaves: kvq_chunk.cuh.
//
// A CTA walks its segments page by page (64 tokens). Per page and tile of 128 query rows
//   S [128 x 64]  = Q [128 x DK] . K^T          (A, B from shared memory; DK = 128, + 128 of the key sketch)
//   O [128 x DV] += P [128 x 64] . V            (A from tensor memory; DV = 128, + 128 of the value sketch)
// with K and V dequantised from the packed page into fp16 (kvq_chunk_dequant.cuh). NT row tiles share a page's dequantisation: two where tensor
// memory holds their sums (O takes 2 x 128 columns, S 2 x 2 x 64), one with a value sketch (O 256).
//
// Warps: 4 per row tile for the softmax (thread = row), 4 or 8 that dequantise keys (and fetch the queries of
// a segment), 4 or 8 for values, 2 that issue the products (S, and P V one page behind; one thread issues an MMA
// about every 50 cycles, so the two kinds run on two warps). K and V pages are staged twice, S twice per
// tile, so that dequantisation, S, softmax and P V of neighbouring pages overlap. P overwrites the first
// 32 columns of its S.
//
// Softmax weights are p = 2^(x - m + 7), m the row's maximum but for steps under 2^8, by which it may lag
// before O is rescaled: p stays under 2^15 in fp16, and a weight is dropped only below 2^-31 of the largest.
#include "kvq_async.cuh"
#include "kvq_chunk_dequant.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

using namespace chunk;

constexpr int kStages = 2;
constexpr int kTileRows = 128;
constexpr float kLag = 8.f, kShift = 7.f;
constexpr uint32_t kColS = 256, kTmemCols = 512;

template <bool KQ, bool VQ>
struct Cfg {
  static constexpr int NT = VQ ? 1 : 2;
  static constexpr int DK = KQ ? 256 : 128, DV = VQ ? 256 : 128;
  // groups of 4 warps that dequantise a side, page n on group n % G: two where a sketch doubles the work
  static constexpr int KG = KQ ? 2 : 1, VG = VQ ? 2 : 1;
  static constexpr int kWarpK = 4 * NT, kWarpV = kWarpK + 4 * KG, kWarpS = kWarpV + 4 * VG, kWarpO = kWarpS + 1;
  static constexpr int kThreads = 32 * (kWarpO + 1);
  static constexpr int kQTile = kTileRows * DK * 2, kKStage = kPage * DK * 2, kVStage = kPage * DV * 2;
  static constexpr int kOffK = NT * kQTile, kOffV = kOffK + kStages * kKStage, kOffEnd = kOffV + kStages * kVStage;
};

template <int NT>
struct Bars {
  uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
  uint64_t sfull[NT][2], pready[NT][2], pvdone[NT][2];
  uint64_t qfull, qempty, done[2];
  unsigned char vbad[kStages][8];  // tokens of the page whose value norm is not finite, a bit each
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
// bounds the softmax; a quarter of them is made here instead.
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

template <bool KQ, bool VQ>
__global__ void __launch_bounds__(Cfg<KQ, VQ>::kThreads, 1) chunk_umma(const __grid_constant__ ChunkParams p) {
  using C = Cfg<KQ, VQ>;
  constexpr int NT = C::NT, DK = C::DK, DV = C::DV;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) Bars<NT> bars;
  const ChunkSet& set = p.set[kWide];
  if (set.head[1] == 0) return;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&bars.kfull[i]), 4);
      mbar_init(smem_addr(&bars.kempty[i]), 1);
      mbar_init(smem_addr(&bars.vfull[i]), 4);
      mbar_init(smem_addr(&bars.vempty[i]), 1);
    }
    for (int t = 0; t < NT; ++t)
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&bars.sfull[t][b]), 1);
        mbar_init(smem_addr(&bars.pready[t][b]), 4);
        mbar_init(smem_addr(&bars.pvdone[t][b]), 1);
      }
    mbar_init(smem_addr(&bars.qfull), 4 * C::KG);
    mbar_init(smem_addr(&bars.qempty), 1);
    mbar_init(smem_addr(&bars.done[0]), 1);
    mbar_init(smem_addr(&bars.done[1]), 1);
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

  if (warp < C::kWarpK) {  // ---- softmax: thread = row
    const int t = warp >> 2, row = tid;  // row of the NT * 128
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tO = tmem + lanes + t * DV, tS = tmem + lanes + kColS + t * 128;
    int n = 0, nv = 0;  // pages this tile, and the CTA, has seen
    while (w.next(p, set)) {
      const Rows r = w.rows;
      const int np = segment_pages(w);
      const bool used = t * kTileRows < r.count && np > 0;
      const bool work = warp * 32 < r.count;
      // rows of no token count as unmasked: what they compute is not kept, and the others' mask may still be empty
      const int last = row < r.count ? min(r.pos0 + row / p.group, r.ctx - 1) : 0x7fffffff;
      float qs = 1.f;
      if (row < r.count)
        qs = p.qscale[(size_t)(r.start + r.first + row / p.group) * p.Hq + w.hk * p.group + row % p.group];
      float m = -INFINITY, ref = 0.f, l = 0.f;
      for (int j = 0; used && j < np; ++j, ++n) {
        const int b = n & 1, st = (nv + j) % kStages;
        wait(bars.sfull[t][b], (n >> 1) & 1);
        tc::fence_after();
        if (work) {
          // two halves of 32 columns, read from tensor memory again for the second pass: a rolled loop (see expand)
          const int reach = last - (w.k0 + j) * kPage;  // the page's tokens 0 .. reach are attended
          const bool full = __all_sync(0xffffffffu, reach >= kPage - 1);
          auto logits = [&](uint32_t (&s)[32], int c) {
            tc::tmem_ld32(tS + 64 * b + c, s);
            tc::wait_ld();
            if (!full) {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = c + i <= reach ? s[i] : 0xff800000u;
            }
          };
          float mx2[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < kPage; c += 32) {
            uint32_t s[32];
            logits(s, c);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              mx2[i & 1] = max3(mx2[i & 1], __uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
          }
          const float mx = fmaxf(mx2[0], mx2[1]) * qs;
          const bool grow = mx > m + kLag || (m == -INFINITY && mx > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = grow ? ex2f(m - mx) : 1.f;
            if (grow) {
              m = mx;
              ref = mx - kShift;
            }
            l *= alpha;
            if (j > 0) {
              wait(bars.pvdone[t][(n - 1) & 1], ((n - 1) >> 1) & 1);
              tc::fence_after();
#pragma unroll 1
              for (int c = 0; c < DV; c += 16) {
                uint32_t o[16];
                tc::tmem_ld16(tO + c, o);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tc::tmem_st16(tO + c, o);
              }
              tc::wait_st();
            }
          }
          F2 sum[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
          const F2 qs2(qs, qs), ref2(-ref, -ref);
#pragma unroll 1
          for (int c = 0; c < kPage; c += 32) {
            uint32_t s[32], ph[16];
            logits(s, c);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              F2 x = fma(F2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), qs2, ref2);
              float a, d;
              if ((i & 3) == 3) {
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
            tc::tmem_st16(tS + 64 * b + c / 2, ph);
          }
          float la, lb;
          add(sum[0], sum[1]).get(la, lb);
          l += la + lb;
          wait(bars.vfull[st], ((nv + j) / kStages) & 1);
          const unsigned long long bad = *reinterpret_cast<const volatile unsigned long long*>(bars.vbad[st]);
          if (bad != 0 && reach >= 0 && (bad & (~0ull >> (63 - min(reach, 63)))) != 0) l = NAN;
          tc::wait_st();
        }
        tc::fence_before();
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(smem_addr(&bars.pready[t][b]));
      }
      nv += np;
      // the segment's state
      if (used) {
        wait(bars.pvdone[t][(n - 1) & 1], ((n - 1) >> 1) & 1);
        tc::fence_after();
      }
      if (work) {
        float* ml = segment_ml(set, w.item, blockIdx.x, DV) + 2 * row;
        float* so = segment_o(set, w.item, blockIdx.x, DV) + (size_t)row * DV;
        if (row < r.count) *reinterpret_cast<float2*>(ml) = make_float2(m == -INFINITY ? m : ref, m == -INFINITY && l == l ? 0.f : l);
#pragma unroll 1
        for (int c = 0; c < DV; c += 16) {
          uint32_t o[16];
          if (used) {
            tc::tmem_ld16(tO + c, o);
            tc::wait_ld();
          }
          if (row < r.count)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(so + c + i) =
                  used ? make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]) : make_uint4(0, 0, 0, 0);
        }
      }
      tc::fence_before();
    }
  } else if (warp < C::kWarpV) {  // ---- keys, and the queries of each segment
    const int all = tid - 32 * C::kWarpK, th = all & 127, grp = all >> 7;
    KeyThread<KQ> keys;
    keys.init(p, th, kPage * 128);
    const uint2 lut = code_halves(p.k);
    int n = 0, seg = 0;
    PageRegs regs = {};
    while (w.next(p, set)) {
      const Rows r = w.rows;
      const int np = segment_pages(w);
      if (np == 0) continue;
      const int first = (grp + C::KG - n % C::KG) % C::KG;  // this group's first page of the segment
      if (first < np) keys.fetch(p, regs, page_tile(p, w, w.k0 + first, page_entry(p, w, w.k0 + first)));
      int entry = page_entry(p, w, w.k0 + first + C::KG);  // of the page after the one in regs
      if (seg > 0) wait(bars.qempty, (seg - 1) & 1);
      ++seg;
      constexpr int kChunks = DK / 8;
      const size_t qrow0 = (size_t)(r.start + r.first) * p.Hq + w.hk * p.group;
#pragma unroll 8
      for (int i = all; i < NT * kTileRows * kChunks; i += 128 * C::KG) {
        const int row = i / kChunks, ch = i % kChunks;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < r.count)
          v = *(reinterpret_cast<const uint4*>(static_cast<const __half*>(p.qprep) +
                                               (qrow0 + (size_t)(row / p.group) * p.Hq + row % p.group) * DK) + ch);
        const int rr = row & (kTileRows - 1);
        *reinterpret_cast<uint4*>(smem + (row / kTileRows) * C::kQTile + (ch >> 3) * (kTileRows * 128) + rr * 128 +
                                  (((ch & 7) ^ (rr & 7)) << 4)) = v;
      }
      arrive_rows(bars.qfull);
      for (int j = first; j < np; j += C::KG) {
        const int nj = n + j, st = nj % kStages;
        const PageRegs cur = regs;
        if (j + C::KG < np) {
          keys.fetch(p, regs, page_tile(p, w, w.k0 + j + C::KG, entry));
          entry = page_entry(p, w, w.k0 + j + 2 * C::KG);
        }
        if (nj >= kStages) wait(bars.kempty[st], (nj / kStages - 1) & 1);
        const uint32_t base = sm + C::kOffK + st * C::kKStage;
        keys.codes(p, cur, lut, base);
        if (KQ) keys.signs(cur, base + 2 * kPage * 128);
        arrive_rows(bars.kfull[st]);
      }
      n += np;
    }
  } else if (warp < C::kWarpS) {  // ---- values: dims 8 k .. + 7 of tokens 8 c .. + 7
    const int th = (tid - 32 * C::kWarpV) & 127, grp = (tid - 32 * C::kWarpV) >> 7;
    ValueThread<VQ> values;
    values.init(th);
    const uint2 lut = code_halves(p.v);
    int n = 0;
    PageRegs regs = {};
    while (w.next(p, set)) {
      const int np = segment_pages(w);
      if (np == 0) continue;
      const int first = (grp + C::VG - n % C::VG) % C::VG;  // this group's first page of the segment
      if (first < np) values.fetch(p, regs, page_tile(p, w, w.k0 + first, page_entry(p, w, w.k0 + first)));
      int entry = page_entry(p, w, w.k0 + first + C::VG);  // of the page after the one in regs
      for (int j = first; j < np; j += C::VG) {
        const int nj = n + j, st = nj % kStages;
        const PageRegs cur = regs;
        const int limit = w.rows.limit - (w.k0 + j) * kPage;
        if (j + C::VG < np) {
          values.fetch(p, regs, page_tile(p, w, w.k0 + j + C::VG, entry));
          entry = page_entry(p, w, w.k0 + j + 2 * C::VG);
        }
        if (nj >= kStages) wait(bars.vempty[st], (nj / kStages - 1) & 1);
        const uint32_t bad = values.store(p, cur, lut, sm + C::kOffV + st * C::kVStage, limit);
        if (th < 8) bars.vbad[st][th] = (unsigned char)bad;
        arrive_rows(bars.vfull[st]);
      }
      n += np;
    }
  } else if (warp == C::kWarpS) {  // ---- S = Q K^T (the whole warp, so that control stays uniform)
    constexpr uint32_t id = tc::idesc_f16(0, 0, 0, kTileRows, kPage);
    int n = 0, seg = 0, nt[NT] = {};
    while (w.next(p, set)) {
      const int np = __shfl_sync(0xffffffffu, segment_pages(w), 0), count = __shfl_sync(0xffffffffu, w.rows.count, 0);
      if (np == 0) continue;
      wait(bars.qfull, seg & 1);
      ++seg;
      for (int j = 0; j < np; ++j, ++n) {
        const int st = n % kStages;
        wait(bars.kfull[st], (n / kStages) & 1);
        const uint64_t kd = desc_sw128(sm + C::kOffK + st * C::kKStage);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (t * kTileRows >= count) continue;
          const int b = nt[t] & 1;
          if (nt[t] >= 2) wait(bars.pvdone[t][b], ((nt[t] >> 1) - 1) & 1);  // P of two pages before is read
          tc::fence_after();
          const uint64_t qd = desc_sw128(sm + t * C::kQTile);
#pragma unroll
          for (int i = 0; i < DK / 64; ++i)
            tc::umma_f16_x4(tmem + kColS + t * 128 + b * 64, qd + ((i * kTileRows * 128) >> 4), kd + ((i * kPage * 128) >> 4), id,
                            i > 0);
          tc::commit_elected(smem_addr(&bars.sfull[t][b]));
          ++nt[t];
        }
        tc::commit_elected(smem_addr(&bars.kempty[st]));
      }
      tc::commit_elected(smem_addr(&bars.qempty));
    }
    tc::commit_elected(smem_addr(&bars.done[0]));
    mbar_wait(smem_addr(&bars.done[0]), 0, p.wait_limit);
  } else {  // ---- O += P V
    constexpr uint32_t id = tc::idesc_f16(0, 0, 0, kTileRows, DV);
    int n = 0, nt[NT] = {};
    while (w.next(p, set)) {
      const int np = __shfl_sync(0xffffffffu, segment_pages(w), 0), count = __shfl_sync(0xffffffffu, w.rows.count, 0);
      for (int j = 0; j < np; ++j, ++n) {
        const int st = n % kStages;
        wait(bars.vfull[st], (n / kStages) & 1);
        const uint64_t vd = desc_sw128(sm + C::kOffV + st * C::kVStage);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (t * kTileRows >= count) continue;
          const int b = nt[t] & 1;
          wait(bars.pready[t][b], (nt[t] >> 1) & 1);
          tc::fence_after();
          tc::umma_f16_ta_x4(tmem + t * DV, tmem + kColS + t * 128 + b * 64, vd, id, j > 0);
          tc::commit_elected(smem_addr(&bars.pvdone[t][b]));
          ++nt[t];
        }
        tc::commit_elected(smem_addr(&bars.vempty[st]));
      }
    }
    tc::commit_elected(smem_addr(&bars.done[1]));
    mbar_wait(smem_addr(&bars.done[1]), 0, p.wait_limit);
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
  const cudaError_t e = cudaFuncSetAttribute(chunk_umma<KQ, VQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  chunk_umma<KQ, VQ><<<p.ctas, Cfg<KQ, VQ>::kThreads, smem, s>>>(p);
  return launched();
}

}  // namespace

int chunk_umma_rows(bool v_qjl) { return kTileRows * (v_qjl ? Cfg<true, true>::NT : Cfg<true, false>::NT); }

cudaError_t launch_chunk_umma(const ChunkParams& p, cudaStream_t s) {
  if (p.k.qjl) return p.v.qjl ? launch<true, true>(p, s) : launch<true, false>(p, s);
  return p.v.qjl ? launch<false, true>(p, s) : launch<false, false>(p, s);
}

}  // namespace kvq
