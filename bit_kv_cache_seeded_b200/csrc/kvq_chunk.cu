// Attention of a ragged batch of new tokens over the packed LM / LM_QJL / SIGN1 cache: plan, query
// prep, the fp32 segment kernel, and the merge (bf16's segment kernels: kvq_chunk_umma.cu, kvq_chunk_narrow.cu).
// ("TurboQuant vs OSCAR vs EpiCache", section "Quantization frontiers: TurboQuant and OSCAR": rotation, Lloyd-Max codes,
// QJL sketch; kernels compatible with paged attention.)
//
// With R = H D / sqrt(d), a key k_t is held as n_t / sqrt(d) R^T (c[code] + kappa gamma_t S^T z_t), kappa =
// sqrt(pi/2) / m. Rotating and sketching the query once (q~ = R q, s = kappa S q~) leaves
//   logit_t = scale n_t / sqrt(d) (<q~, c[code_t]> + gamma_t <s, z_t>),
// and the value sum is rotated back once per row:
//   out = D H / d (sum_t w_t c[code_t] + kappa S^T sum_t w_t gamma_t z_t) / sum_t p_t,  w_t = p_t n_t.
// Launches: prep (plan and queries), segments (kvq_chunk.cuh), merge. fp32 calls have one segment kernel, bf16 ones up to
// three: the wide one, where the call is large enough for it, and the narrow one, with a value sketch in two instances.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_async.cuh"
#include "kvq_chunk.cuh"
#include "kvq_lm_common.cuh"
#include "kvq_quantize_lm.cuh"
#include "kvq_ragged.h"

namespace kvq {
namespace {

using namespace chunk;

constexpr int kPrepThreads = 256;
constexpr int kPrepRows = 32;     // query rows of a prep block: 4 per warp
constexpr float kKappa = lmc::kSqrtHalfPi / kHeadDim;

// Walsh-Hadamard transform of 128 coordinates, lane l holding 4 l .. 4 l + 3 (so that a row is read and written
// 16 or 8 bytes a lane), unnormalised.
__device__ __forceinline__ void fwht(float (&u)[4], int lane) {
#pragma unroll
  for (int b = 0; b < 5; ++b) {
    const bool upper = (lane >> b) & 1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float other = __shfl_xor_sync(0xffffffffu, u[k], 1 << b);
      u[k] = upper ? other - u[k] : u[k] + other;
    }
  }
  const float a0 = u[0] + u[1], a1 = u[0] - u[1], a2 = u[2] + u[3], a3 = u[2] - u[3];
  u[0] = a0 + a2; u[2] = a0 - a2; u[1] = a1 + a3; u[3] = a1 - a3;
}

__device__ __forceinline__ void load4(float (&u)[4], const void* row, bool bf16, int lane) {
  if (bf16) {
    const uint2 v = *(static_cast<const uint2*>(row) + lane);
    u[0] = __uint_as_float(v.x << 16);
    u[1] = __uint_as_float(v.x & 0xffff0000u);
    u[2] = __uint_as_float(v.y << 16);
    u[3] = __uint_as_float(v.y & 0xffff0000u);
  } else {
    const float4 v = *(static_cast<const float4*>(row) + lane);
    u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
  }
}
__device__ __forceinline__ void store4(float* row, const float (&u)[4], int lane) {
  *reinterpret_cast<float4*>(row + 4 * lane) = make_float4(u[0], u[1], u[2], u[3]);
}
template <typename T2>
__device__ __forceinline__ uint2 pack4(T2 a, T2 b) {
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// C [32 x 128] = A [32 x 128] . M [128 x 128] on the tensor cores (mma.sync, fp16 operands, fp32 sums) for the
// bf16 calls' two small products with the sketch matrix: S q~ per query row, S^T z per output row. A row of A
// and all of M (its exponent is the cache's) are brought into fp16's range by powers of two; each rounding is half a step, 2^-11. Warp w of 8
// makes columns 16 w .. + 15 and keeps its fragments of M in registers over the block's row groups. On the CUDA
// cores the products took half of these kernels' time (prep of 131072 rows 207 us, merge of 55000 rows 110;
// 55 and 53 now, with the other steps).
constexpr int kPad = kHeadDim + 4;    // row stride of an fp32 row in shared memory
constexpr int kPadH = kHeadDim + 8;   // of an fp16 row: the 8 rows that ldmatrix reads at once lie in distinct banks

struct Frags {
  uint32_t b[2][8][2];
  float inv;  // 1 / the power of two that M was multiplied by
};
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
// The power of two that a largest magnitude is divided by to come to [2^9, 2^10): from the exponent's bits, within
// fp32's normal numbers (infinities and NaN give some power of two, and stay what they are).
__device__ __forceinline__ int scale_exp(float mx) { return min(max((__float_as_int(mx) >> 23) - 136, -126), 119); }
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ void load_frags(Frags& f, const float* M, int e, int warp, int lane) {
  const float mul = pow2(-e);
  f.inv = pow2(e);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* at = M + (16 * k + 2 * (lane & 3) + 8 * h) * kHeadDim + 16 * warp + 8 * n + (lane >> 2);
        const __half2 v = __floats2half2_rn(__ldg(at) * mul, __ldg(at + kHeadDim) * mul);
        f.b[n][k][h] = *reinterpret_cast<const uint32_t*>(&v);
      }
}
__device__ __forceinline__ void fp16_product(const Frags& f, const __half (*a)[kPadH], float (*c)[kPad], int warp, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float acc[2][4] = {};
    const uint32_t row = (uint32_t)__cvta_generic_to_shared(&a[16 * m + (lane & 15)][8 * (lane >> 4)]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t a0, a1, a2, a3;
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                   : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3) : "r"(row + 32 * k) : "memory");
#pragma unroll
      for (int n = 0; n < 2; ++n)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                     : "+f"(acc[n][0]), "+f"(acc[n][1]), "+f"(acc[n][2]), "+f"(acc[n][3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(f.b[n][k][0]), "r"(f.b[n][k][1]));
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(&c[16 * m + g + 8 * h][16 * warp + 8 * n + 2 * t]) =
            make_float2(acc[n][2 * h] * f.inv, acc[n][2 * h + 1] * f.inv);
  }
}
// One row of A, scaled by its own power of two, which it returns.
__device__ __forceinline__ float store_row(__half* a, const float (&u)[4], int lane) {
  const int e = scale_exp(warp_max(fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3])))));
  const float mul = pow2(-e);
  *reinterpret_cast<uint2*>(a + 4 * lane) =
      pack4(__floats2half2_rn(u[0] * mul, u[1] * mul), __floats2half2_rn(u[2] * mul, u[3] * mul));
  return pow2(e);
}

// Brings a 128 x 128 fp32 matrix into the L1 (256 threads): its rows are needed one after another, and a small call
// has nothing else to hide their latency under.
__device__ __forceinline__ void warm_l1(const float* m) {
#pragma unroll
  for (int i = 0; i < kHeadDim * kHeadDim / 4 / 256; ++i) {
    float a, b, c, d;
    asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];\n"
                 : "=f"(a), "=f"(b), "=f"(c), "=f"(d) : "l"(m + 4 * (256 * i + (int)threadIdx.x)));
  }
}

// One block's plan of a set: row tiles per request, their units, prefix sums of both.
__device__ void plan(const ChunkParams& p, const ChunkSet& s) {
  __shared__ long long s_warp[kPrepThreads / 32];
  __shared__ long long s_run;
  __shared__ int s_most;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = s.rows / p.group;
  auto scan = [&](long long v) {  // exclusive prefix of v over the block, carried in s_run
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long before = s_run;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    __syncthreads();
    if (tid == kPrepThreads - 1) s_run = before + x;
    __syncthreads();
    return before + x - v;
  };
  if (tid == 0) {
    s_run = 0;
    s_most = 0;
  }
  __syncthreads();
  int most = 0;  // tokens of the fullest tile
  for (int b0 = 0; b0 < p.B; b0 += kPrepThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.B) n = max(clamp_start(p, b + 1) - clamp_start(p, b), 0);
    if (n * p.group <= s.above || n * p.group > s.upto) n = 0;
    most = max(most, min(n, per));
    const long long at = scan((n + per - 1) / per);
    // max_tiles holds every tile of a seq_start that does not decrease; another one is cut there
    if (b < p.B) s.tile_start[b] = (int)min(at, (long long)s.max_tiles);
  }
  const int tiles = (int)min(s_run, (long long)s.max_tiles);
  if (most > 0) atomicMax(&s_most, most);
  __syncthreads();
  if (tid == 0) {
    s.tile_start[p.B] = tiles;
    s_run = 0;
  }
  __syncthreads();
  for (int t0 = 0; t0 < tiles; t0 += kPrepThreads) {
    const int t = t0 + tid;
    long long units = 0;
    if (t < tiles) {
      int lo = 0, hi = p.B;  // the last request with tile_start <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.tile_start[mid] <= t) lo = mid;
        else hi = mid;
      }
      const Rows r = tile_rows(p, s, lo, t - s.tile_start[lo]);
      store_rows(s, t, r);
      units = max(1, (r.limit + s.unit - 1) / s.unit);
    }
    const long long at = scan(units);
    if (t < tiles) s.unit_start[t] = at;
  }
  if (tid == 0) {
    s.unit_start[tiles] = s_run;
    s.head[0] = tiles;
    s.head[1] = s_run;
    s.head[2] = (long long)s_most * p.group;
  }
}

// The first blocks plan, one a set; the others rotate (and sketch) kPrepRows query rows each, the logit scale and 1/sqrt(d) of
// the keys folded in. fp32 queries: rows of fp32 [d (+ m)]. bf16 queries: rows of fp16 for the tensor-core
// kernel, in its order and with its scales, divided by a power of two (kept in qscale) that brings the row's
// largest entry to [2^9, 2^10): half a step is 2^-11 of an entry down to 2^-23 of the largest.
template <bool KQ, bool BF16>
__global__ void __launch_bounds__(kPrepThreads, 2) chunk_prep(const __grid_constant__ ChunkParams p) {
  if (blockIdx.x < p.sets) {
    plan(p, p.set[blockIdx.x]);
    return;
  }
  const int block = blockIdx.x - p.sets, blocks = gridDim.x - p.sets;
  __shared__ __align__(16) float s_q[KQ ? kPrepRows : 1][kPad];   // queries, and then (bf16) their sketches
  __shared__ __align__(16) __half s_a[KQ && BF16 ? kPrepRows : 1][kPadH];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = p.n_tokens * p.Hq;  // at most 2^30
  const int shift = 31 - __clz(p.group);  // groups are powers of two
  constexpr int DK = KQ ? 2 * kHeadDim : kHeadDim;
  Frags frags;
  if (KQ && BF16) load_frags(frags, p.St, p.s_exp, warp, lane);
  else if (KQ) warm_l1(p.St);
  float next[4][4];  // the next group's queries, loaded a group ahead
  auto fetch = [&](int group) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = group * kPrepRows + 4 * warp + v;
#pragma unroll
      for (int k = 0; k < 4; ++k) next[v][k] = 0.f;
      if (row < rows) load4(next[v], static_cast<const char*>(p.q) + (size_t)row * kHeadDim * (BF16 ? 2 : 4), BF16, lane);
    }
  };
  fetch(block);
  for (int group = block; group * kPrepRows < rows; group += blocks) {
    const int row0 = group * kPrepRows + 4 * warp;
    int head = row0 % p.Hq;
    float rot[4][4], sk[4][4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        rot[v][k] = next[v][k];
        sk[v][k] = 0.f;
      }
    fetch(group + blocks);
    float back[4];  // powers of two of the product's rows
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float sg[4];
      load4(sg, p.signs + (head >> shift) * p.signs_stride, false, lane);
      if (++head == p.Hq) head = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) rot[v][k] *= sg[k];
      fwht(rot[v], lane);
      // R q * scale / sqrt(d) = H D q * scale / d
#pragma unroll
      for (int k = 0; k < 4; ++k) rot[v][k] *= p.logit_scale * (1.f / kHeadDim);
      if (KQ && BF16) back[v] = store_row(s_a[4 * warp + v], rot[v], lane);
      else if (KQ) store4(s_q[4 * warp + v], rot[v], lane);
    }
    if (KQ && BF16) {  // S q~
      __syncthreads();
      fp16_product(frags, s_a, s_q, warp, lane);
      __syncthreads();
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        load4(sk[v], s_q[4 * warp + v], false, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) sk[v][k] *= back[v];
      }
    } else if (KQ) {  // rows j = 4 lane .. + 3 of S q~, from S^T [i][j]
      __syncwarp();
#pragma unroll 1
      for (int i0 = 0; i0 < kHeadDim; i0 += 16) {
        float part[4][4] = {};
#pragma unroll
        for (int i = i0; i < i0 + 16; ++i) {
          const float4 st = __ldg(reinterpret_cast<const float4*>(p.St + i * kHeadDim) + lane);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float x = s_q[4 * warp + v][i];
            part[v][0] = fmaf(st.x, x, part[v][0]);
            part[v][1] = fmaf(st.y, x, part[v][1]);
            part[v][2] = fmaf(st.z, x, part[v][2]);
            part[v][3] = fmaf(st.w, x, part[v][3]);
          }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int k = 0; k < 4; ++k) sk[v][k] += part[v][k];
      }
      __syncwarp();
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = row0 + v;
      if (row >= rows) break;
#pragma unroll
      for (int k = 0; k < 4; ++k) sk[v][k] *= kKappa;
      if (!BF16) {
        float* dst = static_cast<float*>(p.qprep) + (size_t)row * DK;
        store4(dst, rot[v], lane);
        if (KQ) store4(dst + kHeadDim, sk[v], lane);
        continue;
      }
      float mx = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        rot[v][k] *= kCodeScale;
        sk[v][k] *= kSketchScale;
        mx = fmaxf(mx, fmaxf(fabsf(rot[v][k]), fabsf(sk[v][k])));
      }
      const int e = scale_exp(warp_max(mx));
      const float inv = pow2(-e);
      __half* dst = static_cast<__half*>(p.qprep) + (size_t)row * DK + query_pos(p.k.order, lane);
      if (p.k.order == kOrderOctet) {
        *reinterpret_cast<uint2*>(dst) = pack4(__floats2half2_rn(rot[v][0] * inv, rot[v][1] * inv),
                                               __floats2half2_rn(rot[v][2] * inv, rot[v][3] * inv));
        if (KQ)
          *reinterpret_cast<uint2*>(dst + kHeadDim) = pack4(__floats2half2_rn(sk[v][0] * inv, sk[v][1] * inv),
                                                            __floats2half2_rn(sk[v][2] * inv, sk[v][3] * inv));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dst[8 * k] = __float2half_rn(rot[v][k] * inv);
          if (KQ) dst[kHeadDim + 8 * k] = __float2half_rn(sk[v][k] * inv);
        }
      }
      if (lane == 0) p.qscale[row] = pow2(e);
    }
  }
}

// ---- fp32 segment kernel ------------------------------------------------------------------------------
//
// 64 rows x 64 tokens a step, 256 threads: thread (ty, tx) holds rows 4 ty .. + 3; of the logits tokens
// 4 tx .. + 3, of the value sum dims 4 tx + 64 c .. + 3. Queries, the dequantised key (then value) page and
// the weights lie k-major in shared memory, so every product step is two 16-byte loads (plus one per 64
// value dims) for 16 (16 per 64 dims) FMAs. fp32 throughout.
constexpr int kF32Rows = 64;

// Bits of token `tok` (of 32) at the coordinates 4 quad .. + 3 of the 8 quads part, part + 4, ..: 4 bits each, the first
// lowest. All of a thread's loads are in flight at once: small calls have a page or two a CTA.
__device__ __forceinline__ uint32_t plane_nibbles(const unsigned char* plane, int order, int tok, int part) {
  uint32_t out = 0;
  if (order == kOrderOctet) {  // quads of one t = part: 8 words on end
    const uint32_t* w = reinterpret_cast<const uint32_t*>(plane) + (tok >> 3) * 32 + 8 * part;
    uint32_t x[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = __ldg(w + n) >> (tok & 7);
#pragma unroll
    for (int n = 0; n < 8; ++n)  // word 2 m + h is quad 8 m + 4 h + t
      out |= ((x[n] & 1u) | ((x[n] >> 7) & 2u) | ((x[n] >> 14) & 4u) | ((x[n] >> 21) & 8u)) << (4 * n);
    return out;
  }
  const int step = order == kOrderToken ? 1 : kTile;
  const unsigned char* b = plane + (order == kOrderToken ? tok * 16 : tok) + (part >> 1) * step;
  uint32_t x[8];
#pragma unroll
  for (int n = 0; n < 8; ++n) x[n] = __ldg(b + 2 * n * step);
#pragma unroll
  for (int n = 0; n < 8; ++n) out |= ((x[n] >> (4 * (part & 1))) & 0xFu) << (4 * n);
  return out;
}

// Page `page` of one side as fp32, k-major dst: keys [dim][token], values [token][dim]. Sketch entries are
// +-gamma; tokens at or behind `tokens` give zeros. scale[token] = norm.
template <bool VALUES, bool QJL>
__device__ __forceinline__ void dequant_f32(const ChunkParams& p, const SideLayout& L, const char* region, const Walk& w,
                                            int page, int tokens, const float* cent, float* dst, float* scale) {
  const int tid = threadIdx.x;
  // neighbouring lanes: tokens of a key row, quads of a value row
  const int tok = VALUES ? tid >> 2 : tid & 63, part = VALUES ? tid & 3 : tid >> 6;
  const long ti = tile_index_read(p.table, p.pages_per_seq, p.n_pages, p.tiles_per_seq, p.Hkv, w.rows.b, w.hk, 2 * page, p.err);
  const unsigned char* tb = reinterpret_cast<const unsigned char*>(region) + (size_t)(ti + (tok >> 5)) * L.tile_bytes;
  const int slot = tok & 31;
  constexpr int DIMS = QJL ? 2 * kHeadDim : kHeadDim;
  const bool in = tok < tokens;
  uint32_t code[kMaxBits] = {}, sign = 0;
#pragma unroll
  for (int pp = 0; pp < kMaxBits; ++pp)
    if (pp < L.bits) code[pp] = plane_nibbles(tb + L.off_planes + pp * (kTile * 16), L.order, slot, part);
  if (QJL) sign = plane_nibbles(tb + L.off_sketch, L.order, slot, part);
  float gamma = QJL ? __half2float(reinterpret_cast<const __half*>(tb + L.off_gamma)[slot]) : 0.f;
  const float norm = __half2float(reinterpret_cast<const __half*>(tb + L.off_norm)[slot]);
  if (!in) gamma = 0.f;
  // a residual norm that is not finite (a coded infinity or NaN) makes NaN of the rows that attend to the
  // token, through its scale, and must not reach the rows whose weight is 0 as 0 * NaN
  const bool bad = VALUES && QJL && !isfinite(gamma);
  if (bad) gamma = 0.f;
  if (part == 0) scale[tok] = bad ? NAN : in ? norm : 0.f;
#pragma unroll
  for (int n = 0; n < DIMS / 16; ++n) {
    const int quad = part + 4 * n, at = 4 * (n & 7);
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = at + i;
      if (n < 8) x[i] = cent[((code[0] >> b) & 1u) | (((code[1] >> b) & 1u) << 1) | (((code[2] >> b) & 1u) << 2)];
      else x[i] = (sign >> b) & 1u ? gamma : -gamma;
      if (!in) x[i] = 0.f;
    }
    if (VALUES) {
      *reinterpret_cast<float4*>(dst + tok * DIMS + 4 * quad) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[(4 * quad + i) * 64 + tok] = x[i];
    }
  }
}

template <bool KQ, bool VQ>
struct F32Smem {
  static constexpr int DK = KQ ? 2 * kHeadDim : kHeadDim, DV = VQ ? 2 * kHeadDim : kHeadDim;
  float q[DK][kF32Rows];
  float kv[(DK > DV ? DK : DV) * 64];
  float w[64][kF32Rows];
  float kn[64], vn[64];
  float cent[2][8];  // codes: lanes look up different ones, which constant memory would serve in turn
};

template <bool KQ, bool VQ>
__global__ void __launch_bounds__(256) chunk_f32(const __grid_constant__ ChunkParams p) {
  using Smem = F32Smem<KQ, VQ>;
  constexpr int DK = Smem::DK, DV = Smem::DV, C = DV / 64;
  extern __shared__ __align__(16) unsigned char smem[];
  Smem& sm = *reinterpret_cast<Smem*>(smem);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const ChunkSet& set = p.set[kWide];
  if (tid < 16) sm.cent[tid >> 3][tid & 7] = (tid < 8 ? p.k : p.v).cent[tid & 7];
  grid_dep_wait();
  Walk w;
  w.init(p, set, blockIdx.x);
  while (w.next(set)) {
    const Rows r = w.rows;
    const size_t qrow0 = (size_t)(r.start + r.first) * p.Hq + w.hk * p.group;
    __syncthreads();
    // rows past the last stay as they were: what they give is not kept
    for (int i0 = tid; i0 < r.count * DK; i0 += 8 * 256) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + e * 256, row = i / DK;
        v[e] = 0.f;
        if (i < r.count * DK)
          v[e] = static_cast<const float*>(p.qprep)[(qrow0 + (size_t)(row / p.group) * p.Hq + row % p.group) * DK + i % DK];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + e * 256;
        if (i < r.count * DK) sm.q[i % DK][i / DK] = v[e];
      }
    }
    float m[4], l[4], o[4][C][4];
    int last[4];  // last position row i attends to
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      const int row = 4 * ty + i;
      last[i] = row < r.count ? min(r.pos0 + row / p.group, r.ctx - 1) : -1;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][c][j] = 0.f;
    }
    for (int k = w.k0; k < w.k1; ++k) {
      const int tokens = min(kPage, r.limit - k * kPage);
      if (tokens <= 0) break;  // a tile with no position at all
      __syncthreads();
      dequant_f32<false, KQ>(p, p.k, p.kreg, w, k, tokens, sm.cent[0], sm.kv, sm.kn);
      __syncthreads();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
      const bool rows_here = 4 * (ty & ~1) < r.count;  // of this warp's 8
#pragma unroll 1
      for (int d0 = 0; rows_here && d0 < DK; d0 += 32) {  // 32 products at a time: the sum's rounding grows with the steps behind one
        float part[4][4] = {};
#pragma unroll 8
        for (int d = d0; d < d0 + 32; ++d) {
          const float4 a = *reinterpret_cast<const float4*>(&sm.q[d][4 * ty]);
          const float4 b = *reinterpret_cast<const float4*>(&sm.kv[d * 64 + 4 * tx]);
          const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[i][j] = fmaf(av[i], bv[j], part[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] += part[i][j];
      }
      float alpha[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = k * kPage + 4 * tx + j;
          s[i][j] = t <= last[i] ? s[i][j] * sm.kn[4 * tx + j] : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn;
        alpha[i] = exp2f(m[i] - ref);
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = exp2f(s[i][j] - ref);
          sum += s[i][j];
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l[i] = fmaf(l[i], alpha[i], sum);
      }
      __syncthreads();  // every read of the key page is done
      dequant_f32<true, VQ>(p, p.v, p.vreg, w, k, tokens, sm.cent[1], sm.kv, sm.vn);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = k * kPage + 4 * tx + j;
        const float n = sm.vn[4 * tx + j];
        float4 wv;  // a masked weight is 0 whatever the token's norm
        wv.x = t <= last[0] ? s[0][j] * n : 0.f;
        wv.y = t <= last[1] ? s[1][j] * n : 0.f;
        wv.z = t <= last[2] ? s[2][j] * n : 0.f;
        wv.w = t <= last[3] ? s[3][j] * n : 0.f;
        *reinterpret_cast<float4*>(&sm.w[4 * tx + j][4 * ty]) = wv;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][c][j] *= alpha[i];
#pragma unroll 4
      for (int t = 0; rows_here && t < kPage; ++t) {
        const float4 a = *reinterpret_cast<const float4*>(&sm.w[t][4 * ty]);
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float4 b = *reinterpret_cast<const float4*>(&sm.kv[t * DV + 64 * c + 4 * tx]);
          const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][c][j] = fmaf(av[i], bv[j], o[i][c][j]);
        }
      }
    }
    float* ml = segment_ml(set, w.item, blockIdx.x, DV);
    float* so = segment_o(set, w.item, blockIdx.x, DV);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * ty + i;
      if (tx == 0) *reinterpret_cast<float2*>(ml + 2 * row) = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < C; ++c)
        *reinterpret_cast<float4*>(so + state_pos(kRowShift, kF32Rows, row, 64 * c + 4 * tx)) = make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]);
    }
  }
}

// ---- merge --------------------------------------------------------------------------------------------
//
// A block merges groups of 32 rows of one item (kv-head, row tile): a warp 4 rows, lane l dims 4 l .. + 3.
constexpr int kMergeThreads = 256, kMergeRows = 32;

template <bool VQ, bool BF16>
__global__ void __launch_bounds__(kMergeThreads, VQ ? 2 : 3) chunk_merge(const __grid_constant__ ChunkParams p) {
  constexpr int DV = VQ ? 2 * kHeadDim : kHeadDim;
  __shared__ __align__(16) float s_z[VQ ? kMergeRows : 1][kPad];   // sketch sums; bf16: their products
  __shared__ __align__(16) __half s_a[VQ && BF16 ? kMergeRows : 1][kPadH];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int shift = 31 - __clz(p.group);
  Frags frags;
  if (VQ && BF16) load_frags(frags, p.S, p.s_exp, warp, lane);
  else if (VQ) warm_l1(p.S);
  grid_dep_wait();
  int groups = 0, first[2];  // groups of both sets, one after the other
  for (int i = 0; i < p.sets; ++i) {
    first[i] = groups;
    groups += (int)p.set[i].head[0] * p.Hkv * (p.set[i].rows / kMergeRows);
  }
  for (int g = blockIdx.x; g < groups; g += gridDim.x) {
    const int in = p.sets > 1 && g >= first[1];
    const ChunkSet& set = p.set[in];
    const int group = g - (in ? first[1] : 0), per = set.rows / kMergeRows, tiles = (int)set.head[0];
    const long long units = set.head[1], T = units * p.Hkv, G = cta_count(set, T);
    const int shift_in = BF16 && !in ? kWideShift : kRowShift;
    const int item = group / per;
    const int hk = item / tiles, tile = item % tiles;
    // rotated, so that a block (a number of blocks that `per` may divide) meets full and empty groups in turn
    const int group0 = (group + item) % per * kMergeRows, row0 = group0 + 4 * warp;
    const int4 r = set.tile_rows[2 * tile];  // request, first token in it, rows, the request's first token
    const long long u0 = set.unit_start[tile], u1 = set.unit_start[tile + 1];
    if (group0 >= r.z) continue;
    const int c0 = cta_of(hk * units + u0, T, G);
    const int c1 = cta_of(hk * units + u1 - 1, T, G);
    // the segments' maxima and sums first, a lane per segment; then their rows, four in flight
    float acc[4][4], accz[4][4], l[4], m[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      m[v] = -INFINITY;
      l[v] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[v][k] = accz[v][k] = 0.f;
    }
    for (int c = c0 + lane; c <= c1; c += 32) {
      const float2* ml = reinterpret_cast<const float2*>(segment_ml(set, item, c, DV)) + row0;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (row0 + v >= r.z) continue;
        const float2 s = ml[v];
        const float top = fmaxf(m[v], s.x);
        // a NaN sum (a logit that is NaN: the maximum passes over it) stays, an empty part adds nothing
        l[v] = top == -INFINITY ? l[v] + s.y : l[v] * exp2f(m[v] - top) + s.y * exp2f(s.x - top);
        m[v] = top;
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float top = m[v];
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      l[v] = top == -INFINITY ? l[v] : l[v] * exp2f(m[v] - top);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) l[v] += __shfl_xor_sync(0xffffffffu, l[v], x);
      m[v] = top;
    }
#pragma unroll(BF16 ? 2 : 4)
    for (int c = c0; c <= c1; ++c) {
      const float2* ml = reinterpret_cast<const float2*>(segment_ml(set, item, c, DV)) + row0;
      const float* so = segment_o(set, item, c, DV) + state_pos(shift_in, set.rows, row0, 4 * lane);
      float o[4][4], z[4][4], f[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        f[v] = -INFINITY;
        if (row0 + v >= r.z) continue;
        f[v] = ml[v].x;
        load4(o[v], so + (v << shift_in), false, 0);
        if (VQ) load4(z[v], so + (v << shift_in) + kHeadDim * set.rows, false, 0);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        f[v] = m[v] == -INFINITY ? 0.f : exp2f(f[v] - m[v]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // a part without weight may hold anything
          if (f[v] != 0.f) {
            acc[v][k] = fmaf(f[v], o[v][k], acc[v][k]);
            if (VQ) accz[v][k] = fmaf(f[v], z[v][k], accz[v][k]);
          }
        }
      }
    }
    float back[4];  // powers of two of the product's rows
    if (VQ) {  // acc += kappa S^T accz
      const float zs = kKappa * (BF16 ? kSketchScale / kCodeScale : 1.f);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
#pragma unroll
        for (int k = 0; k < 4; ++k) accz[v][k] *= zs;
        if (BF16) back[v] = store_row(s_a[4 * warp + v], accz[v], lane);
        else store4(s_z[4 * warp + v], accz[v], lane);
      }
    }
    if (VQ && BF16) {
      __syncthreads();
      fp16_product(frags, s_a, s_z, warp, lane);
      __syncthreads();
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        load4(accz[v], s_z[4 * warp + v], false, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[v][k] = fmaf(accz[v][k], back[v], acc[v][k]);
      }
    } else if (VQ) {
      __syncwarp();
#pragma unroll 1
      for (int j0 = 0; j0 < kHeadDim; j0 += 16) {
        float part[4][4] = {};
#pragma unroll
        for (int j = j0; j < j0 + 16; ++j) {
          const float4 sj = __ldg(reinterpret_cast<const float4*>(p.S + j * kHeadDim) + lane);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float x = s_z[4 * warp + v][j];
            part[v][0] = fmaf(sj.x, x, part[v][0]);
            part[v][1] = fmaf(sj.y, x, part[v][1]);
            part[v][2] = fmaf(sj.z, x, part[v][2]);
            part[v][3] = fmaf(sj.w, x, part[v][3]);
          }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[v][k] += part[v][k];
      }
      __syncwarp();
    }
    float sg[4];
    load4(sg, p.signs + hk * p.signs_stride, false, lane);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      fwht(acc[v], lane);
      const int row = row0 + v;
      if (row >= r.z) continue;
      const float f = l[v] > 0.f ? (BF16 ? kCodeScale : 1.f) / (kHeadDim * l[v]) : l[v];  // 0: nothing attended; or NaN
      const size_t at = ((size_t)(r.w + r.y + (row >> shift)) * p.Hq + hk * p.group + (row & (p.group - 1))) * kHeadDim;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[v][k] *= f * sg[k];
      if (BF16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at + 4 * lane) =
            pack4(__floats2bfloat162_rn(acc[v][0], acc[v][1]), __floats2bfloat162_rn(acc[v][2], acc[v][3]));
      else
        store4(static_cast<float*>(p.out) + at, acc[v], lane);
    }
  }
}

// Blocks take groups of rows in turn, as many blocks as fit at once (2 or 3 an SM by their registers), so that a
// block's fragments of the sketch matrix serve many groups.
template <bool KQ, bool BF16>
cudaError_t launch_prep(const ChunkParams& p, cudaStream_t s) {
  const long long groups = ((long long)p.n_tokens * p.Hq + kPrepRows - 1) / kPrepRows;
  chunk_prep<KQ, BF16><<<p.sets + (unsigned)std::min(groups, 2ll * p.sms), kPrepThreads, 0, s>>>(p);
  return launched();
}
template <bool VQ, bool BF16>
cudaError_t launch_merge(const ChunkParams& p, cudaStream_t s) {
  long long groups = 0;
  for (int i = 0; i < p.sets; ++i) groups += (long long)p.set[i].max_tiles * p.Hkv * (p.set[i].rows / kMergeRows);
  return launch_after(chunk_merge<VQ, BF16>, p, (unsigned)std::min(groups, (VQ ? 2ll : 3ll) * p.sms), kMergeThreads, 0, 1, s);
}

template <bool KQ, bool VQ>
cudaError_t launch_f32(const ChunkParams& p, cudaStream_t s) {
  constexpr int smem = (int)sizeof(F32Smem<KQ, VQ>);
  const cudaError_t e = cudaFuncSetAttribute(chunk_f32<KQ, VQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_after(chunk_f32<KQ, VQ>, p, p.set[kWide].ctas, 256, smem, 1, s);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

ChunkLayout chunk_layout(int n_tokens, int batch, int Hq, int Hkv, bool k_qjl, bool v_qjl, bool bf16, int sms) {
  ChunkLayout L;
  L.sets = bf16 ? 2 : 1;
  const int group = Hq / Hkv;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = up256(off + bytes);
    return at;
  };
  for (int i = 0; i < L.sets; ++i) {
    ChunkLayout::Set& s = L.set[i];
    // up to kNarrowRows rows of a kv-head: the narrow kernel (bf16). A call with 16 requests of 7000 tokens, 2 bits and
    // sketches: narrow 129 / wide 232 us at 4 rows, 134 / 236 at 32, 157 / 242 at 48 and 160 at 64, its widest tile
    s.above = bf16 && i == kWide ? kNarrowRows : 0;
    s.upto = i == kNarrow ? kNarrowRows : 0x7fffffff;
    s.rows = i == kNarrow ? kNarrowRows : bf16 ? chunk_umma_rows(v_qjl) : kF32Rows;
    s.unit = i == kNarrow ? 2 * kPage : kPage;
    s.ctas = bf16 && i == kWide ? std::max(sms / 2, 1) : sms;
    // requests of a set have above / group + 1 tokens at least, a tile each and one per `rows` rows
    s.max_tiles = std::min(batch, n_tokens / (s.above / group + 1));
    if (i == kWide) s.max_tiles += n_tokens / (s.rows / group);
    if (n_tokens * (long long)group <= s.above) s.max_tiles = 0;
    s.head = take(3 * sizeof(long long));
    s.unit_start = take(sizeof(long long) * ((size_t)s.max_tiles + 1));
    s.tile_rows = take(2 * sizeof(int4) * (size_t)s.max_tiles);
    s.tile_start = take(sizeof(int) * ((size_t)batch + 1));
    const size_t segments = s.max_tiles ? (size_t)s.max_tiles * Hkv + s.ctas : 0;
    s.part = take(sizeof(float) * segments * s.rows * (2 + kHeadDim * (v_qjl ? 2 : 1)));
  }
  const size_t rows = (size_t)n_tokens * Hq;
  L.qprep = take(rows * kHeadDim * (k_qjl ? 2 : 1) * (bf16 ? sizeof(__half) : sizeof(float)));
  L.qscale = take(bf16 ? sizeof(float) * rows : 0);
  L.total = off;
  return L;
}

cudaError_t launch_chunk_attention(const ChunkParams& p, cudaStream_t s) {
  cudaError_t e;
  if (p.bf16) e = p.k.qjl ? launch_prep<true, true>(p, s) : launch_prep<false, true>(p, s);
  else e = p.k.qjl ? launch_prep<true, false>(p, s) : launch_prep<false, false>(p, s);
  if (e != cudaSuccess) return e;
  if (p.bf16) {
    e = p.set[kWide].max_tiles ? launch_chunk_umma(p, s) : cudaSuccess;
    if (e == cudaSuccess) e = launch_chunk_narrow(p, s);
  } else if (p.k.qjl) e = p.v.qjl ? launch_f32<true, true>(p, s) : launch_f32<true, false>(p, s);
  else {
    e = p.v.qjl ? launch_f32<false, true>(p, s) : launch_f32<false, false>(p, s);
  }
  if (e != cudaSuccess) return e;
  if (p.bf16) return p.v.qjl ? launch_merge<true, true>(p, s) : launch_merge<false, true>(p, s);
  return p.v.qjl ? launch_merge<true, false>(p, s) : launch_merge<false, false>(p, s);
}

}  // namespace kvq
