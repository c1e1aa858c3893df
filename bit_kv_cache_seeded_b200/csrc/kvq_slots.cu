// The ragged serving path's bookkeeping and append: block tables and slot maps from request lengths,
// and an append of a token-major batch into page slots ("TurboQuant vs OSCAR vs EpiCache", OSCAR:
// fused kernels compatible with paged attention and the prefix cache).
//
// extend_block_table. Request b holds held_b tokens and takes new_b more. Its pages grow from
// ceil(held_b / 64) to ceil((held_b + new_b) / 64); the new ones come from the free list in request
// order, at the exclusive prefix sum of the counts. Bound by launch latency: the largest calls move a
// few hundred KB. So one kernel and no exchange between blocks: every block sums the counts of all
// requests before its own (a coalesced round per 256), then writes its own requests' entries.
//
// slot_map. Token t of the ragged batch belongs to the request b with seq_start[b] <= t <
// seq_start[b + 1] (binary search), has position held_b + t - seq_start[b], and goes to slot
// 64 * table[b][position / 64] + position % 64. One thread per token; bound by the 16 bytes it writes.
//
// quantize_slots. The codec's steps 1-7 (kvq_quantize.cu) on vectors [token][kv-head][128], written to
// slots[token]. A block codes TOK tokens of one (kv-head, side) at a time: warps code a token each; the sketch of
// all TOK residuals is one product with S^T on the tensor cores (mma.sync); and the bits go out per run of slots in
// one octet, a run and plane per warp: a whole octet of a key plane is stored, a part of one is merged with
// atomics, since other tokens of the octet may belong to another block.
//
// The product decides signs, so it has to be as good as fp32: residuals and S are each two fp16 numbers, the
// second 2^11 times what the first leaves (22 bits together), and the three products that matter are summed in
// fp32, the small ones apart. On the CUDA cores it took half of the instructions, and the packing on one warp a
// plane a quarter (2200 tokens of 8 heads, 3 bits, a sketch on the keys: 52.3 us; 35 now, bound by
// issue). Small calls take TOK = 8, which spreads them over four times as many blocks as TOK = 32 (launch).
#include <algorithm>

#include <cuda_fp16.h>

#include "kvq_async.cuh"
#include "kvq_quantize_lm.cuh"
#include "kvq_ragged.h"
#include "kvq_tiles.cuh"

namespace kvq {
namespace {

constexpr int kPage = kTile * kTilePair;
constexpr int kTableThreads = 256;

// Inclusive sum over the block of one value per thread (kTableThreads threads), and the block's total.
__device__ __forceinline__ long long block_scan(long long v, long long* total) {
  __shared__ long long s_warp[kTableThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // the previous round's reads of s_warp are done
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kTableThreads / 32; ++w) {
    const long long u = s_warp[w];
    before += w < warp ? u : 0;
    all += u;
  }
  *total = all;
  return v + before;
}

// Pages a request holds and needs; valid: its lengths fit the table.
struct Request {
  int held, n_new, p0, need;
  bool valid;
};
__device__ __forceinline__ Request request(const int* held, const int* n_new, int b, int pages_per_seq) {
  Request r;
  r.held = held[b];
  r.n_new = n_new[b];
  r.valid = r.held >= 0 && r.n_new >= 0 && (long long)r.held + r.n_new <= (long long)pages_per_seq * kPage;
  r.p0 = r.valid ? (int)(((long long)r.held + kPage - 1) / kPage) : 0;
  r.need = r.valid ? (int)(((long long)r.held + r.n_new + kPage - 1) / kPage) - r.p0 : 0;
  return r;
}

// Grid: one block per kOwn requests, a warp each: one block for 256 requests wrote its 23000 entries in 17.7 us, 32
// blocks in 5.
constexpr int kOwn = kTableThreads / 32;

__global__ void __launch_bounds__(kTableThreads)
extend_block_table(const int* __restrict__ held, const int* __restrict__ n_new, int batch, const int* __restrict__ free_pages,
                   int n_free, const int* __restrict__ cursor, int* __restrict__ table, int pages_per_seq,
                   int* __restrict__ seq_start, int* __restrict__ ctx_lens, int* __restrict__ taken) {
  __shared__ int s_first[kOwn], s_need[kOwn], s_p0[kOwn];
  __shared__ int s_sum[2];
  const int tid = threadIdx.x;
  const int begin = blockIdx.x * kOwn;
  const int first = cursor ? *cursor : 0;
  const long long room = first >= 0 && first <= n_free ? n_free - first : -1;  // -1: no page can be given
  long long pages = 0, tokens = 0;  // of the requests before this block's
  for (int b = tid; b < begin; b += kTableThreads) {
    const Request r = request(held, n_new, b, pages_per_seq);
    pages += r.need;
    tokens += max(r.n_new, 0);
  }
  const int b = begin + tid;
  const bool own = tid < kOwn && b < batch;
  Request r{0, 0, 0, 0, true};
  if (own) r = request(held, n_new, b, pages_per_seq);
  long long all_pages, all_tokens, own_pages, own_tokens;
  block_scan(pages, &all_pages);
  block_scan(tokens, &all_tokens);
  const long long end = all_pages + block_scan(r.need, &own_pages);
  const long long tend = all_tokens + block_scan(max(r.n_new, 0), &own_tokens);
  const bool granted = r.valid && (r.need == 0 || end <= room);
  if (tid < 2) s_sum[tid] = 0;
  if (tid < kOwn) {
    s_first[tid] = (int)min(end - r.need, 0x7fffffffll);
    s_need[tid] = granted ? r.need : 0;
    s_p0[tid] = r.p0;
  }
  __syncthreads();
  if (own) {
    if (b == 0) seq_start[0] = 0;
    seq_start[b + 1] = (int)min(tend, 0x7fffffffll);
    ctx_lens[b] = granted ? r.held + r.n_new : (int)min(max((long long)r.held, 0ll), (long long)pages_per_seq * kPage);
  }
  const int i = tid >> 5, n = s_need[i];  // entries: one warp per request
  if (n > 0) {
    int* row = table + (long long)(begin + i) * pages_per_seq + s_p0[i];
    const int* from = free_pages + first + s_first[i];
#pragma unroll 8
    for (int k = tid & 31; k < n; k += 32) row[k] = from[k];
  }
  // totals: the last block sees every request once more
  if (blockIdx.x == gridDim.x - 1) {
    long long run = 0;
    int got = 0, refused = 0;
    for (int b0 = 0; b0 < batch; b0 += kTableThreads) {
      Request q{0, 0, 0, 0, true};
      if (b0 + tid < batch) q = request(held, n_new, b0 + tid, pages_per_seq);
      long long part;
      const long long e = run + block_scan(q.need, &part);
      run += part;
      const bool ok = q.valid && (q.need == 0 || e <= room);
      got += ok ? q.need : 0;
      refused += ok ? 0 : 1;
    }
    atomicAdd(&s_sum[0], got);
    atomicAdd(&s_sum[1], refused);
    __syncthreads();
    if (tid < 2) taken[tid] = s_sum[tid];
  }
}

constexpr int kSlotThreads = 256;

__global__ void __launch_bounds__(kSlotThreads)
slot_map(const int* __restrict__ held, const int* __restrict__ seq_start, const int* __restrict__ ctx_lens, int batch,
         const int* __restrict__ table, int pages_per_seq, int n_pages, int n_tokens, int* __restrict__ seq_ids,
         int* __restrict__ positions, long long* __restrict__ slots) {
  const unsigned at = blockIdx.x * kSlotThreads + threadIdx.x;
  if (at >= (unsigned)n_tokens) return;
  const int t = (int)at;
  if (t < seq_start[0] || t >= seq_start[batch]) return;  // rows of no request stay as they are
  int lo = 0, hi = batch;  // the last b with seq_start[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int start = seq_start[lo], n = seq_start[lo + 1] - start;
  const long long pos = (long long)held[lo] + (t - start);
  long long slot = -1;
  if (pos >= 0 && pos < (long long)pages_per_seq * kPage && (long long)held[lo] + n == ctx_lens[lo]) {
    const int page = table[(long long)lo * pages_per_seq + pos / kPage];
    if (page >= 0 && page < n_pages) slot = (long long)page * kPage + pos % kPage;
  }
  if (seq_ids) seq_ids[t] = lo;
  if (positions) positions[t] = (int)pos;
  slots[t] = slot;
}

__global__ void set_lengths(const __grid_constant__ LengthParams p) {
  const int i = threadIdx.x;
  if (i < p.n) p.lens[p.first + i] = p.value[i];
}

// ---- append by slots --------------------------------------------------------------------------------

constexpr int kAppWarps = 8;
constexpr int kAppThreads = kAppWarps * 32;
constexpr int kPadH = kHeadDim + 8;  // row stride of a half row: the 8 rows that ldmatrix reads lie in distinct banks
constexpr float kSecond = 2048.f;

template <int TOK, bool QJL>
struct AppSmem {
  static constexpr int kRows = TOK < 16 ? 16 : TOK;  // a matrix tile has 16; those past TOK are not looked at
  __half rho[2][QJL ? kRows : 1][kPadH];
  uint32_t planes[TOK][kMaxBits + 1][4];  // code planes, then the sign words
  float n[TOK], gamma[TOK];
  long long slot[TOK];  // -1: not written
};

// x = first + second / 2^11, as halves.
__device__ __forceinline__ __half first_half(float x) { return __float2half_rn(x); }
__device__ __forceinline__ __half second_half(float x) { return __float2half_rn((x - __half2float(__float2half_rn(x))) * kSecond); }
__device__ __forceinline__ uint32_t half_pair(__half a, __half b) {
  const __half2 h = __halves2half2(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Blocks an SM holds: a sketch's fragments of S take 64 registers a thread.
template <bool QJL>
constexpr int kAppBlocks = QJL ? 2 : 4;

// QJL: the side has a sketch, or may have one. other: the call's other side is launched behind this one, to begin as soon
// as it finds room.
template <int TOK, bool QJL>
__global__ void __launch_bounds__(kAppThreads, kAppBlocks<QJL>)
quantize_slots(const __grid_constant__ SlotQuantizeParams p, int first_side, bool other) {
  __shared__ __align__(16) AppSmem<TOK, QJL> sm;
  if (other) grid_dep_launch();
  const int side = first_side + blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const SideLayout& L = p.side[side];
  const int nthr = (1 << L.bits) - 1;
  const int chunks = (p.n_tokens + TOK - 1) / TOK;
  const long long total = (long long)chunks * p.heads;
  const int row0 = p.seq_start ? p.seq_start[0] : 0, row1 = p.seq_start ? p.seq_start[p.batch] : p.n_tokens;
  // this warp's rows 16 warp .. + 15 of S (columns of S^T), divided by 2^s_exp
  uint32_t frag[2][2][8][2];
  const bool qjl = QJL && L.qjl;
  if (qjl) {
    const float mul = exp2f((float)-p.s_exp);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* at = p.St + (16 * k + 2 * (lane & 3) + 8 * h) * kHeadDim + 16 * warp + 8 * n + (lane >> 2);
          const float a = __ldg(at) * mul, b = __ldg(at + kHeadDim) * mul;
          frag[0][n][k][h] = half_pair(first_half(a), first_half(b));
          frag[1][n][k][h] = half_pair(second_half(a), second_half(b));
        }
  }
  float thr[7];
#pragma unroll
  for (int i = 0; i < 7; ++i) thr[i] = i < nthr ? L.thr[i] : INFINITY;
  const float cent_lane = L.cent[(lane & 7) <= nthr ? (lane & 7) : 0];

  for (long long g = blockIdx.x; g < total; g += gridDim.x) {
    const int h = (int)(g % p.heads), first = (int)(g / p.heads) * TOK;
    const int count = min(TOK, p.n_tokens - first);
    float sgn[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) sgn[q] = p.signs[h * p.signs_stride + 32 * q + lane];
    for (int i = warp; i < TOK; i += kAppWarps) {
      // rows of no request are skipped without a look: their slots may be an earlier step's
      long long slot = i < count && first + i >= row0 && first + i < row1 ? p.slots[first + i] : -1;
      if (slot >= (long long)p.n_pages * kPage) {
        if (lane == 0) atomicOr(p.err, kStatusBadPage);
        slot = -1;
      }
      if (lane == 0) sm.slot[i] = slot < 0 ? -1 : slot;
      float rho[4] = {0.f, 0.f, 0.f, 0.f};
      if (slot >= 0) {
        const size_t base = ((size_t)(first + i) * p.heads + h) * kHeadDim;
        float u[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) u[q] = qlm::load_elem(p.src[side], base + 32 * q + lane, p.bf16);
        const float n = sqrtf(qlm::warp_sum(u[0] * u[0] + u[1] * u[1] + u[2] * u[2] + u[3] * u[3]));
#pragma unroll
        for (int q = 0; q < 4; ++q) u[q] *= sgn[q];
#pragma unroll
        for (int b = 0; b < 5; ++b) {  // Walsh-Hadamard butterflies over index bits 0..4
          const bool upper = (lane >> b) & 1;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float other = __shfl_xor_sync(0xffffffffu, u[q], 1 << b);
            u[q] = upper ? other - u[q] : u[q] + other;
          }
        }
        const float a0 = u[0] + u[1], a1 = u[0] - u[1], a2 = u[2] + u[3], a3 = u[2] - u[3];
        u[0] = a0 + a2; u[2] = a0 - a2; u[1] = a1 + a3; u[3] = a1 - a3;
#pragma unroll
        for (int q = 0; q < 4; ++q) u[q] = (n > 0.f) ? u[q] / n : 0.f;
        // the number of thresholds (ascending, infinite where the side has fewer) not above u, bit by bit: what a bit
        // decides is a plane's vote (counted one by one, and the votes taken from the count, 38.8 us in place of 36.3)
        uint32_t plane[kMaxBits];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bool b2 = u[q] >= thr[3];
          const bool b1 = u[q] >= (b2 ? thr[5] : thr[1]);
          const bool b0 = u[q] >= (b2 ? (b1 ? thr[6] : thr[4]) : (b1 ? thr[2] : thr[0]));
          const uint32_t w[kMaxBits] = {__ballot_sync(0xffffffffu, b0), __ballot_sync(0xffffffffu, b1), __ballot_sync(0xffffffffu, b2)};
#pragma unroll
          for (int pp = 0; pp < kMaxBits; ++pp) plane[pp] = q == 0 || lane == q ? w[pp] : plane[pp];
          rho[q] = u[q] - __shfl_sync(0xffffffffu, cent_lane, (b2 ? 4 : 0) + (b1 ? 2 : 0) + (b0 ? 1 : 0));
        }
        if (lane < 4)
#pragma unroll
          for (int pp = 0; pp < kMaxBits; ++pp) sm.planes[i][pp][lane] = plane[pp];
        if (lane == 0) sm.n[i] = n;
        if (qjl) {
          const float gam = sqrtf(qlm::warp_sum(rho[0] * rho[0] + rho[1] * rho[1] + rho[2] * rho[2] + rho[3] * rho[3]));
          if (lane == 0) sm.gamma[i] = gam;
        }
      }
      if (qjl)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sm.rho[0][i][32 * q + lane] = first_half(rho[q]);
          sm.rho[1][i][32 * q + lane] = second_half(rho[q]);
        }
    }
    __syncthreads();

    if (qjl) {
#pragma unroll 1
      for (int m = 0; m < AppSmem<TOK, QJL>::kRows / 16; ++m) {
        float big[2][4] = {}, small[2][4] = {};
        const uint32_t a0 = (uint32_t)__cvta_generic_to_shared(&sm.rho[0][16 * m + (lane & 15)][8 * (lane >> 4)]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                         : "=r"(a[h][0]), "=r"(a[h][1]), "=r"(a[h][2]), "=r"(a[h][3])
                         : "r"(a0 + h * (uint32_t)sizeof(sm.rho[0]) + 32 * k) : "memory");
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            mma16(big[n], a[0], frag[0][n][k]);
            mma16(small[n], a[0], frag[1][n][k]);
            mma16(small[n], a[1], frag[0][n][k]);
          }
        }
        // rows lane / 4 (+ 8), columns 8 n + 2 (lane % 4) + {0, 1} of this warp's 16: half a sign word a row
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t bits = 0;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (fmaf(small[n][2 * h + e], 1.f / kSecond, big[n][2 * h + e]) >= 0.f) bits |= 1u << (8 * n + 2 * (lane & 3) + e);
          bits |= __shfl_xor_sync(0xffffffffu, bits, 1);
          bits |= __shfl_xor_sync(0xffffffffu, bits, 2);
          const int tok = 16 * m + 8 * h + (lane >> 2);
          if ((lane & 3) == 0 && tok < TOK) reinterpret_cast<unsigned short*>(sm.planes[tok][kMaxBits])[warp] = (unsigned short)bits;
        }
      }
      __syncthreads();
    }

    const int nplanes = L.bits + (qjl ? 1 : 0);
    auto tile_base = [&](long long slot) {
      return p.region[side] + (size_t)((slot / kPage * p.heads + h) * 2 + (slot % kPage) / kTile) * L.tile_bytes;
    };
    if (L.order == kOrderOctet) {
      // lane = word 8t + 2m + hh of an octet: byte i is coordinate 32m + 16hh + 4t + i, bit j token j.
      // Tokens of one octet that follow one another in the batch (a run) leave together.
      const int wt = lane >> 3, wm = (lane >> 1) & 3, wh = lane & 1;
      const long long mine = lane < TOK && sm.slot[lane] >= 0 ? sm.slot[lane] >> 3 : -1;
      const long long before = __shfl_up_sync(0xffffffffu, mine, 1);
      const uint32_t starts = __ballot_sync(0xffffffffu, lane < TOK && (lane == 0 || mine != before));
      const int runs = __popc(starts);
      for (int u = warp; u < nplanes * runs; u += kAppWarps) {
        const int pp = u / runs, src = pp < L.bits ? pp : kMaxBits;
        uint32_t left = starts;
        for (int r = u % runs; r > 0; --r) left &= left - 1;
        const int from = __ffs(left) - 1;
        left &= left - 1;
        const int to = left ? __ffs(left) - 1 : TOK;
        const long long slot0 = sm.slot[from];
        if (slot0 < 0) continue;
        uint32_t word = 0, mask = 0;
        for (int i = from; i < to; ++i) {
          const int j = (int)(sm.slot[i] & 7);
          const uint32_t nib = (sm.planes[i][src][wm] >> (16 * wh + 4 * wt)) & 0xFu;
          word = (word & ~(0x01010101u << j)) | (qlm::spread_nibble(nib) << j);
          mask |= 0x01010101u << j;
        }
        const int off = pp < L.bits ? L.off_planes + pp * (kTile * 16) : L.off_sketch;
        uint32_t* dst = reinterpret_cast<uint32_t*>(tile_base(slot0 & ~7ll) + off) + ((slot0 >> 3) & 3) * 32 + lane;
        if (mask == 0xffffffffu) {
          *dst = word;
        } else {
          atomicAnd(dst, ~(mask & ~word));
          atomicOr(dst, word);
        }
      }
    } else {
      constexpr int kShares = TOK / 8;  // of a plane: 8 tokens, byte k of the row, two tokens a step
      for (int u = warp; u < nplanes * kShares; u += kAppWarps) {
        const int pp = u / kShares, src = pp < L.bits ? pp : kMaxBits, k = lane & 15;
        const int off = pp < L.bits ? L.off_planes + pp * (kTile * 16) : L.off_sketch;
        for (int i = 8 * (u % kShares) + lane / 16; i < 8 * (u % kShares) + 8; i += 2) {
          const long long slot = sm.slot[i];
          if (slot < 0) continue;
          const char byte = (char)((sm.planes[i][src][k >> 2] >> (8 * (k & 3))) & 0xFFu);
          char* tb = tile_base(slot) + off;
          const int t = (int)(slot % kTile);
          if (L.order == kOrderToken) tb[t * 16 + k] = byte;
          else tb[k * kTile + t] = byte;
        }
      }
    }
    for (int i = tid; i < 2 * TOK; i += kAppThreads) {
      const int tok = i % TOK;
      const long long slot = sm.slot[tok];
      if (slot < 0) continue;
      char* tb = tile_base(slot) + (slot % kTile) * 2;
      if (i < TOK) *reinterpret_cast<__half*>(tb + L.off_norm) = __float2half_rn(sm.n[tok]);
      else if (qjl) *reinterpret_cast<__half*>(tb + L.off_gamma) = __float2half_rn(sm.gamma[tok]);
    }
    __syncthreads();  // the next tokens reuse the shared buffers
  }
  grid_dep_wait();  // the call's other launch is done when this one is
}

// `sides` sides from `first` on; other: the other side follows; after: it came before.
template <int TOK, bool QJL>
cudaError_t launch_slots(const SlotQuantizeParams& p, int first, int sides, bool other, bool after, cudaStream_t s) {
  const long long blocks = (long long)((p.n_tokens + TOK - 1) / TOK) * p.heads;
  cudaLaunchConfig_t config = {};
  // as many blocks as fit, of a side: they keep their fragments of S from one group to the next
  config.gridDim = dim3((unsigned)std::min<long long>(blocks, p.sms * kAppBlocks<QJL>), sides);
  config.blockDim = dim3(kAppThreads);
  config.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &attr;
  config.numAttrs = after ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&config, quantize_slots<TOK, QJL>, p, first, other);
  const cudaError_t counted = launched();
  return e != cudaSuccess ? e : counted;
}

}  // namespace

cudaError_t launch_extend_block_table(const int* held, const int* n_new, int batch, const int* free_pages, int n_free,
                                      const int* cursor, int* table, int pages_per_seq, int* seq_start, int* ctx_lens,
                                      int* taken, cudaStream_t s) {
  extend_block_table<<<(batch + kOwn - 1) / kOwn, kTableThreads, 0, s>>>(
      held, n_new, batch, free_pages, n_free, cursor, table, pages_per_seq, seq_start, ctx_lens, taken);
  return launched();
}

cudaError_t launch_slot_map(const int* held, const int* seq_start, const int* ctx_lens, int batch, const int* table,
                            int pages_per_seq, int n_pages, int n_tokens, int* seq_ids, int* positions, long long* slots,
                            cudaStream_t s) {
  slot_map<<<(unsigned)((n_tokens + (long long)kSlotThreads - 1) / kSlotThreads), kSlotThreads, 0, s>>>(
      held, seq_start, ctx_lens, batch, table, pages_per_seq, n_pages, n_tokens, seq_ids, positions, slots);
  return launched();
}

cudaError_t launch_set_lengths(const LengthParams& p, cudaStream_t s) {
  set_lengths<<<1, kMaxSeqPerLaunch, 0, s>>>(p);
  return launched();
}

cudaError_t launch_quantize_slots(const SlotQuantizeParams& p, cudaStream_t s) {
  // 2-bit codes and sketches, TOK 8 against 32: 8.2 / 12.7 us at 16 groups, 16.7 / 16.2 at 80, 23.6 / 20.8 at 152, 65.9 /
  // 48.0 at 592. One bit without sketches, the kernel that may have one against the other: 10.6 / 10.5 us at 152 groups,
  // 15.8 / 12.6 at 296, 27.0 / 20.5 at 592; 3 bits and a sketch on one side, both sides at once against a launch each: 22.9 /
  // 24.5 at 296, 39.3 / 35.7 at 592. On 148 SMs: a group an SM, and 2.7 of them
  const long long groups = (long long)((p.n_tokens + 31) / 32) * p.heads;
  const bool k = p.side[0].qjl, v = p.side[1].qjl;
  if (groups < p.sms) return launch_slots<8, true>(p, 0, 2, false, false, s);
  if (!k && !v) return launch_slots<32, false>(p, 0, 2, false, false, s);
  if (k == v || 10 * groups < 27ll * p.sms) return launch_slots<32, true>(p, 0, 2, false, false, s);
  const cudaError_t e = launch_slots<32, true>(p, k ? 0 : 1, 1, true, false, s);
  return e != cudaSuccess ? e : launch_slots<32, false>(p, k ? 1 : 0, 1, false, true, s);
}

}  // namespace kvq
