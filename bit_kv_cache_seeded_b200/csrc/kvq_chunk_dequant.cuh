// Pieces shared by the tensor-core chunk attention kernels: a packed 64-token page turned into fp16 operand rows
// in shared memory.
//
// Operands lie in shared memory as 128-byte-swizzled K-major rows: row r of an atom of 64 K-elements is 128
// bytes, its 16-byte chunk c at chunk c ^ (r % 8). A dequantising thread makes 8 elements of a row at a time
// and stores them as one chunk; 8 neighbouring threads fill 8 different chunks (no bank conflicts). Keys in
// octet order give a thread coordinates 32 m + 16 h + 4 t + i of 8 tokens; the queries are stored in that
// order (query_pos), since the product does not mind which way its K-elements are numbered.
//
// Entries are n c / 4 (a code times the token's norm) and +-n gamma / 16 (a sign bit): the powers of two keep
// every fp16 norm's entries in range, and the queries and the merge carry their inverses. (Norms under 2^-10 give
// entries among fp16's subnormal numbers, with fewer bits.) A value whose norm is
// not finite enters as zeros (0 p would be NaN in every row); the rows that attend to it get a NaN sum from the
// page's mask instead.
#pragma once

#include <cuda_fp16.h>

#include "kvq_async.cuh"
#include "kvq_chunk.cuh"

namespace kvq {
namespace chunk {

__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The bytes of (lo, hi) that the selector's low four nibbles (each under 8) name: one instruction, where __byte_perm
// masks a selector that it does not know.
__device__ __forceinline__ uint32_t pick(uint32_t lo, uint32_t hi, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(r) : "r"(lo), "r"(hi), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t half_bits(float x) { return (uint32_t)__half_as_ushort(__float2half_rn(x)); }

// The code words (one per plane) of 32 elements, element (byte i, bit s): prepared once, then the fp16 pairs of
// bytes 0, 1 and 2, 3 for s = 0 .. 7 in turn, which shifts the words along. Two bits: the code picks one of 4
// halves. Three: the lower two bits, inverted below zero, pick one of 4 magnitudes. A sign word has bytes 1 and 2
// exchanged, so that bits s of a pair lie 16 apart; a product with 2^(15 - s) (bytes 0, 1) or 2^(7 - s) (2, 3) takes
// them to bits 15 and 31. Products rather than shifts: they leave the ALU pipe, which bounds this, to the rest.
__device__ __forceinline__ uint32_t sign_word(uint32_t w) { return __byte_perm(~w, 0, 0x3120); }
constexpr uint32_t kSigns = 0x80008000u;

template <int BITS>
struct Codes {
  uint32_t even, odd, neg;
  __device__ __forceinline__ void set(uint32_t w0, uint32_t w1, uint32_t w2) {
    if (BITS == 1) neg = sign_word(w0);
    if (BITS >= 2) {
      const uint32_t flip = BITS == 3 ? ~w2 : 0u;
      const uint32_t a = w0 ^ flip, b = w1 ^ flip;
      even = (a & 0x55555555u) | ((b & 0x55555555u) << 1);
      odd = ((a >> 1) & 0x55555555u) | (b & 0xAAAAAAAAu);
      if (BITS == 3) neg = sign_word(w2);
    }
  }
  // the next s, of parity `parity`; lo, hi: the 4 halves (one bit: lo holds the magnitude twice); m01 = 2^(15 - s), m23
  // = 2^(7 - s)
  __device__ __forceinline__ void next(int parity, uint32_t lo, uint32_t hi, uint32_t m01, uint32_t m23, uint32_t& p01,
                                       uint32_t& p23) {
    if (BITS == 1) {
      p01 = p23 = lo;
    } else {
      uint32_t& w = parity ? odd : even;
      const uint32_t sel = (w & 0x03030303u) * 0x22u + 0x10101010u;
      w >>= 2;
      p01 = pick(lo, hi, sel);
      p23 = pick(lo, hi, sel >> 16);
    }
    if (BITS != 2) {
      p01 ^= neg * m01 & kSigns;
      p23 ^= neg * m23 & kSigns;
    }
  }
};

// A side's codes as halves (Codes::next), quarters of them.
__device__ __forceinline__ uint2 code_halves(const SideLayout& L) {
  uint32_t lo, hi;
  if (L.bits == 1) {
    lo = hi = half_bits(L.cent[1] * 0.25f) * 0x10001u;
  } else {
    const int at = L.bits == 3 ? 4 : 0;
    lo = half_bits(L.cent[at] * 0.25f) | half_bits(L.cent[at + 1] * 0.25f) << 16;
    hi = half_bits(L.cent[at + 2] * 0.25f) | half_bits(L.cent[at + 3] * 0.25f) << 16;
  }
  return make_uint2(lo, hi);
}

// A thread's share of one side's page: 8 bytes of every plane, and 8 tokens' norms (keys in token order: one).
struct PageRegs {
  uint2 plane[kMaxBits], sketch;
  uint4 norm, gamma;
};

// Loads that stay where they are written: the compiler would move them down to their first use, a page later, and
// leave their latency in the open.
__device__ __forceinline__ uint2 load8(const unsigned char* at) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "l"(at));
  return v;
}
__device__ __forceinline__ uint4 load16(const unsigned char* at) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at));
  return v;
}

template <bool QJL>
__device__ __forceinline__ void load_page(PageRegs& r, const SideLayout& L, const unsigned char* planes, const unsigned char* norms) {
  r.plane[0] = load8(planes);
  if (L.bits > 1) r.plane[1] = load8(planes + kTile * 16);
  if (L.bits > 2) r.plane[2] = load8(planes + 2 * kTile * 16);
  if (QJL) r.sketch = load8(planes + (L.off_sketch - L.off_planes));
  r.norm = load16(norms);
  if (QJL) r.gamma = load16(norms + (L.off_gamma - L.off_norm));
}

__device__ __forceinline__ uint32_t half_at(const uint4& v, int i) {  // i-th of 8
  const uint32_t w = (i >> 1) == 0 ? v.x : (i >> 1) == 1 ? v.y : (i >> 1) == 2 ? v.z : v.w;
  return i & 1 ? w >> 16 : w & 0xFFFFu;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// For s = 0 .. 7 the 8 elements (4 of each word) scaled by a norm, stored as one chunk at d + s * step + 16 (x ^ s).
// ROWS (keys): s is a token, nn[s / 2] holds its norm in half s % 2. Otherwise (values) pair i of tokens has nn[i].
// The loops stay rolled: unrolled, the roles' code missed the instruction cache (38% of all stalls; a page took
// 4500 cycles to dequantise).
template <bool ROWS>
__device__ __forceinline__ void row_factors(const uint32_t (&n)[4], int e, uint32_t (&m)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = ROWS ? __byte_perm(n[0], 0, e ? 0x3232 : 0x1010) : n[i];
}
template <bool ROWS>
__device__ __forceinline__ void next_rows(uint32_t (&n)[4]) {
  if (ROWS) {
    n[0] = n[1]; n[1] = n[2]; n[2] = n[3];
  }
}

// Codes (BITS > 0), signs times ng (SIGNS; `signs` bytes behind the codes' rows, or at d alone), or both in one loop.
template <int BITS, bool SIGNS, bool ROWS>
__device__ __forceinline__ void expand(const PageRegs& r, uint2 lut, const uint32_t (&nn)[4], const uint32_t (&ng)[4], uint32_t d,
                                       int step, uint32_t x, int signs) {
  Codes<BITS> a, b;
  if (BITS > 0) {
    a.set(r.plane[0].x, r.plane[1].x, r.plane[2].x);
    b.set(r.plane[0].y, r.plane[1].y, r.plane[2].y);
  }
  const uint32_t za = SIGNS ? sign_word(r.sketch.x) : 0u, zb = SIGNS ? sign_word(r.sketch.y) : 0u;
  uint32_t n[4] = {nn[0], nn[1], nn[2], nn[3]}, g[4] = {ng[0], ng[1], ng[2], ng[3]};
  uint32_t top = 0x8000u;
#pragma unroll 1
  for (uint32_t s = 0; s < 128; s += 32, d += 2 * step) {  // 16 times the first of two s
    const uint32_t at = d + ((x << 4) ^ s);                 // rows are 128 bytes: x ^ s only turns bits of the chunk within one
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t to = (at ^ (e << 4)) + e * step, m01 = top >> e, m23 = top >> (8 + e);
      uint32_t m[4];
      if (BITS > 0) {
        uint32_t v[4];
        a.next(e, lut.x, lut.y, m01, m23, v[0], v[1]);
        b.next(e, lut.x, lut.y, m01, m23, v[2], v[3]);
        row_factors<ROWS>(n, e, m);
        sts16(to, mul2(v[0], m[0]), mul2(v[1], m[1]), mul2(v[2], m[2]), mul2(v[3], m[3]));
      }
      if (SIGNS) {
        row_factors<ROWS>(g, e, m);
        sts16(to + signs, m[0] ^ (za * m01 & kSigns), m[1] ^ (za * m23 & kSigns), m[2] ^ (zb * m01 & kSigns),
              m[3] ^ (zb * m23 & kSigns));
      }
    }
    top >>= 2;
    if (BITS > 0) next_rows<ROWS>(n);
    if (SIGNS) next_rows<ROWS>(g);
  }
}
template <bool SIGNS, bool ROWS>
__device__ __forceinline__ void expand_codes(int bits, const PageRegs& r, uint2 lut, const uint32_t (&nn)[4], const uint32_t (&ng)[4],
                                             uint32_t d, int step, uint32_t x, int signs) {
  if (bits == 2) expand<2, SIGNS, ROWS>(r, lut, nn, ng, d, step, x, signs);
  else if (bits == 3) expand<3, SIGNS, ROWS>(r, lut, nn, ng, d, step, x, signs);
  else expand<1, SIGNS, ROWS>(r, lut, nn, ng, d, step, x, signs);
}

// Of a warp whose threads have written operand rows: visible to the products, one arrival.
__device__ __forceinline__ void arrive_rows(uint64_t& bar) {
  fence_proxy_async();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&bar));
}

// One of 128 threads that dequantise the pages of a side's keys: octet order: tokens 8 o .. + 7, coordinates of words
// 2 g, 2 g + 1; token order: token th / 2, half a row.
template <bool KQ>
struct KeyThread {
  const unsigned char *planes, *norms;  // of a page's first tile 0
  uint32_t row_off, x;
  int step, tok;
  bool octet;
  // atom: bytes of an operand's atom of 64 K-elements
  __device__ __forceinline__ void init(const ChunkParams& p, int th, int atom) {
    octet = p.k.order == kOrderOctet;
    const int o = th >> 4, g = th & 15;
    tok = th >> 1;
    const unsigned char* tile = reinterpret_cast<const unsigned char*>(p.kreg) + (octet ? o >> 2 : tok >> 5) * p.k.tile_bytes;
    planes = tile + p.k.off_planes + (octet ? (o & 3) * 128 + g * 8 : (tok & 31) * 16 + (th & 1) * 8);
    norms = tile + p.k.off_norm + 2 * (octet ? 8 * (o & 3) : tok & 24);
    row_off = octet ? (g >> 3) * atom + o * 1024 : (th & 1) * atom + tok * 128;
    step = octet ? 128 : 0;
    x = octet ? g & 7 : tok & 7;
  }
  __device__ __forceinline__ void fetch(const ChunkParams& p, PageRegs& r, long ti) const {
    load_page<KQ>(r, p.k, planes + ti * p.k.tile_bytes, norms + ti * p.k.tile_bytes);
  }
  __device__ __forceinline__ void code_norms(const PageRegs& cur, uint32_t (&nn)[4]) const {
    nn[0] = cur.norm.x; nn[1] = cur.norm.y; nn[2] = cur.norm.z; nn[3] = cur.norm.w;
    if (!octet) nn[0] = nn[1] = nn[2] = nn[3] = half_at(cur.norm, tok & 7) * 0x10001u;  // one token
  }
  __device__ __forceinline__ void sign_norms(const PageRegs& cur, uint32_t (&ng)[4]) const {
    const uint32_t nn[4] = {cur.norm.x, cur.norm.y, cur.norm.z, cur.norm.w};
    const uint32_t gg[4] = {cur.gamma.x, cur.gamma.y, cur.gamma.z, cur.gamma.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) ng[i] = mul2(nn[i], mul2(gg[i], 0x2C002C00u));  // n * (gamma / 16)
    if (!octet) ng[0] = ng[1] = ng[2] = ng[3] = half_at(make_uint4(ng[0], ng[1], ng[2], ng[3]), tok & 7) * 0x10001u;
  }
  // the page's rows from `base` on: its codes, its signs, or both, the signs `signs` bytes behind
  __device__ __forceinline__ void codes(const ChunkParams& p, const PageRegs& cur, uint2 lut, uint32_t base) const {
    uint32_t nn[4];
    code_norms(cur, nn);
    expand_codes<false, true>(p.k.bits, cur, lut, nn, nn, base + row_off, step, x, 0);
  }
  __device__ __forceinline__ void signs(const PageRegs& cur, uint32_t base) const {
    uint32_t ng[4];
    sign_norms(cur, ng);
    expand<0, true, true>(cur, make_uint2(0, 0), ng, ng, base + row_off, step, x, 0);
  }
  __device__ __forceinline__ void both(const ChunkParams& p, const PageRegs& cur, uint2 lut, uint32_t base, int signs) const {
    uint32_t nn[4], ng[4] = {};
    code_norms(cur, nn);
    if (KQ) sign_norms(cur, ng);
    expand_codes<KQ, true>(p.k.bits, cur, lut, nn, ng, base + row_off, step, x, signs);
  }
};

// One of the threads that dequantise values: rows are dims, dims 8 k .. + 7 in rows 8 row8 .. + 7, of tokens 8 c .. + 7.
template <bool VQ>
struct ValueThread {
  const unsigned char *planes, *norms;  // of a page's first tile 0
  int c, row8;
  __device__ __forceinline__ void init(const ChunkParams& p, int chunk, int k, int rows8) {
    c = chunk;
    row8 = rows8;
    const unsigned char* tile = reinterpret_cast<const unsigned char*>(p.vreg) + (c >> 2) * p.v.tile_bytes;
    planes = tile + p.v.off_planes + k * kTile + 8 * (c & 3);
    norms = tile + p.v.off_norm + 2 * 8 * (c & 3);
  }
  __device__ __forceinline__ void fetch(const ChunkParams& p, PageRegs& r, long ti) const {
    load_page<VQ>(r, p.v, planes + ti * p.v.tile_bytes, norms + ti * p.v.tile_bytes);
  }
  // the page's dims from `base` on (the signs' `signs` bytes behind the codes'); tokens from `limit` on enter as zeros.
  // Returns this thread's 8 tokens whose norms are not finite, a bit each (zeros too).
  __device__ __forceinline__ uint32_t store(const ChunkParams& p, const PageRegs& cur, uint2 lut, uint32_t base, int signs, int limit) const {
    const int tokens = limit - 8 * c;
    uint32_t nn[4] = {cur.norm.x, cur.norm.y, cur.norm.z, cur.norm.w}, ng[4] = {}, bad = 0;
    if (VQ) {
      ng[0] = cur.gamma.x; ng[1] = cur.gamma.y; ng[2] = cur.gamma.z; ng[3] = cur.gamma.w;
    }
    uint32_t odd = 0;  // an exponent of all ones carries into the sign's place
#pragma unroll
    for (int i = 0; i < 4; ++i) odd |= ((nn[i] & 0x7C007C00u) + 0x04000400u) | ((ng[i] & 0x7C007C00u) + 0x04000400u);
    if ((odd & kSigns) != 0 || tokens < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t half = i & 1 ? 0xFFFF0000u : 0xFFFFu;
        const bool in = i < tokens;
        const bool finite = (((nn[i >> 1] & 0x7C007C00u) + 0x04000400u) | ((ng[i >> 1] & 0x7C007C00u) + 0x04000400u)) & kSigns & half ? false : true;
        if (in && !finite) bad |= 1u << i;
        if (!in || !finite) {
          nn[i >> 1] &= ~half;
          ng[i >> 1] &= ~half;
        }
      }
    }
    if (VQ) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ng[i] = mul2(nn[i], mul2(ng[i], 0x2C002C00u));  // n * (gamma / 16)
    }
    expand_codes<VQ, false>(p.v.bits, cur, lut, nn, ng, base + row8 * 1024, 128, c, signs);
    return bad;
  }
};

// A page's block-table entry (loaded a page before it is looked at: looking waits for the load), and its
// first tile, page 0's for an entry that names none (kvq_tiles.cuh).
__device__ __forceinline__ int page_entry(const ChunkParams& p, const Walk& w, int page) {
  int entry = 0;
  if (p.table && page < p.pages_per_seq)
    asm volatile("ld.global.cg.s32 %0, [%1];\n" : "=r"(entry) : "l"(p.table + (long)w.rows.b * p.pages_per_seq + page));
  return entry;
}
__device__ __forceinline__ long page_tile(const ChunkParams& p, const Walk& w, int page, int entry) {
  if (!p.table) return ((long)w.rows.b * p.Hkv + w.hk) * p.tiles_per_seq + 2 * page;
  if (entry < 0 || entry >= p.n_pages) {
    atomicOr(p.err, kStatusBadPage);
    entry = 0;
  }
  return ((long)entry * p.Hkv + w.hk) * 2;
}

}  // namespace chunk
}  // namespace kvq
