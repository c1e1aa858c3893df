// Pieces shared by the chunk attention kernels: the work plan over ragged requests and the states its
// segments leave behind.
//
// Rows. A kv-head of request b has n_b * group query rows, row r = token r / group, head r % group. A set (ChunkSet)
// takes the requests whose rows are within its bounds. Row tiles of `rows` rows never cross a request; the tiles of
// request b are tile_start[b] .. tile_start[b + 1] - 1, and tile_rows[t] describes tile t, so that a segment starts one
// load after it knows its tile. Below, "CTA" is a pair of them in the wide set.
//
// Units. Tile t attends to the positions below its limit, the last row's position + 1, in units of one or two
// 64-token pages; unit_start[t] is the prefix sum of max(1, ceil(limit / unit)). The units of all kv-heads
// lie end to end (kv-head h's from h * head[1]), and CTA c of G = min(CTAs, T) takes the units floor(c T / G)
// .. floor((c + 1) T / G) - 1 of the T: an even split whatever the lengths, without a host that knows them.
// A CTA's run of units in one tile is a segment; segment number = item + CTA (item = h * tiles + t) is
// distinct, since every step from one segment to the next raises the item or the CTA. A segment writes its
// softmax state, (m, l) [rows][2] and o [rows][value dims]; one kernel then merges the segments of every row,
// folds the value sketch and rotates back.
#pragma once

#include "kvq_ragged.h"
#include "kvq_tiles.cuh"

namespace kvq {
namespace chunk {

constexpr int kPage = kTile * kTilePair;

struct Rows {        // one row tile
  int b;             // request
  int first;         // its first row's token within the request
  int count;         // rows in use
  int start;         // request's first token in the ragged batch
  int pos0;          // position of the tile's first token (may be negative)
  int ctx;           // tokens the request's cache holds
  int limit;         // positions below this are attended by some row
};

__device__ __forceinline__ int clamp_start(const ChunkParams& p, int b) { return min(max(p.seq_start[b], 0), p.n_tokens); }

__device__ __forceinline__ Rows tile_rows(const ChunkParams& p, const ChunkSet& s, int b, int tile) {
  Rows r;
  r.b = b;
  r.start = clamp_start(p, b);
  const int n = max(clamp_start(p, b + 1) - r.start, 0);
  const int per = s.rows / p.group;  // tokens of a row tile
  r.first = tile * per;
  const int tokens = min(per, n - r.first);
  r.count = tokens * p.group;
  const int ctx = p.ctx_lens[b];
  // a refused request's new tokens are not in the cache: no positions, so its rows get zeros
  r.ctx = p.held && (long long)p.held[b] + n != ctx ? 0 : min(max(ctx, 0), p.capacity);
  r.pos0 = r.ctx - n + r.first;
  r.limit = max(0, r.pos0 + tokens);
  return r;
}

__device__ __forceinline__ void store_rows(const ChunkSet& s, int tile, const Rows& r) {
  s.tile_rows[2 * tile] = make_int4(r.b, r.first, r.count, r.start);
  s.tile_rows[2 * tile + 1] = make_int4(r.pos0, r.ctx, r.limit, 0);
}
__device__ __forceinline__ Rows load_rows(const ChunkSet& s, int tile) {
  const int4 x = s.tile_rows[2 * tile], y = s.tile_rows[2 * tile + 1];
  return Rows{x.x, x.y, x.z, x.w, y.x, y.y, y.z};
}

// CTAs that share T units (each has one at least), and the CTA that owns unit u: the largest c with
// floor(c T / G) <= u.
__device__ __forceinline__ long long cta_count(const ChunkSet& s, long long T) { return min((long long)s.ctas, T); }
__device__ __forceinline__ long long cta_first(long long c, long long T, long long G) { return c * T / G; }
__device__ __forceinline__ int cta_of(long long u, long long T, long long G) {
  const long long x = (u + 1) * G;  // the largest c with c T < x: c is small, so fp32 is within one of it
  int c = (int)__fdividef((float)x, (float)T);
  if (c * T >= x) --c;
  if ((c + 1) * T < x) ++c;
  return c;
}

// Walks the segments of one CTA. Every thread (or one per warp) keeps its own copy.
struct Walk {
  long long u, end, units;  // next unit, end of the CTA's range, units of a kv-head
  int tiles, tile, hk;
  // current segment
  long long item;
  int k0, k1;      // its units within the tile: k0 .. k1 - 1
  Rows rows;

  __device__ __forceinline__ void init(const ChunkParams& p, const ChunkSet& s, int cta) {
    tiles = (int)s.head[0];
    units = s.head[1];
    const long long T = units * p.Hkv;
    const long long G = cta_count(s, T);
    u = cta < G ? cta_first(cta, T, G) : 0;
    end = cta < G ? cta_first(cta + 1, T, G) : 0;
    hk = units > 0 ? (int)(u / units) : 0;
    const long long r = u - hk * units;
    int lo = 0, hi = tiles;  // the last tile with unit_start <= r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.unit_start[mid] <= r) lo = mid;
      else hi = mid;
    }
    tile = lo;
  }
  __device__ __forceinline__ bool next(const ChunkSet& s) {
    if (u >= end) return false;
    if (tile == tiles) {
      tile = 0;
      ++hk;
    }
    const long long base = hk * units;
    const long long t0 = base + s.unit_start[tile], t1 = base + s.unit_start[tile + 1];
    const long long stop = min(t1, end);
    k0 = (int)(u - t0);
    k1 = (int)(stop - t0);
    item = (long long)hk * tiles + tile;
    rows = load_rows(s, tile);
    u = stop;
    if (stop == t1) ++tile;
    return true;
  }
};

__device__ __forceinline__ float* segment_ml(const ChunkSet& s, long long item, int cta, int dv) {
  return s.part + (size_t)(item + cta) * s.rows * (2 + dv);
}
__device__ __forceinline__ float* segment_o(const ChunkSet& s, long long item, int cta, int dv) {
  return segment_ml(s, item, cta, dv) + 2 * s.rows;
}
// Where a row's value dim lies in o: [dim / D][row][dim % D], D = 2^shift. The wide kernel's lanes hold a row each: D = 16,
// so that they write whole sectors of neighbouring rows while the merge still reads 64 bytes at once. Mixed batch, wide
// kernel and merge: rows of all dims, 16 bytes a store, 222 and 53 us; 32 bytes a store in blocks of 32 dims 210 and 58,
// of 16 192 and 56, of 8 187 and 61. The other kernels' lanes hold a dim each, or neighbouring ones: D = 128.
constexpr int kWideShift = 4, kRowShift = 7;
__device__ __forceinline__ int state_pos(int shift, int rows, int row, int dim) {
  return (((dim >> shift) * rows + row) << shift) + (dim & ((1 << shift) - 1));
}

// Where the tensor-core kernels keep coordinate 4 lane + k of a query (or of its sketch), so that the keys' order
// in a tile need not change (kvq_chunk_dequant.cuh): the place of k = 0; k is k further in octet order, 8 k in token order.
__device__ __forceinline__ int query_pos(int order, int lane) {
  if (order == kOrderOctet) return 32 * (lane & 3) + 8 * (lane >> 3) + 4 * ((lane >> 2) & 1);
  return 64 * (lane >> 4) + 32 * (lane & 1) + ((lane >> 1) & 7);
}
constexpr float kCodeScale = 4.f, kSketchScale = 16.f;  // their operands hold 1/4 of a code, 1/16 of a sketch entry

// Launches a kernel of the call that starts while its predecessor ends (grid_dep_wait before it reads what that wrote).
inline cudaError_t launch_after(void (*kernel)(ChunkParams), const ChunkParams& p, unsigned blocks, unsigned threads, int smem,
                                int cluster, cudaStream_t s) {
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(blocks);
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  config.attrs = attr;
  config.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&config, kernel, p);
  const cudaError_t counted = launched();
  return e != cudaSuccess ? e : counted;
}

}  // namespace chunk

// The bf16 path's segment kernels: kvq_chunk_umma.cu for the wide set (and the query rows of its tile),
// kvq_chunk_narrow.cu for the narrow one.
int chunk_umma_rows(bool v_qjl);
cudaError_t launch_chunk_umma(const ChunkParams& p, cudaStream_t s);
constexpr int kNarrowRows = 64;
cudaError_t launch_chunk_narrow(const ChunkParams& p, cudaStream_t s);

}  // namespace kvq
