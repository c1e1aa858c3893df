// Parameters and launches of the ragged serving path: slots, appends and chunk attention over the paged packed cache.
#pragma once

#include "kvq_internal.h"

namespace kvq {

// Lengths of up to kMaxSeqPerLaunch sequences, passed by value.
struct LengthParams {
  int* lens;
  int first, n;
  int value[kMaxSeqPerLaunch];
};

// Append of a token-major batch [n_tokens][heads][d] into page slots (kvq_slots.cu).
struct SlotQuantizeParams {
  const void* src[2];       // K, V
  int bf16;
  int n_tokens, heads;
  const long long* slots;   // 64 * page + token of the page; negative: not written
  const int* seq_start;     // [batch + 1]: rows outside [seq_start[0], seq_start[batch]) are not written; or null: all rows count
  int batch;
  char* region[2];
  int n_pages;
  SideLayout side[2];
  const float* signs;
  int signs_stride;
  const float* St;
  int s_exp;                // S / 2^s_exp is within fp16's range
  int* err;
  int sms;
};

// Chunk attention (kvq_chunk.cu): the workspace is laid out by chunk_layout(). The requests of one set are those
// whose query rows of a kv-head lie within its bounds; each set has its own plan, segment kernel and states.
struct ChunkSet {
  int above, upto;          // rows of a request: above < rows <= upto
  int rows;                 // query rows of a row tile
  int unit;                 // tokens of a unit
  int ctas;                 // CTAs (wide set: pairs of them) that share the units
  int max_tiles;            // row tiles of one kv-head the workspace holds
  long long* unit_start;    // [max_tiles + 1]
  int4* tile_rows;          // [max_tiles][2]: the row tiles (chunk::Rows)
  int* tile_start;          // [B + 1]
  long long* head;          // row tiles of a kv-head, their units, rows of the fullest one
  float* part;              // softmax states of the segments
};
constexpr int kWide = 0, kNarrow = 1;  // sets (fp32 calls have the first alone)

struct ChunkParams {
  const void* q;            // [n_tokens, Hq, d]
  void* out;                // the same, in q's type
  int bf16;
  int n_tokens, B, Hq, Hkv, group;
  const int* seq_start;     // [B + 1]
  const int* ctx_lens;      // [B]
  const int* held;          // [B]: a request whose ctx_lens is not held + its new tokens was refused; or null
  int capacity;             // tokens a sequence can hold
  const char* kreg;
  const char* vreg;
  int tiles_per_seq;
  const int* table;
  int pages_per_seq, n_pages;
  SideLayout k, v;
  const float* signs;
  int signs_stride;
  const float* S;
  const float* St;
  int s_exp;                // S / 2^s_exp is within fp16's range
  float logit_scale;        // softmax_scale * log2(e)
  int* err;
  long long wait_limit;
  int sms;
  // workspace
  int sets;
  ChunkSet set[2];
  void* qprep;              // rotated (and sketched) queries
  float* qscale;            // [n_tokens * Hq] (bf16)
};

// A chunk call's workspace: its sets with byte offsets in place of the pointers.
struct ChunkLayout {
  struct Set {
    int above, upto, rows, unit, ctas, max_tiles;
    size_t unit_start, tile_rows, tile_start, head, part;
  } set[2];
  int sets;
  size_t qprep, qscale, total;
};

// Requests of one extend_block_table call: every block sums the counts of all requests before its own, work that
// grows with the square of the batch, in 32-bit request numbers.
constexpr int kMaxTableRequests = 1 << 20;
cudaError_t launch_extend_block_table(const int* held, const int* n_new, int batch, const int* free_pages, int n_free,
                                      const int* cursor, int* table, int pages_per_seq, int* seq_start, int* ctx_lens,
                                      int* taken, cudaStream_t s);
cudaError_t launch_slot_map(const int* held, const int* seq_start, const int* ctx_lens, int batch, const int* table,
                            int pages_per_seq, int n_pages, int n_tokens, int* seq_ids, int* positions, long long* slots,
                            cudaStream_t s);
cudaError_t launch_set_lengths(const LengthParams& p, cudaStream_t s);
cudaError_t launch_quantize_slots(const SlotQuantizeParams& p, cudaStream_t s);
ChunkLayout chunk_layout(int n_tokens, int batch, int Hq, int Hkv, bool k_qjl, bool v_qjl, bool bf16, int sms);
cudaError_t launch_chunk_attention(const ChunkParams& p, cudaStream_t s);

}  // namespace kvq
