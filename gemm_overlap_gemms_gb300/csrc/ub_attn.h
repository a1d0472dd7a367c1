// Internal interface between the host side of the attention operators (ub_attn_api.cu),
// their kernels (ub_kv_append.cu, ub_attn_prompt.cu, ub_attn_decode.cu) and the handle
// (ub_api.cu). Not installed; the public ABI is include/ub.h.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ub.h"

namespace ubk {

// What an attention call takes from its handle: the device, the active token count, the
// launch options, the status word of the bounded waits, and the workspace that the split
// decode attention shares with the split GEMM tiles (calls of a handle are
// stream-ordered, so no two of them use it at once).
struct HandleCall {
    int device;
    int sms;                 // SM count minus UB_OPT_SM_MARGIN
    int pdl;
    int64_t T;               // active tokens
    uint32_t *abort_word;
    int32_t *status;
    uint64_t timeout_ns;
    uint32_t epoch;
    float *ws;
    size_t ws_floats;
    uint32_t *join_counters; // of the decode attention
    int join_words;
    uint32_t *tickets;       // two words, zero between calls
    uint32_t *piece_counters; // of the prompt attention's split items: PROMPT_SLOTS words
    float *ws_rows;          // PROMPT_SLOTS * 512

};

int handle_device(ub_handle_t h);
int64_t handle_tokens(ub_handle_t h);  // active T
// The handle's state for one call on `s` (advances its epoch).
int handle_call(ub_handle_t h, cudaStream_t s, HandleCall *out);
// Kernel timing of UB_OPT_PROFILE around one launch of operation `op`.
int handle_prof_start(ub_handle_t h, int op, cudaStream_t s, bool *timed);
int handle_prof_stop(ub_handle_t h, int op, cudaStream_t s, bool timed);
// Count the tensor maps a call encoded.
void handle_count_maps(ub_handle_t h, int n);
// Record an error message (printf style) and return `code`.
int fail_call(int code, const char *fmt, ...);
// cuTensorMapEncodeTiled for a bf16 tensor of `rank` dimensions (innermost first, its
// stride 1; the others in bytes) in boxes whose innermost extent is 64 elements, with the
// 128-byte swizzle and zero fill.
int encode_nd(CUtensorMap *map, const void *ptr, int rank, const uint64_t *dims, const uint64_t *strides,
              const uint32_t *box);

// The token batch all three operators share (device arrays; see ub_attn_t).
struct SeqBatch {
    const int32_t *seq_starts;
    const int32_t *kv_lens;
    const int32_t *page_table;
    int64_t table_row;       // elements between the table's rows
    int table_width;
    int num_pages;
    int page_shift;          // page_size = 1 << page_shift
    int n_seqs;
    int32_t *status;         // sticky UB_ERR_ARG for a table entry outside the cache
};

struct AppendParams {
    SeqBatch b;
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;
    int64_t kc_page, kc_head, kc_row, vc_page, vc_head, vc_row;
    const float *cos, *sin;  // [max_pos, rot / 2]
    int64_t max_pos;
    int T, heads, kv_heads, head_dim, rot, interleaved;
    int parts;               // warps per token
    int pdl;
};
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t s);

struct DecodeParams {
    CUtensorMap tmK, tmV;    // [pages, kv_heads, head_dim / 64, page_size, 64]
    SeqBatch b;
    const void *q;
    void *out;
    float *lse;
    int64_t q_row, q_head, o_row, o_head;
    int heads, kv_heads, head_dim, group;
    int head_blocks;         // blocks of up to 16 query heads per key/value head
    int many_tiles;          // the table could hold 2^31 units of work or more over all heads
    float scale;
    float *ws;
    uint32_t *counters;      // parts that have come, per item: zero between calls
    uint32_t *times;         // how often all have come: never reset, so at the same place in every call
    uint32_t *abort_word;
    uint64_t timeout_ns;
    uint32_t epoch;
    int pdl;
    __host__ __device__ int32_t *status_word() const { return b.status; }
};
cudaError_t launch_attn_decode(const DecodeParams &p, int grid, cudaStream_t s);
constexpr int DECODE_ITEM_COST = 12;     // tiles that the end of an item counts as in the split
constexpr int DECODE_KEYS = 32;          // keys of one tile
constexpr int DECODE_CTAS_PER_SM = 1;
constexpr int DECODE_HEADS = 16;         // query heads of one pass over a key/value head, at most
constexpr int DECODE_SLOTS = 2;          // workspace slots per CTA
constexpr int DECODE_COUNTERS = 2;       // words per CTA: `counters` and `times`
__host__ __device__ constexpr int decode_slot_floats(int head_dim) { return DECODE_HEADS * (head_dim + 2); }

struct PromptParams {
    CUtensorMap tmQ;         // [T, heads, head_dim], boxes of one q tile's tokens and heads
    CUtensorMap tmK, tmV;    // paged: [pages, kv_heads, page_size, head_dim]; packed: [T, kv_heads, head_dim]
    SeqBatch b;
    int paged;
    void *out;
    float *lse;
    int64_t o_row, o_head;
    int T, heads, kv_heads, head_dim, group;
    int pack_shift;          // 1 << pack_shift query heads of one key/value head share a q tile
    int units;               // kv_heads * (group >> pack_shift)
    float scale;
    uint32_t *tickets;       // work items drawn, CTAs done; zero between calls
    float *ws;               // parts of items split over their keys: `slots` of 256 rows
    float *ws_rows;          // their rows' maxima and sums: 512 per slot
    uint32_t *counters;      // of split items: PROMPT_SLOTS / 2 counts, zero between calls, then as many
                             // that are never reset
    int slots;
    uint32_t *abort_word;
    uint64_t timeout_ns;
    uint32_t epoch;
    int pdl;
};
constexpr int PROMPT_SLOTS = 608;        // parts of split items, at most (half of it for heads of 128)
constexpr int PROMPT_WHOLE_KEYS = 1408;  // items of no more keys are never split
constexpr int PROMPT_ROWS = 128;         // rows (tokens x packed heads) of one q tile, two per CTA
constexpr int PROMPT_KEYS = 128;         // keys of one tile
cudaError_t launch_attn_prompt(const PromptParams &p, int grid, cudaStream_t s);

}  // namespace ubk
