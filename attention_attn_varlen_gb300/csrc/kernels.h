// kernels.h -- host-side declarations shared by the C-ABI layer (api.cu) and
// the kernel translation units.  Parameter blocks are plain structs passed by
// value to the kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

// devices the per-device lazy set-ups (function attributes, symbol addresses) cover
constexpr int kMaxDev = 64;

struct DecodeParams {
    const __nv_bfloat16 *q;      // [B * Sq, Hq, D], row stride q_row_stride
    __nv_bfloat16 *out;          // [B * Sq, Hq, D], row stride out_row_stride
    float *lse;                  // null, or element (row, h) at row * lse_row_stride + h * lse_head_stride
    float *o_part;               // [B * Sq, Hq, S, D]  split partial outputs (normalised)
    float *lse_part;             // [B * Sq, Hq, S]     split partial log2-sum-exp
    const int32_t *cache_seqlens;
    const int32_t *block_table;
    int64_t q_row_stride, out_row_stride;
    int64_t lse_row_stride, lse_head_stride;
    int bt_stride, block_size, rows_per_box, num_splits, split_tokens;
    int64_t num_blocks;
    int Hq, Hkv, G;
    int Sq;                      // query tokens per sequence; Sq * G <= 64
    int ncg;                     // column groups: CTAs per (split, KV head, sequence), 16 columns each
    int causal;                  // bottom-right: token t sees keys j <= L - Sq + t
    int max_seqlen;              // cache_seqlens outside [0, max_seqlen] are clamped and reported
    int v16;                     // 1: V tiles are the fp16 V / 16 cache (PV on one fp16 term P' = 16 P)
    float scale_log2;            // softmax_scale * log2(e)
    uint32_t *err;
};

struct PrefillParams {
    const __nv_bfloat16 *v;      // contiguous [total_k, Hkv, D] (row stride v_row_stride) or the V cache
    __half *v16;                 // workspace: V / 16 in fp16, [total_k, Hkv, D] by logical key
    __nv_bfloat16 *out;          // [total_q, Hq, D], row stride out_row_stride
    float *lse;                  // [Hq, total_q] or null
    const int32_t *cu_q, *cu_k;
    const int32_t *seqused_q;    // null, or [batch]: sequence b uses the first seqused_q[b] rows of its range
    const int32_t *seqused_k;    // null, or [batch]: the same for its keys
    const int32_t *block_table;  // null: contiguous K/V
    int64_t total_q, total_k, out_row_stride, v_row_stride;
    int64_t num_blocks;
    int bt_stride, block_size, rows_per_box;
    int batch, Hq, Hkv, G, causal, head_dim, max_seqlen_k;
    int max_pairs;               // slot pairs per sequence at max_seqlen_q
    int v16_paged;               // 1: V' tiles come from a paged fp16 V / 16 cache through the block
                                 //    table (written by store_kvcache); no conversion pass
    int num_ctas;                // grid size: persistent CTAs (one per SM, at most the possible units)
    int one_slot;                // 1: max_seqlen_q <= 128 / G, every sequence fits one query slot
    int v_cvt;                   // 1 (one-slot launches without a V' cache): V tiles are loaded as bf16
                                 //    from v and converted to V' in shared memory; no conversion pass
    int2 *units;                 // workspace: (sequence, pair | kv_head << 16), scheduled order
    int *unit_count;             // workspace: [0] number of units
    float scale_log2;            // softmax_scale * log2(e), > 0
    uint32_t *err;
};

cudaError_t launch_store_kvcache(const void *k, const void *v, void *k_cache, void *v_cache, void *v16_cache,
                                 const int64_t *slot_mapping, int64_t num_tokens, int row_elems,
                                 int64_t k_stride, int64_t v_stride, int64_t num_slots, int num_sms,
                                 uint32_t *err, cudaStream_t stream);

cudaError_t launch_decode(const CUtensorMap &kmap, const CUtensorMap &vmap, const DecodeParams &p, int batch,
                          int head_dim, cudaStream_t stream);

// static scratch of the allocation-free decode entry point (device address on
// the current device, looked up on first use)
cudaError_t decode_noalloc_scratch(float **ptr, size_t *bytes);

// rows per query slot of the prefill kernel (a slot packs 128 / G tokens x G heads)
constexpr int kPrefillSlotRows = 128;
constexpr int kPrefillKeyTile = 128;

// measurement hook: record the caller's events (if set on this thread) right
// before and right after the main kernel of a call
void main_kernel_event_before(cudaStream_t stream);
void main_kernel_event_after(cudaStream_t stream);

cudaError_t launch_softmax_rows(const void *x, void *y, int64_t rows, int cols, int64_t x_row_stride,
                                int64_t y_row_stride, int bf16, int sms, uint32_t *err, cudaStream_t stream);

cudaError_t launch_padded_cu(int batch, int seqlen_q, int seqlen_k, int32_t *cu_q, int32_t *cu_k,
                             cudaStream_t stream);

cudaError_t launch_kvcache_cu(const int32_t *cache_seqlens, int batch, int seqlen_q, int max_cache_seqlen,
                              int32_t *cu_q, int32_t *cu_k, uint32_t *err, cudaStream_t stream);

// step_tables.cu: growing and trimming page tables on the GPU
constexpr int kTablesMaxBatch = 65535;
struct TablesParams {
    const int32_t *rows;         // null (entry b is row b), or [batch]: request row of each entry
    const int32_t *lens;         // [batch]: new tokens (grow) or tokens to keep (trim)
    int32_t *seq_lens;           // [num_rows]: cached tokens of each request
    int32_t *page_table;         // [num_rows, max_blocks]
    int32_t *free_pages;         // [num_pages]: the first *num_free entries are free pages
    int32_t *num_free;
    int batch, num_rows, max_blocks, bs_log2, num_pages;
    int64_t max_tokens;          // grow: entries of slot_mapping and positions
    int32_t *block_table;        // grow, outputs: [batch, max_blocks]
    int64_t *slot_mapping;       //   [max_tokens]
    int32_t *positions;          //   [max_tokens]
    int32_t *cu_q, *cu_k;        //   [batch + 1]
    int32_t *cache_seqlens;      //   [batch]: tokens after the step
    int32_t *context_lens;       //   [batch]: tokens before it
    int vec_rows, vec_tokens;    // grow: table rows, tokens take 16-byte accesses
    int32_t *before;             // workspace [batch]: length found for the entry, -1: unusable; then (trim)
                                 // before[0]: the release's CTAs that are done
    int4 *info;                  // workspace [batch] (grow)
    int4 *span;                  // workspace [batch] (trim): kept pages, pages before, place, row
    uint32_t *err;
};
cudaError_t launch_step_tables(const TablesParams &p, int num_sms, cudaStream_t stream);
cudaError_t launch_trim_pages(const TablesParams &p, int num_sms, cudaStream_t stream);

// rope_store.cu: rotary positions fused with the paged store
constexpr int kRopeMaxPairs = 128;
constexpr int kRopeMaxAxes = 4;
struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;   // [N, H, D]; row strides below; v null: nothing of V is stored
    __nv_bfloat16 *q_out, *k_out;     // k_out null: k goes to the cache only
    __nv_bfloat16 *k_cache, *v_cache; // null: no cache
    __half *v16_cache;
    const int64_t *slot_mapping;
    const int32_t *positions;         // axis a of token t at positions[a * axis_stride + t]
    const float *inv_freq;            // [half]
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride, axis_stride;
    int64_t num_tokens, num_slots;
    int Hq, Hkv, D, half, num_axes;
    int interleaved;
    float scale;
    uint8_t axis[kRopeMaxPairs];      // position axis of each pair
    uint32_t *err;
};
cudaError_t launch_rope_store(const RopeParams &p, bool vec, int num_sms, cudaStream_t stream);

// linear_attn.cu: linear attention with a decay for each head
struct LinearParams {
    const __nv_bfloat16 *q, *k, *v;   // [T, H, D] with row strides
    __nv_bfloat16 *out;
    const float *log_decay;           // [Hkv]
    const int32_t *cu;                // [batch + 1], or null (recurrent form): sequence b is row b
    float *state;                     // [num_slots, Hkv, D, D], rows along the value dimension; null: none kept
    const int32_t *slots;             // [batch]; < 0: no state
    const int32_t *context_lens;      // [batch] or null; 0: the sequence starts from a zero state
    const int32_t *cache_seqlens;     // [batch] or null; not above context_lens: refused, no state
    int64_t q_stride, k_stride, v_stride, out_stride, total_tokens, num_slots;
    int batch, Hq, Hkv, G, D, max_seqlen;
    int start_zero;                   // context_lens is null and every sequence starts from zero
    float scale;
    // prompts: the work list and the states at segment starts, in the workspace
    int seg_len;                      // a longer sequence is cut into segments of this many tokens (a multiple of 64)
    int max_units, state_rows;        // entries of units, rows of states
    int num_sms;                      // CTAs of the prompt kernel at most
    void *units;                      // kLinearUnitBytes each
    int *unit_count;
    float *decay;                     // [Hkv, kLinearDecayRow]
    float *states;                    // [state_rows, Hkv, D, D]
    uint32_t *err;
};
constexpr int kLinearDecayRow = 136, kLinearUnitBytes = 32;
cudaError_t launch_linear_varlen(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                 const CUtensorMap &omap, const LinearParams &p, cudaStream_t stream);
cudaError_t launch_linear_decode(const LinearParams &p, cudaStream_t stream);

cudaError_t launch_prefill(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                           const CUtensorMap &omap, const PrefillParams &p, int head_dim, cudaStream_t stream);

}  // namespace attn
