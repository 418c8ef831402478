// Launchers behind the libkvarn C-ABI (host side, not exported).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace kvarn {

// Launch facts cached per device, so that a call makes no driver query after the first one on a
// device (they cost host time on every call otherwise).
constexpr int kMaxCachedDevices = 64;

// The calling thread's device and its SM count (queried once per device).
cudaError_t current_device(int* dev, int* sms);

// Raise the kernel's dynamic shared-memory limit to bytes (and, with max_carveout, prefer the
// largest shared-memory carveout) unless an earlier call already did so for this kernel (by address)
// on this device with at least bytes.
cudaError_t set_smem_limit_once(const void* kernel, int bytes, bool max_carveout, int dev);
template <typename Kern>
cudaError_t set_smem_limit_once(Kern kern, int bytes, bool max_carveout, int dev) {
    return set_smem_limit_once(reinterpret_cast<const void*>(kern), bytes, max_carveout, dev);
}

// Read a kernel family's device error word (symbol: its address on the host) and clear it where it was set: a copy
// from the device synchronises and takes 8.5 us, the clearing one 4, and the words are nearly always 0.
inline cudaError_t read_and_clear_word(const void* symbol, unsigned int* out) {
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, symbol, sizeof(v));
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(symbol, &zero, sizeof(zero));
    if (e == cudaSuccess) *out = v;
    return e;
}

size_t encode_smem_bytes();
cudaError_t read_and_clear_device_error(unsigned int* out);
cudaError_t read_and_clear_decode_error(unsigned int* out);
cudaError_t launch_encode(int bits, int kind, const void* x, int64_t n_tiles, void* codes,
                          void* params, float* tile_scale, int iters, int rotate, int normalize,
                          cudaStream_t stream);

// K tiles then V tiles in one grid.  dest (optional, device, [n_k] with n_k == n_v): input tile u of
// either kind goes to output slot dest[u], and is skipped when dest[u] < 0.
cudaError_t launch_encode_kv(int k_bits, int v_bits, const void* k_x, int64_t n_k, void* k_codes,
                             void* k_params, float* k_scale, const void* v_x, int64_t n_v, void* v_codes,
                             void* v_params, float* v_scale, int iters, int rotate, int normalize,
                             cudaStream_t stream, const int32_t* dest = nullptr);

cudaError_t launch_dequant(int bits, int kind, const void* codes, const void* params,
                           const float* tile_scale, int64_t n_tiles, int original_basis,
                           int rotate, float* out, cudaStream_t stream);

// Split-K layout for decode attention: piece granularity P (minimum piece and tiles per partial
// slot block), slot count and workspace size.
struct DecodePlan {
    int piece;
    int splits;
    size_t workspace_bytes;
};
DecodePlan plan_decode(int B, int Hq, int Hkv, int max_tiles);

cudaError_t launch_decode(int k_bits, int v_bits, int group, const void* q, int B, int Hq, int Hkv,
                          const void* k_codes, const void* k_params, const float* k_scale,
                          const void* v_codes, const void* v_params, const float* v_scale,
                          const int32_t* block_table, int max_tiles, const int32_t* seq_lens,
                          const void* k_sink, const void* v_sink, int sink_len, const void* k_tail,
                          const void* v_tail, float softmax_scale, int rotate, int full_tail,
                          void* workspace, const DecodePlan& plan, float* out, cudaStream_t stream);

// Appending tokens: arguments of the append kernel (all device pointers).
struct AppendArgs {
    int Hkv, n_new, max_tiles, full_tail;
    const __nv_bfloat16* k_new;  // [B][Hkv][n_new][128]
    const __nv_bfloat16* v_new;
    const int32_t* n_accept;     // [B] or null (all offered tokens)
    int32_t* seq_lens;           // [B], updated
    __nv_bfloat16* k_tail;       // [B][Hkv][128][128], updated
    __nv_bfloat16* v_tail;
    const int32_t* block_table;  // [B][Hkv][max_tiles]
    __nv_bfloat16* k_stage;      // workspace: [B * Hkv][128][128], slot b * Hkv + h
    __nv_bfloat16* v_stage;
    int32_t* dest;               // workspace: [B * Hkv] pool tile of each staged block, -1 if none
};
size_t append_workspace_bytes(int B, int Hkv);
cudaError_t launch_append(const AppendArgs& a, int B, int k_bits, int v_bits, int iters, int rotate,
                          int normalize, void* k_codes, void* k_params, float* k_scale, void* v_codes,
                          void* v_params, float* v_scale, cudaStream_t stream);
cudaError_t read_and_clear_append_error(unsigned int* out);

// Launch with programmatic stream serialisation: the grid may start before the previous kernel in the
// stream completes; the kernel executes griddepcontrol.wait before it reads or writes global memory.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kern, args...);
}

// The same with clusters of `cluster` CTAs; past 8 the kernel needs allow_large_cluster_once.
template <typename... P, typename... A>
cudaError_t launch_pdl_cluster(void (*kern)(P...), dim3 grid, int cluster, dim3 block, size_t smem, cudaStream_t stream,
                               const A&... args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 2;
    return cudaLaunchKernelEx(&lc, kern, args...);
}

// Allow the kernel clusters past the portable 8 CTAs, unless an earlier call did so on this device.
cudaError_t allow_large_cluster_once(const void* kernel, int dev);
template <typename Kern>
cudaError_t allow_large_cluster_once(Kern kern, int dev) {
    return allow_large_cluster_once(reinterpret_cast<const void*>(kern), dev);
}

// A step's tables: see kvarn_step_tables for the arrays.
constexpr int kMaxTableSeqs = 16384;  // three prefix sums per sequence in shared memory
struct StepTablesArgs {
    int B, max_pages, page_size, free_capacity, n_rows, Hkv;
    int page_shift;  // set by the launcher: log2 of a page size that is a power of two, else -1
    const int32_t* seq_lens;
    const int32_t* n_new;
    const int32_t* page_counts;
    int32_t* page_table;
    int32_t* free_pages;
    const int32_t* free_count;
    int32_t* kv_lens;
    int32_t* page_counts_out;
    int32_t* free_count_out;
    int32_t* cu_tokens;
    int32_t* positions;
    int32_t* slot_map;
    int32_t* block_table;
    int32_t* status;
};
cudaError_t launch_step_tables(const StepTablesArgs& a, cudaStream_t stream);
cudaError_t read_and_clear_tables_error(unsigned int* out);

// Norm, rotation and cache write: see kvarn_rope_qkv.  Strides in elements.
struct RopeArgs {
    int n_tokens, Hq, Hkv, rot_dim, interleaved, page_size, n_slots;
    int passes;  // set by the launcher: times four rows that a warp takes of a token
    float rope_scale, eps;
    const void* q;
    const void* k;
    const void* v;
    int64_t q_token_stride, q_head_stride, kv_token_stride, kv_head_stride;
    const int32_t* positions;
    const double* inv_freq;
    const float* q_weight;
    const float* k_weight;
    void* q_out;
    int64_t qo_token_stride, qo_head_stride;
    void* k_cache;
    void* v_cache;
    int64_t page_stride, head_stride, token_stride;
    const int32_t* slot_map;
};
cudaError_t launch_rope_qkv(const RopeArgs& a, int x_dtype, int out_dtype, cudaStream_t stream);
cudaError_t read_and_clear_rope_error(unsigned int* out);

// Attention over a paged 16-bit cache: see kvarn_paged_attention.  Strides in elements.
struct PagedAttnArgs {
    int B, Hq, Hkv, page_size, max_pages, max_len, window, out_dtype;
    int64_t n_pages;
    // set by the launcher: query heads per kv head and (at most) per unit, units per kv head and per
    // sequence, log2 of a page size that is a power of two (else -1), whether first units of warps wait
    // in shared memory for their join
    int group, rows, row_blocks, units, page_shift, heads_near;
    float scale, softcap, inv_softcap;
    float lift;  // set by the launcher: log2 of the factor that a row's sum carries
    const void* q;
    int64_t q_token_stride, q_head_stride;
    const void* k_cache;
    const void* v_cache;
    int64_t page_stride, head_stride, token_stride;
    const int8_t* k_exp;  // [n_pages][Hkv][page_size] exponents of an 8-bit cache (strides in bytes), else null
    const int8_t* v_exp;
    const int32_t* page_table;
    const int32_t* kv_lens;
    const int32_t* kv_starts;
    const float* slopes;
    void* workspace;
    void* out;
    float* lse;
};
size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv);
cudaError_t launch_paged_attention(PagedAttnArgs a, int dtype, cudaStream_t stream);
cudaError_t read_and_clear_paged_attn_error(unsigned int* out);
cudaError_t launch_paged_attention_q8(PagedAttnArgs a, int dtype, cudaStream_t stream);
cudaError_t read_and_clear_paged_q8_error(unsigned int* out);

// Keys and values into a paged 8-bit cache: see kvarn_quantize_kv.  Input strides in elements, cache strides in bytes.
struct QuantizeArgs {
    int n_tokens, Hkv, page_size, n_slots;
    unsigned n_rows;  // set by the launcher: keys and values, a row of 128 channels each
    int page_shift;  // set by the launcher: log2 of a page size that is a power of two, else -1
    const void* k;
    const void* v;
    int64_t kv_token_stride, kv_head_stride;
    void* k_cache;
    void* v_cache;
    int64_t page_stride, head_stride, token_stride;
    int8_t* k_exp;
    int8_t* v_exp;
    const int32_t* slot_map;
};
cudaError_t launch_quantize_kv(QuantizeArgs a, int x_dtype, cudaStream_t stream);
cudaError_t read_and_clear_quantize_error(unsigned int* out);

// Attention of the new tokens of packed sequences over a paged 16-bit cache: see kvarn_prompt_attention.  Strides
// in elements.
constexpr int kMaxPromptSeqs = 16384;  // tiles of each sequence in shared memory
struct PromptArgs {
    int B, T, Hq, Hkv, page_size, max_pages, max_len, window, causal;
    int64_t n_pages;
    // set by the launcher: query heads per kv head, tokens of a copy, rows of a partial slot, log2 of a page size that
    // is a power of two (else -1), whether rows come and go by tiled copies
    int group, box, slot_rows, page_shift, tiled_rows, tiled_out;
    int ctas;                     // of the split
    uint32_t group_mul, group_shift;  // division by the group
    uint64_t grid_mul;                // and by the split's CTAs: 2^64 / ctas, rounded up (0: one CTA)
    float scale, softcap;
    // set by the launcher: of scores in the log2 domain, for capped ones (cap_near), of the maxima in partial slots
    float score_scale, cap, cap_scale, near[4], join_scale;
    const void* q;
    int64_t q_token_stride, q_head_stride;
    const void* k_cache;
    const void* v_cache;
    int64_t page_stride, head_stride, token_stride;
    const int32_t* page_table;
    const int32_t* cu;
    const int32_t* kv_lens;
    const int32_t* kv_starts;
    const float* slopes;
    const float* own_out;  // a part of each row's result that is joined with this one, and its log-sum-exp, or null:
    const float* own_lse;  // [T][Hq][128] and [T][Hq]
    void* workspace;
    void* out;
    float* lse;
};
size_t prompt_attention_workspace_bytes(int64_t T, int Hq, int Hkv);
cudaError_t launch_prompt_attention(PromptArgs a, int dtype, cudaStream_t stream);
cudaError_t read_and_clear_prompt_error(unsigned int* out);
cudaError_t read_and_clear_prompt_page_error(unsigned int* out);

// Self-check: one kernel whose bounded mbarrier wait runs out after limit_us (see bounded_wait.cu).
cudaError_t launch_bounded_wait_check(uint32_t limit_us, cudaStream_t stream);
cudaError_t read_and_clear_selftest_error(unsigned int* out);

}  // namespace kvarn
