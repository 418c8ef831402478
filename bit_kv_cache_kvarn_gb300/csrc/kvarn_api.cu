// libkvarn C-ABI: argument validation and kernel launches.  See include/kvarn.h for the contract.
#include <float.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <string>

#include "../../include/kvarn.h"
#include "kvarn_internal.h"

namespace kvarn {

cudaError_t current_device(int* dev, int* sms) {
    static std::atomic<int> sm_count[kMaxCachedDevices] = {};  // 0: not queried yet
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return e;
    const bool cached = *dev >= 0 && *dev < kMaxCachedDevices;
    if (cached) {
        const int v = sm_count[*dev].load(std::memory_order_relaxed);
        if (v > 0) {
            *sms = v;
            return cudaSuccess;
        }
    }
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
    if (e == cudaSuccess && cached) sm_count[*dev].store(*sms, std::memory_order_relaxed);
    return e;
}

cudaError_t set_smem_limit_once(const void* kernel, int bytes, bool max_carveout, int dev) {
    struct Entry {
        const void* kernel;
        int dev, bytes;
    };
    static std::mutex mutex;
    static Entry done[256];  // a few dozen kernels x devices in practice
    static int n_done = 0;
    std::lock_guard<std::mutex> lock(mutex);
    for (int i = 0; i < n_done; ++i)
        if (done[i].kernel == kernel && done[i].dev == dev && done[i].bytes >= bytes) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && max_carveout)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e == cudaSuccess && n_done < 256) done[n_done++] = Entry{kernel, dev, bytes};
    return e;
}

cudaError_t allow_large_cluster_once(const void* kernel, int dev) {
    struct Entry {
        const void* kernel;
        int dev;
    };
    static std::mutex mutex;
    static Entry done[256];
    static int n_done = 0;
    std::lock_guard<std::mutex> lock(mutex);
    for (int i = 0; i < n_done; ++i)
        if (done[i].kernel == kernel && done[i].dev == dev) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && n_done < 256) done[n_done++] = Entry{kernel, dev};
    return e;
}

}  // namespace kvarn

namespace {

thread_local std::string g_last_error;

kvarn_status fail(kvarn_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
kvarn_status fail(kvarn_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

kvarn_status ok() {
    g_last_error.clear();
    return KVARN_OK;
}

kvarn_status cuda_fail(cudaError_t e, const char* what) {
    cudaGetLastError();  // consume
    return fail(KVARN_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

kvarn_status check_cfg(const kvarn_config* cfg) {
    if (!cfg) return fail(KVARN_ERR_INVALID_ARG, "cfg is NULL");
    if (cfg->k_bits != 2 && cfg->k_bits != 4)
        return fail(KVARN_ERR_INVALID_ARG, "k_bits = %d; supported: 2, 4", cfg->k_bits);
    if (cfg->v_bits != 2 && cfg->v_bits != 4)
        return fail(KVARN_ERR_INVALID_ARG, "v_bits = %d; supported: 2, 4", cfg->v_bits);
    if (cfg->sinkhorn_iters < 0 || cfg->sinkhorn_iters > 64)
        return fail(KVARN_ERR_INVALID_ARG, "sinkhorn_iters = %d; allowed 0..64", cfg->sinkhorn_iters);
    if (cfg->flags & ~(KVARN_FLAG_NO_ROTATE | KVARN_FLAG_NO_NORMALIZE | KVARN_FLAG_FULL_TAIL))
        return fail(KVARN_ERR_INVALID_ARG, "unknown flag bits 0x%x", cfg->flags);
    return KVARN_OK;
}

kvarn_status check_ptr(const void* p, size_t align, const char* name) {
    if (!p) return fail(KVARN_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, align)) return fail(KVARN_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
    return KVARN_OK;
}

#define KV_TRY(expr)                     \
    do {                                 \
        kvarn_status _s = (expr);        \
        if (_s != KVARN_OK) return _s;   \
    } while (0)

}  // namespace

extern "C" {

kvarn_status kvarn_config_from_preset(const char* name, kvarn_config* out) {
    if (!name || !out) return fail(KVARN_ERR_INVALID_ARG, "name or out is NULL");
    struct Preset {
        const char* name;
        kvarn_config cfg;
    };
    static const Preset kPresets[] = {
        {"kvarn_k4v2_g128", {4, 2, 8, 0u}},
        {"kvarn_k2v2_g128", {2, 2, 8, 0u}},
        {"kvarn_k4v4_g128", {4, 4, 8, 0u}},
        {"kvarn_k2v4_g128", {2, 4, 8, 0u}},
        {"hadamard_k2v2_g128", {2, 2, 0, KVARN_FLAG_NO_NORMALIZE}},
        {"kivi_k2v2_g128", {2, 2, 0, KVARN_FLAG_NO_ROTATE | KVARN_FLAG_NO_NORMALIZE}},
    };
    for (const Preset& p : kPresets) {
        if (strcmp(name, p.name) == 0) {
            *out = p.cfg;
            return ok();
        }
    }
    return fail(KVARN_ERR_INVALID_ARG,
                "unknown preset '%s' (known: kvarn_k4v2_g128, kvarn_k2v2_g128, kvarn_k4v4_g128, "
                "kvarn_k2v4_g128, hadamard_k2v2_g128, kivi_k2v2_g128)",
                name);
}

size_t kvarn_tile_code_bytes(int bits) {
    return (bits == 2 || bits == 4) ? (size_t)KVARN_TILE_TOKENS * 16 * bits : 0;
}

size_t kvarn_tile_param_bytes(void) { return KVARN_PARAM_BYTES; }

kvarn_status kvarn_encode_blocks(const kvarn_config* cfg, kvarn_kind kind, const void* x_bf16,
                                 int64_t n_tiles, void* codes, void* params, float* tile_scale,
                                 kvarn_stream_t stream) {
    KV_TRY(check_cfg(cfg));
    if (kind != KVARN_KIND_K && kind != KVARN_KIND_V)
        return fail(KVARN_ERR_INVALID_ARG, "kind = %d; expected KVARN_KIND_K or KVARN_KIND_V", (int)kind);
    if (n_tiles < 0) return fail(KVARN_ERR_INVALID_ARG, "n_tiles = %lld < 0", (long long)n_tiles);
    if (n_tiles == 0) return ok();
    KV_TRY(check_ptr(x_bf16, 16, "x_bf16"));
    KV_TRY(check_ptr(codes, 16, "codes"));
    KV_TRY(check_ptr(params, 16, "params"));
    KV_TRY(check_ptr(tile_scale, 4, "tile_scale"));
    const int bits = kind == KVARN_KIND_K ? cfg->k_bits : cfg->v_bits;
    cudaError_t e = kvarn::launch_encode(bits, (int)kind, x_bf16, n_tiles, codes, params, tile_scale,
                                         cfg->sinkhorn_iters, !(cfg->flags & KVARN_FLAG_NO_ROTATE),
                                         !(cfg->flags & KVARN_FLAG_NO_NORMALIZE), (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "encode launch");
    return ok();
}

kvarn_status kvarn_encode_kv_blocks(const kvarn_config* cfg, const void* k_bf16, const void* v_bf16,
                                    int64_t n_tiles, void* k_codes, void* k_params, float* k_scale,
                                    void* v_codes, void* v_params, float* v_scale,
                                    kvarn_stream_t stream) {
    KV_TRY(check_cfg(cfg));
    if (n_tiles < 0) return fail(KVARN_ERR_INVALID_ARG, "n_tiles = %lld < 0", (long long)n_tiles);
    if (n_tiles == 0) return ok();
    KV_TRY(check_ptr(k_bf16, 16, "k_bf16"));
    KV_TRY(check_ptr(v_bf16, 16, "v_bf16"));
    KV_TRY(check_ptr(k_codes, 16, "k_codes"));
    KV_TRY(check_ptr(k_params, 16, "k_params"));
    KV_TRY(check_ptr(k_scale, 4, "k_scale"));
    KV_TRY(check_ptr(v_codes, 16, "v_codes"));
    KV_TRY(check_ptr(v_params, 16, "v_params"));
    KV_TRY(check_ptr(v_scale, 4, "v_scale"));
    cudaError_t e = kvarn::launch_encode_kv(cfg->k_bits, cfg->v_bits, k_bf16, n_tiles, k_codes, k_params,
                                            k_scale, v_bf16, n_tiles, v_codes, v_params, v_scale,
                                            cfg->sinkhorn_iters, !(cfg->flags & KVARN_FLAG_NO_ROTATE),
                                            !(cfg->flags & KVARN_FLAG_NO_NORMALIZE), (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "encode launch");
    return ok();
}

kvarn_status kvarn_dequant(const kvarn_config* cfg, kvarn_kind kind, const void* codes,
                           const void* params, const float* tile_scale, int64_t n_tiles,
                           int original_basis, float* out, kvarn_stream_t stream) {
    KV_TRY(check_cfg(cfg));
    if (kind != KVARN_KIND_K && kind != KVARN_KIND_V)
        return fail(KVARN_ERR_INVALID_ARG, "kind = %d; expected KVARN_KIND_K or KVARN_KIND_V", (int)kind);
    if (n_tiles < 0 || n_tiles > 0x7fffffffLL)
        return fail(KVARN_ERR_INVALID_ARG, "n_tiles = %lld outside 0..2^31-1", (long long)n_tiles);
    if (original_basis != 0 && original_basis != 1)
        return fail(KVARN_ERR_INVALID_ARG, "original_basis = %d; expected 0 or 1", original_basis);
    if (n_tiles == 0) return ok();
    KV_TRY(check_ptr(codes, 16, "codes"));
    KV_TRY(check_ptr(params, 16, "params"));
    KV_TRY(check_ptr(tile_scale, 4, "tile_scale"));
    KV_TRY(check_ptr(out, 16, "out"));
    const int bits = kind == KVARN_KIND_K ? cfg->k_bits : cfg->v_bits;
    cudaError_t e = kvarn::launch_dequant(bits, (int)kind, codes, params, tile_scale, n_tiles,
                                          original_basis, !(cfg->flags & KVARN_FLAG_NO_ROTATE), out,
                                          (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "dequant launch");
    return ok();
}

static kvarn_status check_decode_shape(const kvarn_config* cfg, int B, int Hq, int Hkv, int max_tiles) {
    KV_TRY(check_cfg(cfg));
    if (B < 0 || B > 65535) return fail(KVARN_ERR_INVALID_ARG, "B = %d outside 0..65535", B);
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
        return fail(KVARN_ERR_INVALID_ARG, "Hq = %d, Hkv = %d: need Hq a positive multiple of Hkv", Hq, Hkv);
    if (Hq > 65535) return fail(KVARN_ERR_INVALID_ARG, "Hq = %d outside 1..65535", Hq);
    if (max_tiles < 0 || max_tiles > (1 << 24))
        return fail(KVARN_ERR_INVALID_ARG, "max_tiles = %d outside 0..2^24", max_tiles);
    return KVARN_OK;
}

size_t kvarn_decode_workspace_size(const kvarn_config* cfg, int B, int Hq, int Hkv, int max_tiles) {
    if (check_decode_shape(cfg, B, Hq, Hkv, max_tiles) != KVARN_OK) return 0;
    return kvarn::plan_decode(B, Hq, Hkv, max_tiles).workspace_bytes;
}

namespace {

kvarn_status decode_impl(const kvarn_config* cfg, const void* q_bf16, int B, int Hq, int Hkv,
                         const void* k_codes, const void* k_params, const float* k_scale,
                         const void* v_codes, const void* v_params, const float* v_scale,
                         const int32_t* block_table, int max_tiles, const int32_t* seq_lens,
                         const int32_t* seq_lens_host, const void* k_sink_bf16, const void* v_sink_bf16,
                         int sink_len, const void* k_tail_bf16, const void* v_tail_bf16,
                         float softmax_scale, void* workspace, size_t workspace_bytes, float* out,
                         kvarn_stream_t stream) {
    KV_TRY(check_decode_shape(cfg, B, Hq, Hkv, max_tiles));
    if (!isfinite(softmax_scale)) return fail(KVARN_ERR_INVALID_ARG, "softmax_scale is not finite");
    if (sink_len < 0 || sink_len > KVARN_TILE_TOKENS)
        return fail(KVARN_ERR_INVALID_ARG, "sink_len = %d outside 0..128", sink_len);
    if (B == 0) return ok();
    KV_TRY(check_ptr(q_bf16, 16, "q_bf16"));
    KV_TRY(check_ptr(seq_lens, 4, "seq_lens"));
    KV_TRY(check_ptr(k_tail_bf16, 16, "k_tail_bf16"));
    KV_TRY(check_ptr(v_tail_bf16, 16, "v_tail_bf16"));
    KV_TRY(check_ptr(out, 16, "out"));
    if (sink_len > 0) {
        KV_TRY(check_ptr(k_sink_bf16, 16, "k_sink_bf16"));
        KV_TRY(check_ptr(v_sink_bf16, 16, "v_sink_bf16"));
    }
    if (max_tiles > 0) {
        KV_TRY(check_ptr(k_codes, 16, "k_codes"));
        KV_TRY(check_ptr(k_params, 16, "k_params"));
        KV_TRY(check_ptr(k_scale, 4, "k_scale"));
        KV_TRY(check_ptr(v_codes, 16, "v_codes"));
        KV_TRY(check_ptr(v_params, 16, "v_params"));
        KV_TRY(check_ptr(v_scale, 4, "v_scale"));
        KV_TRY(check_ptr(block_table, 4, "block_table"));
    }
    if (seq_lens_host) {
        const long long cap = (long long)sink_len + (long long)max_tiles * KVARN_TILE_TOKENS +
                              ((cfg->flags & KVARN_FLAG_FULL_TAIL) ? KVARN_TILE_TOKENS : KVARN_TILE_TOKENS - 1);
        for (int b = 0; b < B; ++b)
            if (seq_lens_host[b] < 0 || seq_lens_host[b] > cap)
                return fail(KVARN_ERR_INVALID_ARG, "seq_lens[%d] = %d outside 0..%lld", b, seq_lens_host[b], cap);
    }
    const kvarn::DecodePlan plan = kvarn::plan_decode(B, Hq, Hkv, max_tiles);
    KV_TRY(check_ptr(workspace, 16, "workspace"));
    if (workspace_bytes < plan.workspace_bytes)
        return fail(KVARN_ERR_WORKSPACE, "workspace_bytes = %zu < required %zu", workspace_bytes,
                    plan.workspace_bytes);
    cudaError_t e = kvarn::launch_decode(cfg->k_bits, cfg->v_bits, Hq / Hkv, q_bf16, B, Hq, Hkv, k_codes,
                                         k_params, k_scale, v_codes, v_params, v_scale, block_table,
                                         max_tiles, seq_lens, k_sink_bf16, v_sink_bf16, sink_len, k_tail_bf16,
                                         v_tail_bf16, softmax_scale, !(cfg->flags & KVARN_FLAG_NO_ROTATE),
                                         (cfg->flags & KVARN_FLAG_FULL_TAIL) != 0, workspace, plan, out,
                                         (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "decode attention launch");
    return ok();
}

}  // namespace

kvarn_status kvarn_decode_attention(const kvarn_config* cfg, const void* q_bf16, int B, int Hq,
                                    int Hkv, const void* k_codes, const void* k_params,
                                    const float* k_scale, const void* v_codes,
                                    const void* v_params, const float* v_scale,
                                    const int32_t* block_table, int max_tiles,
                                    const int32_t* seq_lens, const int32_t* seq_lens_host,
                                    const void* k_tail_bf16, const void* v_tail_bf16,
                                    float softmax_scale, void* workspace, size_t workspace_bytes,
                                    float* out, kvarn_stream_t stream) {
    return decode_impl(cfg, q_bf16, B, Hq, Hkv, k_codes, k_params, k_scale, v_codes, v_params, v_scale,
                       block_table, max_tiles, seq_lens, seq_lens_host, nullptr, nullptr, 0, k_tail_bf16,
                       v_tail_bf16, softmax_scale, workspace, workspace_bytes, out, stream);
}

kvarn_status kvarn_decode_attention_sink(const kvarn_config* cfg, const void* q_bf16, int B, int Hq,
                                         int Hkv, const void* k_codes, const void* k_params,
                                         const float* k_scale, const void* v_codes, const void* v_params,
                                         const float* v_scale, const int32_t* block_table, int max_tiles,
                                         const int32_t* seq_lens, const int32_t* seq_lens_host,
                                         const void* k_sink_bf16, const void* v_sink_bf16, int sink_len,
                                         const void* k_tail_bf16, const void* v_tail_bf16,
                                         float softmax_scale, void* workspace, size_t workspace_bytes,
                                         float* out, kvarn_stream_t stream) {
    return decode_impl(cfg, q_bf16, B, Hq, Hkv, k_codes, k_params, k_scale, v_codes, v_params, v_scale,
                       block_table, max_tiles, seq_lens, seq_lens_host, k_sink_bf16, v_sink_bf16, sink_len,
                       k_tail_bf16, v_tail_bf16, softmax_scale, workspace, workspace_bytes, out, stream);
}

// Whether a serving-step call of this process was enqueued or captured: without one its error words are 0
// and not read (54 us -> 91 with them and a clearing copy for every word; now 37, with them 64).
static std::atomic<bool> g_serving_used = {false};
static std::atomic<bool> g_prompt_used = {false};  // the same for the calls with many queries,
static std::atomic<bool> g_q8_used = {false};      // and for those with 8-bit caches

kvarn_status kvarn_device_error(uint32_t* code_out) {
    if (!code_out) return fail(KVARN_ERR_INVALID_ARG, "code_out is NULL");
    unsigned int v = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "device synchronize");
    e = kvarn::read_and_clear_device_error(&v);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    unsigned int w = 0;
    e = kvarn::read_and_clear_decode_error(&w);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    unsigned int x = 0;
    e = kvarn::read_and_clear_append_error(&x);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    unsigned int y = 0;
    e = kvarn::read_and_clear_selftest_error(&y);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    unsigned int serving[3] = {0, 0, 0};
    if (g_serving_used.load()) {
        e = kvarn::read_and_clear_tables_error(&serving[0]);
        if (e != cudaSuccess) return cuda_fail(e, "device error word");
        e = kvarn::read_and_clear_rope_error(&serving[1]);
        if (e != cudaSuccess) return cuda_fail(e, "device error word");
        e = kvarn::read_and_clear_paged_attn_error(&serving[2]);
        if (e != cudaSuccess) return cuda_fail(e, "device error word");
    }
    unsigned int prompt = 0;
    if (g_prompt_used.load()) {
        unsigned int page = 0;
        e = kvarn::read_and_clear_prompt_page_error(&page);
        if (e != cudaSuccess) return cuda_fail(e, "device error word");
        e = kvarn::read_and_clear_prompt_error(&prompt);
        if (e != cudaSuccess) return cuda_fail(e, "device error word");
        serving[2] |= page;
    }
    if (g_q8_used.load()) {
        unsigned int slot = 0, page = 0;
        e = kvarn::read_and_clear_quantize_error(&slot);
        if (e != cudaSuccess) return cuda_fail(e, "device error word");
        e = kvarn::read_and_clear_paged_q8_error(&page);
        if (e != cudaSuccess) return cuda_fail(e, "device error word");
        serving[1] |= slot;
        serving[2] |= page;
    }
    *code_out = v | (w << 1) | (x << 2) | (y << 3) | (serving[0] << 4) | (serving[1] << 5) | (serving[2] << 6) | (prompt << 7);
    if (*code_out & KVARN_DEVICE_TIMEOUT_BITS)
        return fail(KVARN_ERR_TIMEOUT, "a bounded device wait gave up (device error bits 0x%x)", *code_out);
    return ok();
}

kvarn_status kvarn_check_bounded_wait(uint32_t limit_us, kvarn_stream_t stream) {
    if (limit_us < 1 || limit_us > 1000000)
        return fail(KVARN_ERR_INVALID_ARG, "limit_us = %u outside 1..1000000", limit_us);
    cudaError_t e = kvarn::launch_bounded_wait_check(limit_us, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "bounded-wait check launch");
    return ok();
}

size_t kvarn_append_workspace_size(int B, int Hkv) {
    if (B < 0 || B > 65535 || Hkv < 1 || Hkv > 1024) return 0;
    return kvarn::append_workspace_bytes(B, Hkv);
}

kvarn_status kvarn_append_tokens(const kvarn_config* cfg, int B, int Hkv, const void* k_new_bf16,
                                 const void* v_new_bf16, int n_new, const int32_t* n_accept,
                                 int32_t* seq_lens, void* k_tail_bf16, void* v_tail_bf16, void* k_codes,
                                 void* k_params, float* k_scale, void* v_codes, void* v_params,
                                 float* v_scale, const int32_t* block_table, int max_tiles, void* workspace,
                                 size_t workspace_bytes, kvarn_stream_t stream) {
    KV_TRY(check_cfg(cfg));
    if (B < 0 || B > 65535) return fail(KVARN_ERR_INVALID_ARG, "B = %d outside 0..65535", B);
    if (Hkv < 1 || Hkv > 1024) return fail(KVARN_ERR_INVALID_ARG, "Hkv = %d outside 1..1024", Hkv);
    if (n_new < 1 || n_new > KVARN_TILE_TOKENS) return fail(KVARN_ERR_INVALID_ARG, "n_new = %d outside 1..128", n_new);
    if (max_tiles < 0 || max_tiles > (1 << 24))
        return fail(KVARN_ERR_INVALID_ARG, "max_tiles = %d outside 0..2^24", max_tiles);
    if (B == 0) return ok();
    KV_TRY(check_ptr(k_new_bf16, 16, "k_new_bf16"));
    KV_TRY(check_ptr(v_new_bf16, 16, "v_new_bf16"));
    if (n_accept) KV_TRY(check_ptr(n_accept, 4, "n_accept"));
    KV_TRY(check_ptr(seq_lens, 4, "seq_lens"));
    KV_TRY(check_ptr(k_tail_bf16, 16, "k_tail_bf16"));
    KV_TRY(check_ptr(v_tail_bf16, 16, "v_tail_bf16"));
    if (max_tiles > 0) {
        KV_TRY(check_ptr(k_codes, 16, "k_codes"));
        KV_TRY(check_ptr(k_params, 16, "k_params"));
        KV_TRY(check_ptr(k_scale, 4, "k_scale"));
        KV_TRY(check_ptr(v_codes, 16, "v_codes"));
        KV_TRY(check_ptr(v_params, 16, "v_params"));
        KV_TRY(check_ptr(v_scale, 4, "v_scale"));
        KV_TRY(check_ptr(block_table, 4, "block_table"));
    }
    KV_TRY(check_ptr(workspace, 256, "workspace"));
    const size_t need = kvarn::append_workspace_bytes(B, Hkv);
    if (workspace_bytes < need)
        return fail(KVARN_ERR_WORKSPACE, "workspace_bytes = %zu < required %zu", workspace_bytes, need);
    kvarn::AppendArgs a;
    a.Hkv = Hkv;
    a.n_new = n_new;
    a.max_tiles = max_tiles;
    a.full_tail = (cfg->flags & KVARN_FLAG_FULL_TAIL) != 0;
    a.k_new = static_cast<const __nv_bfloat16*>(k_new_bf16);
    a.v_new = static_cast<const __nv_bfloat16*>(v_new_bf16);
    a.n_accept = n_accept;
    a.seq_lens = seq_lens;
    a.k_tail = static_cast<__nv_bfloat16*>(k_tail_bf16);
    a.v_tail = static_cast<__nv_bfloat16*>(v_tail_bf16);
    a.block_table = block_table;
    const size_t tiles = (size_t)B * Hkv;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.k_stage = reinterpret_cast<__nv_bfloat16*>(w);
    a.v_stage = reinterpret_cast<__nv_bfloat16*>(w + tiles * KVARN_TILE_TOKENS * KVARN_TILE_TOKENS * 2);
    a.dest = reinterpret_cast<int32_t*>(w + 2 * tiles * KVARN_TILE_TOKENS * KVARN_TILE_TOKENS * 2);
    cudaError_t e = kvarn::launch_append(a, B, cfg->k_bits, cfg->v_bits, cfg->sinkhorn_iters,
                                         !(cfg->flags & KVARN_FLAG_NO_ROTATE),
                                         !(cfg->flags & KVARN_FLAG_NO_NORMALIZE), k_codes, k_params, k_scale,
                                         v_codes, v_params, v_scale, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "append launch");
    return ok();
}

// ---- decode attention with library-owned scratch (no allocation by the caller or the library) ----
// The split-K partials normally live in a caller-supplied workspace.  This variant keeps them in a
// fixed device array instead, for callers that have no way to obtain device memory at this point.
// Every GPU that loads the library holds the array (KVARN_STATIC_WS_BYTES) until the process exits.
static __device__ __align__(256) unsigned char g_kvarn_static_ws[KVARN_STATIC_WS_BYTES];

namespace {
constexpr int kMaxDevices = 256;
std::mutex g_static_ws_mutex;
void* g_static_ws_ptr[kMaxDevices] = {};  // device address of g_kvarn_static_ws, per device
}  // namespace

kvarn_status kvarn_decode_attention_static_ws(
    const kvarn_config* cfg, const void* q_bf16, int B, int Hq, int Hkv, const void* k_codes,
    const void* k_params, const float* k_scale, const void* v_codes, const void* v_params,
    const float* v_scale, const int32_t* block_table, int max_tiles, const int32_t* seq_lens,
    const int32_t* seq_lens_host, const void* k_tail_bf16, const void* v_tail_bf16,
    float softmax_scale, float* out, kvarn_stream_t stream) {
    const size_t need = kvarn_decode_workspace_size(cfg, B, Hq, Hkv, max_tiles);
    if (need > (size_t)KVARN_STATIC_WS_BYTES)
        return fail(KVARN_ERR_WORKSPACE,
                    "this shape needs %zu bytes of split-K scratch; the static scratch holds %zu "
                    "(use kvarn_decode_attention with a caller workspace)",
                    need, (size_t)KVARN_STATIC_WS_BYTES);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(KVARN_ERR_UNSUPPORTED, "device index %d", dev);
    void* ws = nullptr;
    {
        // First call on this device (with it current): look up the array's device address once.
        std::lock_guard<std::mutex> lock(g_static_ws_mutex);
        if (!g_static_ws_ptr[dev]) {
            e = cudaGetSymbolAddress(&g_static_ws_ptr[dev], g_kvarn_static_ws);
            if (e != cudaSuccess) {
                g_static_ws_ptr[dev] = nullptr;
                return cuda_fail(e, "cudaGetSymbolAddress(static scratch)");
            }
        }
        ws = g_static_ws_ptr[dev];
    }
    // Every partial the kernels read is written earlier in the same call, so the array needs no
    // clearing between calls.
    return kvarn_decode_attention(cfg, q_bf16, B, Hq, Hkv, k_codes, k_params, k_scale, v_codes,
                                  v_params, v_scale, block_table, max_tiles, seq_lens, seq_lens_host,
                                  k_tail_bf16, v_tail_bf16, softmax_scale, ws,
                                  (size_t)KVARN_STATIC_WS_BYTES, out, stream);
}

// ---- a serving step around the caches ----

kvarn_status kvarn_step_tables(int B, int max_pages, int page_size, const int32_t* seq_lens,
                               const int32_t* n_new, const int32_t* page_counts, int32_t* page_table,
                               int32_t* free_pages, const int32_t* free_count, int free_capacity,
                               int32_t* kv_lens, int32_t* page_counts_out, int32_t* free_count_out,
                               int32_t* cu_tokens, int32_t* positions, int32_t* slot_map, int n_rows,
                               int32_t* block_table, int Hkv, int32_t* status, kvarn_stream_t stream) {
    if (B < 0 || B > kvarn::kMaxTableSeqs)
        return fail(KVARN_ERR_INVALID_ARG, "B = %d outside 0..%d", B, kvarn::kMaxTableSeqs);
    if (page_size < 1 || page_size > 65536) return fail(KVARN_ERR_INVALID_ARG, "page_size = %d outside 1..65536", page_size);
    if (max_pages < 1 || (int64_t)B * max_pages > (1LL << 30))
        return fail(KVARN_ERR_INVALID_ARG, "max_pages = %d: need at least 1 and B * max_pages <= 2^30", max_pages);
    if (n_rows < 0 || n_rows > (1 << 30)) return fail(KVARN_ERR_INVALID_ARG, "n_rows = %d outside 0..2^30", n_rows);
    if (free_capacity < 0 || free_capacity > (1 << 30))
        return fail(KVARN_ERR_INVALID_ARG, "free_capacity = %d outside 0..2^30", free_capacity);
    if (Hkv < 0 || Hkv > 1024) return fail(KVARN_ERR_INVALID_ARG, "Hkv = %d outside 0..1024", Hkv);
    if ((Hkv > 0) != (block_table != nullptr))
        return fail(KVARN_ERR_INVALID_ARG, "Hkv = %d: block_table goes with Hkv > 0, and only with it", Hkv);
    if (B == 0) return ok();
    const struct {
        const void* p;
        const char* name;
    } arrays[] = {{seq_lens, "seq_lens"},     {n_new, "n_new"},
                  {page_counts, "page_counts"}, {page_table, "page_table"},
                  {free_count, "free_count"}, {kv_lens, "kv_lens"},
                  {page_counts_out, "page_counts_out"}, {free_count_out, "free_count_out"},
                  {cu_tokens, "cu_tokens"},   {status, "status"}};
    for (const auto& x : arrays) KV_TRY(check_ptr(x.p, 4, x.name));
    if (free_capacity > 0) KV_TRY(check_ptr(free_pages, 4, "free_pages"));
    if (n_rows > 0) {
        KV_TRY(check_ptr(positions, 4, "positions"));
        KV_TRY(check_ptr(slot_map, 4, "slot_map"));
    }
    if (block_table) KV_TRY(check_ptr(block_table, 4, "block_table"));
    kvarn::StepTablesArgs a = {};
    a.B = B;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.free_capacity = free_capacity;
    a.n_rows = n_rows;
    a.Hkv = Hkv;
    a.seq_lens = seq_lens;
    a.n_new = n_new;
    a.page_counts = page_counts;
    a.page_table = page_table;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.kv_lens = kv_lens;
    a.page_counts_out = page_counts_out;
    a.free_count_out = free_count_out;
    a.cu_tokens = cu_tokens;
    a.positions = positions;
    a.slot_map = slot_map;
    a.block_table = block_table;
    a.status = status;
    g_serving_used.store(true);
    cudaError_t e = kvarn::launch_step_tables(a, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "step tables launch");
    return ok();
}

kvarn_status kvarn_rope_frequencies(const kvarn_rope_config* cfg, double* freqs, float* rope_scale) {
    if (!cfg || !freqs || !rope_scale) return fail(KVARN_ERR_INVALID_ARG, "cfg, freqs or rope_scale is NULL");
    const int R = cfg->rot_dim;
    if (R < 16 || R > KVARN_HEAD_DIM || R % 16 != 0)
        return fail(KVARN_ERR_INVALID_ARG, "rot_dim = %d; need a multiple of 16, 16..128", R);
    if (cfg->scaling < KVARN_ROPE_PLAIN || cfg->scaling > KVARN_ROPE_YARN)
        return fail(KVARN_ERR_INVALID_ARG, "scaling = %d; expected 0..4", cfg->scaling);
    if (!(cfg->base > 1.0) || !isfinite(cfg->base)) return fail(KVARN_ERR_INVALID_ARG, "base = %g; need a finite base > 1", cfg->base);
    const double s = cfg->scaling == KVARN_ROPE_PLAIN ? 1.0 : cfg->factor;
    if (!(s >= 1.0) || !isfinite(s)) return fail(KVARN_ERR_INVALID_ARG, "factor = %g; need a finite factor >= 1", s);
    const bool mixed = cfg->scaling == KVARN_ROPE_BANDS || cfg->scaling == KVARN_ROPE_YARN;
    if (mixed && (!(cfg->original_len > 0.0) || !isfinite(cfg->original_len)))
        return fail(KVARN_ERR_INVALID_ARG, "original_len = %g; need a finite length > 0", cfg->original_len);
    if (mixed && !(cfg->low > 0.0 && cfg->low < cfg->high && isfinite(cfg->high)))
        return fail(KVARN_ERR_INVALID_ARG, "low = %g, high = %g; need 0 < low < high", cfg->low, cfg->high);
    const double two_pi = 6.28318530717958647692;
    const double base = cfg->scaling == KVARN_ROPE_NTK ? cfg->base * pow(s, R / (R - 2.0)) : cfg->base;
    // YaRN: the (fractional) channel pair that makes n turns over the trained context
    auto pair_of = [&](double turns) { return R * log(cfg->original_len / (turns * two_pi)) / (2.0 * log(base)); };
    double first = 0.0, last = 0.0;
    if (cfg->scaling == KVARN_ROPE_YARN) {
        first = fmax(floor(pair_of(cfg->high)), 0.0);
        last = fmin(ceil(pair_of(cfg->low)), R - 1.0);
        if (!(last > first)) last = first + 0.001;
    }
    for (int i = 0; i < R / 2; ++i) {
        const double f = pow(base, -2.0 * i / R);
        double keep = 1.0;  // share of the unstretched frequency
        if (cfg->scaling == KVARN_ROPE_LINEAR) {
            keep = 0.0;
        } else if (cfg->scaling == KVARN_ROPE_BANDS) {
            keep = fmin(fmax((cfg->original_len * f / two_pi - cfg->low) / (cfg->high - cfg->low), 0.0), 1.0);
        } else if (cfg->scaling == KVARN_ROPE_YARN) {
            keep = 1.0 - fmin(fmax((i - first) / (last - first), 0.0), 1.0);
        }
        freqs[i] = keep * f + (1.0 - keep) * (f / s);
    }
    *rope_scale = cfg->scaling == KVARN_ROPE_YARN ? (float)(0.1 * log(s) + 1.0) : 1.0f;
    return ok();
}

namespace {

bool is_16bit(int t) { return t == KVARN_DTYPE_BF16 || t == KVARN_DTYPE_FP16; }

kvarn_status check_strides(const char* name, int64_t token, int64_t head, int multiple) {
    if (token < 0 || head < 0 || token % multiple != 0 || head % multiple != 0)
        return fail(KVARN_ERR_INVALID_ARG, "%s strides %lld, %lld: need non-negative multiples of %d", name,
                    (long long)token, (long long)head, multiple);
    return KVARN_OK;
}

kvarn_status check_cache(const void* k, const void* v, int64_t n_pages, int Hkv, int page_size, int64_t page_stride,
                         int64_t head_stride, int64_t token_stride, int multiple = 8) {
    if (page_size < 1 || n_pages < 1 || n_pages > 0x7fffffffLL / page_size)
        return fail(KVARN_ERR_INVALID_ARG, "n_pages = %lld, page_size = %d: need positive sizes and n_pages * page_size <= 2^31 - 1",
                    (long long)n_pages, page_size);
    KV_TRY(check_ptr(k, 16, "k_cache"));
    KV_TRY(check_ptr(v, 16, "v_cache"));
    // sorted by stride, each axis has to step over the whole of the axes below it
    struct Axis {
        int64_t stride, size;
    } ax[3] = {{page_stride, n_pages}, {head_stride, Hkv}, {token_stride, page_size}};
    for (int i = 0; i < 3; ++i)  // the stride of a single entry is never used
        if (ax[i].size > 1 && (ax[i].stride <= 0 || ax[i].stride % multiple != 0 || ax[i].stride > (1LL << 40)))
            return fail(KVARN_ERR_INVALID_ARG, "cache strides %lld, %lld, %lld: need positive multiples of %d up to 2^40",
                        (long long)page_stride, (long long)head_stride, (long long)token_stride, multiple);
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (ax[j].stride > ax[j + 1].stride || (ax[j].stride == ax[j + 1].stride && ax[j].size > ax[j + 1].size)) {
                const Axis t = ax[j];
                ax[j] = ax[j + 1];
                ax[j + 1] = t;
            }
    int64_t extent = KVARN_HEAD_DIM;
    for (int i = 0; i < 3; ++i) {
        if (ax[i].size == 1) continue;
        if (ax[i].stride < extent)
            return fail(KVARN_ERR_INVALID_ARG, "cache strides %lld, %lld, %lld: elements would coincide",
                        (long long)page_stride, (long long)head_stride, (long long)token_stride);
        if (ax[i].size - 1 > (1LL << 48) / ax[i].stride)
            return fail(KVARN_ERR_INVALID_ARG, "the cache spans more than 2^48 elements");
        extent += (ax[i].size - 1) * ax[i].stride;
    }
    return KVARN_OK;
}

}  // namespace

kvarn_status kvarn_rope_qkv(kvarn_dtype x_dtype, kvarn_dtype out_dtype, int n_tokens, int Hq, int Hkv,
                            const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                            const void* v, int64_t kv_token_stride, int64_t kv_head_stride,
                            const int32_t* positions, const double* inv_freq, int rot_dim,
                            int interleaved, float rope_scale, const float* q_weight,
                            const float* k_weight, float eps, void* q_out, int64_t qo_token_stride,
                            int64_t qo_head_stride, void* k_cache, void* v_cache, int64_t n_pages,
                            int page_size, int64_t page_stride, int64_t head_stride,
                            int64_t token_stride, const int32_t* slot_map, kvarn_stream_t stream) {
    if (!is_16bit(out_dtype)) return fail(KVARN_ERR_INVALID_ARG, "out_dtype = %d; expected bf16 or fp16", (int)out_dtype);
    if (x_dtype != out_dtype && x_dtype != KVARN_DTYPE_FP32)
        return fail(KVARN_ERR_INVALID_ARG, "x_dtype = %d; expected out_dtype (%d) or fp32", (int)x_dtype, (int)out_dtype);
    if (n_tokens < 0) return fail(KVARN_ERR_INVALID_ARG, "n_tokens = %d < 0", n_tokens);
    if (Hq < 0 || Hq > 65535 || Hkv < 0 || Hkv > 65535)
        return fail(KVARN_ERR_INVALID_ARG, "Hq = %d, Hkv = %d: allowed 0..65535", Hq, Hkv);
    if (rot_dim < 0 || rot_dim > KVARN_HEAD_DIM || rot_dim % 16 != 0)
        return fail(KVARN_ERR_INVALID_ARG, "rot_dim = %d; need a multiple of 16, 0..128", rot_dim);
    if (interleaved != 0 && interleaved != 1)
        return fail(KVARN_ERR_INVALID_ARG, "interleaved = %d; expected 0 or 1", interleaved);
    if (!isfinite(rope_scale)) return fail(KVARN_ERR_INVALID_ARG, "rope_scale is not finite");
    if (!(eps >= 0.f) || !isfinite(eps)) return fail(KVARN_ERR_INVALID_ARG, "eps = %g; need a finite eps >= 0", eps);
    if (n_tokens == 0 || (Hq == 0 && Hkv == 0)) return ok();
    KV_TRY(check_ptr(positions, 4, "positions"));
    if (rot_dim > 0) KV_TRY(check_ptr(inv_freq, 8, "inv_freq"));
    const int x_step = x_dtype == KVARN_DTYPE_FP32 ? 4 : 8;
    if (Hq > 0) {
        KV_TRY(check_ptr(q, 16, "q"));
        KV_TRY(check_ptr(q_out, 16, "q_out"));
        KV_TRY(check_strides("q", q_token_stride, q_head_stride, x_step));
        KV_TRY(check_strides("q_out", qo_token_stride, qo_head_stride, 8));
        if (q_weight) KV_TRY(check_ptr(q_weight, 16, "q_weight"));
        const int64_t lo = qo_token_stride < qo_head_stride ? qo_token_stride : qo_head_stride;
        const int64_t hi = qo_token_stride < qo_head_stride ? qo_head_stride : qo_token_stride;
        const int64_t n_lo = qo_token_stride < qo_head_stride ? n_tokens : Hq;
        const int64_t n_hi = qo_token_stride < qo_head_stride ? Hq : n_tokens;
        if ((n_lo > 1 && lo < KVARN_HEAD_DIM) || (n_hi > 1 && hi < (n_lo > 1 ? (n_lo - 1) * lo : 0) + KVARN_HEAD_DIM))
            return fail(KVARN_ERR_INVALID_ARG, "q_out strides %lld, %lld: rows would coincide",
                        (long long)qo_token_stride, (long long)qo_head_stride);
        if (q == q_out && (x_dtype != out_dtype || q_token_stride != qo_token_stride || q_head_stride != qo_head_stride))
            return fail(KVARN_ERR_INVALID_ARG, "q_out may be q only with its type and strides");
    }
    if (Hkv > 0) {
        KV_TRY(check_ptr(k, 16, "k"));
        KV_TRY(check_ptr(v, 16, "v"));
        KV_TRY(check_strides("k, v", kv_token_stride, kv_head_stride, x_step));
        KV_TRY(check_cache(k_cache, v_cache, n_pages, Hkv, page_size, page_stride, head_stride, token_stride));
        if (k_cache == v_cache) return fail(KVARN_ERR_INVALID_ARG, "k_cache and v_cache are the same array");
        if (k_weight) KV_TRY(check_ptr(k_weight, 16, "k_weight"));
        if (slot_map) KV_TRY(check_ptr(slot_map, 4, "slot_map"));
        else if (n_tokens > n_pages * page_size)
            return fail(KVARN_ERR_INVALID_ARG, "n_tokens = %d rows without a slot_map; the cache has %lld slots", n_tokens,
                        (long long)(n_pages * page_size));
    }
    kvarn::RopeArgs a;
    a.n_tokens = n_tokens;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.rot_dim = rot_dim;
    a.interleaved = interleaved;
    a.page_size = Hkv > 0 ? page_size : 1;
    a.n_slots = Hkv > 0 ? (int)(n_pages * page_size) : 0;
    a.passes = 0;
    a.rope_scale = rope_scale;
    a.eps = eps;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.kv_token_stride = kv_token_stride;
    a.kv_head_stride = kv_head_stride;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.q_out = q_out;
    a.qo_token_stride = qo_token_stride;
    a.qo_head_stride = qo_head_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_stride = page_stride;
    a.head_stride = head_stride;
    a.token_stride = token_stride;
    a.slot_map = slot_map;
    g_serving_used.store(true);
    cudaError_t e = kvarn::launch_rope_qkv(a, (int)x_dtype, (int)out_dtype, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "rope launch");
    return ok();
}

static kvarn_status check_softcap(float softcap) {
    // the reciprocal of a cap below the normal numbers may be infinite
    if (softcap != 0.f && (!(softcap >= FLT_MIN) || !isfinite(softcap)))
        return fail(KVARN_ERR_INVALID_ARG, "softcap = %g; need 0 or a finite cap of at least 2^-126", softcap);
    return KVARN_OK;
}

static kvarn_status check_paged_shape(int B, int Hq, int Hkv) {
    if (B < 0 || B > 65535) return fail(KVARN_ERR_INVALID_ARG, "B = %d outside 0..65535", B);
    if (Hq <= 0 || Hkv <= 0 || Hq > 65535 || Hq % Hkv != 0)
        return fail(KVARN_ERR_INVALID_ARG, "Hq = %d, Hkv = %d: need Hq a positive multiple of Hkv, up to 65535", Hq, Hkv);
    return KVARN_OK;
}

size_t kvarn_paged_attention_workspace_size(int B, int Hq, int Hkv) {
    if (check_paged_shape(B, Hq, Hkv) != KVARN_OK) return 0;
    return kvarn::paged_attention_workspace_bytes(B, Hq, Hkv);
}

static kvarn_status paged_impl(bool q8, const int8_t* k_exp, const int8_t* v_exp, kvarn_dtype dtype, int B, int Hq,
                               int Hkv, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                               const void* k_cache, const void* v_cache, int64_t n_pages, int page_size,
                               int64_t page_stride, int64_t head_stride, int64_t token_stride,
                               const int32_t* page_table, int max_pages, const int32_t* kv_lens,
                               const int32_t* kv_starts, int window, float softmax_scale, float softcap,
                               const float* slopes, void* workspace, size_t workspace_bytes, kvarn_dtype out_dtype,
                               void* out, float* lse, kvarn_stream_t stream) {
    KV_TRY(check_paged_shape(B, Hq, Hkv));
    if (!is_16bit(dtype)) return fail(KVARN_ERR_INVALID_ARG, "dtype = %d; expected bf16 or fp16", (int)dtype);
    if (out_dtype != KVARN_DTYPE_FP32 && out_dtype != dtype)
        return fail(KVARN_ERR_INVALID_ARG, "out_dtype = %d; expected fp32 or dtype (%d)", (int)out_dtype, (int)dtype);
    if (!isfinite(softmax_scale)) return fail(KVARN_ERR_INVALID_ARG, "softmax_scale is not finite");
    KV_TRY(check_softcap(softcap));
    if (window < 0) return fail(KVARN_ERR_INVALID_ARG, "window = %d < 0", window);
    if (page_size < 16 || page_size % 16 != 0)
        return fail(KVARN_ERR_INVALID_ARG, "page_size = %d; need a positive multiple of 16", page_size);
    if (max_pages < 1 || (int64_t)max_pages * page_size > 0x7fffffffLL - 63)
        return fail(KVARN_ERR_INVALID_ARG, "max_pages = %d: need at least 1 and max_pages * page_size <= 2^31 - 64", max_pages);
    if (B == 0) return ok();
    KV_TRY(check_ptr(q, 16, "q"));
    KV_TRY(check_strides("q", q_token_stride, q_head_stride, 8));
    KV_TRY(check_cache(k_cache, v_cache, n_pages, Hkv, page_size, page_stride, head_stride, token_stride, q8 ? 16 : 8));
    if (q8) {
        KV_TRY(check_ptr(k_exp, 16, "k_exp"));
        KV_TRY(check_ptr(v_exp, 16, "v_exp"));
    }
    KV_TRY(check_ptr(page_table, 4, "page_table"));
    KV_TRY(check_ptr(kv_lens, 4, "kv_lens"));
    if (kv_starts) KV_TRY(check_ptr(kv_starts, 4, "kv_starts"));
    if (slopes) KV_TRY(check_ptr(slopes, 4, "slopes"));
    KV_TRY(check_ptr(out, 16, "out"));
    if (lse) KV_TRY(check_ptr(lse, 4, "lse"));
    KV_TRY(check_ptr(workspace, 16, "workspace"));
    const size_t need = kvarn::paged_attention_workspace_bytes(B, Hq, Hkv);
    if (workspace_bytes < need)
        return fail(KVARN_ERR_WORKSPACE, "workspace_bytes = %zu < required %zu", workspace_bytes, need);
    kvarn::PagedAttnArgs a = {};
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.max_len = max_pages * page_size;
    a.window = window;
    a.out_dtype = (int)out_dtype;
    a.n_pages = n_pages;
    a.scale = softmax_scale;
    a.softcap = softcap;
    a.q = q;
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_stride = page_stride;
    a.head_stride = head_stride;
    a.token_stride = token_stride;
    a.k_exp = k_exp;
    a.v_exp = v_exp;
    a.page_table = page_table;
    a.kv_lens = kv_lens;
    a.kv_starts = kv_starts;
    a.slopes = slopes;
    a.workspace = workspace;
    a.out = out;
    a.lse = lse;
    g_serving_used.store(true);
    if (q8) g_q8_used.store(true);
    cudaError_t e = q8 ? kvarn::launch_paged_attention_q8(a, (int)dtype, (cudaStream_t)stream)
                       : kvarn::launch_paged_attention(a, (int)dtype, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
    return ok();
}

kvarn_status kvarn_paged_attention(kvarn_dtype dtype, int B, int Hq, int Hkv, const void* q, int64_t q_token_stride,
                                   int64_t q_head_stride, const void* k_cache, const void* v_cache, int64_t n_pages,
                                   int page_size, int64_t page_stride, int64_t head_stride, int64_t token_stride,
                                   const int32_t* page_table, int max_pages, const int32_t* kv_lens,
                                   const int32_t* kv_starts, int window, float softmax_scale, float softcap,
                                   const float* slopes, void* workspace, size_t workspace_bytes, kvarn_dtype out_dtype,
                                   void* out, float* lse, kvarn_stream_t stream) {
    return paged_impl(false, nullptr, nullptr, dtype, B, Hq, Hkv, q, q_token_stride, q_head_stride, k_cache, v_cache,
                      n_pages, page_size, page_stride, head_stride, token_stride, page_table, max_pages, kv_lens,
                      kv_starts, window, softmax_scale, softcap, slopes, workspace, workspace_bytes, out_dtype, out,
                      lse, stream);
}

kvarn_status kvarn_paged_attention_q8(kvarn_dtype dtype, int B, int Hq, int Hkv, const void* q, int64_t q_token_stride,
                                      int64_t q_head_stride, const void* k_cache, const void* v_cache,
                                      const int8_t* k_exp, const int8_t* v_exp, int64_t n_pages, int page_size,
                                      int64_t page_stride, int64_t head_stride, int64_t token_stride,
                                      const int32_t* page_table, int max_pages, const int32_t* kv_lens,
                                      const int32_t* kv_starts, int window, float softmax_scale, float softcap,
                                      const float* slopes, void* workspace, size_t workspace_bytes,
                                      kvarn_dtype out_dtype, void* out, float* lse, kvarn_stream_t stream) {
    return paged_impl(true, k_exp, v_exp, dtype, B, Hq, Hkv, q, q_token_stride, q_head_stride, k_cache, v_cache,
                      n_pages, page_size, page_stride, head_stride, token_stride, page_table, max_pages, kv_lens,
                      kv_starts, window, softmax_scale, softcap, slopes, workspace, workspace_bytes, out_dtype, out,
                      lse, stream);
}

kvarn_status kvarn_quantize_kv(kvarn_dtype x_dtype, int n_tokens, int Hkv, const void* k, const void* v,
                               int64_t kv_token_stride, int64_t kv_head_stride, void* k_cache, void* v_cache,
                               int64_t n_pages, int page_size, int64_t page_stride, int64_t head_stride,
                               int64_t token_stride, int8_t* k_exp, int8_t* v_exp, const int32_t* slot_map,
                               kvarn_stream_t stream) {
    if (!is_16bit(x_dtype) && x_dtype != KVARN_DTYPE_FP32)
        return fail(KVARN_ERR_INVALID_ARG, "x_dtype = %d; expected bf16, fp16 or fp32", (int)x_dtype);
    if (n_tokens < 0) return fail(KVARN_ERR_INVALID_ARG, "n_tokens = %d < 0", n_tokens);
    if (Hkv < 1 || Hkv > 65535) return fail(KVARN_ERR_INVALID_ARG, "Hkv = %d outside 1..65535", Hkv);
    if (n_tokens == 0) return ok();
    KV_TRY(check_ptr(k, 16, "k"));
    KV_TRY(check_ptr(v, 16, "v"));
    KV_TRY(check_strides("k, v", kv_token_stride, kv_head_stride, x_dtype == KVARN_DTYPE_FP32 ? 4 : 8));
    KV_TRY(check_cache(k_cache, v_cache, n_pages, Hkv, page_size, page_stride, head_stride, token_stride, 16));
    if (k_cache == v_cache) return fail(KVARN_ERR_INVALID_ARG, "k_cache and v_cache are the same array");
    KV_TRY(check_ptr(k_exp, 1, "k_exp"));
    KV_TRY(check_ptr(v_exp, 1, "v_exp"));
    if (k_exp == v_exp) return fail(KVARN_ERR_INVALID_ARG, "k_exp and v_exp are the same array");
    if (slot_map) KV_TRY(check_ptr(slot_map, 4, "slot_map"));
    else if (n_tokens > n_pages * page_size)
        return fail(KVARN_ERR_INVALID_ARG, "n_tokens = %d rows without a slot_map; the cache has %lld slots", n_tokens,
                    (long long)(n_pages * page_size));
    if ((int64_t)n_tokens * Hkv > (1LL << 30))
        return fail(KVARN_ERR_INVALID_ARG, "n_tokens = %d, Hkv = %d: need n_tokens * Hkv <= 2^30", n_tokens, Hkv);
    kvarn::QuantizeArgs a = {};
    a.n_tokens = n_tokens;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.n_slots = (int)(n_pages * page_size);
    a.k = k;
    a.v = v;
    a.kv_token_stride = kv_token_stride;
    a.kv_head_stride = kv_head_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_stride = page_stride;
    a.head_stride = head_stride;
    a.token_stride = token_stride;
    a.k_exp = k_exp;
    a.v_exp = v_exp;
    a.slot_map = slot_map;
    g_q8_used.store(true);
    cudaError_t e = kvarn::launch_quantize_kv(a, (int)x_dtype, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "quantize launch");
    return ok();
}

static kvarn_status check_prompt_shape(int64_t T, int Hq, int Hkv) {
    if (T < 0 || T > 0x7fffffffLL) return fail(KVARN_ERR_INVALID_ARG, "T = %lld outside 0..2^31 - 1", (long long)T);
    if (Hq <= 0 || Hkv <= 0 || Hq > 65535 || Hq % Hkv != 0)
        return fail(KVARN_ERR_INVALID_ARG, "Hq = %d, Hkv = %d: need Hq a positive multiple of Hkv, up to 65535", Hq, Hkv);
    if (T * (Hq / Hkv) > 0x7fffffffLL - 1023)
        return fail(KVARN_ERR_INVALID_ARG, "T = %lld: need T * Hq / Hkv <= 2^31 - 1024", (long long)T);
    return KVARN_OK;
}

// What kvarn_prompt_attention and kvarn_prefix_attention ask of the cache: the strides of a tiled copy.
static kvarn_status check_tiled_cache(const void* k, const void* v, int64_t n_pages, int Hkv, int page_size, int64_t page_stride,
                                      int64_t head_stride, int64_t token_stride) {
    if (page_size < 16 || page_size % 16 != 0)
        return fail(KVARN_ERR_INVALID_ARG, "page_size = %d; need a positive multiple of 16", page_size);
    KV_TRY(check_cache(k, v, n_pages, Hkv, page_size, page_stride, head_stride, token_stride));
    const int64_t most = 1LL << 38;
    if (token_stride > most || (Hkv > 1 && head_stride > most) || (n_pages > 1 && page_stride > most))
        return fail(KVARN_ERR_UNSUPPORTED, "cache strides %lld, %lld, %lld: allowed up to 2^38", (long long)page_stride,
                    (long long)head_stride, (long long)token_stride);
    return KVARN_OK;
}

size_t kvarn_prompt_attention_workspace_size(int64_t T, int Hq, int Hkv) {
    if (check_prompt_shape(T, Hq, Hkv) != KVARN_OK) return 0;
    return kvarn::prompt_attention_workspace_bytes(T, Hq, Hkv);
}

kvarn_status kvarn_prompt_attention(kvarn_dtype dtype, int B, int T, int Hq, int Hkv, const void* q, int64_t q_token_stride,
                                    int64_t q_head_stride, const void* k_cache, const void* v_cache, int64_t n_pages,
                                    int page_size, int64_t page_stride, int64_t head_stride, int64_t token_stride,
                                    const int32_t* page_table, int max_pages, const int32_t* cu_tokens,
                                    const int32_t* kv_lens, const int32_t* kv_starts, int causal, int window,
                                    float softmax_scale, float softcap, const float* slopes, void* workspace,
                                    size_t workspace_bytes, void* out, float* lse, kvarn_stream_t stream) {
    KV_TRY(check_prompt_shape(T, Hq, Hkv));
    if (B < 0 || B > kvarn::kMaxPromptSeqs)
        return fail(KVARN_ERR_INVALID_ARG, "B = %d outside 0..%d", B, kvarn::kMaxPromptSeqs);
    if (!is_16bit(dtype)) return fail(KVARN_ERR_INVALID_ARG, "dtype = %d; expected bf16 or fp16", (int)dtype);
    if (!isfinite(softmax_scale)) return fail(KVARN_ERR_INVALID_ARG, "softmax_scale is not finite");
    KV_TRY(check_softcap(softcap));
    if (causal != 0 && causal != 1) return fail(KVARN_ERR_INVALID_ARG, "causal = %d; expected 0 or 1", causal);
    if (window < 0) return fail(KVARN_ERR_INVALID_ARG, "window = %d < 0", window);
    if (!causal && window > 0) return fail(KVARN_ERR_INVALID_ARG, "window = %d: a window goes with causal = 1", window);
    if (!causal && slopes) return fail(KVARN_ERR_INVALID_ARG, "slopes go with causal = 1");
    if (max_pages < 1 || (int64_t)max_pages * page_size > 0x7fffffffLL - 255)
        return fail(KVARN_ERR_INVALID_ARG, "max_pages = %d: need at least 1 and max_pages * page_size <= 2^31 - 256", max_pages);
    if (B == 0 || T == 0) return ok();
    KV_TRY(check_ptr(q, 16, "q"));
    KV_TRY(check_strides("q", q_token_stride, q_head_stride, 8));
    KV_TRY(check_tiled_cache(k_cache, v_cache, n_pages, Hkv, page_size, page_stride, head_stride, token_stride));
    KV_TRY(check_ptr(page_table, 4, "page_table"));
    KV_TRY(check_ptr(cu_tokens, 4, "cu_tokens"));
    KV_TRY(check_ptr(kv_lens, 4, "kv_lens"));
    if (kv_starts) KV_TRY(check_ptr(kv_starts, 4, "kv_starts"));
    if (slopes) KV_TRY(check_ptr(slopes, 4, "slopes"));
    KV_TRY(check_ptr(out, 16, "out"));
    if (lse) KV_TRY(check_ptr(lse, 4, "lse"));
    KV_TRY(check_ptr(workspace, 16, "workspace"));
    const size_t need = kvarn::prompt_attention_workspace_bytes(T, Hq, Hkv);
    if (workspace_bytes < need)
        return fail(KVARN_ERR_WORKSPACE, "workspace_bytes = %zu < required %zu", workspace_bytes, need);
    kvarn::PromptArgs a = {};
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.max_len = max_pages * page_size;
    a.window = window < a.max_len ? window : 0;  // (a wider one hides nothing, and position + 1 - window keeps to 32 bits)
    a.causal = causal;
    a.n_pages = n_pages;
    a.scale = softmax_scale;
    a.softcap = softcap;
    a.q = q;
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_stride = page_stride;
    a.head_stride = head_stride;
    a.token_stride = token_stride;
    a.page_table = page_table;
    a.cu = cu_tokens;
    a.kv_lens = kv_lens;
    a.kv_starts = kv_starts;
    a.slopes = slopes;
    a.workspace = workspace;
    a.out = out;
    a.lse = lse;
    g_prompt_used.store(true);
    cudaError_t e = kvarn::launch_prompt_attention(a, (int)dtype, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "prompt attention launch");
    return ok();
}

namespace {

// Parts of kvarn_prefix_attention's workspace, one after the other.
struct PrefixWorkspace {
    size_t prompt, paged, out, lse, total;  // bytes of each
    PrefixWorkspace(int B, int Hq, int Hkv) {
        auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
        prompt = kvarn::prompt_attention_workspace_bytes(B, Hq, Hkv);
        paged = kvarn::paged_attention_workspace_bytes(B, Hq, Hkv);
        out = up((size_t)B * Hq * KVARN_HEAD_DIM * sizeof(float));
        lse = up((size_t)B * Hq * sizeof(float));
        total = prompt + paged + out + lse;
    }
};

}  // namespace

size_t kvarn_prefix_attention_workspace_size(int B, int Hq, int Hkv) {
    if (B > kvarn::kMaxPromptSeqs || check_paged_shape(B, Hq, Hkv) != KVARN_OK || check_prompt_shape(B, Hq, Hkv) != KVARN_OK) return 0;
    return PrefixWorkspace(B, Hq, Hkv).total;
}

kvarn_status kvarn_prefix_attention(kvarn_dtype dtype, int B, int n_groups, int Hq, int Hkv, const void* q,
                                    int64_t q_token_stride, int64_t q_head_stride, const void* k_cache,
                                    const void* v_cache, int64_t n_pages, int page_size, int64_t page_stride,
                                    int64_t head_stride, int64_t token_stride, const int32_t* prefix_table,
                                    int max_prefix_pages, const int32_t* prefix_lens, const int32_t* cu_seqs,
                                    const int32_t* page_table, int max_pages, const int32_t* kv_lens,
                                    float softmax_scale, float softcap, void* workspace, size_t workspace_bytes,
                                    void* out, float* lse, kvarn_stream_t stream) {
    KV_TRY(check_paged_shape(B, Hq, Hkv));
    KV_TRY(check_prompt_shape(B, Hq, Hkv));
    if (B > kvarn::kMaxPromptSeqs) return fail(KVARN_ERR_INVALID_ARG, "B = %d outside 0..%d", B, kvarn::kMaxPromptSeqs);
    if (n_groups < 0 || n_groups > kvarn::kMaxPromptSeqs)
        return fail(KVARN_ERR_INVALID_ARG, "n_groups = %d outside 0..%d", n_groups, kvarn::kMaxPromptSeqs);
    if (!is_16bit(dtype)) return fail(KVARN_ERR_INVALID_ARG, "dtype = %d; expected bf16 or fp16", (int)dtype);
    if (!isfinite(softmax_scale)) return fail(KVARN_ERR_INVALID_ARG, "softmax_scale is not finite");
    KV_TRY(check_softcap(softcap));
    const struct {
        int pages;
        const char* name;
    } widths[] = {{max_prefix_pages, "max_prefix_pages"}, {max_pages, "max_pages"}};
    for (const auto& w : widths)
        if (w.pages < 1 || (int64_t)w.pages * page_size > 0x7fffffffLL - 255)
            return fail(KVARN_ERR_INVALID_ARG, "%s = %d: need at least 1 and %s * page_size <= 2^31 - 256", w.name, w.pages, w.name);
    if (B == 0) return ok();
    KV_TRY(check_ptr(q, 16, "q"));
    KV_TRY(check_strides("q", q_token_stride, q_head_stride, 8));
    KV_TRY(check_tiled_cache(k_cache, v_cache, n_pages, Hkv, page_size, page_stride, head_stride, token_stride));
    if (n_groups > 0) {
        KV_TRY(check_ptr(prefix_table, 4, "prefix_table"));
        KV_TRY(check_ptr(prefix_lens, 4, "prefix_lens"));
        KV_TRY(check_ptr(cu_seqs, 4, "cu_seqs"));
    }
    KV_TRY(check_ptr(page_table, 4, "page_table"));
    KV_TRY(check_ptr(kv_lens, 4, "kv_lens"));
    KV_TRY(check_ptr(out, 16, "out"));
    if (lse) KV_TRY(check_ptr(lse, 4, "lse"));
    KV_TRY(check_ptr(workspace, 16, "workspace"));
    const PrefixWorkspace need(B, Hq, Hkv);
    if (workspace_bytes < need.total)
        return fail(KVARN_ERR_WORKSPACE, "workspace_bytes = %zu < required %zu", workspace_bytes, need.total);
    uint8_t* at = static_cast<uint8_t*>(workspace);
    kvarn::PromptArgs p = {};
    p.B = n_groups;
    p.T = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.page_size = page_size;
    p.max_pages = max_prefix_pages;
    p.max_len = max_prefix_pages * page_size;
    p.n_pages = n_pages;
    p.scale = softmax_scale;
    p.softcap = softcap;
    p.q = q;
    p.q_token_stride = q_token_stride;
    p.q_head_stride = q_head_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.page_stride = page_stride;
    p.head_stride = head_stride;
    p.token_stride = token_stride;
    p.page_table = prefix_table;
    p.cu = cu_seqs;
    p.kv_lens = prefix_lens;
    kvarn::PagedAttnArgs a = {};
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.max_len = max_pages * page_size;
    a.out_dtype = KVARN_DTYPE_FP32;
    a.n_pages = n_pages;
    a.scale = softmax_scale;
    a.softcap = softcap;
    a.q = q;
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_stride = page_stride;
    a.head_stride = head_stride;
    a.token_stride = token_stride;
    a.page_table = page_table;
    a.kv_lens = kv_lens;
    // the sequences' own tokens first; the prefixes' part is joined with that
    a.workspace = at + need.prompt;
    if (n_groups == 0) {
        a.out_dtype = (int)dtype;
        a.out = out;
        a.lse = lse;
    } else {
        a.out_dtype = KVARN_DTYPE_FP32;
        a.out = at + need.prompt + need.paged;
        a.lse = reinterpret_cast<float*>(at + need.prompt + need.paged + need.out);
    }
    p.own_out = static_cast<const float*>(a.out);
    p.own_lse = a.lse;
    p.workspace = at;
    p.out = out;
    p.lse = lse;
    g_serving_used.store(true);
    g_prompt_used.store(true);
    cudaError_t e = kvarn::launch_paged_attention(a, (int)dtype, (cudaStream_t)stream);
    if (e == cudaSuccess && n_groups > 0) e = kvarn::launch_prompt_attention(p, (int)dtype, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "prefix attention launch");
    return ok();
}

const char* kvarn_status_string(kvarn_status status) {
    switch (status) {
        case KVARN_OK: return "KVARN_OK";
        case KVARN_ERR_INVALID_ARG: return "KVARN_ERR_INVALID_ARG: an argument is out of range";
        case KVARN_ERR_UNSUPPORTED: return "KVARN_ERR_UNSUPPORTED: valid but not implemented";
        case KVARN_ERR_CUDA: return "KVARN_ERR_CUDA: a CUDA call or kernel launch failed";
        case KVARN_ERR_WORKSPACE: return "KVARN_ERR_WORKSPACE: workspace too small";
        case KVARN_ERR_TIMEOUT: return "KVARN_ERR_TIMEOUT: a bounded device wait gave up";
    }
    return "unknown kvarn_status";
}

const char* kvarn_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
