// Keys and values of new tokens into a paged 8-bit cache: E4M3 values times a power of two for each token and head.
//
// Mathematics, per token and head, over the row's 128 channels: e = ceil(log2(max |x| / 448)) (448: E4M3's largest),
// at least -127, and code = round(x / 2^e) to E4M3, to nearest, ties to even.  x / 2^e is exact, so a code is off by
// that one rounding, and the same inputs give the same codes everywhere.
//
// What bounds it: 256 bytes read and 129 written per row (16-bit inputs): HBM.  Half a warp takes a row, 16 bytes a
// lane, so that the maximum takes four shuffles and a store is 8 bytes a lane of one row, and has kAhead rows in flight;
// they stay packed until they are used (unpacked at the load they took 26.4 us below, kept packed 20.4).  A warp does its
// rows and ends: a grid of resident CTAs that loops took 27.8 us.
//
// Measured: 16384 tokens of 8 heads, bf16, 101 MB: 20.4 us (4.9 TB/s; kAhead 2: 21.9); 64 tokens 2.9 us.
#include <type_traits>

#include "kvarn_common.cuh"
#include "kvarn_internal.h"

namespace kvarn {

// Set when a slot lies outside the cache.  Read by kvarn_device_error.
__device__ unsigned int g_quantize_error = 0;

namespace {

constexpr int kWarps = 4;
constexpr int kAhead = 4;  // rows that half a warp loads at once

// eight neighbouring channels, as they lie in memory until they are used
template <typename T>
struct Eight {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                const uint32_t w[4] = {v[i >> 1].x, v[i >> 1].y, v[i >> 1].z, v[i >> 1].w};
                x[2 * i] = __uint_as_float(w[2 * (i & 1)]), x[2 * i + 1] = __uint_as_float(w[2 * (i & 1) + 1]);
            } else {
                const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
                if constexpr (std::is_same<T, __half>::value) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                    x[2 * i] = f.x, x[2 * i + 1] = f.y;
                } else {
                    x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            }
        }
    }
};

// Rows in the order (token, keys or values, head).
template <typename T>
__global__ void __launch_bounds__(32 * kWarps, 10) quantize_kv_kernel(QuantizeArgs a) {
    const int lane = threadIdx.x & 31, part = lane & 15;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const unsigned first = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * (2 * kAhead) + (lane >> 4), per_token = 2u * a.Hkv;
    unsigned token = first / per_token, r = first - token * per_token;  // the only division; the other rows go on from there
    Eight<T> in[kAhead];
    int slot[kAhead], kind[kAhead], head[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        slot[i] = -1;
        if (first + 2 * i < a.n_rows) {
            kind[i] = r >= (unsigned)a.Hkv;
            head[i] = (int)r - (kind[i] ? a.Hkv : 0);
            slot[i] = a.slot_map != nullptr ? __ldg(a.slot_map + token) : (int)token;
            in[i].load(static_cast<const T*>(kind[i] ? a.v : a.k) + (int64_t)token * a.kv_token_stride + (int64_t)head[i] * a.kv_head_stride + 8 * part);
        }
        r += 2;
        if (r >= per_token) r -= per_token, ++token;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        float top = 0.f, x[8];
        in[i].values(x);
#pragma unroll
        for (int c = 0; c < 8; ++c) top = fmaxf(top, fabsf(x[c]));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (slot[i] < 0 || slot[i] >= a.n_slots) {
            if (slot[i] != -1 && part == 0) atomicOr(&g_quantize_error, 1u);
            continue;
        }
        // top = 1.f 2^E, 448 = 1.75 2^8
        const uint32_t bits = __float_as_uint(top);
        const int e = max((int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), -127);
        const float scale = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h] * scale, x[4 * h + 1] * scale), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h + 2] * scale, x[4 * h + 3] * scale), __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | hi << 16;
        }
        const int page = a.page_shift >= 0 ? slot[i] >> a.page_shift : slot[i] / a.page_size, in_page = slot[i] - page * a.page_size;
        uint8_t* dst = static_cast<uint8_t*>(kind[i] ? a.v_cache : a.k_cache) + (int64_t)page * a.page_stride +
                       (int64_t)head[i] * a.head_stride + (int64_t)in_page * a.token_stride;
        *reinterpret_cast<uint2*>(dst + 8 * part) = make_uint2(w[0], w[1]);
        if (part == 0) (kind[i] ? a.v_exp : a.k_exp)[((int64_t)page * a.Hkv + head[i]) * a.page_size + in_page] = (int8_t)e;
    }
}

}  // namespace

cudaError_t read_and_clear_quantize_error(unsigned int* out) { return read_and_clear_word(&g_quantize_error, out); }

cudaError_t launch_quantize_kv(QuantizeArgs a, int x_dtype, cudaStream_t stream) {
    a.n_rows = (unsigned)a.n_tokens * 2u * (unsigned)a.Hkv;
    a.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz((unsigned)a.page_size) : -1;
    const unsigned ctas = (a.n_rows + kWarps * 2 * kAhead - 1) / (kWarps * 2 * kAhead);
    const auto kern = x_dtype == KVARN_DTYPE_FP32 ? quantize_kv_kernel<float>
                      : x_dtype == KVARN_DTYPE_FP16 ? quantize_kv_kernel<__half> : quantize_kv_kernel<__nv_bfloat16>;
    return launch_pdl(kern, dim3(ctas), dim3(32 * kWarps), 0, stream, a);
}

}  // namespace kvarn
