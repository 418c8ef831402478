// Per-head RMS norm and position rotation of a step's queries and keys, with the write of keys and
// values into the paged cache, in one pass.
//
// Mathematics, per token and head x[128] (fp32 from the load to the one rounding at the store):
//   y = x w / sqrt(mean(x^2) + eps) (only with a weight w), then over the first R channels, in pairs
//   (a, b) = (i, i + R/2) or (2i, 2i + 1):  y_a' = s (y_a cos t - y_b sin t),
//   y_b' = s (y_b cos t + y_a sin t),  t = position * f_i.
// The angle is reduced exactly: F = round(2^64 f / 2 pi) is the frequency as a fraction of a turn, and
// position * F mod 2^64 is the fraction of the turn that is left, off by at most 2^31 * 2^-65 turns
// (plus the 2^-53 of the fp64 frequency itself) at any position; an fp32 product would be off by 0.06
// radians at position 10^6.  cos and sin of that fraction are then taken in fp32.
//
// What bounds it: every element is read and written once and nothing is read again, so HBM for
// chunks of thousands of tokens and launch latency for a decode step.  Eight lanes hold a head, two
// 16-byte pieces each, chosen so that both channels of every pair are in the same lane in either
// layout: no element is exchanged between lanes, only the three shuffles of the sum of squares.
#include "kvarn_common.cuh"
#include "kvarn_internal.h"

namespace kvarn {

// Set when a slot of the slot map lies outside the cache (that row's key and value are not
// written).  Read by kvarn_device_error.
__device__ unsigned int g_rope_error = 0;

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHalf = kTile / 2;  // most pairs a head has

// 8 consecutive channels of a row, as fp32
__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b, __nv_bfloat16) {
    a = __uint_as_float(u << 16);
    b = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    a = f.x;
    b = f.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename X>
struct Raw8 {  // 8 channels as loaded
    uint4 u;
    __device__ __forceinline__ void load(const X* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        unpack2(u.x, f[0], f[1], X());
        unpack2(u.y, f[2], f[3], X());
        unpack2(u.z, f[4], f[5], X());
        unpack2(u.w, f[6], f[7], X());
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};

template <typename O>
__device__ __forceinline__ void store8(O* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1], O()), pack2(f[2], f[3], O()),
                                              pack2(f[4], f[5], O()), pack2(f[6], f[7], O()));
}

// X: type of q, k, v; O: type of q_out and the cache.  A warp takes a.passes times four of the
// Hq + 2 Hkv rows of a token and works alone; a token is a.slices warps.
template <typename X, typename O, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 7) rope_qkv_kernel(RopeArgs a) {
    __shared__ float2 s_turn[kWarps][kHalf];  // (cos, sin) * rope_scale of the warp's token
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned id = blockIdx.x * kWarps + warp;
    const int t = (int)(id / (unsigned)a.slices), slice = (int)(id - (unsigned)t * (unsigned)a.slices);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= a.n_tokens) return;
    const int rows = a.Hq + 2 * a.Hkv, pairs = a.rot_dim >> 1;
    const int sub = lane >> 3, j = lane & 7;
    const bool turned = j < (a.rot_dim >> 4);
    const int ca = 8 * (INTERLEAVED || !turned ? 2 * j : j);
    const int cb = INTERLEAVED || !turned ? ca + 8 : ca + pairs;
    const X* q = static_cast<const X*>(a.q) + t * a.q_token_stride;
    const X* k = static_cast<const X*>(a.k) + t * a.kv_token_stride;
    const X* v = static_cast<const X*>(a.v) + t * a.kv_token_stride;
    O* qo = static_cast<O*>(a.q_out) + t * a.qo_token_stride;

    auto load = [&](int r, Raw8<X>& ra, Raw8<X>& rb) {
        if (r >= rows) return;
        const X* src = r < a.Hq           ? q + r * a.q_head_stride
                       : r < a.Hq + a.Hkv ? k + (r - a.Hq) * a.kv_head_stride
                                          : v + (r - a.Hq - a.Hkv) * a.kv_head_stride;
        ra.load(src + ca);
        rb.load(src + cb);
    };
    // the first rows are on their way while the angles are made
    int r = 4 * slice * a.passes + sub;
    Raw8<X> ra = {}, rb = {};
    load(r, ra, rb);
    const int pos = a.positions[t];
    const int slot = a.Hkv == 0 ? -1 : a.slot_map != nullptr ? a.slot_map[t] : t;
    if (pos < 0) return;  // a padding row: nothing of it is written
    for (int p = lane; p < pairs; p += 32) {
        // 2^64 f / 2 pi modulo 2^64: whole turns per position drop out
        const double turns = a.inv_freq[p] * 0.15915494309189533577;
        const double frac = turns - floor(turns);
        const unsigned long long F = __double2ull_rn(frac * 18446744073709551616.0);
        const unsigned long long at = F * (unsigned long long)(unsigned)pos;
        // nearest fraction of a turn in [-1/2, 1/2), as half turns for sincospif
        const float half_turns = (float)(int)((at + 0x80000000ull) >> 32) * 4.656612873077393e-10f;
        float sn, cs;
        sincospif(half_turns, &sn, &cs);
        s_turn[warp][p] = make_float2(cs * a.rope_scale, sn * a.rope_scale);
    }
    O* kdst = nullptr;
    O* vdst = nullptr;
    if (slot >= 0 && slot < a.n_slots) {
        const int page = slot / a.page_size, off = slot - page * a.page_size;
        const int64_t o = page * a.page_stride + off * a.token_stride;
        kdst = static_cast<O*>(a.k_cache) + o;
        vdst = static_cast<O*>(a.v_cache) + o;
    } else if (slot >= 0 && lane == 0) {
        atomicOr(&g_rope_error, 1u);
    }
    __syncwarp();

    for (int pass = 0; pass < a.passes; ++pass, r += 4) {
        Raw8<X> na = {}, nb = {};  // the next four rows
        if (pass + 1 < a.passes) load(r + 4, na, nb);
        float fa[8], fb[8];
        ra.get(fa);
        rb.get(fb);
        ra = na, rb = nb;
        const bool is_q = r < a.Hq, is_k = !is_q && r < a.Hq + a.Hkv;
        const float* w = is_q ? a.q_weight : is_k ? a.k_weight : nullptr;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(fa[i], fa[i], fmaf(fb[i], fb[i], sq));
#pragma unroll
        for (int s = 1; s < 8; s <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, s);
        O* dst = nullptr;
        if (is_q) dst = qo + r * a.qo_head_stride;
        else if (is_k) dst = kdst != nullptr ? kdst + (r - a.Hq) * a.head_stride : nullptr;
        else if (r < rows) dst = vdst != nullptr ? vdst + (r - a.Hq - a.Hkv) * a.head_stride : nullptr;
        if (dst == nullptr) continue;
        if (w != nullptr) {
            const float inv = 1.0f / sqrtf(sq * (1.0f / kTile) + a.eps);
            float wa[8], wb[8];
            Raw8<float> t8;
            t8.load(w + ca);
            t8.get(wa);
            t8.load(w + cb);
            t8.get(wb);
#pragma unroll
            for (int i = 0; i < 8; ++i) fa[i] *= inv * wa[i], fb[i] *= inv * wb[i];
        }
        if (turned && (is_q || is_k)) {
            const float2* cs = &s_turn[warp][8 * j];
            if (INTERLEAVED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 c = cs[i], d = cs[i + 4];
                    const float x = fa[2 * i], y = fa[2 * i + 1], z = fb[2 * i], u = fb[2 * i + 1];
                    fa[2 * i] = x * c.x - y * c.y;
                    fa[2 * i + 1] = y * c.x + x * c.y;
                    fb[2 * i] = z * d.x - u * d.y;
                    fb[2 * i + 1] = u * d.x + z * d.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 c = cs[i];
                    const float x = fa[i], y = fb[i];
                    fa[i] = x * c.x - y * c.y;
                    fb[i] = y * c.x + x * c.y;
                }
            }
        }
        store8(dst + ca, fa);
        store8(dst + cb, fb);
    }
}

template <typename X, typename O>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    const cudaError_t e = current_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    // a warp takes the whole token once there are tokens enough for 28 warps on every SM, so that the
    // angles are made once; with fewer, a token is spread over more warps
    const int quads = (a.Hq + 2 * a.Hkv + 3) / 4;
    const int64_t passes = (int64_t)a.n_tokens * quads / (28 * (int64_t)sms);
    a.passes = (int)(passes < 1 ? 1 : passes < quads ? passes : quads);
    a.slices = (quads + a.passes - 1) / a.passes;
    a.passes = (quads + a.slices - 1) / a.slices;
    const int64_t warps = (int64_t)a.n_tokens * a.slices;
    const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps));
    return a.interleaved ? launch_pdl(rope_qkv_kernel<X, O, true>, grid, dim3(kThreads), 0, stream, a)
                         : launch_pdl(rope_qkv_kernel<X, O, false>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t read_and_clear_rope_error(unsigned int* out) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(v));
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

cudaError_t launch_rope_qkv(const RopeArgs& a, int x_dtype, int out_dtype, cudaStream_t stream) {
    if (out_dtype == KVARN_DTYPE_BF16)
        return x_dtype == KVARN_DTYPE_FP32 ? launch<float, __nv_bfloat16>(a, stream)
                                           : launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
    return x_dtype == KVARN_DTYPE_FP32 ? launch<float, __half>(a, stream) : launch<__half, __half>(a, stream);
}

}  // namespace kvarn
