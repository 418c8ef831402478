// Per-head RMS norm and position rotation of a step's queries and keys, with the write of keys and
// values into the paged cache, in one pass.
//
// Mathematics, per token and head x[128] (fp32 from the load to the one rounding at the store):
//   y = x w / sqrt(mean(x^2) + eps) (only with a weight w), then over the first R channels, in pairs
//   (a, b) = (i, i + R/2) or (2i, 2i + 1):  y_a' = s (y_a cos t - y_b sin t),
//   y_b' = s (y_b cos t + y_a sin t),  t = position * f_i.
// The angle is reduced exactly: F = 2^64 f / 2 pi mod 2^64 is the frequency as a fraction of a turn, and
// position * F mod 2^64 is the fraction of the turn that is left, off by at most 2^31 * 2^-63 turns at
// any position; an fp32 product would be off by 0.06 radians at position 10^6.  F comes from the
// frequency's bits by one 64 x 64 bit product (fp64 runs at 2 operations per SM and clock here: 1.3 us
// for a step of 256 tokens).  cos and sin of that fraction are then taken in fp32.
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

__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
__device__ __forceinline__ uint32_t pack2(float2 v, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float2 v, __half) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 neighbouring channels of a row, as loaded
template <typename X>
struct Raw8 {
    uint4 u;
    __device__ __forceinline__ void load(const X* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        f[0] = unpack2(u.x, X());
        f[1] = unpack2(u.y, X());
        f[2] = unpack2(u.z, X());
        f[3] = unpack2(u.w, X());
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
        f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
    }
};

template <typename O>
__device__ __forceinline__ void store8(O* p, const float2 (&f)[4]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], O()), pack2(f[1], O()), pack2(f[2], O()), pack2(f[3], O()));
}

// 2^64 f / 2 pi mod 2^64, truncated: f = m 2^e with a 53-bit m, and 1 / 2 pi = c 2^-66 with c = 2^64 (2 / pi).
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f), c = 0xa2f9836e4e44152aull;
    const int ex = (int)(bits >> 52) & 0x7ff;
    const unsigned long long m = (bits & ((1ull << 52) - 1)) | (ex > 0 ? 1ull << 52 : 0ull);
    const unsigned long long hi = __umul64hi(m, c), lo = m * c;
    const int down = 2 - ((ex > 0 ? ex : 1) - 1075);  // m c 2^(64 - 66 + e)
    unsigned long long r;
    if (down >= 64) r = down < 128 ? hi >> (down - 64) : 0ull;
    else if (down > 0) r = (hi << (64 - down)) | (lo >> down);
    else r = down > -64 ? lo << -down : 0ull;
    return (long long)bits < 0 ? 0ull - r : r;
}

// X: type of q, k, v; O: type of q_out and the cache.  A warp takes a.passes times four of the
// Hq + 2 Hkv rows of a token and works alone; a token is a.slices warps.
template <typename X, typename O, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_qkv_kernel(RopeArgs a) {
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
        const unsigned long long at = turn_fraction(a.inv_freq[p]) * (unsigned long long)(unsigned)pos;
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

    // this lane's 8 pairs, kept in registers: from shared memory in every pass, 64 bytes apart, they
    // were the bound (85% of the L1 rate, three quarters of it bank conflicts)
    float2 cs[4], sn[4];  // of neighbouring pairs
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cs[i] = sn[i] = make_float2(0.f, 0.f);
        if (turned) {
            const float2 c = s_turn[warp][8 * j + 2 * i], d = s_turn[warp][8 * j + 2 * i + 1];
            cs[i] = make_float2(c.x, d.x);
            sn[i] = make_float2(c.y, d.y);
        }
    }
    float2 wa[4], wb[4];  // and its weights, of the queries' or the keys' norm
    const float* held = nullptr;

    for (int pass = 0; pass < a.passes; ++pass, r += 4) {
        Raw8<X> na = {}, nb = {};  // the next four rows
        if (pass + 1 < a.passes) load(r + 4, na, nb);
        float2 fa[4], fb[4];
        ra.get(fa);
        rb.get(fb);
        ra = na, rb = nb;
        const bool is_q = r < a.Hq, is_k = !is_q && r < a.Hq + a.Hkv;
        const float* w = is_q ? a.q_weight : is_k ? a.k_weight : nullptr;
        float2 sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) sq = ffma2(fa[i], fa[i], ffma2(fb[i], fb[i], sq));
        float sum = sq.x + sq.y;
#pragma unroll
        for (int s = 1; s < 8; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        O* dst = nullptr;
        if (is_q) dst = qo + r * a.qo_head_stride;
        else if (is_k) dst = kdst != nullptr ? kdst + (r - a.Hq) * a.head_stride : nullptr;
        else if (r < rows) dst = vdst != nullptr ? vdst + (r - a.Hq - a.Hkv) * a.head_stride : nullptr;
        if (dst == nullptr) continue;
        if (w != nullptr) {
            if (w != held) {
                held = w;
                Raw8<float> t8;
                t8.load(w + ca);
                t8.get(wa);
                t8.load(w + cb);
                t8.get(wb);
            }
            const float inv = rsqrtf(sum * (1.0f / kTile) + a.eps);
            const float2 inv2 = make_float2(inv, inv);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fa[i] = fmul2(fa[i], fmul2(inv2, wa[i]));
                fb[i] = fmul2(fb[i], fmul2(inv2, wb[i]));
            }
        }
        if (turned && (is_q || is_k)) {
            if (INTERLEAVED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // pairs 8 j + i of the first piece and 8 j + 4 + i of the second
                    const float c = i & 1 ? cs[i / 2].y : cs[i / 2].x, n = i & 1 ? sn[i / 2].y : sn[i / 2].x;
                    const float d = i & 1 ? cs[i / 2 + 2].y : cs[i / 2 + 2].x, e = i & 1 ? sn[i / 2 + 2].y : sn[i / 2 + 2].x;
                    fa[i] = make_float2(fa[i].x * c - fa[i].y * n, fa[i].y * c + fa[i].x * n);
                    fb[i] = make_float2(fb[i].x * d - fb[i].y * e, fb[i].y * d + fb[i].x * e);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = fa[i], y = fb[i];
                    fa[i] = ffma2(x, cs[i], fmul2(y, make_float2(-sn[i].x, -sn[i].y)));
                    fb[i] = ffma2(y, cs[i], fmul2(x, sn[i]));
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
