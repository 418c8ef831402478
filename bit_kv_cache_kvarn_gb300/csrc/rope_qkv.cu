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
// chunks of thousands of tokens and launch latency for a decode step.  Rows come into a ring in shared
// memory that each warp fills and reads alone; from there eight lanes hold a row, two runs of eight
// channels each, chosen so that both channels of every pair are in the same lane in either layout: past
// the ring the lanes of a row exchange nothing but the three shuffles of the sum of squares.
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

// Channels c .. c + 7 of a row in shared memory, whose 16-byte piece p lies at p ^ (p / 8 mod 4).
template <typename X>
__device__ __forceinline__ void take8(const uint4* row, int c, float2 (&f)[4]) {
    const int p = c * (int)sizeof(X) / 16;
    const uint4 u = row[p ^ ((p >> 3) & 3)];
    if constexpr (sizeof(X) == 2) {
        f[0] = unpack2(u.x, X());
        f[1] = unpack2(u.y, X());
        f[2] = unpack2(u.z, X());
        f[3] = unpack2(u.w, X());
    } else {
        const uint4 w = row[(p + 1) ^ ((p >> 3) & 3)];
        f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
        f[2] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        f[3] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
}
__device__ __forceinline__ void load8(const float* p, float2 (&f)[4]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
}

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

// X: type of q, k, v; O: type of q_out and the cache; SHARE: warps that share a token and its angles.  A
// warp takes a.passes times four of a token's Hq + 2 Hkv rows.
template <typename X, typename O, int SHARE, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 4) rope_qkv_kernel(RopeArgs a) {
    constexpr int kDepth = sizeof(X) == 4 ? 3 : 4;     // passes in flight per warp
    constexpr int kPieces = kTile * sizeof(X) / 16;  // 16-byte pieces of a row; piece p lies at p ^ (p / 8 mod 4),
                                                     // so that the lanes of a row never meet in a bank
    __shared__ float2 s_turns[kWarps / SHARE][kHalf];  // (cos, sin) * rope_scale of the tokens
    __shared__ uint4 s_raw[kWarps][kDepth][4][kPieces];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2* s_turn = s_turns[warp / SHARE];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // this warp's (or CTA's) tokens: every `stride`th; grid.y: the slices of a token
    const unsigned n_tokens = (unsigned)a.n_tokens, stride = gridDim.x * (kWarps / SHARE);
    unsigned t = blockIdx.x * (kWarps / SHARE) + warp / SHARE;
    if (t >= n_tokens) return;  // SHARE > 1: the whole CTA
    const int rows = a.Hq + 2 * a.Hkv, pairs = a.rot_dim >> 1;
    const int sub = lane >> 3, j = lane & 7;
    const bool turned = j < (a.rot_dim >> 4);
    const int ca = 8 * (INTERLEAVED || !turned ? 2 * j : j);
    const int cb = INTERLEAVED || !turned ? ca + 8 : ca + pairs;
    constexpr int kStep = 4 * SHARE;  // rows from one pass to the next

    // Rows come through a ring in shared memory that each warp fills and reads alone; kept in registers,
    // passes ahead would cost the warps that the rate needs.  The copies go along the row: with each lane
    // copying its own pieces, the interleaved layout and fp32 took half sectors, and twice the L2 traffic.
    // Addresses are carried from pass to pass inside a section (queries, keys, values): made anew for
    // each row they were half of the kernel's instructions.
    constexpr uint32_t kEntry = sizeof(s_raw[0][0]);
    const uint32_t ring = smem_addr(s_raw[warp][0][sub]);
    const int first_row = SHARE == 1 ? sub : 4 * ((int)blockIdx.y * a.passes * SHARE + warp % SHARE) + sub;
    unsigned in_t = t;
    int in_pass = 0, in_row = first_row, in_end = 0;
    const uint4* src = nullptr;
    int64_t src_step = 0;
    uint32_t in_at = 0;
    auto load = [&]() {
        if (in_t < n_tokens) {
            if (in_row >= in_end && in_row < rows) {  // the first row, or one of another section
                const X* p;
                int64_t head = a.kv_head_stride;
                if (in_row < a.Hq) {
                    head = a.q_head_stride, in_end = a.Hq;
                    p = static_cast<const X*>(a.q) + in_t * a.q_token_stride + in_row * head;
                } else {
                    const bool key = in_row < a.Hq + a.Hkv;
                    const int h = in_row - (key ? a.Hq : a.Hq + a.Hkv);
                    in_end = key ? a.Hq + a.Hkv : rows;
                    p = static_cast<const X*>(key ? a.k : a.v) + in_t * a.kv_token_stride + h * head;
                }
                src = reinterpret_cast<const uint4*>(p) + j;
                src_step = kStep * head * (int64_t)sizeof(X) / 16;
            }
            if (in_row < rows) {
#pragma unroll
                for (int i = 0; i < kPieces / 8; ++i)
                    cp_async16(ring + in_at + 16 * ((j + 8 * i) ^ (i & 3)), src + 8 * i, true);
            }
            src += src_step;
            in_row += kStep;
            if (++in_pass == a.passes) {  // on to the next token: the ring does not run dry between them
                in_t += stride;
                in_pass = 0, in_row = first_row, in_end = 0;
            }
        }
        in_at = in_at + kEntry < kDepth * kEntry ? in_at + kEntry : 0;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i) load();  // on their way while the angles are made
    const uint4* entry = s_raw[warp][0][sub];
    int out_at = 0;
    int pos = a.positions[t], slot = a.Hkv == 0 ? -1 : a.slot_map != nullptr ? a.slot_map[t] : (int)t;

    constexpr int kPairs = kHalf / (32 * SHARE) > 0 ? kHalf / (32 * SHARE) : 1;  // of a lane, to make angles for
    unsigned long long freq[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int p = lane + 32 * (warp % SHARE + SHARE * i);
        freq[i] = p < pairs ? turn_fraction(a.inv_freq[p]) : 0;
    }

    for (;;) {
        // the next token's position and slot come while this one is turned
        const unsigned next = t + stride;
        int next_pos = 0, next_slot = 0;
        if (next < n_tokens) {
            next_pos = a.positions[next];
            next_slot = a.Hkv == 0 ? -1 : a.slot_map != nullptr ? a.slot_map[next] : (int)next;
        }
        const bool padding = pos < 0;  // nothing of the row is written
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int p = lane + 32 * (warp % SHARE + SHARE * i);
            const unsigned long long at = freq[i] * (unsigned long long)(unsigned)max(pos, 0);
            // nearest fraction of a turn in [-1/2, 1/2), as half turns for sincospif
            const float half_turns = (float)(int)((at + 0x80000000ull) >> 32) * 4.656612873077393e-10f;
            float sn, cs;
            sincospif(half_turns, &sn, &cs);
            if (p < pairs) s_turn[p] = make_float2(cs * a.rope_scale, sn * a.rope_scale);
        }
        int64_t cache_at = -1;  // of the token's slot
        if (slot >= 0 && slot < a.n_slots) {
            const int page = slot / a.page_size, off = slot - page * a.page_size;
            cache_at = page * a.page_stride + off * a.token_stride;
        } else if (slot != -1 && !padding && lane == 0) {
            atomicOr(&g_rope_error, 1u);
        }
        if (SHARE == kWarps) __syncthreads();
        else __syncwarp();

        // This lane's 8 pairs, kept in registers: from shared memory in every pass, 64 bytes apart, they
        // were the bound (85% of the L1 rate, three quarters of it bank conflicts).
        float2 cs[4], sn[4];  // of neighbouring pairs
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cs[i] = sn[i] = make_float2(0.f, 0.f);
            if (turned) {
                const float2 c = s_turn[8 * j + 2 * i], d = s_turn[8 * j + 2 * i + 1];
                cs[i] = make_float2(c.x, d.x);
                sn[i] = make_float2(c.y, d.y);
            }
        }
        float2 wa[4], wb[4];  // and its weights, where the section has a norm
        bool normed = false, turn = false, kept = false;
        int r = first_row, end = 0;
        O* dst = nullptr;
        int64_t dst_step = 0;

        for (int pass = 0; pass < a.passes; ++pass, r += kStep) {
            cp_async_wait<kDepth - 1>();
            __syncwarp();
            float2 fa[4], fb[4];
            take8<X>(entry + out_at, ca, fa);
            take8<X>(entry + out_at, cb, fb);
            out_at = out_at + 4 * kPieces < kDepth * 4 * kPieces ? out_at + 4 * kPieces : 0;
            if (r >= end && r < rows) {
                const float* w = nullptr;
                if (r < a.Hq) {
                    dst = static_cast<O*>(a.q_out) + t * a.qo_token_stride + r * a.qo_head_stride;
                    dst_step = kStep * a.qo_head_stride;
                    end = a.Hq, w = a.q_weight, turn = turned, kept = !padding;
                } else {
                    const bool key = r < a.Hq + a.Hkv;
                    const int h = r - (key ? a.Hq : a.Hq + a.Hkv);
                    dst = static_cast<O*>(key ? a.k_cache : a.v_cache) + cache_at + h * a.head_stride;
                    dst_step = kStep * a.head_stride;
                    end = key ? a.Hq + a.Hkv : rows, w = key ? a.k_weight : nullptr, turn = key && turned, kept = cache_at >= 0 && !padding;
                }
                normed = w != nullptr;
                if (normed) {
                    load8(w + ca, wa);
                    load8(w + cb, wb);
                }
            }
            float2 sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) sq = ffma2(fa[i], fa[i], ffma2(fb[i], fb[i], sq));
            float sum = sq.x + sq.y;
#pragma unroll
            for (int s = 1; s < 8; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            load();  // into the entry that the warp has just read
            if (normed) {
                const float inv = rsqrtf(sum * (1.0f / kTile) + a.eps);
                const float2 inv2 = make_float2(inv, inv);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    fa[i] = fmul2(fa[i], fmul2(inv2, wa[i]));
                    fb[i] = fmul2(fb[i], fmul2(inv2, wb[i]));
                }
            }
            if (turn) {
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
                        const float2 x = fa[i], y = fb[i], z = fmul2(y, sn[i]);
                        fa[i] = ffma2(x, cs[i], make_float2(-z.x, -z.y));
                        fb[i] = ffma2(y, cs[i], fmul2(x, sn[i]));
                    }
                }
            }
            if (kept && r < rows) {
                store8(dst + ca, fa);
                store8(dst + cb, fb);
            }
            dst += dst_step;
        }
        if (next >= n_tokens) break;
        t = next, pos = next_pos, slot = next_slot;
    }
}

template <typename X, typename O, int SHARE>
cudaError_t launch(RopeArgs a, int slices, int dev, int sms, cudaStream_t stream) {
    const int rounds = (a.Hq + 2 * a.Hkv + 4 * SHARE - 1) / (4 * SHARE);
    slices = slices < 1 ? 1 : slices < rounds ? slices : rounds;
    a.passes = (rounds + slices - 1) / slices;
    int64_t ctas = ((int64_t)a.n_tokens * SHARE + kWarps - 1) / kWarps;
    // past 16 CTAs for an SM (four run at once) warps go on from token to token, eight CTAs for an SM
    if (SHARE == 1 && ctas > 16 * (int64_t)sms) ctas = 8 * (int64_t)sms;
    const auto kern = a.interleaved ? rope_qkv_kernel<X, O, SHARE, true> : rope_qkv_kernel<X, O, SHARE, false>;
    const cudaError_t e = set_smem_limit_once(kern, 0, true, dev);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)ctas, (unsigned)((rounds + a.passes - 1) / a.passes)), dim3(kThreads), 0, stream, a);
}

// Measured, bf16 with norm, device time (us), the same inputs each time (in L2) and, in brackets, inputs from
// HBM; a warp per token / four sharing it:
//   32 + 2 x 8 heads:  3 tokens 6.3 / 2.2 (the same), 256 6.5 / 3.7 (7.2 / 4.3), 600 8.8 / 4.4 (9.1 / 5.7),
//     1000 10.0 / 7.4 (10.8 / 9.3), 1215 7.6 / 7.8 (8.7 / 9.9), 1500 10.5 / 10.2 (11.4 / 12.3), 2000 10.7 / 13.0
//     (11.9 / 15.6), 5003 25.5 / 32.2 (25.8 / 32.3), 16384 66 / 96 (66 / 96)
//   1 + 2 x 1:  600 3.3 / 2.8, 1000 3.5 / 4.7, 1215 3.0 / 5.1, 2000 3.6 / 8.5
//   128 + 2 x 8:  1000 25 / 13, 1215 18 / 15, 1500 27 / 21, 2000 27.5 / 27.6, 5003 66 / 61, 16384 204 / 188
// A warp per token is fastest where its CTAs, four tokens each, come out even on the SMs: 1215 tokens are two
// on every SM, and take less time than 1000.  The rule is taken from the first row, with 48 rows a token; with 3 the
// crossing lies before 1000 tokens, with 144 past 2000.  Four that share are sliced further while that leaves
// at most four CTAs for an SM.  The slices are the grid's second dimension: as one index, divided in the kernel,
// 3 tokens took 2.8 and 256 4.1.
template <typename X, typename O>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    const cudaError_t e = current_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    if (a.n_tokens < 8 * sms) return launch<X, O, kWarps>(a, 4 * sms / a.n_tokens, dev, sms, stream);
    return launch<X, O, 1>(a, 1, dev, sms, stream);
}

}  // namespace

cudaError_t read_and_clear_rope_error(unsigned int* out) { return read_and_clear_word(&g_rope_error, out); }

cudaError_t launch_rope_qkv(const RopeArgs& a, int x_dtype, int out_dtype, cudaStream_t stream) {
    if (out_dtype == KVARN_DTYPE_BF16)
        return x_dtype == KVARN_DTYPE_FP32 ? launch<float, __nv_bfloat16>(a, stream)
                                           : launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
    return x_dtype == KVARN_DTYPE_FP32 ? launch<float, __half>(a, stream) : launch<__half, __half>(a, stream);
}

}  // namespace kvarn
