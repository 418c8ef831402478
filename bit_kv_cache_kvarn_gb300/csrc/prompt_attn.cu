// Attention of many new tokens per sequence over a paged 16-bit cache, on the 5th-generation tensor cores.
//
// Mathematics, per sequence and query head, for the new token i at position p_i = L - n + i:
//   s_ij = scale q_i.k_j;  s_ij = cap tanh(s_ij / cap)  (cap > 0);  s_ij += slope (j - p_i);
//   out_i = sum_j e^{s_ij - m} v_j / l,  l = sum_j e^{s_ij - m},  lse = m + log l,
// over the visible keys j: start <= j, and p_i - window < j <= p_i when causal, else j < L.  One pass over the
// keys: with (m, l, o) of the keys so far, a tile's scores give m' = max(m, max s), and l and o are scaled by
// e^{m - m'} before its probabilities are added.
#include <cuda.h>
#include <math_constants.h>

#include <type_traits>

#include "kvarn_common.cuh"
#include "kvarn_internal.h"
#include "tcgen05.cuh"

namespace kvarn {

// Timeouts of the kernel's waits, and page table entries outside the cache.  Read by kvarn_device_error.
__device__ unsigned int g_prompt_error = 0;
__device__ unsigned int g_prompt_page_error = 0;

namespace {

constexpr int kHalf = 128;                       // rows of a tile: a (token, query head) pair each
constexpr int kUnit = 2 * kHalf;                 // rows that share a pass over the keys
constexpr int kThreads = 384;                    // two warpgroups of softmax, one of the four warps below
constexpr int kLoadWarp = 8, kMmaWarp = 9, kRowWarp = 10, kEdgeWarp = 11;
constexpr int kStages = 5;
constexpr int kStageBytes = kTile * kTile * 2;   // keys or values of a tile
constexpr int kSpan = kStageBytes / 2;           // 64 channels of it
constexpr int kRowBytes = kHalf * kTile * 2;     // queries of a half
constexpr int kSmem = 2 * kRowBytes + kStages * kStageBytes + 1024;
constexpr int kMaxCtas = 160;
constexpr int kMinPart = 2;                      // tiles of a unit that a CTA takes, at least
constexpr int kColS = 0, kColO = 256, kCols = 512;  // tensor memory: scores of the halves, then their outputs
constexpr float kGrow = 8.f;                     // how far (in powers of two) scores may pass the maximum in use
constexpr float kHalfLift = 7.f;                 // fp16 probabilities are multiplied by 2^7
constexpr int kJoinRows = 32, kJoinThreads = 256;

struct Join {
    int b, h, u, last;  // the unit that slot 1 begins and the last CTA that holds a part; b = -1: none
};
__host__ __device__ constexpr size_t slot_floats(int rows) { return ((size_t)rows * (kTile + 2) + 7) & ~(size_t)7; }

struct Workspace {
    float* base;
    size_t stride;
    int ctas;
    __device__ __forceinline__ float* slot(int cta, int which) const { return base + (2 * (size_t)cta + which) * stride; }
    __device__ __forceinline__ Join* joins() const { return reinterpret_cast<Join*>(slot(ctas, 0)); }
};

// A sequence: its rows of q, its length and its first visible key.
struct Seq {
    int b, q0, n, len, start;
};
__device__ __forceinline__ Seq load_seq(const PromptArgs& a, int b) {
    Seq s;
    s.b = b;
    s.q0 = min(max(a.cu[b], 0), a.T);
    s.n = min(max(a.cu[b + 1], s.q0), a.T) - s.q0;
    s.len = min(max(a.kv_lens[b], 0), a.max_len);
    s.start = a.kv_starts != nullptr ? max(a.kv_starts[b], 0) : 0;
    return s;
}
__device__ __forceinline__ int units_of(const PromptArgs& a, const Seq& s) {
    return (int)(((unsigned)s.n * (unsigned)a.group + kUnit - 1) / kUnit);
}

// Keys that some row of [f0, f1) sees, f = token * group + head.
struct Keys {
    int lo, hi;
    __device__ __forceinline__ int first() const { return lo / kTile; }
    __device__ __forceinline__ int past() const { return hi > lo ? (hi + kTile - 1) / kTile : lo / kTile; }
};
__device__ __forceinline__ Keys keys_of(const PromptArgs& a, const Seq& s, unsigned f0, unsigned f1) {
    Keys k = {s.start, s.len};
    if (f1 <= f0) k.hi = k.lo;
    if (a.causal && f1 > f0) {
        const int shift = s.len - s.n;
        const int p0 = shift + (int)(f0 / (unsigned)a.group), p1 = shift + (int)((f1 - 1) / (unsigned)a.group);
        k.hi = min(k.hi, p1 + 1);
        if (a.window > 0) k.lo = max(k.lo, p0 + 1 - a.window);
    }
    return k;
}
// Tiles of a unit in the stream of work: at least one, so that a unit without visible keys has its place.
__device__ __forceinline__ int cost_of(const PromptArgs& a, const Seq& s, int u) {
    const unsigned f0 = (unsigned)u * kUnit;
    const Keys k = keys_of(a, s, f0, min(f0 + kUnit, (unsigned)s.n * (unsigned)a.group));
    return max(k.past() - k.first(), 1);
}

// A CTA's share of one unit: the tiles [t0, t1), and of them those of each half.
struct Piece {
    Seq s;
    int h, u;
    unsigned f0;
    int rows;        // of the unit
    int t0, t1;
    int a0[2], a1[2];
    Keys keys;       // of the unit
    bool starts, ends;
    long long past;  // end of the unit in the stream
    __device__ __forceinline__ bool active(int half, int t) const { return t >= a0[half] && t < a1[half]; }
    __device__ __forceinline__ bool active(int t) const { return active(0, t) || active(1, t); }
    __device__ __forceinline__ int half_rows(int half) const { return min(max(rows - half * kHalf, 0), kHalf); }
};

// A place in the stream of tiles, ordered by (sequence, kv head, unit, tile); run by whole warps.
struct Walk {
    Seq s;
    int h, u, o, units;
    long long at, end;
    __device__ __forceinline__ bool next(const PromptArgs& a, Piece& p, int lane) {
        if (at >= end) return false;
        while (u >= units) {
            u = 0;
            if (units > 0 && ++h < a.Hkv) break;
            h = 0;
            // sequences without rows are passed over 32 at a time
            int b = s.b + 1;
            for (;;) {
                const int mine = b + lane;
                const bool some = mine < a.B && load_seq(a, mine).n > 0;
                const unsigned any = __ballot_sync(0xffffffffu, some);
                if (any != 0) {
                    b += __ffs(any) - 1;
                    break;
                }
                b += 32;
                if (b >= a.B) return false;
            }
            s = load_seq(a, b);
            units = units_of(a, s);
        }
        p.s = s, p.h = h, p.u = u;
        p.f0 = (unsigned)u * kUnit;
        const unsigned past = min(p.f0 + kUnit, (unsigned)s.n * (unsigned)a.group);
        p.rows = (int)(past - p.f0);
        p.keys = keys_of(a, s, p.f0, past);
        const int first = p.keys.first(), cost = max(p.keys.past() - first, 1);
        const int o1 = (int)min((long long)cost, o + (end - at));
        p.t0 = first + o, p.t1 = first + o1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const Keys k = keys_of(a, s, min(p.f0 + half * kHalf, past), min(p.f0 + (half + 1) * kHalf, past));
            p.a0[half] = max(k.first(), p.t0);
            p.a1[half] = min(k.past(), p.t1);
        }
        p.starts = o == 0, p.ends = o1 == cost;
        p.past = at - o + cost;
        at += o1 - o;
        o = 0;
        ++u;
        return true;
    }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack2(float x, float y, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float x, float y, __half) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 32 bytes, aligned so where wide says it
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                     "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
        static_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
        : "memory");
}

struct Barriers {
    uint64_t full[kStages], raw[kStages], empty[kStages];
    uint64_t q_full[2], q_free[2], s_full[2], p_full[2], o_full[2];
    uint64_t gave_up;
};

// T: type of q and the cache; O: type of the output; GEN: scores are capped or biased, or the scale has a sign or
// size for which the maximum cannot be taken before it.
template <typename T, typename O, bool GEN>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_split_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, PromptArgs a) {
    constexpr bool kIsHalf = std::is_same<T, __half>::value;
    constexpr float kLift = kIsHalf ? kHalfLift : 0.f;
    constexpr uint32_t kIdescS = kIsHalf ? tc::idesc_f16_f32(128, 128) : tc::idesc_as_bf16(tc::idesc_f16_f32(128, 128));
    constexpr uint32_t kIdescO = kIsHalf ? tc::idesc_f16_f32_bmn(128, 128) : tc::idesc_as_bf16(tc::idesc_f16_f32_bmn(128, 128));
    extern __shared__ uint8_t dsm_raw[];
    __shared__ Barriers bar;
    __shared__ uint32_t s_tmem;
    __shared__ long long s_scan[kThreads / 32];
    __shared__ long long s_at[2];          // the boundaries of this CTA's share
    __shared__ int s_seq[2], s_place[3];   // their sequences; kv head, unit and tile of the first one
    __shared__ long long s_in[2];
    uint8_t* dsm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* rows_smem = dsm;
    uint8_t* ring = dsm + 2 * kRowBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == kMmaWarp) tc::alloc(&s_tmem, kCols);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&bar.full[i], 1), mbar_init(&bar.raw[i], 1), mbar_init(&bar.empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1), mbar_init(&bar.q_free[i], 1), mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4), mbar_init(&bar.o_full[i], 1);
        }
        mbar_init(&bar.gave_up, 1);
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- this CTA's share: the tiles of all units form one stream, cut into equal pieces ----
    long long* s_cost = reinterpret_cast<long long*>(ring);  // tiles of a sequence's units, of one kv head
    for (int base = warp * 32; base < a.B; base += kThreads) {
        const bool in = base + lane < a.B;
        const Seq s = in ? load_seq(a, base + lane) : Seq{0, 0, 0, 0, 0};
        const int n = units_of(a, s);
        long long cost = 0;
        if (n <= 4)
            for (int u = 0; u < n; ++u) cost += cost_of(a, s, u);
        for (unsigned many = __ballot_sync(0xffffffffu, n > 4); many != 0; many &= many - 1) {  // by the whole warp
            const int k = __ffs(many) - 1;
            Seq w;
            w.b = 0, w.q0 = 0;
            w.n = __shfl_sync(0xffffffffu, s.n, k);
            w.len = __shfl_sync(0xffffffffu, s.len, k);
            w.start = __shfl_sync(0xffffffffu, s.start, k);
            const int nw = units_of(a, w);
            long long sum = 0;
            for (int u = lane; u < nw; u += 32) sum += cost_of(a, w, u);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (lane == k) cost = sum;
        }
        if (in) s_cost[base + lane] = cost;
    }
    __syncthreads();
    const int seg = (a.B + kThreads - 1) / kThreads, seg0 = min(tid * seg, a.B), seg1 = min(seg0 + seg, a.B);
    long long mine = 0;
    for (int b = seg0; b < seg1; ++b) mine += s_cost[b] * a.Hkv;
    long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += v;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) inc += s_scan[w];
        total += s_scan[w];
    }
    const long long piece = max((total + gridDim.x - 1) / gridDim.x, (long long)kMinPart);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const long long pos = min(piece * (blockIdx.x + which), total);
        if (pos >= total) {
            if (tid == 0) s_seq[which] = -1;
        } else if (pos >= inc - mine && pos < inc) {
            long long in_seq = pos - (inc - mine);
            int b = seg0;
            for (; in_seq >= s_cost[b] * a.Hkv; ++b) in_seq -= s_cost[b] * a.Hkv;
            s_seq[which] = b;
            s_in[which] = in_seq;
        }
    }
    __syncthreads();
    if (warp < 2) {
        const int b = s_seq[warp];
        long long pos = min(piece * (blockIdx.x + warp), total);
        if (b >= 0) {
            const Seq s = load_seq(a, b);
            const int units = units_of(a, s);
            const long long per_head = s_cost[b];
            const int h = (int)(s_in[warp] / per_head);
            const long long want = s_in[warp] - h * per_head;
            long long before = 0;
            int u = 0, o = 0, cost = 0;
            for (int u0 = 0; u0 < units; u0 += 32) {
                const int c = u0 + lane < units ? cost_of(a, s, u0 + lane) : 0;
                long long sum = c;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const long long v = __shfl_up_sync(0xffffffffu, sum, d);
                    if (lane >= d) sum += v;
                }
                const unsigned ends_later = __ballot_sync(0xffffffffu, before + sum > want);
                if (ends_later != 0) {
                    const int k = __ffs(ends_later) - 1;
                    u = u0 + k;
                    cost = __shfl_sync(0xffffffffu, c, k);
                    o = (int)(want - (before + __shfl_sync(0xffffffffu, sum, k) - cost));
                    break;
                }
                before += __shfl_sync(0xffffffffu, sum, 31);
            }
            // parts of a unit have kMinPart tiles at least: the boundary moves to the unit's begin or end
            if (o < kMinPart) {
                pos -= o;
                o = 0;
            } else if (cost - o < kMinPart) {
                pos += cost - o;
                o = 0;
                ++u;
            }
            if (warp == 0 && lane == 0) s_place[0] = h, s_place[1] = u, s_place[2] = o;
        }
        if (lane == 0) s_at[warp] = pos;
    }
    fence_proxy_async();  // s_cost lies where the copies go
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    const Workspace ws = {static_cast<float*>(a.workspace), slot_floats(a.slot_rows), (int)gridDim.x};
    Walk walk;
    walk.at = s_at[0], walk.end = s_at[1];
    walk.units = 0;
    if (walk.at < walk.end) {
        walk.s = load_seq(a, s_seq[0]);
        walk.h = s_place[0], walk.u = s_place[1], walk.o = s_place[2];
        walk.units = units_of(a, walk.s);
    }
    if (tid == 0) ws.joins()[blockIdx.x].b = -1;
    unsigned int* const err = &g_prompt_error;

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---- softmax: a thread has a row of its half ----
        const int half = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t t_s = tmem + lanes + kColS + half * kTile, t_o = tmem + lanes + kColO + half * kTile;
        uint32_t s_parity = 0, o_parity = 0;
        const float c = GEN ? 1.f : a.scale * kLog2e;
        bool fine = true;
        Piece p;
        while (fine && walk.next(a, p, lane)) {
            const int rows = p.half_rows(half);
            const bool real = r < rows;
            const unsigned f = p.f0 + half * kHalf + r;
            const int token = (int)(f / (unsigned)a.group), head = p.h * a.group + (int)(f - (unsigned)token * a.group);
            const int pos = p.s.len - p.s.n + token;
            int lo = p.s.start, hi = p.s.len;
            if (a.causal) {
                hi = min(hi, pos + 1);
                if (a.window > 0) lo = max(lo, pos + 1 - a.window);
            }
            if (!real) hi = lo;
            const float slope = GEN && a.slopes != nullptr && real ? a.slopes[head] : 0.f;
            float m = -CUDART_INF_F, l = 0.f;
            const int first = p.a0[half], past = p.a1[half];
            for (int t = first; t < past; ++t) {
                if (!mbar_wait(&bar.s_full[half], s_parity, err)) {
                    fine = false;
                    break;
                }
                s_parity ^= 1;
                tc::fence_after();
                if ((warp & 3) * 32 < rows) {
                    uint32_t x[4][32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tc::ld32(t_s + 32 * i, x[i]);
                    tc::wait_ld();
                    const int lo_in = lo - t * kTile, hi_in = hi - t * kTile;
                    if (GEN) {
                        const float d0 = (float)(t * kTile - pos);
#pragma unroll
                        for (int i = 0; i < 128; ++i) {
                            float v = __uint_as_float(x[i >> 5][i & 31]) * a.scale;
                            if (a.softcap > 0.f) v = a.softcap * tanhf(v * a.inv_softcap);
                            x[i >> 5][i & 31] = __float_as_uint(fmaf(slope, d0 + i, v) * kLog2e);
                        }
                    }
                    if (__any_sync(0xffffffffu, lo_in > 0 || hi_in < kTile)) {
#pragma unroll
                        for (int i = 0; i < 128; ++i)
                            if (i < lo_in || i >= hi_in) x[i >> 5][i & 31] = 0xff800000u;
                    }
                    float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int i = 0; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(x[i >> 5][i & 31]));
                    const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), m);
                    if (__any_sync(0xffffffffu, (top - m) * c > kGrow)) {
                        const float scale = top > m ? exp2_fast((m - top) * c) : 1.f;
                        m = top;
                        l *= scale;
                        if (t > first) {
#pragma unroll 1
                            for (int i = 0; i < 4; ++i) {
                                uint32_t o[32];
                                tc::ld32(t_o + 32 * i, o);
                                tc::wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * scale);
                                tc::st32(t_o + 32 * i, o);
                            }
                        }
                    }
                    const float ref = (m == -CUDART_INF_F ? 0.f : m * c) - kLift;
                    const float2 c2 = make_float2(c, c), ref2 = make_float2(-ref, -ref);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t w[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const int e = 64 * i + 2 * k;
                            float2 v = make_float2(__uint_as_float(x[e >> 5][e & 31]), __uint_as_float(x[e >> 5][(e & 31) + 1]));
                            v = ffma2(v, c2, ref2);
                            v.x = exp2_fast(v.x);
                            v.y = exp2_fast(v.y);
                            sum[k & 1] = fadd2(sum[k & 1], v);
                            w[k] = pack2(v.x, v.y, T());
                        }
                        tc::st32(t_s + 32 * i, w);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tc::wait_st();
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[half]);
            }
            if (!fine) break;
            const bool any = past > first;
            if (any) {
                if (!mbar_wait(&bar.o_full[half], o_parity, err)) {
                    fine = false;
                    break;
                }
                o_parity ^= 1;
                tc::fence_after();
            }
            const bool whole = p.starts && p.ends;
            const int64_t row = (int64_t)(p.s.q0 + token) * a.Hq + head;
            float* slot = ws.slot(blockIdx.x, p.starts ? 1 : 0);
            const int rr = half * kHalf + r;
            const float inv = l != 0.f ? 1.f / l : 0.f;
            if ((warp & 3) * 32 < rows) {
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    uint32_t o[32];
                    if (any) {
                        tc::ld32(t_o + 32 * i, o);
                        tc::wait_ld();
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0u;
                    }
                    if (!real) continue;
                    if (whole && sizeof(O) == 2) {
                        O* out = static_cast<O*>(a.out) + row * kTile + 32 * i;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float x0 = __uint_as_float(o[16 * k + 2 * e]) * inv, x1 = __uint_as_float(o[16 * k + 2 * e + 1]) * inv;
                                w[e] = pack2(l != 0.f ? x0 : 0.f, l != 0.f ? x1 : 0.f, T());
                            }
                            store32(out + 16 * k, w, a.wide_out);
                        }
                    } else {
                        float* out = whole ? static_cast<float*>(a.out) + row * kTile + 32 * i : slot + rr * kTile + 32 * i;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float x0 = __uint_as_float(o[8 * k + e]);
                                w[e] = __float_as_uint(whole ? (l != 0.f ? x0 * inv : 0.f) : x0);
                            }
                            store32(out + 8 * k, w, a.wide_out);
                        }
                    }
                }
            }
            if (real) {
                if (whole) {
                    if (a.lse != nullptr)
                        a.lse[row] = l != 0.f ? (m * c + (log2f(l) - kLift)) * 0.69314718055994531f : -CUDART_INF_F;
                } else {
                    slot[a.slot_rows * kTile + rr] = m == -CUDART_INF_F ? m : m * c;
                    slot[a.slot_rows * kTile + a.slot_rows + rr] = l;
                }
            }
            if (tid == 0 && p.starts && !p.ends) {
                // the CTA that takes the unit's last tile; its boundary may have moved to the unit's end
                int last = (int)((p.past - 1) / piece);
                if (p.past - piece * last < kMinPart) --last;
                ws.joins()[blockIdx.x] = Join{p.s.b, p.h, p.u, last};
            }
            tc::fence_before();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        Piece p;
        if (warp == kLoadWarp) {
            // ---- keys and values, a tile at a time, page by page ----
            uint32_t stage = 0, parity = 1;
            bool fine = true;
            const int boxes = kTile / a.box;
            uint64_t* last[kStages] = {};  // barrier of each stage's last copy, and its parity
            uint32_t last_parity = 0, raw_parity = 0;
            while (fine && walk.next(a, p, lane)) {
                for (int t = p.t0; fine && t < p.t1; ++t) {
                    if (!p.active(t)) continue;
                    // lane i: box i of the tile
                    const int tok = t * kTile + lane * a.box;
                    const bool want = lane < boxes && tok < p.keys.hi && tok + a.box > p.keys.lo;
                    const int entry = tok / a.page_size, in_page = tok - entry * a.page_size;
                    const int page = want ? a.page_table[(int64_t)p.s.b * a.max_pages + entry] : 0;
                    const bool bad = want && (page < 0 || page >= a.n_pages);
                    const unsigned good = __ballot_sync(0xffffffffu, want && !bad), zero = __ballot_sync(0xffffffffu, bad);
                    const uint32_t bytes = (uint32_t)__popc(good) * (uint32_t)a.box * (kTile * 2);
                    const bool edge = t * kTile < p.keys.lo || (t + 1) * kTile > p.keys.hi;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (!mbar_wait(&bar.empty[stage], parity, err)) {
                            fine = false;
                            break;
                        }
                        uint8_t* dst = ring + stage * kStageBytes;
                        if (zero != 0) {  // keys and values of pages outside the cache count as zeros
                            if (lane == 0) atomicOr(&g_prompt_page_error, 1u);
                            for (unsigned z = zero; z != 0; z &= z - 1) {
                                const int r0 = (__ffs(z) - 1) * a.box;
                                for (int i = lane; i < a.box * 16; i += 32)
                                    *reinterpret_cast<uint4*>(dst + (i & 1) * kSpan + r0 * kTile + (i >> 1) * 16) = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async();
                            __syncwarp();
                        }
                        // values with rows that nobody may see go through the edge warp
                        uint64_t* b = kv == 1 && edge ? &bar.raw[stage] : &bar.full[stage];
                        if (lane == 0) {
                            if (bytes > 0) mbar_expect_tx(b, bytes);
                            else mbar_arrive(b);
                        }
                        __syncwarp();
                        const uint32_t bit = 1u << stage, phase = b == &bar.raw[stage] ? raw_parity & bit : parity != 0 ? 0u : bit;
#pragma unroll
                        for (int i = 0; i < kStages; ++i)
                            if (i == (int)stage) last[i] = b;
                        last_parity = (last_parity & ~bit) | phase;
                        if (b == &bar.raw[stage]) raw_parity ^= bit;
                        if (want && !bad) {
                            const CUtensorMap* map = kv == 0 ? &k_map : &v_map;
                            uint8_t* d = dst + lane * a.box * kTile;
                            tma_load4(d, map, 0, in_page, p.h, page, b);
                            tma_load4(d + kSpan, map, 64, in_page, p.h, page, b);
                        }
                        __syncwarp();
                        if (++stage == kStages) stage = 0, parity ^= 1;
                    }
                }
            }
            // no copy and no arrival is on its way when the CTA leaves
            for (int i = 0; fine && i < kStages; ++i) {
                fine = mbar_wait(&bar.empty[stage], parity, err);
                if (++stage == kStages) stage = 0, parity ^= 1;
            }
            if (!fine) {
#pragma unroll
                for (int i = 0; i < kStages; ++i)
                    if (last[i] != nullptr) mbar_drain(last[i], last_parity >> i & 1u);
            }
        } else if (warp == kMmaWarp) {
            // ---- products: S of the halves' next tile between the two halves' P V of this one ----
            uint32_t stage = 0, parity = 0;  // of the ring
            uint32_t q_parity[2] = {0, 0}, p_parity[2] = {0, 0};
            const uint32_t ring_addr = smem_addr(ring), q_addr = smem_addr(rows_smem);
            bool fine = true;
            Piece cur, nxt;
            int t = 0, tn = 0;
            auto next_stage = [&]() {
                if (++stage == kStages) stage = 0, parity ^= 1;
            };
            // the next tile that some half takes: of piece q from tile i on, or of a later piece
            auto seek = [&](Piece& q, int& i, bool have) {
                for (;;) {
                    if (have)
                        for (; i < q.t1; ++i)
                            if (q.active(i)) return true;
                    if (!walk.next(a, q, lane)) return false;
                    i = q.t0;
                    have = true;
                }
            };
            auto scores = [&](const Piece& q, int i, int half, uint32_t kb) {
                if (i == q.a0[half]) {
                    if (!mbar_wait(&bar.q_full[half], q_parity[half], err)) return false;
                    q_parity[half] ^= 1;
                    tc::fence_after();
                }
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t off = (k >> 2) * kSpan + (k & 3) * 32;
                        tc::mma_f16_ss(tmem + kColS + half * kTile, tc::smem_desc_sw128(q_addr + half * kRowBytes + off, 16, 1024),
                                       tc::smem_desc_sw128(kb + off, 16, 1024), kIdescS, k > 0);
                    }
                    tc::commit(&bar.s_full[half]);
                    if (i + 1 == q.a1[half]) tc::commit(&bar.q_free[half]);
                }
                __syncwarp();
                return true;
            };
            bool have = seek(cur, t, false);
            if (have) {
                fine = mbar_wait(&bar.full[stage], parity, err);
                tc::fence_after();
                for (int half = 0; fine && half < 2; ++half)
                    if (cur.active(half, t)) fine = scores(cur, t, half, ring_addr + stage * kStageBytes);
                if (fine && lane == 0) tc::commit(&bar.empty[stage]);
                next_stage();
            }
            while (fine && have) {
                const uint32_t v_stage = stage, v_parity = parity;
                next_stage();
                nxt = cur;
                tn = t + 1;
                have = seek(nxt, tn, true);
                const uint32_t k_stage = stage, k_parity = parity;
                if (have) next_stage();
                bool v_in = false, k_in = false;
                for (int half = 0; fine && half < 2; ++half) {
                    if (cur.active(half, t)) {
                        if (!v_in) fine = mbar_wait(&bar.full[v_stage], v_parity, err);
                        v_in = true;
                        if (!fine || !mbar_wait(&bar.p_full[half], p_parity[half], err)) {
                            fine = false;
                            break;
                        }
                        p_parity[half] ^= 1;
                        tc::fence_after();
                        if (lane == 0) {
                            const uint32_t vb = ring_addr + v_stage * kStageBytes;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                tc::mma_f16_ts(tmem + kColO + half * kTile, tmem + kColS + half * kTile + 8 * k,
                                               tc::smem_desc_sw128(vb + k * 2048, kSpan, 1024), kIdescO, k > 0 || t > cur.a0[half]);
                            if (t + 1 == cur.a1[half]) tc::commit(&bar.o_full[half]);
                        }
                        __syncwarp();
                    }
                    if (have && nxt.active(half, tn)) {
                        if (!k_in) {
                            fine = mbar_wait(&bar.full[k_stage], k_parity, err);
                            tc::fence_after();
                        }
                        k_in = true;
                        if (fine) fine = scores(nxt, tn, half, ring_addr + k_stage * kStageBytes);
                    }
                }
                if (fine && lane == 0) {
                    tc::commit(&bar.empty[v_stage]);
                    if (have) tc::commit(&bar.empty[k_stage]);
                }
                __syncwarp();
                cur = nxt;
                t = tn;
            }
            if (!fine) {
                if (lane == 0) tc::commit(&bar.gave_up);
                __syncwarp();
                mbar_drain(&bar.gave_up, 0);
            }
        } else if (warp == kRowWarp) {
            // ---- queries: rows of 256 bytes, gathered, chunk i of a row at i ^ (row mod 8) ----
            uint32_t free_parity[2] = {1, 1};
            bool fine = true;
            while (fine && walk.next(a, p, lane)) {
                for (int half = 0; fine && half < 2; ++half) {
                    if (p.a0[half] >= p.a1[half]) continue;
                    if (!mbar_wait(&bar.q_free[half], free_parity[half], err)) {
                        fine = false;
                        break;
                    }
                    free_parity[half] ^= 1;
                    const int rows = p.half_rows(half), chunk = lane & 15;
                    const uint32_t dst = smem_addr(rows_smem + half * kRowBytes) + (chunk >> 3) * kSpan;
#pragma unroll 4
                    for (int i = 0; i < kHalf / 2; ++i) {
                        const int r = 2 * i + (lane >> 4);
                        const bool real = r < rows;
                        const unsigned f = real ? p.f0 + half * kHalf + r : p.f0;
                        const unsigned token = f / (unsigned)a.group, g = f - token * a.group;
                        const T* src = static_cast<const T*>(a.q) + (int64_t)(p.s.q0 + token) * a.q_token_stride +
                                       (int64_t)(p.h * a.group + g) * a.q_head_stride + 8 * chunk;
                        cp_async16(dst + r * kTile + (((chunk & 7) ^ (r & 7)) << 4), src, real);
                    }
                    cp_async_commit();
                    cp_async_wait<0>();
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.q_full[half]);
                }
            }
            for (int half = 0; fine && half < 2; ++half) fine = mbar_wait(&bar.q_free[half], free_parity[half], err);
        } else {
            // ---- values at the edges of what a unit sees: rows outside are zeros ----
            uint32_t stage = 0, raw_parity = 0;  // a bit for each stage
            bool fine = true;
            while (fine && walk.next(a, p, lane)) {
                for (int t = p.t0; fine && t < p.t1; ++t) {
                    if (!p.active(t)) continue;
                    if (++stage == kStages) stage = 0;  // the keys' stage
                    if (t * kTile < p.keys.lo || (t + 1) * kTile > p.keys.hi) {
                        fine = mbar_wait(&bar.raw[stage], (raw_parity >> stage) & 1, err);
                        if (!fine) break;
                        raw_parity ^= 1u << stage;
                        uint8_t* v = ring + stage * kStageBytes;
                        const int lo = p.keys.lo - t * kTile, hi = p.keys.hi - t * kTile;
                        for (int i = lane; i < kTile * 16; i += 32) {
                            const int r = i >> 4;
                            if (r < lo || r >= hi)
                                *reinterpret_cast<uint4*>(v + ((i >> 3) & 1) * kSpan + r * kTile + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.full[stage]);
                    }
                    if (++stage == kStages) stage = 0;
                }
            }
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) tc::dealloc(tmem, kCols);
}

// Parts of the units that several CTAs share, joined: CTA (c, y) takes kJoinRows rows of the unit that begins in the
// split's CTA c and goes on after it, a warp a row at a time, a lane four channels.
template <typename T, typename O>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(PromptArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Workspace ws = {static_cast<float*>(a.workspace), slot_floats(a.slot_rows), (int)gridDim.x};
    const int c0 = blockIdx.x;
    const Join jn = ws.joins()[c0];
    if (jn.b < 0) return;
    const Seq s = load_seq(a, jn.b);
    const unsigned f0 = (unsigned)jn.u * kUnit;
    const int rows = (int)(min(f0 + kUnit, (unsigned)s.n * (unsigned)a.group) - f0);
    const int past = min(rows, (int)(blockIdx.y + 1) * kJoinRows);
    for (int r = blockIdx.y * kJoinRows + warp; r < past; r += kJoinThreads / 32) {
        float m = -CUDART_INF_F, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = c0; c <= jn.last; ++c) {
            const float* slot = ws.slot(c, c == c0 ? 1 : 0);
            const float4 po = *reinterpret_cast<const float4*>(slot + r * kTile + 4 * lane);
            const float pm = slot[a.slot_rows * kTile + r], pl = slot[a.slot_rows * kTile + a.slot_rows + r];
            const float top = fmaxf(m, pm), ref = top == -CUDART_INF_F ? 0.f : top;
            const float x = exp2f(m - ref), y = exp2f(pm - ref);
            m = top;
            l = fmaf(y, pl, x * l);
            o.x = fmaf(y, po.x, x * o.x);
            o.y = fmaf(y, po.y, x * o.y);
            o.z = fmaf(y, po.z, x * o.z);
            o.w = fmaf(y, po.w, x * o.w);
        }
        const unsigned f = f0 + r;
        const int token = (int)(f / (unsigned)a.group), head = jn.h * a.group + (int)(f - (unsigned)token * a.group);
        const int64_t row = (int64_t)(s.q0 + token) * a.Hq + head;
        const float inv = 1.f / l;
        o = l != 0.f ? make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (sizeof(O) == 2)
            *reinterpret_cast<uint2*>(static_cast<O*>(a.out) + row * kTile + 4 * lane) = make_uint2(pack2(o.x, o.y, T()), pack2(o.z, o.w, T()));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kTile + 4 * lane) = o;
        if (a.lse != nullptr && lane == 0)
            a.lse[row] = l != 0.f ? (m + (log2f(l) - (std::is_same<T, __half>::value ? kHalfLift : 0.f))) * 0.69314718055994531f : -CUDART_INF_F;
    }
}

// Two parts of every row, each with its log-sum-exp, into one: the prefix's where the row has one.
template <typename T>
__global__ void __launch_bounds__(256) prefix_merge_kernel(PrefixMergeArgs a) {
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (int64_t)a.B * a.Hq) return;
    const int b = (int)(row / a.Hq);
    const bool some = b >= a.cu[0] && b < a.cu[a.n_groups];  // rows outside the groups have no prefix
    const float x = some ? a.prefix_lse[row] : -CUDART_INF_F, y = a.own_lse[row], top = fmaxf(x, y);
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    const float wx = exp2f((x - ref) * kLog2e), wy = exp2f((y - ref) * kLog2e), sum = wx + wy;
    const float4 p = some ? *reinterpret_cast<const float4*>(a.prefix_out + row * kTile + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 o = *reinterpret_cast<const float4*>(a.own_out + row * kTile + 4 * lane);
    const float inv = sum != 0.f ? 1.f / sum : 0.f, fx = wx * inv, fy = wy * inv;
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * kTile + 4 * lane) =
        make_uint2(pack2(fmaf(fx, p.x, fy * o.x), fmaf(fx, p.y, fy * o.y), T()), pack2(fmaf(fx, p.z, fy * o.z), fmaf(fx, p.w, fy * o.w), T()));
    if (a.lse != nullptr && lane == 0) a.lse[row] = sum != 0.f ? top + log2f(sum) * 0.69314718055994531f : -CUDART_INF_F;
}

struct Kernels {
    void (*split)(CUtensorMap, CUtensorMap, PromptArgs);
    void (*join)(PromptArgs);
};
template <typename T>
Kernels pick(bool general, bool wide) {
    if (wide) return {general ? prompt_split_kernel<T, float, true> : prompt_split_kernel<T, float, false>, prompt_join_kernel<T, float>};
    return {general ? prompt_split_kernel<T, T, true> : prompt_split_kernel<T, T, false>, prompt_join_kernel<T, T>};
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
    static std::atomic<void*> known{nullptr};
    void* p = known.load(std::memory_order_relaxed);
    if (p == nullptr) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        known.store(p, std::memory_order_relaxed);
    }
    return reinterpret_cast<EncodeTiled>(p);
}

// Keys or values of the cache as channels x tokens of a page x heads x pages, in boxes of 64 channels of `box` tokens.
cudaError_t cache_map(CUtensorMap* map, const PromptArgs& a, int dtype, const void* cache) {
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t sizes[4] = {kTile, (cuuint64_t)a.page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_pages};
    // the stride of an axis with one entry is never used, but has to be one that the encoding takes
    const cuuint64_t strides[3] = {(cuuint64_t)a.token_stride * 2, a.Hkv > 1 ? (cuuint64_t)a.head_stride * 2 : 256,
                                   a.n_pages > 1 ? (cuuint64_t)a.page_stride * 2 : 256};
    const cuuint32_t box[4] = {64, (cuuint32_t)a.box, 1, 1}, step[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, dtype == KVARN_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                              const_cast<void*>(cache), sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int slot_rows(int64_t T, int Hq, int Hkv) {
    const int64_t rows = T * (Hq / Hkv);
    return (int)(rows < 1 ? 1 : rows < kUnit ? rows : kUnit);
}

}  // namespace

size_t prompt_attention_workspace_bytes(int64_t T, int Hq, int Hkv) {
    const size_t bytes = 2 * kMaxCtas * slot_floats(slot_rows(T, Hq, Hkv)) * sizeof(float) + kMaxCtas * sizeof(Join);
    return (bytes + 255) & ~(size_t)255;
}

cudaError_t read_and_clear_prompt_error(unsigned int* out) { return read_and_clear_word(&g_prompt_error, out); }
cudaError_t read_and_clear_prompt_page_error(unsigned int* out) { return read_and_clear_word(&g_prompt_page_error, out); }

cudaError_t launch_prompt_attention(PromptArgs a, int dtype, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = current_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    a.group = a.Hq / a.Hkv;
    a.slot_rows = slot_rows(a.T, a.Hq, a.Hkv);
    a.inv_softcap = a.softcap > 0.f ? 1.f / a.softcap : 0.f;
    a.box = a.page_size % 128 == 0 ? 128 : a.page_size % 64 == 0 ? 64 : a.page_size % 32 == 0 ? 32 : 16;
    a.wide_out = ((uintptr_t)a.out & 31) == 0 && ((uintptr_t)a.workspace & 31) == 0;
    const float c = a.scale * kLog2e;
    const bool general = a.softcap > 0.f || a.slopes != nullptr || !(c >= 1e-30f && c <= 1e30f);
    const bool wide = a.out_dtype == KVARN_DTYPE_FP32;
    const Kernels k = dtype == KVARN_DTYPE_FP16 ? pick<__half>(general, wide) : pick<__nv_bfloat16>(general, wide);
    CUtensorMap k_map, v_map;
    e = cache_map(&k_map, a, dtype, a.k_cache);
    if (e == cudaSuccess) e = cache_map(&v_map, a, dtype, a.v_cache);
    if (e == cudaSuccess) e = set_smem_limit_once(k.split, kSmem, false, dev);
    if (e != cudaSuccess) return e;
    // no more CTAs than parts of kMinPart tiles that the call can have
    const int64_t units = (int64_t)a.Hkv * (((int64_t)a.T * a.group + kUnit - 1) / kUnit + a.B);
    const int64_t parts = units * (((int64_t)a.max_len + 2 * kTile - 1) / kTile);
    const int most = sms < kMaxCtas ? sms : kMaxCtas;
    const int ctas = (int)(parts < 1 ? 1 : parts < most ? parts : most);
    e = launch_pdl(k.split, dim3(ctas), dim3(kThreads), kSmem, stream, k_map, v_map, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(k.join, dim3(ctas, (a.slot_rows + kJoinRows - 1) / kJoinRows), dim3(kJoinThreads), 0, stream, a);
}

cudaError_t launch_prefix_merge(const PrefixMergeArgs& a, int dtype, cudaStream_t stream) {
    const int64_t ctas = ((int64_t)a.B * a.Hq + 7) / 8;
    return launch_pdl(dtype == KVARN_DTYPE_FP16 ? prefix_merge_kernel<__half> : prefix_merge_kernel<__nv_bfloat16>,
                      dim3((unsigned)ctas), dim3(256), 0, stream, a);
}

}  // namespace kvarn
