// Attention of one new token per sequence over a paged 16-bit cache, or one of 8-bit values with an exponent for each
// token and head, split over the cache's length and joined.
//
// Mathematics, per sequence and query head, over the visible keys j in [lo, L):
//   s_j = scale q.k_j;  s_j = cap tanh(s_j / cap)  (cap > 0);  s_j += slope (j - (L - 1));
//   out = sum_j e^{s_j - m} v_j / l,  l = sum_j e^{s_j - m},  m = max_j s_j,  lse = m + log l,
// with lo = max(start, L - window).  (m, l, sum) of two disjoint parts join as
//   m = max(m1, m2), l = l1 e^{m1 - m} + l2 e^{m2 - m}, and the sums alike.
//
// What bounds it: every visible key and value is read once (512 bytes per kv head and token) for 512
// operations per query head: HBM.  So the work is arranged around keeping bytes in flight:
//   - the visible tokens of all (sequence, kv head, block of 16 query heads) units, in groups of 16,
//     form one stream that is cut into equal contiguous pieces, one per warp of a persistent grid (one
//     CTA of 12 warps per SM, 8 for 9 to 16 query heads), so the load is even whatever the lengths;
//   - a warp is on its own: it fetches its next group into its own ring in shared memory (16-byte
//     asynchronous copies, 8 KB per group, 96 to 192 KB in flight per SM) across the ends of units, and
//     never waits for another warp until its piece is done.  12 warps with two groups each took 88 us
//     where 8 with three took 98 (256 sequences of 1 to 900 tokens), 305 and 318 (16 x 32k);
//   - both products are taken transposed, m16n8k16: scores^T = K Q^T with the group's 16 tokens as rows
//     (K as it lies, ldmatrix) and 8 query heads as columns, out^T = V^T P^T with 16 channels as rows
//     (V through the transposing ldmatrix) and the probabilities turned in registers (movmatrix).  With
//     query heads as the 16 rows instead, half of every product, exponential and addition was padding
//     for groups of up to 8 heads.  A group of 8 KB is 24 or 32 such products per 8 heads, a small part
//     of what an SM's warps can issue while HBM brings it, so these products, which need no hand-over
//     between warps, fit better than 128-row tensor-memory tiles;
//   - units that cross warps of a CTA are joined in shared memory at its end, units that cross CTAs by
//     a second launch of one CTA per boundary.
// Rounding: the products take the cache's type exactly; scores, maximum, sums and outputs are fp32.
// A probability enters the second product in 16-bit pieces that add up to it.  bf16: two pieces are off
// by up to 2^-16, on average 2.3e-6 of an output whose other errors are 4e-7, so an fp32 output takes
// three pieces (2^-24) and a bf16 output, which rounds by 2^-8 itself, two.  fp16: two pieces (2^-22) of
// 2^15 p, since p itself would lose its digits below 2^-14 (sums and outputs carry the factor alike).  Each
// group's P V is added to the running output by an fp32 addition, to nearest.
//
// Measured (among others, us): 16 x 32k tokens, 32 over 8 heads 312 (6.87 TB/s), 256 x 1-900 tokens, 64 over 8,
// fp16, capped 93 to 99 by the lengths drawn (5.2 TB/s at 93; without the cap 1 less), one sequence of 4k 10.4.
#include <cooperative_groups.h>
#include <math_constants.h>

#include <type_traits>

#include "kvarn_common.cuh"
#include "kvarn_internal.h"

namespace kvarn {

namespace {

#ifndef KVARN_PAGED_Q8
#define KVARN_PAGED_Q8 0
#endif
constexpr bool kQ8 = KVARN_PAGED_Q8;  // which caches this unit is compiled for

// Set when a page table entry lies outside the cache (its keys and values count as zeros).  Read by
// kvarn_device_error.
__device__ unsigned int g_paged_attn_error = 0;

namespace cg = cooperative_groups;

constexpr int kGroup = 16;                             // tokens per step
constexpr int kRows = 16;                              // query heads per unit, at most
constexpr int kMaxCtas = 160;                          // CTAs of a grid, at most
constexpr int kMaxWarps = 12;                          // warps of a CTA, at most
constexpr int kSmemLimit = 227 * 1024 - 2048;          // dynamic shared memory of a CTA, beside the static

// Warps of a CTA and groups in a warp's ring, by the eights of query heads in a unit.
template <int NT, bool Q8 = false>
struct Shape {
    static constexpr int kWarps = NT == 1 ? 12 : 8, kStages = Q8 ? (NT == 1 ? 4 : 6) : NT == 1 ? 2 : 3;
    static constexpr int kRowBytes = Q8 ? kTile : 2 * kTile;                  // a token's keys or values
    static constexpr int kHalf = kGroup * kRowBytes;                          // keys or values of a group
    static constexpr int kStage = 2 * kHalf + (Q8 ? 2 * kGroup : 0);          // with the 8-bit ones' exponents
    static constexpr int kThreads = 32 * kWarps, kRing = kStages * kStage;    // bytes of a warp
};
constexpr float kHalfLift = 15.f;                      // fp16 probabilities are multiplied by 2^15,
constexpr float kGrow = 4.f;                           // over 8-bit caches by 2^11, as scores may pass the maximum by 2^4 there
constexpr int kJoinWarps = 16;
constexpr int kAhead = 2;                              // parts that a warp of the join loads at once

// Workspace: partial slots, each o[rows][128] then m[rows] and l[rows] (fp32; a slot is a multiple of 16
// bytes, joins read four channels at a time): two per CTA (slot 0: the unit that began before the CTA's
// pieces, slot 1: the one that begins in them and goes on after them), then one per warp (the unit that
// began before its piece and ends inside it; in shared memory where that fits beside the rings); then one
// Join per CTA.
struct Join {
    int b, u;  // sequence and unit that slot 1 begins; b = -1: none
    int last;  // the last CTA that holds a part
    int pad;
};

__host__ __device__ constexpr size_t slot_floats(int rows) { return ((size_t)rows * (kTile + 2) + 3) & ~(size_t)3; }

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// the 8 x 8 matrix of 16-bit pairs that the warp holds (row lane / 4), transposed
__device__ __forceinline__ uint32_t turn8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// d += a (16 x 16) b (16 x 8)
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// (x, y) to 16 bits; x and y become what is left
__device__ __forceinline__ uint32_t take2(float& x, float& y, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
    x -= __uint_as_float(u << 16);
    y -= __uint_as_float(u & 0xffff0000u);
    return u;
}
__device__ __forceinline__ uint32_t take2(float& x, float& y, __half) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    x -= f.x;
    y -= f.y;
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}
__device__ __forceinline__ void store4(__half* p, float4 v) {
    const __half2 x = __floats2half2_rn(v.x, v.y), y = __floats2half2_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// Visible keys [lo, len) of a sequence and its groups of 16 tokens: [lo / 16, ceil(len / 16)).
struct Span {
    int lo, len;
    __device__ __forceinline__ int first() const { return lo / kGroup; }
    __device__ __forceinline__ int groups() const { return lo < len ? (len + kGroup - 1) / kGroup - lo / kGroup : 0; }
};
__device__ __forceinline__ Span load_span(const PagedAttnArgs& a, int b) {
    Span s;
    s.len = min(max(a.kv_lens[b], 0), a.max_len);
    s.lo = a.kv_starts != nullptr ? max(a.kv_starts[b], 0) : 0;
    if (a.window > 0) s.lo = max(s.lo, s.len - a.window);
    return s;
}

// A place in the stream of groups, ordered by (sequence, unit, group).
struct Cursor {
    int b, u, g, n;  // sequence, unit, group of the unit, groups per unit
    Span s;
    // By the whole warp, and only where the stream goes on: the unused slots behind a batch's last sequence are
    // never walked through.  Empty sequences before the next one are passed over 32 at a time: one by one they cost
    // 95 ns each (2048 slots, two of them in use at the start: 186 us, now 16).
    __device__ __forceinline__ void next(const PagedAttnArgs& a, int lane) {
        if (++g < n) return;
        g = 0;
        if (++u < a.units) return;
        u = 0;
        s = load_span(a, ++b);
        n = s.groups();
        while (n == 0 && b + 1 < a.B) {
            const int mine = b + 1 + lane;
            const Span other = mine < a.B ? load_span(a, mine) : Span{0, 0};
            const unsigned some = __ballot_sync(0xffffffffu, other.groups() > 0);
            const int k = some != 0 ? __ffs(some) - 1 : 31;
            b += 1 + k;
            s.lo = __shfl_sync(0xffffffffu, other.lo, k);
            s.len = __shfl_sync(0xffffffffu, other.len, k);
            n = s.groups();
        }
    }
    __device__ __forceinline__ int token() const { return (s.first() + g) * kGroup; }
};

template <bool CAP, bool SCALED>
__device__ __forceinline__ float score(const PagedAttnArgs& a, float dot, float slope, float dist) {
    // in the log2 domain
    float s = SCALED ? dot : dot * a.scale;
    if (CAP) s = a.softcap * tanhf(s * a.inv_softcap);
    return fmaf(slope, dist, s) * kLog2e;
}

// A partial of one row as a lane holds it: channels 4 lane .. 4 lane + 3.
struct RowPart {
    float m, l;
    float4 o;
};
__device__ __forceinline__ RowPart load_part(const float* slot, int rows, int r, int lane) {
    RowPart p;
    p.o = *reinterpret_cast<const float4*>(slot + r * kTile + 4 * lane);
    p.m = slot[rows * kTile + r];
    p.l = slot[rows * kTile + rows + r];
    return p;
}
// s joined with p; m = -inf: nothing yet (o and l are 0), or only scores of -inf
__device__ __forceinline__ void join_part(RowPart& s, const RowPart& p) {
    const float m = fmaxf(s.m, p.m);
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    const float a = exp2f(s.m - ref), b = exp2f(p.m - ref);
    s.m = m;
    s.l = fmaf(b, p.l, a * s.l);
    s.o.x = fmaf(b, p.o.x, a * s.o.x);
    s.o.y = fmaf(b, p.o.y, a * s.o.y);
    s.o.z = fmaf(b, p.o.z, a * s.o.z);
    s.o.w = fmaf(b, p.o.w, a * s.o.w);
}
// Natural log of the row's sum; l carries the factor 2^lift.  l = 0: no key, or only scores of -inf.
__device__ __forceinline__ float lse_of(const PagedAttnArgs& a, float m, float l) {
    return l != 0.f ? (m + (log2f(l) - a.lift)) * 0.69314718055994531f : -CUDART_INF_F;
}
template <typename O>
__device__ __forceinline__ void store_row(const PagedAttnArgs& a, int64_t row, const RowPart& s, int lane) {
    const float inv = s.l != 0.f ? 1.f / s.l : 0.f;
    store4(static_cast<O*>(a.out) + row * kTile + 4 * lane, make_float4(s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv));
    if (a.lse != nullptr && lane == 0) a.lse[row] = lse_of(a, s.m, s.l);
}

// x / y, both at least 0: 64-bit division takes five times as long as the 32-bit one, which nearly
// always suffices
__device__ __forceinline__ long long divide(long long x, long long y) {
    return (x | y) >> 32 ? x / y : (long long)((unsigned)x / (unsigned)y);
}

// Query heads of a unit: the first one and how many (the last block of a kv head's may be short).
struct Heads {
    int kvh, first, rows;
};
__device__ __forceinline__ Heads heads_of(const PagedAttnArgs& a, int u) {
    Heads h;
    h.kvh = u / a.row_blocks;
    const int rb = u - h.kvh * a.row_blocks;
    h.first = h.kvh * a.group + rb * kRows;
    h.rows = min(a.group - rb * kRows, kRows);
    return h;
}

struct Workspace {
    float* base;
    size_t stride;
    int ctas, warps;  // of the split's grid and of its CTAs
    __device__ __forceinline__ float* cta_slot(int cta, int which) const { return base + (2 * (size_t)cta + which) * stride; }
    __device__ __forceinline__ float* warp_slot(int worker) const { return base + (2 * (size_t)ctas + worker) * stride; }
    __device__ __forceinline__ Join* joins() const { return reinterpret_cast<Join*>(warp_slot(ctas * warps)); }
};

// What a warp leaves for the join at its CTA's end.
struct Left {
    int b, u;
    unsigned flags;
    int pad;
    long long end;  // stream position of the last group of the open unit (where it starts here)
};
constexpr unsigned kOpen = 1;    // the warp's last unit is in its ring:
constexpr unsigned kStarts = 2;  //   it begins in this warp's piece
constexpr unsigned kEnds = 4;    //   it ends with this warp's piece
constexpr unsigned kHead = 8;    // its first unit began before its piece, ended inside it, and is in its head slot

// two E4M3 pairs to fp16 pairs, exactly
__device__ __forceinline__ void halves_of(uint32_t& low, uint32_t& high, uint32_t x) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(low), "=r"(high)
        : "r"(x));
}
// 2^e for e of -127..127
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float(e > -127 ? (e + 127) << 23 : 1 << 22); }

// T: type of q and the cache; O: type of the output; NT: eights of query heads in a unit; CAP: scores are
// capped.
// Q8: the cache holds E4M3 values c and an exponent e for each token and head, x = c 2^e.  The products take c as
// fp16, exactly, and queries as fp16 with a power of two of their own (so that a bf16 query keeps its eight digits down to
// 2^-31 of its largest element, and the last of them goes at 2^-39); keys' exponents scale the scores.  Values' exponents
// go into the probabilities: with their own maximum m' = max(s + e), 2^(s + e - m') is at most 1 for fp16, while l keeps
// 2^(s - m), and the factor 2^(m' - m) joins them at the end of a unit.
// Half the bytes but as many products: instruction issue is near HBM as a bound (505 instructions a warp and group,
// 55% of the issue slots).  So maxima are shared between lanes only when one has grown by 2^kGrow, and a channel's order
// inside a product is the one that the bytes have.  Measured: 16 sequences of 32k tokens, 32 over 8 heads, 189 us
// (5.7 TB/s; with a maximum per group and its shuffles 237); 200 of 1 to 1200 tokens 75 to 77 us by the
// lengths drawn.  (16 warps a CTA in 128 registers: 182 and 79.)
// CLUSTER: a thread-block cluster takes one unit, its CTAs equal parts of it, and the parts are joined
// through the cluster's shared memory: no second launch.
template <typename T, typename O, int NT, bool CAP, bool CLUSTER, bool Q8>
__global__ void __launch_bounds__(Shape<NT, Q8>::kThreads, 1) paged_split_kernel(PagedAttnArgs a) {
    constexpr int kWarps = Shape<NT, Q8>::kWarps, kThreads = Shape<NT, Q8>::kThreads, kRing = Shape<NT, Q8>::kRing;
    constexpr int kStages = Shape<NT, Q8>::kStages, kStageBytes = Shape<NT, Q8>::kStage, kHalfBytes = Shape<NT, Q8>::kHalf;
    constexpr int kRowBytes = Shape<NT, Q8>::kRowBytes;
    using P = typename std::conditional<Q8, __half, T>::type;  // of the products
    using C = typename std::conditional<Q8, uint8_t, T>::type;  // of the cache
    constexpr float kLift = Q8 ? kHalfLift - kGrow : std::is_same<P, __half>::value ? kHalfLift : 0.f;  // log2 of the probabilities' factor
    constexpr int PIECES = sizeof(O) == 4 && std::is_same<P, __nv_bfloat16>::value ? 3 : 2;  // of a probability
    extern __shared__ __align__(1024) uint8_t dsm[];
    __shared__ long long s_scan[kWarps];
    __shared__ Left s_left[kWarps];
    long long* s_pre = reinterpret_cast<long long*>(dsm);  // before anything is fetched
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- this warp's piece of the stream: equal pieces for the CTAs, cut into equal ones for the warps ----
    Cursor at = {};
    long long piece = 1, begin = 0, seq_begin = 0;  // piece: groups of a CTA
    int len = 0;
    auto cut = [&](long long total) {
        piece = max(divide(total + gridDim.x - 1, gridDim.x), 1LL);
        const long long own = divide(piece + kWarps - 1, kWarps), first = min(total, piece * blockIdx.x);
        const long long past = min(total, first + piece);
        begin = min(past, first + own * warp);
        len = (int)(min(past, begin + own) - begin);
    };
    const int n_parts = CLUSTER ? (int)cg::this_cluster().num_blocks() : 1, part = CLUSTER ? blockIdx.x % n_parts : 0;
    if (CLUSTER) {
        const int unit = blockIdx.x / n_parts;
        at.b = unit / a.units, at.u = unit - at.b * a.units;
        at.s = load_span(a, at.b), at.n = at.s.groups();
        piece = (at.n + n_parts - 1) / n_parts;
        const int own = ((int)piece + kWarps - 1) / kWarps, past = min(at.n, (int)piece * (part + 1));
        at.g = min(past, (int)piece * part + own * warp);
        len = min(past, at.g + own) - at.g;
    } else if (a.B <= 32) {  // every warp by itself
        const Span s = lane < a.B ? load_span(a, lane) : Span{0, 0};
        long long inc = (long long)s.groups() * a.units;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        const long long total = __shfl_sync(0xffffffffu, inc, 31);
        cut(total);
        const int b = min(__popc(__ballot_sync(0xffffffffu, inc <= begin)), 31);
        at.b = b;
        at.s.lo = __shfl_sync(0xffffffffu, s.lo, b);
        at.s.len = __shfl_sync(0xffffffffu, s.len, b);
        at.n = at.s.groups();
        seq_begin = __shfl_sync(0xffffffffu, inc, b) - (long long)at.n * a.units;
    } else {
        long long total = -1, carry = 0;
        if (a.B > kThreads) {  // else the one chunk below gives it
            long long sum = 0;
            for (int b = tid; b < a.B; b += kThreads) sum += load_span(a, b).groups();
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            if (lane == 0) s_scan[warp] = sum;
            __syncthreads();
            total = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) total += s_scan[w];
            total *= a.units;
            __syncthreads();
        }
        for (int base = 0; base < a.B; base += kThreads) {
            const int b = base + tid;
            long long inc = b < a.B ? (long long)load_span(a, b).groups() * a.units : 0;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, inc, s);
                if (lane >= s) inc += o;
            }
            if (base > 0) __syncthreads();  // s_scan and s_pre are reused
            if (lane == 31) s_scan[warp] = inc;
            __syncthreads();
            const long long chunk_begin = carry;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) inc += s_scan[w];
                carry += s_scan[w];
            }
            s_pre[tid] = chunk_begin + inc;  // end of sequence b in the stream
            __syncthreads();
            if (base == 0) {
                if (total < 0) total = carry;
                cut(total);
            }
            if (begin >= chunk_begin && begin < carry) {
                int skip = 0;  // sequences of this chunk that end at or before the piece's begin
#pragma unroll
                for (int i = 0; i < kThreads / 32; ++i)
                    skip += __popc(__ballot_sync(0xffffffffu, s_pre[32 * i + lane] <= begin));
                at.b = base + skip;
                at.s = load_span(a, at.b);
                at.n = at.s.groups();
                seq_begin = s_pre[skip] - (long long)at.n * a.units;
            }
        }
        __syncthreads();  // s_pre lies in the rings
    }
    const int at_n = at.n;  // groups of the cluster's unit
    const Workspace ws = {static_cast<float*>(a.workspace), slot_floats(a.rows), (int)gridDim.x, kWarps};
    if (!CLUSTER && len > 0) {
        const long long in_seq = begin - seq_begin;
        at.u = (int)divide(in_seq, at.n);
        at.g = (int)(in_seq - (long long)at.u * at.n);
    }

    // ---- fetching ----
    uint8_t* own = dsm + warp * kRing;
    const uint32_t ring = smem_addr(own);
    constexpr int kCopyRows = Q8 ? 4 : 2, kCopies = kGroup / kCopyRows;  // a copy instruction covers that many rows
    const int c_row = Q8 ? lane >> 3 : lane >> 4, c_chunk = Q8 ? lane & 7 : lane & 15;
    const int64_t c_off = c_row * a.token_stride + 16 / (int)sizeof(C) * c_chunk;
    const C* kbase = static_cast<const C*>(a.k_cache) + c_off;
    const C* vbase = static_cast<const C*>(a.v_cache) + c_off;
    uint32_t c_dst[8 / kCopyRows];  // row r of a copy: kRowBytes r + 16 (chunk ^ (r mod 8)), r = kCopyRows i + c_row
#pragma unroll
    for (int i = 0; i < 8 / kCopyRows; ++i)
        c_dst[i] = ring + (kCopyRows * i + c_row) * kRowBytes + ((c_chunk ^ (kCopyRows * i + c_row)) << 4);
    Cursor in = at;  // next group to fetch: its token, its page's place in the table, and its page
    auto entry_of = [&](int b, int t) {
        return (int64_t)b * a.max_pages + (a.page_shift >= 0 ? t >> a.page_shift : t / a.page_size);
    };
    int in_t = in.token();
    int64_t entry = entry_of(in.b, in_t);
    int page = len > 0 ? a.page_table[entry] : 0;
    int fetched = 0;
    uint32_t in_stage = 0;
    auto fetch = [&]() {
        if (fetched < len) {
            const bool bad = page < 0 || page >= a.n_pages;
            if (bad && lane == 0) atomicOr(&g_paged_attn_error, 1u);
            const int in_page = a.page_shift >= 0 ? in_t & (a.page_size - 1) : in_t % a.page_size;
            const int64_t o = (int64_t)(bad ? 0 : page) * a.page_stride + (int64_t)(in.u / a.row_blocks) * a.head_stride +
                              (int64_t)in_page * a.token_stride;
            const C* ks = kbase + o;
            const C* vs = vbase + o;
            if (!bad && in_t >= in.s.lo && in_t + kGroup <= in.s.len) {
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const uint32_t d = c_dst[i % (8 / kCopyRows)] + in_stage + (i / (8 / kCopyRows)) * 8 * kRowBytes;
                    cp_async16(d, ks, true);
                    cp_async16(d + kHalfBytes, vs, true);
                    ks += kCopyRows * a.token_stride;
                    vs += kCopyRows * a.token_stride;
                }
            } else {  // rows that are not visible are not read but zero
#pragma unroll 1
                for (int i = 0; i < kCopies; ++i) {
                    const int r = kCopyRows * i + c_row, t = in_t + r;
                    const bool read = !bad && t >= in.s.lo && t < in.s.len;
                    const uint32_t d = ring + in_stage + r * kRowBytes + ((c_chunk ^ (r & 7)) << 4);
                    cp_async16(d, read ? ks : kbase, read);
                    cp_async16(d + kHalfBytes, read ? vs : vbase, read);
                    ks += kCopyRows * a.token_stride;
                    vs += kCopyRows * a.token_stride;
                }
            }
            if constexpr (Q8) {  // the group's 16 exponents of keys, and of values
                const int8_t* es = (lane == 0 ? a.k_exp : a.v_exp) +
                                   ((int64_t)(bad ? 0 : page) * a.Hkv + in.u / a.row_blocks) * a.page_size + in_page;
                if (lane < 2) cp_async16(ring + in_stage + 2 * kHalfBytes + lane * kGroup, es, !bad);
            }
            in_stage = in_stage + kStageBytes < kRing ? in_stage + kStageBytes : 0;
            if (++fetched < len) {
                in.next(a, lane);
                in_t = in.token();
                const int64_t e = entry_of(in.b, in_t);
                if (e != entry) page = a.page_table[e];  // mostly the same page
                entry = e;
            }
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) fetch();

    // sequences with nothing visible: zeros, log-sum-exp -inf
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (load_span(a, b).groups() > 0) continue;
        for (int i = tid; i < a.Hq * kTile / 4; i += kThreads)
            store4(static_cast<O*>(a.out) + (int64_t)b * a.Hq * kTile + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
        if (a.lse != nullptr)
            for (int h = tid; h < a.Hq; h += kThreads) a.lse[(int64_t)b * a.Hq + h] = -CUDART_INF_F;
    }

    // ---- consuming ----
    // products' layout: a lane holds tokens lane / 4 and lane / 4 + 8 (scores) or those channels (output)
    // of the query heads 2 (lane mod 4) and + 1 of each eight
    const int row0 = lane >> 2, col0 = 2 * (lane & 3);
    const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row that this lane addresses
    const int k_row = ((mi & 1) << 3) + mr, k_sel = mi >> 1;
    const int v_row = ((mi >> 1) << 3) + mr, v_sel = mi & 1;
    // where warp w leaves its first unit: beside the rings where that fits
    auto head_slot = [&](int w) -> float* {
        return a.heads_near ? reinterpret_cast<float*>(dsm + kWarps * kRing) + w * ws.stride
                       : ws.warp_slot(blockIdx.x * kWarps + w);
    };
    int done = 0;
    uint32_t stage = 0;
    Left left = {};
    while (done < len) {
        const int b = at.b, u = at.u, g_begin = at.g, n = at.n;
        const Span span = at.s;
        const int steps = min(n - g_begin, len - done);
        const Heads hd = heads_of(a, u);
        const int rows = hd.rows;
        // the unit's queries as the products' right operand, zeros past the last head
        uint32_t qf[NT][8][2];
        float slope[NT][2], q_scale[NT][2];  // (q_scale: Q8, the factor of a head's scores)
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            const int r = 8 * e + row0;
            const T* q = static_cast<const T*>(a.q) + (int64_t)b * a.q_token_stride +
                         (int64_t)(hd.first + (r < rows ? r : 0)) * a.q_head_stride + (Q8 ? 2 * col0 : col0);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qf[e][kk][i] = r < rows ? *reinterpret_cast<const uint32_t*>(q + 16 * kk + (Q8 ? 2 : 8) * i) : 0u;
            if constexpr (Q8) {
                float own_scale = 1.f;
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                        for (int i = 0; i < 2; ++i) top = max(top, max(qf[e][kk][i] & 0x7fffu, (qf[e][kk][i] >> 16) & 0x7fffu));
#pragma unroll
                    for (int d = 1; d < 4; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                    // by 2^-lift the largest lies in [2^14, 2^15)
                    const int lift = min(max((int)(top >> 7) - 127 - 14, -126), 126);
                    const float down = power_of_two(-lift);
                    own_scale = power_of_two(lift);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t x = qf[e][kk][i];
                            const __half2 h = __floats2half2_rn(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xffff0000u) * down);
                            qf[e][kk][i] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) q_scale[e][i] = a.scale * __shfl_sync(0xffffffffu, own_scale, 4 * (col0 + i));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                slope[e][i] = a.slopes != nullptr && 8 * e + col0 + i < rows ? a.slopes[hd.first + 8 * e + col0 + i] : 0.f;
        }
        float o[NT][8][4];
        float m[NT][2], l[NT][2];
        float mo[NT][2];  // the maximum that the output carries: m, or Q8's m'
#pragma unroll
        for (int e = 0; e < NT; ++e) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[e][i][c] = 0.f;
            m[e][0] = m[e][1] = mo[e][0] = mo[e][1] = -CUDART_INF_F;
            l[e][0] = l[e][1] = 0.f;
        }

        for (int st = 0; st < steps; ++st) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            fetch();  // into the stage consumed in the step before
            const uint32_t kb = ring + stage, vb = kb + kHalfBytes;
            stage = stage + kStageBytes < kRing ? stage + kStageBytes : 0;
            float s[NT][2][4] = {};  // [eight][chain]
            int v_exp[2] = {0, 0};    // Q8: exponents of this lane's two tokens' values
            if constexpr (Q8) {
#pragma unroll
                for (int c2 = 0; c2 < 4; ++c2) {  // 32 channels: a lane has four neighbouring ones of each 16
                    uint32_t f[4];
                    ldm4(f, kb + k_row * kRowBytes + (((2 * c2 + k_sel) ^ mr) << 4));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t w[4];
                        halves_of(w[0], w[2], f[2 * i]);
                        halves_of(w[1], w[3], f[2 * i + 1]);
#pragma unroll
                        for (int e = 0; e < NT; ++e) mma(s[e][i], w, qf[e][2 * c2 + i][0], qf[e][2 * c2 + i][1], P());
                    }
                }
                const int8_t* es = reinterpret_cast<const int8_t*>(own + (kb - ring) + 2 * kHalfBytes);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float k_scale = power_of_two(es[row0 + 8 * i]);
                    v_exp[i] = es[kGroup + row0 + 8 * i];
#pragma unroll
                    for (int e = 0; e < NT; ++e)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            s[e][0][2 * i + c] = (s[e][0][2 * i + c] + s[e][1][2 * i + c]) * (k_scale * q_scale[e][c]), s[e][1][2 * i + c] = 0.f;
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    uint32_t f[4];
                    ldm4(f, kb + k_row * kRowBytes + (((2 * kk + k_sel) ^ mr) << 4));
#pragma unroll
                    for (int e = 0; e < NT; ++e) mma(s[e][kk & 1], f, qf[e][kk][0], qf[e][kk][1], P());
                }
            }
            const int t0 = (span.first() + g_begin + st) * kGroup + row0;
            const bool seen[2] = {t0 >= span.lo && t0 < span.len, t0 + 8 >= span.lo && t0 + 8 < span.len};
            const float dist = (float)(t0 - (span.len - 1));
            float mx[NT][2], mv[NT][2];
            bool grew = false;
#pragma unroll
            for (int e = 0; e < NT; ++e) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float x = score<CAP, Q8>(a, s[e][0][c] + s[e][1][c], slope[e][c & 1], dist + 8 * (c >> 1));
                    s[e][0][c] = seen[c >> 1] ? x : -CUDART_INF_F;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mx[e][i] = fmaxf(fmaxf(s[e][0][i], s[e][0][i + 2]), m[e][i]);
                    if constexpr (Q8) {  // this lane's tokens only: the others' are asked when some score passes its maximum by kGrow
                        mv[e][i] = fmaxf(fmaxf(s[e][0][i] + v_exp[0], s[e][0][i + 2] + v_exp[1]), mo[e][i]);
                        grew |= mx[e][i] > m[e][i] + kGrow || mv[e][i] > mo[e][i] + kGrow;
                    } else {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx[e][i] = fmaxf(mx[e][i], __shfl_xor_sync(0xffffffffu, mx[e][i], d));
                        grew |= mx[e][i] > m[e][i];
                    }
                }
            }
            if (__any_sync(0xffffffffu, grew)) {
                if constexpr (Q8) {
#pragma unroll
                    for (int e = 0; e < NT; ++e)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) {
                                mx[e][i] = fmaxf(mx[e][i], __shfl_xor_sync(0xffffffffu, mx[e][i], d));
                                mv[e][i] = fmaxf(mv[e][i], __shfl_xor_sync(0xffffffffu, mv[e][i], d));
                            }
                }
#pragma unroll
                for (int e = 0; e < NT; ++e) {
                    float al[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        al[i] = mx[e][i] > m[e][i] ? exp2f(m[e][i] - mx[e][i]) : 1.f;
                        m[e][i] = mx[e][i];
                        l[e][i] *= al[i];
                        if constexpr (Q8) {
                            al[i] = mv[e][i] > mo[e][i] ? exp2f(mo[e][i] - mv[e][i]) : 1.f;
                            mo[e][i] = mv[e][i];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[e][i][c] *= al[c & 1];
                }
            }
            uint32_t p[NT][PIECES][2];
#pragma unroll
            for (int e = 0; e < NT; ++e) {
                // a row whose scores are all -inf so far has no maximum to subtract
                const float ref[2] = {m[e][0] == -CUDART_INF_F ? 0.f : m[e][0], m[e][1] == -CUDART_INF_F ? 0.f : m[e][1]};
                const float ref_o[2] = {mo[e][0] == -CUDART_INF_F ? 0.f : mo[e][0], mo[e][1] == -CUDART_INF_F ? 0.f : mo[e][1]};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // The lift is added to the difference: a maximum past 2^24 less 15 may be rounded to the maximum
                    // less 16, and 2^16 is no fp16 number any more.
                    float x0 = s[e][0][2 * h] - ref[0], x1 = s[e][0][2 * h + 1] - ref[1];
                    if constexpr (Q8) {
                        l[e][0] += exp2f(x0);
                        l[e][1] += exp2f(x1);
                        x0 = s[e][0][2 * h] + v_exp[h] - ref_o[0];
                        x1 = s[e][0][2 * h + 1] + v_exp[h] - ref_o[1];
                    }
                    if constexpr (kLift != 0.f) x0 += kLift, x1 += kLift;
                    float p0 = exp2f(x0), p1 = exp2f(x1);
                    if constexpr (!Q8) {
                        l[e][0] += p0;
                        l[e][1] += p1;
                    }
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) p[e][i][h] = turn8(take2(p0, p1, P()));
                }
            }
            auto add = [&](int cc, const uint32_t(&f)[4]) {
#pragma unroll
                for (int e = 0; e < NT; ++e) {
                    float d[4] = {};
                    if constexpr (Q8) {
                        mma_first(d, f, p[e][1][0], p[e][1][1]);
                        mma(d, f, p[e][0][0], p[e][0][1], P());
                    } else {
#pragma unroll
                        for (int i = PIECES - 1; i >= 0; --i) mma(d, f, p[e][i][0], p[e][i][1], P());  // the small pieces first
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[e][cc][c] += d[c];
                }
            };
            if constexpr (Q8) {
#pragma unroll
                for (int c2 = 0; c2 < 4; ++c2) {
                    // turned as pairs of channels: a lane has channels 2 j and 2 j + 1 of two tokens, j = lane / 4, and
                    // takes the even channels as the product's rows 0..7 and the odd ones as 8..15
                    uint32_t g[4];
                    ldm4t(g, vb + k_row * kRowBytes + (((2 * c2 + k_sel) ^ mr) << 4));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t x = __byte_perm(g[2 * i], 0, 0x3120), y = __byte_perm(g[2 * i + 1], 0, 0x3120);
                        uint32_t f[4];
                        halves_of(f[0], f[1], x);
                        halves_of(f[2], f[3], y);
                        add(2 * c2 + i, f);
                    }
                }
            } else {
#pragma unroll
                for (int cc = 0; cc < 8; ++cc) {
                    uint32_t f[4];
                    ldm4t(f, vb + v_row * kRowBytes + (((2 * cc + v_sel) ^ mr) << 4));
                    add(cc, f);
                }
            }
            __syncwarp();  // the stage is read before a later step fetches into it
            if (done + st + 1 < len) at.next(a, lane);
        }
        done += steps;

        // ---- end of the unit, or of this warp's part of it ----
        const bool starts = g_begin == 0, ends = g_begin + steps == n;
        const bool whole = !CLUSTER && starts && ends, last = done == len;
        // the last unit of the piece, if not whole, waits in shared memory (this warp's ring is read out) for
        // the join at the CTA's end; one that ended before goes to the workspace
        if (!whole && last) cp_async_wait<0>();
        float* slot = last ? reinterpret_cast<float*>(own) : warp == 0 ? ws.cta_slot(blockIdx.x, 0) : head_slot(warp);
        const int ch0 = Q8 ? 2 * row0 : row0, ch1 = Q8 ? 1 : 8;  // channels of a lane in each 16: the first, and how far the second
#pragma unroll
        for (int e = 0; e < NT; ++e) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (Q8) {  // from the output's maximum and lift to the sum's
                    const float f = mo[e][i] == -CUDART_INF_F ? 0.f : exp2f(mo[e][i] - m[e][i] - kLift);
#pragma unroll
                    for (int cc = 0; cc < 8; ++cc) o[e][cc][i] *= f, o[e][cc][i + 2] *= f;
                }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[e][i] += __shfl_xor_sync(0xffffffffu, l[e][i], d);
                const int r = 8 * e + col0 + i;
                if (r >= rows) continue;
                if (whole) {
                    const int64_t row = (int64_t)b * a.Hq + hd.first + r;
                    const float inv = l[e][i] != 0.f ? 1.f / l[e][i] : 0.f;
                    O* out = static_cast<O*>(a.out) + row * kTile + ch0;
#pragma unroll
                    for (int cc = 0; cc < 8; ++cc) {
                        store1(out + 16 * cc, o[e][cc][i] * inv);
                        store1(out + 16 * cc + ch1, o[e][cc][i + 2] * inv);
                    }
                    if (a.lse != nullptr && row0 == 0) a.lse[row] = lse_of(a, m[e][i], l[e][i]);
                } else {
#pragma unroll
                    for (int cc = 0; cc < 8; ++cc) {
                        slot[r * kTile + 16 * cc + ch0] = o[e][cc][i];
                        slot[r * kTile + 16 * cc + ch0 + ch1] = o[e][cc][i + 2];
                    }
                    if (row0 == 0) {
                        slot[a.rows * kTile + r] = m[e][i];
                        slot[a.rows * kTile + a.rows + r] = l[e][i];
                    }
                }
            }
        }
        if (!whole && last) {
            left.b = b, left.u = u;
            left.flags |= kOpen | (starts ? kStarts : 0u) | (ends ? kEnds : 0u);
            left.end = begin + done - steps + n - 1;
        } else if (!whole) {
            left.flags |= kHead;
        }
    }

    // ---- join of the units that cross warps of this CTA: chains of warps, a row at a time ----
    if (lane == 0) s_left[warp] = left;
    const int cta = blockIdx.x;
    if (!CLUSTER && tid == 0) ws.joins()[cta].b = -1;
    float* near = reinterpret_cast<float*>(dsm);  // warp 0's ring: where a cluster's CTA leaves its part
    if (CLUSTER && len == 0 && warp == 0) {       // no groups of the unit are this CTA's
        for (int r = 0; r < a.rows; ++r) {
            store4(near + r * kTile + 4 * lane, make_float4(0.f, 0.f, 0.f, 0.f));
            if (lane == 0) near[a.rows * kTile + r] = -CUDART_INF_F, near[a.rows * kTile + a.rows + r] = 0.f;
        }
    }
    __syncthreads();
    const unsigned flags = lane < kWarps ? s_left[lane].flags : 0u;
    const unsigned open = __ballot_sync(0xffffffffu, flags & kOpen), begins = __ballot_sync(0xffffffffu, flags & kStarts);
    const unsigned closes = __ballot_sync(0xffffffffu, flags & kEnds), heads = __ballot_sync(0xffffffffu, flags & kHead);
    const unsigned goes_on = open & ~begins;  // warps whose open unit is that of the warp before
    int task = 0;
    for (unsigned firsts = open & (begins | 1u); firsts != 0; firsts &= firsts - 1) {
        // members: the rings of w0 .. w1, and the head slot of w1 + 1 where the unit ends in it
        const int w0 = __ffs(firsts) - 1;
        int w1 = w0;
        while (!(closes >> w1 & 1u) && (goes_on >> (w1 + 1) & 1u)) ++w1;
        const bool tail = !(closes >> w1 & 1u) && (heads >> (w1 + 1) & 1u);
        const bool starts = begins >> w0 & 1u, ends = (closes >> w1 & 1u) || tail;
        const int b = s_left[w0].b, u = s_left[w0].u;
        const Heads hd = heads_of(a, u);
        for (int r = 0; r < hd.rows; ++r, ++task) {
            if (task % kWarps != warp) continue;
            RowPart s = load_part(reinterpret_cast<const float*>(dsm + w0 * kRing), a.rows, r, lane);
            if (tail) join_part(s, load_part(head_slot(w1 + 1), a.rows, r, lane));
#pragma unroll 1
            for (int w = w0 + 1; w <= w1; ++w)
                join_part(s, load_part(reinterpret_cast<const float*>(dsm + w * kRing), a.rows, r, lane));
            if (!CLUSTER && starts && ends) {
                store_row<O>(a, (int64_t)b * a.Hq + hd.first + r, s, lane);
            } else {
                // (in a cluster over row r of warp 0's part, which only this warp reads)
                float* slot = CLUSTER ? near : ws.cta_slot(cta, starts ? 1 : 0);
                __syncwarp();
                *reinterpret_cast<float4*>(slot + r * kTile + 4 * lane) = s.o;
                if (lane == 0) {
                    slot[a.rows * kTile + r] = s.m;
                    slot[a.rows * kTile + a.rows + r] = s.l;
                }
            }
        }
        if (!CLUSTER && starts && !ends && tid == 0) ws.joins()[cta] = Join{b, u, (int)divide(s_left[w0].end, piece), 0};
    }
    if constexpr (CLUSTER) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();  // every CTA's part is in its shared memory
        const int unit = cta / n_parts, b = unit / a.units;
        const Heads hd = heads_of(a, unit - b * a.units);
        for (int r = part + n_parts * warp; at_n > 0 && r < hd.rows; r += n_parts * kWarps) {  // the CTAs first
            RowPart s = load_part(cluster.map_shared_rank(near, 0), a.rows, r, lane);
#pragma unroll 4
            for (int i = 1; i < n_parts; ++i) join_part(s, load_part(cluster.map_shared_rank(near, i), a.rows, r, lane));
            store_row<O>(a, (int64_t)b * a.Hq + hd.first + r, s, lane);
        }
        cluster.sync();  // no CTA leaves while its part is read
    }
}

// One CTA per CTA of the split whose last unit goes on in others.  A warp takes a row, or its share of a
// row's parts where there are fewer rows than warps.  The first parts are loaded before it is known
// whether they are needed: one round trip instead of two.
template <typename O>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(PagedAttnArgs a) {
    __shared__ RowPart s_part[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Workspace ws = {static_cast<float*>(a.workspace), slot_floats(a.rows), (int)gridDim.x, a.rows <= 8 ? Shape<1>::kWarps : Shape<2>::kWarps};
    const int c0 = blockIdx.x;
    static_assert(kRows <= kJoinWarps, "a warp for every row");
    const int share = kJoinWarps / a.rows, sub = warp % share;
    auto load = [&](int i, int r) {  // part 0 is slot 1 of c0, part i slot 0 of c0 + i
        return load_part(ws.cta_slot(min(c0 + i, ws.ctas - 1), i == 0 ? 1 : 0), a.rows, r, lane);
    };
    const Join jn = ws.joins()[c0];
    RowPart ahead[kAhead];
    int r = warp / share;
    if (r < a.rows) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) ahead[k] = load(sub + k * share, r);
    }
    if (jn.b < 0) return;
    const Heads hd = heads_of(a, jn.u);
    const int parts = jn.last - c0 + 1;
    // At most once a warp; written as an `if` it compiles to 32 registers instead of 62, and 256 sequences of 1 to
    // 900 tokens take 99.3 us instead of 98.3.
    for (; r < a.rows; r += kJoinWarps) {
        RowPart s = {-CUDART_INF_F, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        for (int i = sub; i < parts; i += kAhead * share) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i + k * share < parts) join_part(s, ahead[k]);
            if (i + kAhead * share < parts) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) ahead[k] = load(i + (kAhead + k) * share, r);
            }
        }
        if (share == 1) {
            if (r < hd.rows) store_row<O>(a, (int64_t)jn.b * a.Hq + hd.first + r, s, lane);
        } else {
            s_part[warp][lane] = s;
        }
    }
    if (share == 1) return;
    __syncthreads();
    r = warp / share;
    if (sub != 0 || r >= hd.rows) return;
    RowPart s = s_part[warp][lane];
    for (int i = 1; i < share; ++i) join_part(s, s_part[warp + i][lane]);
    store_row<O>(a, (int64_t)jn.b * a.Hq + hd.first + r, s, lane);
}

struct Kernels {
    void (*split)(PagedAttnArgs);
    void (*join)(PagedAttnArgs);
    int ring;  // bytes of a warp's
};
template <typename T, typename O, int NT, bool Q8>
Kernels pick(const PagedAttnArgs& a, bool cluster) {
    const bool cap = a.softcap > 0.f;
    return {cluster ? (cap ? paged_split_kernel<T, O, NT, true, true, Q8> : paged_split_kernel<T, O, NT, false, true, Q8>)
                    : (cap ? paged_split_kernel<T, O, NT, true, false, Q8> : paged_split_kernel<T, O, NT, false, false, Q8>),
            paged_join_kernel<O>, Shape<NT, Q8>::kRing};
}
template <typename T, typename O>
Kernels pick(const PagedAttnArgs& a, bool cluster) {
    return a.rows <= 8 ? pick<T, O, 1, kQ8>(a, cluster) : pick<T, O, 2, kQ8>(a, cluster);
}

// How many clusters of n = 1, 2, 4, 8, 16 of the split's CTAs (one to an SM) run at once; queried once per
// device, since it depends on how a chip's SMs are grouped (152, 76, 36, 15, 7 on the one measured).
cudaError_t cluster_room(int log2n, int dev, int sms, int* room) {
    static std::atomic<int> known[kMaxCachedDevices][5] = {};
    const bool cached = dev >= 0 && dev < kMaxCachedDevices;
    *room = log2n == 0 ? sms : cached ? known[dev][log2n].load(std::memory_order_relaxed) : 0;
    if (*room != 0) return cudaSuccess;
    const auto kern = paged_split_kernel<__nv_bfloat16, float, 1, false, true, kQ8>;
    const int smem = Shape<1, kQ8>::kWarps * Shape<1, kQ8>::kRing;
    cudaError_t e = set_smem_limit_once(kern, smem, false, dev);
    if (e == cudaSuccess) e = allow_large_cluster_once(kern, dev);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1 << log2n;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(1 << log2n);
    lc.blockDim = dim3(Shape<1>::kThreads);
    lc.dynamicSmemBytes = smem;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(room, kern, &lc) != cudaSuccess) {
        cudaGetLastError();  // no such cluster on this device
        *room = 0;
    }
    if (cached) known[dev][log2n].store(*room > 0 ? *room : -1, std::memory_order_relaxed);
    return cudaSuccess;
}

// CTAs of a cluster that takes one unit, 0: the stream is split instead.  A cluster needs no second launch
// (10.8 -> 6.6 us at B 1, 8 kv heads, 512 tokens; 14.3 -> 10.0 at B 16), but a long unit has only its own
// SMs: taken while no warp gets more than four groups, when even one long sequence among empty ones costs
// no more than the split stream (about 10 us).
cudaError_t cluster_ctas(const PagedAttnArgs& a, int64_t unit_groups, int warps, int dev, int sms, int* ctas) {
    const int64_t units = (int64_t)a.B * a.units;
    *ctas = 0;
    for (int log2n = 4; log2n >= 0; --log2n) {
        const int64_t n = 1ll << log2n;
        if (units * n > sms || (log2n > 0 && n / 2 * warps >= unit_groups)) continue;  // a group for every warp
        if (unit_groups > 4 * n * warps) return cudaSuccess;  // nor with a smaller one
        int room = 0;
        const cudaError_t e = cluster_room(log2n, dev, sms, &room);
        if (e != cudaSuccess) return e;
        if (units > room) continue;
        *ctas = (int)n;
        return cudaSuccess;
    }
    return cudaSuccess;
}

int grid_ctas(int64_t max_groups, int warps, int sms) {
    const int64_t fill = (max_groups + warps - 1) / warps;
    const int most = sms < kMaxCtas ? sms : kMaxCtas;
    return (int)(fill < 1 ? 1 : fill < most ? fill : most);
}

}  // namespace

#if !KVARN_PAGED_Q8
size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv) {
    (void)B;
    const int group = Hq / Hkv, rows = group < kRows ? group : kRows;
    const size_t slots = (size_t)kMaxCtas * (kMaxWarps + 2);
    const size_t bytes = slots * slot_floats(rows) * sizeof(float) + kMaxCtas * sizeof(Join);
    return (bytes + 255) & ~(size_t)255;
}

cudaError_t read_and_clear_paged_attn_error(unsigned int* out) { return read_and_clear_word(&g_paged_attn_error, out); }

cudaError_t launch_paged_attention(PagedAttnArgs a, int dtype, cudaStream_t stream) {
#else
cudaError_t read_and_clear_paged_q8_error(unsigned int* out) { return read_and_clear_word(&g_paged_attn_error, out); }

cudaError_t launch_paged_attention_q8(PagedAttnArgs a, int dtype, cudaStream_t stream) {
#endif
    int dev = 0, sms = 0;
    cudaError_t e = current_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    a.group = a.Hq / a.Hkv;
    a.rows = a.group < kRows ? a.group : kRows;
    a.row_blocks = (a.group + kRows - 1) / kRows;
    a.units = a.Hkv * a.row_blocks;
    a.lift = dtype == KVARN_DTYPE_FP16 && !kQ8 ? kHalfLift : 0.f;
    a.inv_softcap = a.softcap > 0.f ? 1.f / a.softcap : 0.f;
    a.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz((unsigned)a.page_size) : -1;
    const bool wide = a.out_dtype == KVARN_DTYPE_FP32;
    const int64_t most = a.window > 0 && a.window < a.max_len ? (int64_t)a.window + kGroup : a.max_len;
    const int64_t unit_groups = (most + kGroup - 1) / kGroup;
    const int warps = a.rows <= 8 ? Shape<1>::kWarps : Shape<2>::kWarps;
    int parts = 0;
    e = cluster_ctas(a, unit_groups, warps, dev, sms, &parts);
    if (e != cudaSuccess) return e;
    const Kernels k = dtype == KVARN_DTYPE_FP16
                          ? (wide ? pick<__half, float>(a, parts > 0) : pick<__half, __half>(a, parts > 0))
                          : (wide ? pick<__nv_bfloat16, float>(a, parts > 0) : pick<__nv_bfloat16, __nv_bfloat16>(a, parts > 0));
    size_t smem = (size_t)warps * k.ring;
    if (parts > 0) {
        e = set_smem_limit_once(k.split, (int)smem, false, dev);
        if (e == cudaSuccess && parts > 8) e = allow_large_cluster_once(k.split, dev);
        if (e != cudaSuccess) return e;
        return launch_pdl_cluster(k.split, dim3(a.B * a.units * parts), parts, dim3(32 * warps), smem, stream, a);
    }
    const int ctas = grid_ctas((int64_t)a.B * a.units * unit_groups, warps, sms);
    const size_t heads = warps * slot_floats(a.rows) * sizeof(float);
    a.heads_near = smem + heads <= kSmemLimit;
    if (a.heads_near) smem += heads;
    e = set_smem_limit_once(k.split, (int)smem, false, dev);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k.split, dim3(ctas), dim3(32 * warps), smem, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(k.join, dim3(ctas), dim3(32 * kJoinWarps), 0, stream, a);
}

}  // namespace kvarn
