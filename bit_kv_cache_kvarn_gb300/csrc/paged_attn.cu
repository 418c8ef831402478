// Attention of one new token per sequence over a paged 16-bit cache, split over the cache's length and
// joined.
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
//     form one stream that is cut into equal contiguous pieces, one per warp of a persistent grid
//     (one CTA of 8 warps per SM), so the load is even whatever the lengths;
//   - a warp is on its own: it fetches its next groups into its own 3-stage ring in shared memory
//     (16-byte asynchronous copies, 8 KB per group, 128 to 192 KB in flight per SM) across the ends of
//     units, and never waits for another warp until its piece is done;
//   - the query heads of a kv head are the 16 rows of m16n8k16 products: scores from K as it lies
//     (ldmatrix), then P V with the probabilities taken from the score registers.  A group of 8 KB is
//     48 such products, a quarter of what an SM's warps can issue in the time HBM needs to bring it, so
//     the warp-level products, which need no hand-over between warps, fit better than 128-row
//     tensor-memory tiles that would be at most one eighth full.
// Rounding: the products take the cache's type exactly; scores, maximum, sums and outputs are fp32.
// A probability enters the second product as two 16-bit pieces (p = hi + lo, error 2^-18 for bf16 and
// 2^-22 for fp16), because one piece alone (2^-9) would be the largest error of an fp32 result.  Each
// group's P V is added to the running output by an fp32 addition, rounded to nearest.
#include <math_constants.h>

#include "kvarn_common.cuh"
#include "kvarn_internal.h"

namespace kvarn {

// Set when a page table entry lies outside the cache (its keys and values count as zeros).  Read by
// kvarn_device_error.
__device__ unsigned int g_paged_attn_error = 0;

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kGroup = 16;                             // tokens per step
constexpr int kRows = 16;                              // query heads per unit
constexpr int kHalfBytes = kGroup * kTile * 2;         // K or V of a group
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kMaxCtas = 160;                          // CTAs of a grid, at most
constexpr int kMergeThreads = 128;

// Workspace: partial slots [worker][2], each o[rows][128] then m[rows] and l[rows] (fp32; a slot is a
// multiple of 16 bytes, the join reads four channels at a time), then one Join per worker.  A worker (warp) writes slot 0 for a unit that began before its piece, slot 1 for
// one that begins in its piece and goes on after it.
struct Join {
    int unit_b, unit_u;  // sequence and unit to join, -1: none
    int last;            // the last worker that holds a part
    int pad;
};

__host__ __device__ constexpr size_t slot_floats(int rows) { return ((size_t)rows * (kTile + 2) + 3) & ~(size_t)3; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
    const int n = read ? 16 : 0;  // 0: the 16 bytes are zero-filled
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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
// (x, y) as two 16-bit pieces each: hi + lo
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
    lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo, __half) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ void store2(const PagedAttnArgs& a, int64_t at, float x, float y) {
    if (a.out_dtype == KVARN_DTYPE_FP32) {
        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(x, y);
    } else if (a.out_dtype == KVARN_DTYPE_BF16) {
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at) = __floats2bfloat162_rn(x, y);
    } else {
        *reinterpret_cast<__half2*>(static_cast<__half*>(a.out) + at) = __floats2half2_rn(x, y);
    }
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
    __device__ __forceinline__ void next(const PagedAttnArgs& a) {
        if (++g < n) return;
        g = 0;
        if (++u < a.units) return;
        u = 0;
        do {
            if (++b >= a.B) return;
            s = load_span(a, b);
            n = s.groups();
        } while (n == 0);
    }
    __device__ __forceinline__ int token() const { return (s.first() + g) * kGroup; }
};

__device__ __forceinline__ float score(const PagedAttnArgs& a, float dot, float slope, float dist) {
    // in the log2 domain
    float s = dot * a.scale;
    if (a.softcap > 0.f) {
        // tanh(x) = 1 - 2 / (1 + e^{2x}); saturates to +-1 through e^{2x} = 0 or inf
        const float x = s * a.inv_softcap;
        s = a.softcap * (1.f - 2.f / (1.f + exp2f(x * (2.f * kLog2e))));
    }
    return fmaf(slope, dist, s) * kLog2e;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) paged_split_kernel(PagedAttnArgs a) {
    extern __shared__ __align__(1024) uint8_t dsm[];
    __shared__ long long s_scan[kWarps];
    __shared__ long long s_pre[kThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- this warp's piece of the stream ----
    long long sum = 0;
    for (int b = tid; b < a.B; b += kThreads) sum += load_span(a, b).groups();
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    if (lane == 0) s_scan[warp] = sum;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += s_scan[w];
    total *= a.units;
    const int workers = gridDim.x * kWarps;
    const long long piece = max((total + workers - 1) / workers, 1LL);
    const int worker = blockIdx.x * kWarps + warp;
    const long long begin = min(total, piece * worker);
    const int len = (int)(min(total, begin + piece) - begin);

    Cursor at = {};
    long long seq_begin = 0;  // stream position of the sequence the piece begins in
    {
        long long carry = 0;
        bool found = false;
        for (int base = 0; base < a.B; base += kThreads) {
            const int b = base + tid;
            long long own = b < a.B ? (long long)load_span(a, b).groups() * a.units : 0, inc = own;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, inc, s);
                if (lane >= s) inc += o;
            }
            __syncthreads();  // s_scan and s_pre are reused
            if (lane == 31) s_scan[warp] = inc;
            __syncthreads();
            long long before = carry;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += s_scan[w];
                carry += s_scan[w];
            }
            s_pre[tid] = before + inc;  // end of sequence base + tid
            __syncthreads();
            if (!found && begin < carry) {
                found = true;
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
    }
    // sequences with nothing visible: zeros, log-sum-exp -inf
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (load_span(a, b).groups() > 0) continue;
        for (int i = tid; i < a.Hq * kTile / 2; i += kThreads) store2(a, (int64_t)b * a.Hq * kTile + 2 * i, 0.f, 0.f);
        if (a.lse != nullptr)
            for (int h = tid; h < a.Hq; h += kThreads) a.lse[(int64_t)b * a.Hq + h] = -CUDART_INF_F;
    }
    float* slots = static_cast<float*>(a.workspace);
    Join* joins = reinterpret_cast<Join*>(slots + 2 * (size_t)workers * slot_floats(a.rows));
    if (lane == 0) joins[worker].unit_b = -1;
    if (len == 0) return;
    {
        const long long in_seq = begin - seq_begin;
        at.u = (int)(in_seq / at.n);
        at.g = (int)(in_seq - (long long)at.u * at.n);
    }

    // ---- fetching ----
    const uint32_t ring = smem_addr(dsm) + warp * kStages * kStageBytes;
    const int c_row = lane >> 4, c_chunk = lane & 15;  // a copy instruction covers two rows
    const T* kbase = static_cast<const T*>(a.k_cache) + 8 * c_chunk;
    const T* vbase = static_cast<const T*>(a.v_cache) + 8 * c_chunk;
    Cursor in = at;  // next group to fetch, and its page
    auto page_of = [&](const Cursor& c) { return a.page_table[(int64_t)c.b * a.max_pages + c.token() / a.page_size]; };
    int page = page_of(in);
    int fetched = 0;
    auto fetch = [&]() {
        if (fetched < len) {
            const int t0 = in.token();
            const uint32_t dst = ring + (fetched % kStages) * kStageBytes;
            const bool bad = page < 0 || page >= a.n_pages;
            if (bad && lane == 0) atomicOr(&g_paged_attn_error, 1u);
            const int64_t o = (int64_t)(bad ? 0 : page) * a.page_stride + (int64_t)(in.u / a.row_blocks) * a.head_stride +
                              (int64_t)(t0 % a.page_size) * a.token_stride;
#pragma unroll
            for (int i = 0; i < kGroup / 2; ++i) {
                const int r = 2 * i + c_row, t = t0 + r;
                const bool read = !bad && t >= in.s.lo && t < in.s.len;
                const uint32_t d = dst + r * (kTile * 2) + ((c_chunk ^ (r & 7)) << 4);
                const int64_t src = o + (int64_t)r * a.token_stride;
                cp_async16(d, read ? kbase + src : kbase, read);
                cp_async16(d + kHalfBytes, read ? vbase + src : vbase, read);
            }
            if (++fetched < len) {
                in.next(a);
                page = page_of(in);
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();

    // ---- consuming ----
    const int row0 = lane >> 2, col0 = 2 * (lane & 3);
    const int k_row = ((lane >> 4) << 3) + (lane & 7), k_sel = (lane >> 3) & 1;  // ldmatrix rows of K
    const int v_row = (((lane >> 3) & 1) << 3) + (lane & 7), v_sel = lane >> 4;  // and of V
    int done = 0;
    bool first_unit = true;
    while (done < len) {
        const int b = at.b, u = at.u, g_begin = at.g, n = at.n;
        const Span span = at.s;
        const int steps = min(n - g_begin, len - done);
        const int kvh = u / a.row_blocks, head0 = kvh * a.group + (u - kvh * a.row_blocks) * kRows;
        const int rows = min(a.group - (u - kvh * a.row_blocks) * kRows, kRows);
        // the unit's queries as the products' left operand, zero rows below
        uint32_t qf[8][4];
        {
            const T* q = static_cast<const T*>(a.q) + (int64_t)b * a.q_token_stride + col0;
            const T* q0 = q + (int64_t)(head0 + row0) * a.q_head_stride;
            const T* q1 = q + (int64_t)(head0 + row0 + 8) * a.q_head_stride;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                qf[kk][0] = row0 < rows ? *reinterpret_cast<const uint32_t*>(q0 + 16 * kk) : 0u;
                qf[kk][1] = row0 + 8 < rows ? *reinterpret_cast<const uint32_t*>(q1 + 16 * kk) : 0u;
                qf[kk][2] = row0 < rows ? *reinterpret_cast<const uint32_t*>(q0 + 16 * kk + 8) : 0u;
                qf[kk][3] = row0 + 8 < rows ? *reinterpret_cast<const uint32_t*>(q1 + 16 * kk + 8) : 0u;
            }
        }
        float slope[2] = {0.f, 0.f};
        if (a.slopes != nullptr) {
            if (row0 < rows) slope[0] = a.slopes[head0 + row0];
            if (row0 + 8 < rows) slope[1] = a.slopes[head0 + row0 + 8];
        }
        float o[16][4];
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};

        for (int st = 0; st < steps; ++st, ++done) {
            cp_wait<kStages - 2>();
            __syncwarp();
            fetch();  // into the stage consumed in the step before
            const uint32_t kb = ring + (done % kStages) * kStageBytes, vb = kb + kHalfBytes;
            float s[2][2][4] = {};  // [chain][token half]
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t f[4];
                ldm4(f, kb + k_row * (kTile * 2) + (((2 * kk + k_sel) ^ (k_row & 7)) << 4));
                mma(s[kk & 1][0], qf[kk], f[0], f[1], T());
                mma(s[kk & 1][1], qf[kk], f[2], f[3], T());
            }
            const int t0 = (span.first() + g_begin + st) * kGroup;
            float mx[2] = {m[0], m[1]};
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int t = t0 + 8 * j + col0 + (c & 1);
                    const float x = score(a, s[0][j][c] + s[1][j][c], slope[c >> 1], (float)(t - (span.len - 1)));
                    s[0][j][c] = t >= span.lo && t < span.len ? x : -CUDART_INF_F;
                    mx[c >> 1] = fmaxf(mx[c >> 1], s[0][j][c]);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            }
            if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
                float al[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    al[h] = mx[h] > m[h] ? exp2f(m[h] - mx[h]) : 1.f;
                    m[h] = mx[h];
                    l[h] *= al[h];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[i][0] *= al[0], o[i][1] *= al[0];
                    o[i][2] *= al[1], o[i][3] *= al[1];
                }
            }
            // a row whose scores are all -inf so far has no maximum to subtract
            const float ref[2] = {m[0] == -CUDART_INF_F ? 0.f : m[0], m[1] == -CUDART_INF_F ? 0.f : m[1]};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = exp2f(s[0][j][2 * h] - ref[h]), p1 = exp2f(s[0][j][2 * h + 1] - ref[h]);
                    l[h] += p0 + p1;
                    split2(p0, p1, hi[2 * j + h], lo[2 * j + h], T());
                }
#pragma unroll
            for (int cc = 0; cc < 8; ++cc) {
                uint32_t f[4];
                ldm4t(f, vb + v_row * (kTile * 2) + (((2 * cc + v_sel) ^ (v_row & 7)) << 4));
                float d0[4] = {}, d1[4] = {};
                mma(d0, lo, f[0], f[1], T());
                mma(d1, lo, f[2], f[3], T());
                mma(d0, hi, f[0], f[1], T());
                mma(d1, hi, f[2], f[3], T());
#pragma unroll
                for (int c = 0; c < 4; ++c) o[2 * cc][c] += d0[c], o[2 * cc + 1][c] += d1[c];
            }
            __syncwarp();  // the stage is read before a later step fetches into it
            at.next(a);
        }

        // ---- end of the unit, or of this warp's part of it ----
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        const bool starts_here = g_begin == 0, ends_here = g_begin + steps == n;
        if (starts_here && ends_here) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = row0 + 8 * h;
                if (r >= rows) continue;
                const int64_t row = (int64_t)b * a.Hq + head0 + r;
                const float inv = l[h] != 0.f ? 1.f / l[h] : 0.f;  // 0: no key, or only scores of -inf
#pragma unroll
                for (int i = 0; i < 16; ++i) store2(a, row * kTile + 8 * i + col0, o[i][2 * h] * inv, o[i][2 * h + 1] * inv);
                if (a.lse != nullptr && (lane & 3) == 0)
                    a.lse[row] = l[h] != 0.f ? (m[h] + log2f(l[h])) * 0.69314718055994531f : -CUDART_INF_F;
            }
        } else {
            const int which = first_unit && !starts_here ? 0 : 1;
            float* slot = slots + (2 * (size_t)worker + which) * slot_floats(a.rows);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = row0 + 8 * h;
                if (r >= rows) continue;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    *reinterpret_cast<float2*>(slot + r * kTile + 8 * i + col0) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
                if ((lane & 3) == 0) {
                    slot[a.rows * kTile + r] = m[h];
                    slot[a.rows * kTile + a.rows + r] = l[h];
                }
            }
            if (which == 1 && lane == 0) {
                // the unit's last group, in the stream, tells the last worker that holds a part
                const long long end = begin + done - steps + n - 1;
                joins[worker] = Join{b, u, (int)(end / piece), 0};
            }
        }
        first_unit = false;
    }
}

// One CTA per worker whose last unit goes on in other pieces: a warp takes a query head, a lane four
// channels.
__global__ void __launch_bounds__(kMergeThreads) paged_join_kernel(PagedAttnArgs a, int workers) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float* slots = static_cast<const float*>(a.workspace);
    const size_t stride = slot_floats(a.rows);
    const Join* joins = reinterpret_cast<const Join*>(slots + 2 * (size_t)workers * stride);
    const int w0 = blockIdx.x;
    const Join jn = joins[w0];
    if (jn.unit_b < 0) return;
    const int kvh = jn.unit_u / a.row_blocks, rb = jn.unit_u - kvh * a.row_blocks;
    const int head0 = kvh * a.group + rb * kRows, rows = min(a.group - rb * kRows, kRows);
    const int parts = jn.last - w0 + 1;
    // part 0 is slot 1 of w0, part i slot 0 of w0 + i
    auto part = [&](int i) { return slots + (2 * (size_t)(w0 + i) + (i == 0 ? 1 : 0)) * stride; };
    for (int r = blockIdx.y * (kMergeThreads / 32) + warp; r < rows; r += gridDim.y * (kMergeThreads / 32)) {
        float mx = -CUDART_INF_F;
        for (int i = lane; i < parts; i += 32) mx = fmaxf(mx, part(i)[a.rows * kTile + r]);
        mx = warp_max(mx);
        const float ref = mx == -CUDART_INF_F ? 0.f : mx;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
            const float* p = part(i);
            const float wgt = exp2f(p[a.rows * kTile + r] - ref);
            const float4 v = *reinterpret_cast<const float4*>(p + r * kTile + 4 * lane);
            l = fmaf(wgt, p[a.rows * kTile + a.rows + r], l);
            acc.x = fmaf(wgt, v.x, acc.x);
            acc.y = fmaf(wgt, v.y, acc.y);
            acc.z = fmaf(wgt, v.z, acc.z);
            acc.w = fmaf(wgt, v.w, acc.w);
        }
        const int64_t row = (int64_t)jn.unit_b * a.Hq + head0 + r;
        const float inv = l != 0.f ? 1.f / l : 0.f;
        store2(a, row * kTile + 4 * lane, acc.x * inv, acc.y * inv);
        store2(a, row * kTile + 4 * lane + 2, acc.z * inv, acc.w * inv);
        if (a.lse != nullptr && lane == 0) a.lse[row] = l != 0.f ? (ref + log2f(l)) * 0.69314718055994531f : -CUDART_INF_F;
    }
}

int grid_ctas(int64_t max_groups, int sms) {
    const int64_t fill = (max_groups + kWarps - 1) / kWarps;
    const int most = sms < kMaxCtas ? sms : kMaxCtas;
    return (int)(fill < 1 ? 1 : fill < most ? fill : most);
}

}  // namespace

size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv) {
    (void)B;
    const int group = Hq / Hkv, rows = group < kRows ? group : kRows;
    const size_t workers = (size_t)kMaxCtas * kWarps;
    const size_t bytes = 2 * workers * slot_floats(rows) * sizeof(float) + workers * sizeof(Join);
    return (bytes + 255) & ~(size_t)255;
}

cudaError_t read_and_clear_paged_attn_error(unsigned int* out) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_paged_attn_error, sizeof(v));
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_paged_attn_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

cudaError_t launch_paged_attention(PagedAttnArgs a, int dtype, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = current_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    a.group = a.Hq / a.Hkv;
    a.rows = a.group < kRows ? a.group : kRows;
    a.row_blocks = (a.group + kRows - 1) / kRows;
    a.units = a.Hkv * a.row_blocks;
    a.inv_softcap = a.softcap > 0.f ? 1.f / a.softcap : 0.f;
    const int64_t cap = a.window > 0 && a.window < a.max_len ? (int64_t)a.window + kGroup : a.max_len;
    const int ctas = grid_ctas((int64_t)a.B * a.units * ((cap + kGroup - 1) / kGroup), sms);
    const size_t smem = (size_t)kWarps * kStages * kStageBytes;
    auto kern = dtype == KVARN_DTYPE_BF16 ? paged_split_kernel<__nv_bfloat16> : paged_split_kernel<__half>;
    e = set_smem_limit_once(kern, (int)smem, false, dev);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, stream, a);
    if (e != cudaSuccess) return e;
    const int workers = ctas * kWarps;
    return launch_pdl(paged_join_kernel, dim3(workers, (a.rows + 3) / 4), dim3(kMergeThreads), 0, stream, a, workers);
}

}  // namespace kvarn
