// A serving step's page tables and slot maps, built on the device from the requests' lengths.
//
// Mathematics: three exclusive prefix sums over the sequences (tokens added, pages taken, pages given
// back) turn every output into a lookup.  Token t belongs to the last sequence whose prefix is <= t;
// the k-th page taken, counted over the sequences in order, is entry top - 1 - k of the page stack,
// whose part at and above the caller's count is the pages given back in the same order.  So no thread
// waits for another's allotment, and the result does not depend on the schedule.
//
// What bounds it: latency.  A step moves a few words per token and per new page (at most some MB for a
// long prefill) and is a chain of dependent round trips (lengths, stack entry, page table, store) around
// one block-wide scan and one barrier.  One launch, one cluster: every CTA scans all sequences itself,
// which is cheaper than handing prefixes over; the one cluster barrier stands between everything that
// reads the lengths, counts and stack size and their update, which may be in place, and between the
// page table's new entries and the rows that look them up.
#include <cooperative_groups.h>

#include "kvarn_common.cuh"
#include "kvarn_internal.h"

namespace kvarn {

// Set when a step's tables could not be built (status word non-zero).  Read by kvarn_device_error.
__device__ unsigned int g_tables_error = 0;

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxThreads = 1024;
constexpr int kCluster = 16;
constexpr int kPerThread = 8;                // rows in flight per thread
constexpr unsigned kMost = 0x7fffffffu;

// Sums over sequences: new tokens and pages taken (both saturating, beyond every allowed total), pages
// given back (<= B * max_pages <= 2^30).
struct Sums {
    int add, fresh, given;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
    return {(int)min((unsigned)a.add + (unsigned)b.add, kMost), (int)min((unsigned)a.fresh + (unsigned)b.fresh, kMost),
            a.given + b.given};
}
__device__ __forceinline__ Sums shfl_up(Sums v, int s) {
    return {__shfl_up_sync(0xffffffffu, v.add, s), __shfl_up_sync(0xffffffffu, v.fresh, s),
            __shfl_up_sync(0xffffffffu, v.given, s)};
}
__device__ __forceinline__ Sums warp_inclusive(Sums v, int lane) {
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const Sums o = shfl_up(v, s);
        if (lane >= s) v = v + o;
    }
    return v;
}

struct Seq {
    int len, n_new, count;
};

__device__ __forceinline__ Seq load_seq(const StepTablesArgs& a, int b) {
    return {a.seq_lens[b], a.n_new[b], a.page_counts[b]};
}

__device__ __forceinline__ int page_of(const StepTablesArgs& a, int pos) {
    return a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size;
}
__device__ __forceinline__ Sums seq_sums(const StepTablesArgs& a, Seq s, unsigned& bad) {
    if (s.len < 0 || s.count < 0 || s.count > a.max_pages) {
        bad |= KVARN_TABLES_INVALID;
        return {0, 0, 0};
    }
    if (s.n_new < 0) return {0, 0, s.count};
    const long long kv = (long long)s.len + s.n_new;
    int pages;
    if (kv > (long long)kMost) {
        bad |= KVARN_TABLES_INVALID;
        pages = (int)min((kv + a.page_size - 1) / a.page_size, (long long)kMost);
    } else {
        pages = kv > 0 ? page_of(a, (int)kv - 1) + 1 : 0;
    }
    if (pages > a.max_pages) bad |= KVARN_TABLES_ROW_FULL;
    return {s.n_new, max(pages - s.count, 0), 0};
}

// last i in [lo, hi) with pre[i] <= x; pre[lo] <= x
__device__ __forceinline__ int last_at_most(const int* pre, int lo, int hi, int x) {
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The same for the whole warp at once, one x: 32 probes a round.  All lanes return it.
__device__ __forceinline__ int warp_last_at_most(const int* pre, int n, int x, int lane) {
    int lo = 0, width = n;  // the answer is in [lo, lo + width)
    while (width > 1) {
        const int step = (width + 31) >> 5, i = lo + lane * step;
        const unsigned in = __ballot_sync(0xffffffffu, lane * step < width && pre[i] <= x);
        const int k = 31 - __clz(in);  // pre rises, so the set lanes are the first ones; lane 0 is set
        lo += k * step;
        width = min(step, width - k * step);
    }
    return lo;
}

__global__ void __launch_bounds__(kMaxThreads) step_tables_kernel(StepTablesArgs a) {
    extern __shared__ int dsm[];
    __shared__ Sums s_warp[32];
    __shared__ unsigned s_bad;
    int* pre_add = dsm;             // [B] tokens of the sequences before b
    int* pre_fresh = dsm + a.B;     // [B] pages they take
    int* pre_given = dsm + 2 * a.B; // [B] pages they give back
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) s_bad = 0;
    if (tid < 32) s_warp[tid] = Sums{0, 0, 0};
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int F = *a.free_count;
    __syncthreads();

    // prefix sums, one sequence per thread at a time
    Sums carry = {0, 0, 0};
    unsigned bad = 0;
    int my_len = 0;  // of the sequence that the thread took last
    for (int base = 0; base < a.B; base += threads) {
        const int b = base + tid;
        Sums own = {0, 0, 0};
        if (b < a.B) {
            const Seq s = load_seq(a, b);
            my_len = s.len;
            own = seq_sums(a, s, bad);
        }
        const Sums inc = warp_inclusive(own, lane);
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        const Sums all = warp_inclusive(s_warp[lane], lane);
        Sums before;
        before.add = __shfl_sync(0xffffffffu, all.add, max(warp - 1, 0));
        before.fresh = __shfl_sync(0xffffffffu, all.fresh, max(warp - 1, 0));
        before.given = __shfl_sync(0xffffffffu, all.given, max(warp - 1, 0));
        if (warp == 0) before = Sums{0, 0, 0};
        before = carry + before;
        const Sums prev = shfl_up(inc, 1);
        if (lane > 0) before = before + prev;
        if (b < a.B) pre_add[b] = before.add, pre_fresh[b] = before.fresh, pre_given[b] = before.given;
        Sums total;
        total.add = __shfl_sync(0xffffffffu, all.add, 31);
        total.fresh = __shfl_sync(0xffffffffu, all.fresh, 31);
        total.given = __shfl_sync(0xffffffffu, all.given, 31);
        carry = carry + total;
        if (base + threads < a.B) __syncthreads();  // s_warp is reused
    }
    if (bad) atomicOr(&s_bad, bad);
    __syncthreads();
    unsigned status = s_bad;
    const long long left = (long long)F + carry.given - carry.fresh;
    if (F < 0 || F > a.free_capacity) status |= KVARN_TABLES_INVALID;
    if (left < 0) status |= KVARN_TABLES_NO_PAGES;
    if (left > a.free_capacity) status |= KVARN_TABLES_FREE_FULL;
    if (carry.add > a.n_rows) status |= KVARN_TABLES_ROWS;
    const bool ok = status == 0;
    const int total = ok ? (int)carry.add : 0, fresh = ok ? (int)carry.fresh : 0;
    // ok: top = left + fresh <= 2^31, and every index of the stack fits 32 bits
    const unsigned top = (unsigned)F + (unsigned)carry.given, held = (unsigned)F;

    // entry j of the page stack: the caller's, then the pages given back in order
    auto stack = [&](unsigned j) {
        if (j < held) return a.free_pages[j];
        const int r = (int)(j - held);
        const int b = last_at_most(pre_given, 0, a.B, r);
        return a.page_table[(size_t)b * a.max_pages + (r - pre_given[b])];
    };

    const int n_ctas = gridDim.x;
    const int first = blockIdx.x * threads + tid, step = n_ctas * threads;
    const int n_warps = step >> 5, warp_id = first >> 5;

    // ---- pages: taken, and given back for good; one lookup each, all in one round where they fit ----
    const int kept = ok && left > F ? (int)(left - F) : 0;
    for (unsigned k = first; k < (unsigned)fresh + (unsigned)kept; k += step) {
        if (k >= (unsigned)fresh) {
            const unsigned j = held + (k - (unsigned)fresh);
            a.free_pages[j] = stack(j);
            continue;
        }
        const int b = last_at_most(pre_fresh, 0, a.B, (int)k);
        const int i = a.page_counts[b] + ((int)k - pre_fresh[b]);
        const int page = stack(top - 1u - k);
        a.page_table[(size_t)b * a.max_pages + i] = page;
        for (int h = 0; h < a.Hkv; ++h)
            a.block_table[((size_t)b * a.Hkv + h) * a.max_pages + i] = page * a.Hkv + h;
    }
    for (int b = first; b <= a.B; b += step) a.cu_tokens[b] = !ok ? 0 : b < a.B ? pre_add[b] : total;

    // From here on the lengths and counts may be overwritten in place: the old lengths move to shared memory.
    __syncthreads();
    int* old_len = pre_given;
    if (a.B <= threads) {
        if (tid < a.B) old_len[tid] = my_len;
    } else {
        for (int b = tid; b < a.B; b += threads) old_len[b] = a.seq_lens[b];
    }
    if (n_ctas > 1) cg::this_cluster().sync();
    else __syncthreads();

    for (int b = first; b < a.B; b += step) {
        const int len = old_len[b], n_new = a.n_new[b], count = a.page_counts[b];
        int kv = len, pages = count;
        if (ok) {
            kv = n_new < 0 ? 0 : len + n_new;
            pages = n_new < 0 ? 0 : max(count, kv > 0 ? page_of(a, kv - 1) + 1 : 0);
        }
        a.kv_lens[b] = kv;
        a.page_counts_out[b] = pages;
    }
    if (first == 0) {
        *a.free_count_out = ok ? (int)left : F;
        *a.status = (int)status;
        if (!ok) atomicOr(&g_tables_error, 1u);
    }

    // ---- rows ----
    // The rows are cut evenly over the warps, at multiples of 32, and a warp takes 32 * kPerThread at a time:
    // their sequences lie between those of the first and the last, found by the whole warp, and the lookups of
    // a thread's rows overlap.  Every page is in the table by now, written by any CTA of the cluster, hence the
    // loads from L2.
    const int per_warp = ((a.n_rows + n_warps - 1) / n_warps + 31) & ~31;
    const int row_begin = (int)min((long long)warp_id * per_warp, (long long)a.n_rows);
    const int row_end = min(row_begin + per_warp, a.n_rows);
    for (int run = row_begin; run < row_end; run += 32 * kPerThread) {
        const int last = min(min(run + 32 * kPerThread, row_end), total);  // rows run .. last - 1 hold tokens
        int pos[kPerThread], page[kPerThread];
        if (run < total) {
            int b_lo = 0, b_hi = a.B;
            if (a.B > 64) {  // a whole warp's search is two to three probes, a thread's log2(B)
                b_lo = warp_last_at_most(pre_add, a.B, run, lane);
                b_hi = warp_last_at_most(pre_add, a.B, last - 1, lane) + 1;
            }
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                if (run + 32 * i >= last) break;
                const int t = min(run + 32 * i + lane, last - 1);
                const int b = last_at_most(pre_add, b_lo, b_hi, t);
                pos[i] = old_len[b] + (t - pre_add[b]);
                page[i] = __ldcg(a.page_table + (size_t)b * a.max_pages + page_of(a, pos[i]));
            }
        }
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int t = run + 32 * i + lane;
            if (t >= row_end) break;
            int slot = -1;
            if (t < last) slot = (int)((unsigned)page[i] * (unsigned)a.page_size + (unsigned)(pos[i] - page_of(a, pos[i]) * a.page_size));
            a.positions[t] = t < last ? pos[i] : -1;
            a.slot_map[t] = slot;
        }
    }
}

}  // namespace

cudaError_t read_and_clear_tables_error(unsigned int* out) { return read_and_clear_word(&g_tables_error, out); }

cudaError_t launch_step_tables(const StepTablesArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = current_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)3 * a.B * sizeof(int);
    e = set_smem_limit_once(step_tables_kernel, 3 * kMaxTableSeqs * (int)sizeof(int), false, dev);
    if (e == cudaSuccess) e = allow_large_cluster_once(step_tables_kernel, dev);
    if (e != cudaSuccess) return e;
    // One CTA, as small as the step is, until it would take more than two rounds, then the cluster, with more
    // threads once there is a round of four rows for each (us): 64 sequences and rows 2.8, 256 4.3, 1259 rows
    // 3.8 (4.1 in one CTA), 3262 4.8 (5.4 with 1024 threads), 4901 5.5 (6.3), 70778 8.8 (10.6 with 512; 12.0 in a
    // cluster of 8).
    const int most = a.n_rows > a.B ? a.n_rows : a.B;
    const int ctas = most > kMaxThreads ? kCluster : 1;
    const int threads = most <= 128 ? 128 : most > 4 * kCluster * kMaxThreads / 2 ? kMaxThreads : kMaxThreads / 2;
    StepTablesArgs args = a;
    args.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz((unsigned)a.page_size) : -1;
    return launch_pdl_cluster(step_tables_kernel, dim3(ctas), ctas, dim3(threads), smem, stream, args);
}

}  // namespace kvarn
