// Attention of many new tokens per sequence over a paged 16-bit cache, on the 5th-generation tensor cores.
//
// Mathematics, per sequence and query head, for the new token i at position p_i = L - n + i:
//   s_ij = scale q_i.k_j;  s_ij = cap tanh(s_ij / cap)  (cap > 0);  s_ij += slope (j - p_i);
//   out_i = sum_j e^{s_ij - m} v_j / l,  l = sum_j e^{s_ij - m},  lse = m + log l,
// over the visible keys j: start <= j, and p_i - window < j <= p_i when causal, else j < L.  One pass over the
// keys: with (m, l, o) of the keys so far, a tile's scores give m' = max(m, max s), and l and o are scaled by
// e^{m - m'} before its probabilities are added.
//
// What bounds it: 4 * 128 operations for each (row, key), 8.4 M for a tile of 128 rows x 128 keys, against 64 KB of keys
// and values for 256 rows: the tensor cores, or HBM where few rows meet many keys.  So:
//   - the rows of a kv head, (token, query head) pairs, are taken 256 at a time (a unit), whatever the heads per kv head,
//     as two halves of 128 rows = 128 lanes of tensor memory.  Scores (fp32, 128 columns), the probabilities over them (16
//     bit, 64 columns) and the output (fp32, 128 columns) of both halves fill the 512 columns, and a tile's keys and values
//     are read from shared memory for both;
//   - while one half's softmax runs, the other half's P V and next Q K^T do.  The two halves' products take turns: left to
//     themselves they interleaved, both halves finished late and then waited together (1503 us for 2000 rows behind 60k
//     keys, with turns 1341);
//   - a warp for each job: products of a half, copies of keys, of values, queries of a half, the plan, the edges; eight
//     warps of softmax with a row a thread, so that no maximum or sum crosses a thread;
//   - the maximum in use may lag by 2^8: then nothing is scaled, which the output (in tensor memory) mostly spares;
//   - the tiles of all units form one stream that is cut into equal shares, one per SM, whatever the lengths; a unit counts
//     as kUnitCost tiles more than it has (without that 24 packed prompts of 1 to 2000 tokens took 384 us, with it 254).
//     Units that several CTAs share leave partial sums, joined by a second launch;
//   - pages come by tiled copies with the 128-byte swizzle that the products want, in the largest boxes that pages allow.
// A tile of 256 rows takes 3070 to 3250 cycles, 2048 of them at the tensor cores' full rate (63 to 67%): what is left is one
// half's chain, scores -> softmax (1200 cycles) -> P V -> Q K^T (1400 with their latency) and the hand-overs between them.
// The softmax threads' 200 registers do not quite hold a tile's row: 56 to 80 bytes a thread are spilled.  Not kept: the
// probabilities handed over in two parts, turns passed on before a half's Q K^T, spinning waits, and sixteen softmax warps
// with half a row each, whose registers did not suffice.
// Rounding: products are exact in fp32 but for their sums; scores, maxima, sums and outputs are fp32.  Probabilities enter
// P V rounded to the cache's type, as the operand has to be: off by half a step each, at random, so that an output of
// many keys is off by as much as by its own rounding (kvarn_paged_attention, which HBM bounds, takes two or three operands
// for a probability; here a second one would cost half as many products again).  l keeps them unrounded.  fp16 ones are multiplied by 2^7, so that
// with the maximum's lag of 2^8 they use the range of fp16 (p below 2^-21 of the largest lose digits, those below 2^-31 go).
//
// Measured (us): 2000 rows behind 60k keys, 32 over 8 heads, 1300 to 1380 in short runs (1450 to 1540 TFLOP/s, 75 to 79% of
// cuBLAS's burst) and 1520 in long ones, whose clocks the power cap lowers (76% of cuBLAS's sustained rate, 68% of its burst);
// a 16k prompt 1455 and 1490 (78% of the burst, 86% of the sustained rate); 24 prompts of 1 to 2000 tokens 258 (850 TFLOP/s);
// one token 10.
#include <cuda.h>
#include <float.h>
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
constexpr int kThreads = 512;                    // two warpgroups of softmax, then a warp for each of:
constexpr int kKeyWarp = 8, kValueWarp = 9;      //   copies of keys, and of values,
constexpr int kMmaWarp = 10;                     //   products of a half (and 11),
constexpr int kRowWarp = 12;                     //   queries of a half (and 13),
constexpr int kPlanWarp = 14;                    //   the plan, and (15) values at the edges of what a unit sees
constexpr int kPieces = 4, kReaders = 15;        // the planning warp's ring, and the warps that read it
constexpr int kStages = 4;                       // tiles of keys or values on their way (a fifth one gained nothing)
constexpr int kStageBytes = kTile * kTile * 2;   // keys or values of a tile
constexpr int kSpan = kStageBytes / 2;           // 64 channels of it
constexpr int kRowBytes = kHalf * kTile * 2;     // queries of a half
constexpr int kTurnBytes = 32 * 128;             // where a softmax warp lays out 32 rows of 64 channels for a tiled store
constexpr int kSmem = 2 * kRowBytes + kStages * kStageBytes + 8 * kTurnBytes + 1024;
constexpr int kMaxCtas = 160;
constexpr int kMinPart = 2;                      // tiles of a unit that a CTA takes, at least (8 drafts: 2 24, 4 30 us)
constexpr int kUnitCost = 2;                     // what a unit costs beside its tiles, in tiles (24 packed prompts: 0 384,
                                                 // 2 252, 4 261, 5 265 us)
constexpr int kColS = 0, kColO = 256, kCols = 512;  // tensor memory: scores of the halves, then their outputs
constexpr float kGrow = 8.f;                     // how far (in powers of two) scores may pass the maximum in use
constexpr float kLarge = 1048576.f;              // log2 domain; see softmax_tile
constexpr float kHalfLift = 7.f;                 // fp16 probabilities are multiplied by 2^7
constexpr int kSerialUnits = 16;                 // of a sequence, whose tiles one lane counts
constexpr int kJoinRows = 8, kJoinThreads = 256, kJoinAhead = 5, kJoinGrid = 8;
constexpr float kLn2 = 0.69314718055994531f;

struct alignas(16) Join {
    int last;       // the last CTA that holds a part of the unit that slot 1 begins; -1: none
    int h, u;       // the unit,
    int q0, n;      // and its sequence's rows (from here they come a round trip to L2 earlier)
    int unused[3];
};
__host__ __device__ constexpr size_t slot_floats(int rows) { return ((size_t)rows * (kTile + 2) + 7) & ~(size_t)7; }

// Workspace: partial slots (fp32), two per CTA: slot 0 for the unit that began before the CTA's share, slot 1 for the
// one that begins in it and goes on after it; then one Join per CTA, and their `last` once more.  A slot holds o as [32 groups of four
// channels][rows][4], so that neighbouring rows' threads read and write neighbouring 16 bytes, then m[rows] (before
// the scale) and l[rows].
struct Workspace {
    float* base;
    size_t stride;
    int ctas;
    __device__ __forceinline__ float* slot(int cta, int which) const { return base + (2 * (size_t)cta + which) * stride; }
    __device__ __forceinline__ Join* joins() const { return reinterpret_cast<Join*>(slot(ctas, 0)); }
    __device__ __forceinline__ int* lasts() const { return reinterpret_cast<int*>(joins() + ctas); }  // theirs again, side by side
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
// f / group for f below 2^31
__device__ __forceinline__ unsigned token_of(const PromptArgs& a, unsigned f) {
    return a.group == 1 ? f : __umulhi(f, a.group_mul) >> a.group_shift;
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
        k.hi = min(k.hi, shift + (int)token_of(a, f1 - 1) + 1);
        if (a.window > 0) k.lo = max(k.lo, shift + (int)token_of(a, f0) + 1 - a.window);
    }
    return k;
}
// Keys that all of these rows see, of a sequence whose first row has the position `shift`.
__device__ __forceinline__ Keys common_keys(const PromptArgs& a, int start, int len, int shift, unsigned f0, unsigned f1) {
    Keys k = {start, len};
    if (a.causal) {
        k.hi = min(len, shift + (int)token_of(a, f0) + 1);
        if (a.window > 0) k.lo = max(start, shift + (int)token_of(a, f1 - 1) + 1 - a.window);
    }
    return k;
}
// A unit's length in the stream of work: kUnitCost, then its tiles.
__device__ __forceinline__ int cost_of(const PromptArgs& a, const Seq& s, int u) {
    const unsigned f0 = (unsigned)u * kUnit;
    const Keys k = keys_of(a, s, f0, min(f0 + kUnit, (unsigned)s.n * (unsigned)a.group));
    return k.past() - k.first() + kUnitCost;
}

// A CTA's share of one unit, as the planning warp hands it to the others: the tiles [t0, t1), and of them those of
// each half.
struct Piece {
    int t0, t1;          // t1 < t0: nothing more comes
    int a0[2], a1[2];
    int lo, hi;          // keys that some row of the unit sees,
    int all_lo, all_hi;  // and those that all of its rows see
    int b, h, u;
    int q0, shift, len, start, f0;  // the sequence's first row of q, the position of its first row, ...
    int rows;            // of the unit
    int starts, ends;
    int last;            // where the unit begins here and goes on: the last CTA that has a part
    __device__ __forceinline__ int half_rows(int half) const { return min(max(rows - half * kHalf, 0), kHalf); }
};

// A place in the stream of tiles, ordered by (sequence, kv head, unit, tile); run by a whole warp.
struct Walk {
    Seq s;
    int h, u, o, units;
    long long at, end, piece;
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
        p.b = s.b, p.h = h, p.u = u;
        p.q0 = s.q0, p.shift = s.len - s.n, p.len = s.len, p.start = s.start;
        const unsigned f0 = (unsigned)u * kUnit, past = min(f0 + kUnit, (unsigned)s.n * (unsigned)a.group);
        p.f0 = (int)f0;
        p.rows = (int)(past - f0);
        const Keys keys = keys_of(a, s, f0, past);
        p.lo = keys.lo, p.hi = keys.hi;
        const Keys all = common_keys(a, s.start, s.len, p.shift, f0, past);
        p.all_lo = all.lo, p.all_hi = all.hi;
        const int first = keys.first(), cost = keys.past() - first + kUnitCost;
        const int o1 = (int)min((long long)cost, o + (end - at));
        p.t0 = first + max(o - kUnitCost, 0), p.t1 = first + o1 - kUnitCost;
        // the halves: lanes 0 and 1
        const Keys k = keys_of(a, s, min(f0 + (lane & 1) * kHalf, past), min(f0 + ((lane & 1) + 1) * kHalf, past));
        const int a0 = max(k.first(), p.t0), a1 = min(k.past(), p.t1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            p.a0[half] = __shfl_sync(0xffffffffu, a0, half);
            p.a1[half] = __shfl_sync(0xffffffffu, a1, half);
        }
        p.starts = o == 0, p.ends = o1 == cost;
        p.last = 0;
        if (p.starts && !p.ends) {
            // the CTA that takes the unit's last tile; its boundary may have moved to the unit's end
            const long long unit_end = at - o + cost;
            p.last = blockIdx.x;
            while (unit_end - piece * (p.last + 1) >= kMinPart) ++p.last;
        }
        at += o1 - o;
        o = 0;
        ++u;
        return true;
    }
};

// the low n bits (none for n <= 0, all for n >= 32)
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
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
// sum + 0 x, two 16-bit numbers at a time
__device__ __forceinline__ uint32_t add_zero_times(uint32_t x, uint32_t sum, __nv_bfloat16) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0), "r"(sum));
    return r;
}
__device__ __forceinline__ uint32_t add_zero_times(uint32_t x, uint32_t sum, __half) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0), "r"(sum));
    return r;
}
// The waits are in as few instructions as possible: the kernel has three dozen of these, and with each poll loop unrolled
// its code was 145 KB, with these 80 KB (24 packed prompts 437 and 431 us).  A wait for a step of a tile has a second.  One
// that may last for a whole unit has kUnitUs, twice what 2^31 keys take (2 us for 128); it ends with the first of the
// others that gives up.
constexpr uint32_t kUnitUs = 64u << 20;
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, unsigned int* err) {
    return mbar_wait_warp(bar, parity, err, (uint32_t)(kWaitNs / 1000));
}
__device__ __forceinline__ bool wait_unit(uint64_t* bar, uint32_t parity, unsigned int* err) {
    return mbar_wait_warp(bar, parity, err, kUnitUs);
}
// The same with an answer of each lane's own, for a warp that asks for several before it votes.  QUIET: by time only,
// without an error word.
template <bool QUIET = false>
__device__ __forceinline__ bool lane_wait_for(uint64_t* bar, uint32_t parity, unsigned int* err) {
    const uint32_t addr = smem_addr(bar);
    uint32_t began = 0;
#pragma unroll 1
    for (uint32_t i = 0; i < (uint32_t)kSpinLimit; ++i) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done)
            : "r"(addr), "r"(parity)
            : "memory");
        if (done) return true;
        if ((i & 255) == 0) {
            if (!QUIET && *reinterpret_cast<volatile unsigned int*>(err)) return false;
            uint32_t now;
            asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(now));
            if (i == 0) began = now;
            else if (now - began > (uint32_t)kWaitNs) break;
        }
    }
    if (!QUIET) atomicOr(err, kErrTmaTimeout);
    return false;
}
// after a wait that gave up: for a copy or products of this CTA, by time only
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
    lane_wait_for<true>(bar, parity, nullptr);
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

__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_store3(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(c0), "r"(c1),
                 "r"(c2), "r"(smem_addr(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// this thread's stores have read their shared memory, or are done
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct Barriers {
    uint64_t full[kStages], raw[kStages], empty[kStages];
    uint64_t q_full[2], q_free[2], s_full[2], p_full[2], o_full[2], turn[2];
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t gave_up;
};

// The ring of pieces as one of its readers goes through it.
struct Reader {
    uint32_t slot = 0, parity = 0, n = 0;  // n: pieces taken
    // A whole warp waits for the next piece and copies what it needs by `take`; false: nothing more
    template <typename F>
    __device__ __forceinline__ bool next(const Piece* ring, Barriers& bar, unsigned int* err, int lane, F take) {
        if (!wait_unit(&bar.piece_full[slot], parity, err)) return false;
        const Piece& p = ring[slot];
        const bool some = p.t1 >= p.t0;
        if (some) take(p);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.piece_empty[slot]);
        if (++slot == kPieces) slot = 0, parity ^= 1;
        ++n;
        return some;
    }
};

template <typename V>
__device__ __forceinline__ V warp_scan(V v, int lane) {
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const V o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}
// Tiles of a CTA's share, but for the shifts of its boundaries to those of units.
__device__ __forceinline__ long long piece_of(const PromptArgs& a, long long total) {
    // a division by the grid, exact below 2^56
    return max(gridDim.x == 1 ? total : (long long)__umul64hi((unsigned long long)(total + gridDim.x - 1), a.grid_mul), (long long)kMinPart);
}
// Tiles of one kv head's units of sequence base + lane; by a whole warp, a long sequence by all of its lanes.
__device__ __forceinline__ long long seq_cost(const PromptArgs& a, int base, int lane) {
    const bool in = base + lane < a.B;
    const Seq s = in ? load_seq(a, base + lane) : Seq{0, 0, 0, 0, 0};
    const int n = units_of(a, s);
    long long cost = 0;
    if (n <= kSerialUnits)
#pragma unroll 1
        for (int u = 0; u < n; ++u) cost += cost_of(a, s, u);
    for (unsigned many = __ballot_sync(0xffffffffu, n > kSerialUnits); many != 0; many &= many - 1) {
        const int k = __ffs(many) - 1;
        Seq w;
        w.b = 0, w.q0 = 0;
        w.n = __shfl_sync(0xffffffffu, s.n, k);
        w.len = __shfl_sync(0xffffffffu, s.len, k);
        w.start = __shfl_sync(0xffffffffu, s.start, k);
        const int nw = units_of(a, w);
        long long sum = 0;
#pragma unroll 1
        for (int u = 0; u < nw; u += 32) sum += __reduce_add_sync(0xffffffffu, u + lane < nw ? (unsigned)cost_of(a, w, u + lane) : 0u);
        if (lane == k) cost = sum;
    }
    return cost;
}
// Begin (which = 0, with the walk from there) or end of this CTA's share, by one warp, from the sequences' tiles.
__device__ __forceinline__ void plan(const PromptArgs& a, Walk& walk, int which, const long long* s_cost, int lane) {
    long long total = 0;
#pragma unroll 1
    for (int i = lane; i < a.B; i += 32) total += s_cost[i];
    total = __shfl_sync(0xffffffffu, warp_scan(total, lane), 31) * a.Hkv;
    walk.piece = piece_of(a, total);
    long long pos = min(walk.piece * (blockIdx.x + which), total);
    walk.at = pos;
    if (pos >= total) return;
    int b = 0;
    long long in_seq = pos, per_head = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const long long mine = b0 + lane < a.B ? s_cost[b0 + lane] : 0;
        const long long inc = warp_scan(mine, lane) * a.Hkv, all = __shfl_sync(0xffffffffu, inc, 31);
        if (in_seq < all) {
            const int k = __popc(__ballot_sync(0xffffffffu, inc <= in_seq));
            b = b0 + k;
            per_head = __shfl_sync(0xffffffffu, mine, k);
            in_seq -= __shfl_sync(0xffffffffu, inc, k) - per_head * a.Hkv;
            break;
        }
        in_seq -= all;
    }
    const Seq s = load_seq(a, b);
    const int units = units_of(a, s);
    int h = 0;  // in_seq / per_head
#pragma unroll 1
    for (int i = 1; i < a.Hkv; i += 32)
        h += __popc(__ballot_sync(0xffffffffu, i + lane < a.Hkv && (i + lane) * per_head <= in_seq));
    const long long want = in_seq - h * per_head;
    long long before = 0;
    int u = 0, o = 0, cost = 0;
#pragma unroll 1
    for (int u0 = 0; u0 < units; u0 += 32) {
        const unsigned c = u0 + lane < units ? (unsigned)cost_of(a, s, u0 + lane) : 0u;  // (32 of them fit 32 bits)
        const unsigned all = __reduce_add_sync(0xffffffffu, c);
        if (before + all > want) {
            const unsigned sum = warp_scan(c, lane), in = (unsigned)(want - before);
            const int k = __popc(__ballot_sync(0xffffffffu, sum <= in));
            u = u0 + k;
            cost = (int)__shfl_sync(0xffffffffu, c, k);
            o = (int)(in - __shfl_sync(0xffffffffu, sum - c, k));
            break;
        }
        before += all;
    }
    // parts of a unit have kMinPart tiles at least: the boundary moves to the unit's begin or end
    if (o < kUnitCost + kMinPart) {
        pos -= o;
        o = 0;
    } else if (cost - o < kMinPart) {
        pos += cost - o;
        o = 0;
        ++u;
    }
    walk.s = s, walk.h = h, walk.u = u, walk.o = o, walk.units = units;
    walk.at = pos;
}
// lane 0's value, which the compiler then knows to be the same in all lanes
template <typename V>
__device__ __forceinline__ V uniform(V v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ void pair_sync() { asm volatile("bar.sync 1, 64;" ::: "memory"); }  // of the planning and the edge warp

// A tile of a thread's row: its 128 scores at t_s become probabilities there, with the running maximum m and sum l; the
// output at t_o is scaled where the maximum went on by more than kGrow.
__device__ __forceinline__ void scale_output(uint32_t t_o, float top, float c, bool first, float& m, float& l) {
    const float scale = top > m ? exp2_fast((m - top) * c) : 1.f;
    m = top;
    l *= scale;
    if (first) return;
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
// scores x of 32 columns to packed probabilities, added to sum
template <typename T>
__device__ __forceinline__ void probabilities(const uint32_t (&x)[32], uint32_t (&w)[16], float2 c2, float2 ref2, float2 (&sum)[2]) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float2 v = ffma2(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), c2, ref2);
        v.x = exp2_fast(v.x);
        v.y = exp2_fast(v.y);
        sum[k & 1] = fadd2(sum[k & 1], v);
        w[k] = pack2(v.x, v.y, T());
    }
}
__device__ __forceinline__ float max32(const uint32_t (&x)[32], float top) {
    float mx[4] = {top, top, top, top};
#pragma unroll
    for (int k = 0; k < 32; k += 2) mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
    return max3(max3(mx[0], mx[1], mx[2]), mx[3], top);
}
// cap tanh(s / cap), in the log2 domain.  Up to |y| = |s / cap| = 1/4 it is s (1 + z P(z)), z = y^2: P is the polynomial of
// degree 2 whose 1 + z P(z) has the least relative error against tanh(y) / y there (3e-9, by Remez exchange), so that
// such a score is off by its roundings, whatever the cap, and is s itself under a large one.  Beyond that it takes
// tanh y = 1 - 2 / (e^2y + 1), off by 2^-22 or so, 2^-20 of the score at most (near 0 it would be all of a score that is
// small against the cap).  A warp takes the polynomial for a whole tile, and where some score of it is larger the tile
// again, choosing for each score: a 4k prompt under a cap of 50 takes 169 us (by the second formula alone 214, with the
// library's tanhf 361), under one of 5, where every tile is taken again, 293.  A polynomial up to 1/2 takes a degree more:
// 181 and 301; a warp that leaves the polynomial out after such tiles 181 and 253.
constexpr float kNear = 0.0625f;  // of z
__device__ __forceinline__ float2 cap_near(const PromptArgs& a, float2 x, float2& y, float2& z) {
    y = fmul2(x, make_float2(a.cap_scale, a.cap_scale));
    z = fmul2(y, y);
    float2 p = ffma2(z, make_float2(a.near[3], a.near[3]), make_float2(a.near[2], a.near[2]));
    p = ffma2(p, z, make_float2(a.near[1], a.near[1]));
    p = ffma2(p, z, make_float2(a.near[0], a.near[0]));
    return fmul2(x, p);
}
__device__ __forceinline__ float2 cap_far(const PromptArgs& a, float2 y) {
    const float2 e = fmul2(y, make_float2(2.f * kLog2e, 2.f * kLog2e));
    const float2 d = fadd2(make_float2(exp2_fast(e.x), exp2_fast(e.y)), make_float2(1.f, 1.f));
    return ffma2(make_float2(rcp_fast(d.x), rcp_fast(d.y)), make_float2(-2.f * a.cap, -2.f * a.cap), make_float2(a.cap, a.cap));
}
// The scores stay in registers, and their scale waits until the maximum is subtracted.  Columns lo .. hi - 1 are seen.
// GEN: the scores are scaled, capped (CAP) and biased first (d0: position of column 0 less the row's), and c is 1.
// x c - m c takes m c rounded: off by half a step of m c, which no longer matters to the row's sums, but a probability of
// more than 2^16 is no fp16 number, and past 2^31 even fp32 has no room.  So a maximum past 2^20 becomes the row's base
// (`based`: some row of the warp has one), which is subtracted from the scores first; m lies beside it.
template <typename T, bool GEN, bool CAP>
__device__ __forceinline__ void softmax_tile(const PromptArgs& a, uint32_t t_s, uint32_t t_o, int lo, int hi, float c, float slope,
                                             float d0, bool first, float& m, float& l, float& base, bool& based) {
    constexpr float kLift = std::is_same<T, __half>::value ? kHalfLift : 0.f;
    uint32_t x[4][32];
    const bool partial = __any_sync(0xffffffffu, lo > 0 || hi < kTile);
    float less = base;
again:
    if (!GEN && (partial || based)) {
        // hidden scores become -inf in tensor memory, 32 columns at a time: unrolled over the registers below, these
        // instructions, which a unit runs once or twice, cost their fetching (a masked tile took twice a whole one's time)
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const uint32_t seen = bits_below(hi - 32 * i) & ~bits_below(lo - 32 * i);
            if (__all_sync(0xffffffffu, seen == 0xffffffffu) && !based) continue;
            tc::ld32(t_s + 32 * i, x[0]);
            tc::wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) x[0][k] = (seen & (1u << k)) != 0 ? __float_as_uint(__uint_as_float(x[0][k]) - less) : 0xff800000u;
            tc::st32(t_s + 32 * i, x[0]);
        }
        tc::wait_st();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) tc::ld32(t_s + 32 * i, x[i]);
    tc::wait_ld();
    if constexpr (GEN) {
        const float scale = a.score_scale;
        if constexpr (CAP) {
            float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                uint32_t &x0 = x[i >> 4][2 * (i & 15)], &x1 = x[i >> 4][2 * (i & 15) + 1];
                float2 y, z;
                const float2 v = cap_near(a, make_float2(__uint_as_float(x0), __uint_as_float(x1)), y, z);
                top[i & 3] = max3(top[i & 3], z.x, z.y);
                x0 = __float_as_uint(v.x), x1 = __float_as_uint(v.y);
            }
            if (__any_sync(0xffffffffu, fmaxf(max3(top[0], top[1], top[2]), top[3]) > kNear)) {
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    tc::ld32(t_s + 32 * i, x[0]);
                    tc::wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float2 y, z;
                        const float2 near = cap_near(a, make_float2(__uint_as_float(x[0][k]), __uint_as_float(x[0][k + 1])), y, z);
                        const float2 far = cap_far(a, y);
                        x[0][k] = __float_as_uint(z.x <= kNear ? near.x : far.x);
                        x[0][k + 1] = __float_as_uint(z.y <= kNear ? near.y : far.y);
                    }
                    tc::st32(t_s + 32 * i, x[0]);
                }
                tc::wait_st();
#pragma unroll
                for (int i = 0; i < 4; ++i) tc::ld32(t_s + 32 * i, x[i]);
                tc::wait_ld();
            }
        } else {
#pragma unroll
            for (int i = 0; i < 128; ++i) x[i >> 5][i & 31] = __float_as_uint(__uint_as_float(x[i >> 5][i & 31]) * scale);
        }
        if (a.slopes != nullptr) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
                x[i >> 5][i & 31] = __float_as_uint(fmaf(slope, d0 + i, __uint_as_float(x[i >> 5][i & 31])));
        }
    }
    if (GEN && partial) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t seen = bits_below(hi - 32 * i) & ~bits_below(lo - 32 * i);
            if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
#pragma unroll
            for (int k = 0; k < 32; ++k) x[i][k] = (seen & (1u << k)) != 0 ? x[i][k] : 0xff800000u;
        }
    }
    const float top = max3(max3(max32(x[0], m), max32(x[1], m), max32(x[2], m)), max32(x[3], m), m);
    if (__any_sync(0xffffffffu, (top - m) * c > kGrow)) {
        // a large maximum becomes the base, and the tile is taken again without it
        const bool large = !GEN && fabsf(top * c) > kLarge && top != -CUDART_INF_F;
        if (!GEN && __any_sync(0xffffffffu, large)) {
            less = large ? top : 0.f;
            base += less, m -= less;
            based = true;
            goto again;
        }
        scale_output(t_o, top, c, first, m, l);
    }
    // (GEN's scores are rounded as much as their maximum; a lift that is lost to a large one makes probabilities smaller)
    const float ref = GEN ? __fsub_ru(m == -CUDART_INF_F ? 0.f : m, kLift) : (m == -CUDART_INF_F ? 0.f : m * c) - kLift;
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w[2][16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            probabilities<T>(x[2 * i + k], w[k], make_float2(c, c), make_float2(-ref, -ref), sum);
            tc::st16(t_s + 32 * i + 16 * k, w[k]);
        }
    }
    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    tc::wait_st();
}
// Two parts of a row by their log-sum-exps x and y: their shares fx and fy of the whole and its log-sum-exp.
__device__ __forceinline__ float join_lse(float x, float y, float& fx, float& fy) {
    const float top = fmaxf(x, y), ref = top == -CUDART_INF_F ? 0.f : top;
    const float wx = exp2f((x - ref) * kLog2e), wy = exp2f((y - ref) * kLog2e), sum = wx + wy;
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    fx = wx * inv, fy = wy * inv;
    return sum != 0.f ? top + log2f(sum) * kLn2 : -CUDART_INF_F;
}

// The infinities and NaNs among the values of the tokens [from, past), which a row sees, in tiles that not all rows see
// whole (the others' were in the products), added to its output or to its part in a slot: its probabilities are positive,
// whatever they round to.  Rare: straight from the cache, a token after the other.
template <typename T>
__device__ __forceinline__ void add_odd(const PromptArgs& a, int b, int h, int from, int past, Keys all, T* out, float* part,
                                        size_t part_stride) {
    constexpr uint32_t kOdd = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;  // such a value's exponent
#pragma unroll 1
    for (int t = from; t < past; ++t) {
        const int tile = t / kTile * kTile;
        if (tile >= all.lo && tile + kTile <= all.hi) {
            t = all.hi / kTile * kTile - 1;
            continue;
        }
        const int entry = a.page_shift >= 0 ? t >> a.page_shift : t / a.page_size;
        const int page = a.page_table[(int64_t)b * a.max_pages + entry];
        if (page < 0 || page >= a.n_pages) continue;
        const uint16_t* v = reinterpret_cast<const uint16_t*>(static_cast<const T*>(a.v_cache) + (int64_t)page * a.page_stride +
                                                              (int64_t)h * a.head_stride + (int64_t)(t - entry * a.page_size) * a.token_stride);
#pragma unroll 1
        for (int c = 0; c < kTile; ++c) {
            const uint32_t bits = __ldg(v + c), size = bits & 0x7fffu;
            if (size < kOdd) continue;
            const float x = size > kOdd ? CUDART_NAN_F : bits != size ? -CUDART_INF_F : CUDART_INF_F;
            if (out != nullptr) out[c] = T((float)__ldcg(out + c) + x);
            else part[(c >> 2) * part_stride + (c & 3)] += x;
        }
    }
    __syncwarp();
}

// T: type of q, the cache and the output; OWN: each row is joined with a part of its own (kvarn_prefix_attention); GEN:
// scores are capped or biased, or the scale has a sign or size for which the maximum cannot be taken before it; CAP: they
// are capped (with both in one kernel a biased 4k prompt took 173 us for 166).
template <typename T, bool OWN, bool GEN, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_split_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                        const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap o_map, PromptArgs a) {
    constexpr bool kIsHalf = std::is_same<T, __half>::value;
    constexpr float kLift = kIsHalf ? kHalfLift : 0.f;
    constexpr uint32_t kIdescS = kIsHalf ? tc::idesc_f16_f32(128, 128) : tc::idesc_as_bf16(tc::idesc_f16_f32(128, 128));
    constexpr uint32_t kIdescO = kIsHalf ? tc::idesc_f16_f32_bmn(128, 128) : tc::idesc_as_bf16(tc::idesc_f16_f32_bmn(128, 128));
    extern __shared__ uint8_t dsm_raw[];
    __shared__ Barriers bar;
    __shared__ Piece s_piece[kPieces];
    __shared__ int2 s_odd[2 * kPieces];  // tiles of a piece in which the edge warp found values that are no numbers
    __shared__ uint32_t s_tmem;
    __shared__ long long s_end;  // of this CTA's share
    uint8_t* dsm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* rows_smem = dsm;
    uint8_t* ring = dsm + 2 * kRowBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == kMmaWarp) tc::alloc(&s_tmem, kCols);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&bar.full[i], 1), mbar_init(&bar.raw[i], 1), mbar_init(&bar.empty[i], 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1), mbar_init(&bar.q_free[i], 1), mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4), mbar_init(&bar.o_full[i], 1), mbar_init(&bar.turn[i], 1);
        }
        for (int i = 0; i < kPieces; ++i) mbar_init(&bar.piece_full[i], 1), mbar_init(&bar.piece_empty[i], kReaders);
        mbar_init(&bar.gave_up, 2);
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // the tiles of all units form one stream, which is cut into equal pieces: first the tiles of each sequence
    long long* s_cost = reinterpret_cast<long long*>(ring);  // of its units, for one kv head
    static_assert(kMaxPromptSeqs * sizeof(long long) <= (size_t)kStages * kStageBytes, "all sequences' tiles lie in the ring");
#pragma unroll 1
    for (int base = warp * 32; base < a.B; base += kThreads) {
        const long long cost = seq_cost(a, base, lane);
        if (base + lane < a.B) s_cost[base + lane] = cost;
    }
    fence_proxy_async();  // s_cost lies where the copies go
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;
    const Workspace ws = {static_cast<float*>(a.workspace), slot_floats(a.slot_rows), (int)gridDim.x};
    if (tid == 0) ws.joins()[blockIdx.x].last = -1, ws.lasts()[blockIdx.x] = -1;
    unsigned int* const err = &g_prompt_error;

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---- softmax: a thread has a row of its half ----
        const int half = warp >> 2, r = tid & 127;
        uint8_t* const turn = ring + kStages * kStageBytes + warp * kTurnBytes;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t t_s = tmem + lanes + kColS + half * kTile, t_o = tmem + lanes + kColO + half * kTile;
        uint32_t s_parity = 0, o_parity = 0;
        const float c = GEN ? 1.f : a.scale * kLog2e;
        bool fine = true;
        Reader reader;
        struct {
            int first, past, rows, b, h, u, q0, shift, len, start, f0, starts, ends, last;
        } p;
        while (fine && reader.next(s_piece, bar, err, lane, [&](const Piece& from) {
            p.first = from.a0[half], p.past = from.a1[half], p.rows = from.half_rows(half);
            p.b = from.b, p.h = from.h, p.u = from.u, p.q0 = from.q0, p.shift = from.shift, p.len = from.len;
            p.start = from.start, p.f0 = from.f0, p.starts = from.starts, p.ends = from.ends, p.last = from.last;
        })) {
            const int rows = p.rows;
            const bool real = r < rows;
            const unsigned f = (unsigned)p.f0 + half * kHalf + r;
            const int token = (int)token_of(a, f), head = p.h * a.group + (int)(f - (unsigned)token * a.group);
            const int pos = p.shift + token;
            int lo = p.start, hi = p.len;
            if (a.causal) {
                hi = min(hi, pos + 1);
                if (a.window > 0) lo = max(lo, pos + 1 - a.window);
            }
            if (!real) hi = lo;
            const float slope = GEN && a.slopes != nullptr && real ? a.slopes[head] * kLog2e : 0.f;
            float m = -CUDART_INF_F, l = 0.f, base = 0.f;
            bool based = false;
            const int first = p.first, past = p.past;
#pragma unroll 1
            for (int t = first; t < past; ++t) {
                if (!wait_for(&bar.s_full[half], s_parity, err)) {
                    fine = false;
                    break;
                }
                s_parity ^= 1;
                tc::fence_after();
                if ((warp & 3) * 32 < rows) {
                    const int lo_in = lo - t * kTile, hi_in = hi - t * kTile;
                    softmax_tile<T, GEN, CAP>(a, t_s, t_o, lo_in, hi_in, c, slope, (float)(t * kTile - pos), t == first, m, l, base, based);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[half]);
            }
            if (!fine) break;
            const bool any = past > first;
            if (any) {
                if (!wait_for(&bar.o_full[half], o_parity, err)) {
                    fine = false;
                    break;
                }
                o_parity ^= 1;
                tc::fence_after();
            }
            const bool whole = p.starts && p.ends;
            const int64_t row = (int64_t)(p.q0 + token) * a.Hq + head;
            float* slot = ws.slot(blockIdx.x, p.starts ? 1 : 0);
            const int rr = half * kHalf + r;
            float inv = l != 0.f ? 1.f / l : 0.f, lse = l != 0.f ? ((m + base) * c + (log2f(l) - kLift)) * kLn2 : -CUDART_INF_F, own = 0.f;
            if (OWN && real && whole) {
                float share;
                lse = join_lse(lse, a.own_lse[row], share, own);
                inv *= share;
            }
            if ((warp & 3) * 32 < rows) {
                const bool tiled = whole && a.tiled_out && rows >= ((warp & 3) + 1) * 32;  // all of the warp's rows
                T* const out = static_cast<T*>(a.out) + row * kTile;
                const bool zero = whole && __any_sync(0xffffffffu, l == 0.f);  // no key, or only scores of -inf
                const float by = whole ? inv : 1.f;
                // (rolled: code that runs once a unit costs its fetching)
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    uint32_t o[32];
                    if (any) {
                        tc::ld32(t_o + 32 * i, o);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0u;
                    }
                    tc::wait_ld();
                    if (tiled && (i & 1) == 0) {  // the warp's 4 KB are free again
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by);
                    if (zero) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = l != 0.f ? o[k] : 0u;
                    }
                    if (OWN && real && whole) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 w = *reinterpret_cast<const float4*>(a.own_out + row * kTile + 32 * i + 4 * k);
                            o[4 * k] = __float_as_uint(fmaf(own, w.x, __uint_as_float(o[4 * k])));
                            o[4 * k + 1] = __float_as_uint(fmaf(own, w.y, __uint_as_float(o[4 * k + 1])));
                            o[4 * k + 2] = __float_as_uint(fmaf(own, w.z, __uint_as_float(o[4 * k + 2])));
                            o[4 * k + 3] = __float_as_uint(fmaf(own, w.w, __uint_as_float(o[4 * k + 3])));
                        }
                    }
                    if (!whole) {
                        if (real) {
                            uint4* part = reinterpret_cast<uint4*>(slot) + (size_t)8 * i * a.slot_rows + rr;
#pragma unroll
                            for (int k = 0; k < 8; ++k) part[(size_t)k * a.slot_rows] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        }
                        continue;
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) w[k] = pack2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]), T());
                    if (tiled) {
                        uint8_t* const mine = turn + lane * 128;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4*>(mine + (((4 * (i & 1) + k) ^ (lane & 7)) << 4)) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                        if ((i & 1) == 1) {
                            fence_proxy_async();
                            __syncwarp();
                            if (lane == 0) tma_store3(&o_map, turn, 32 * (i - 1), head, p.q0 + token);
                        }
                    } else if (real) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(out + 32 * i)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    }
                }
            }
            const int2 odd = s_odd[(reader.n - 1) % (2 * kPieces)];
            if (any && odd.y >= odd.x) {
                if (lane == 0) bulk_wait_all();
                __syncwarp();
                const unsigned unit = (unsigned)p.f0, unit_past = min(unit + kUnit, (unsigned)(p.len - p.shift) * (unsigned)a.group);
                add_odd<T>(a, p.b, p.h, max(max(odd.x, first) * kTile, lo), l != 0.f ? min(min(odd.y + 1, past) * kTile, hi) : lo,
                           common_keys(a, p.start, p.len, p.shift, unit, unit_past), whole ? static_cast<T*>(a.out) + row * kTile : nullptr,
                           slot + 4 * (size_t)rr, 4 * (size_t)a.slot_rows);
            }
            if (real) {
                if (whole) {
                    if (a.lse != nullptr) a.lse[row] = lse;
                } else {
                    slot[a.slot_rows * kTile + rr] = m + base;
                    slot[a.slot_rows * kTile + a.slot_rows + rr] = l;
                }
            }
            if (tid == 0 && p.starts && !p.ends) {
                ws.joins()[blockIdx.x] = Join{p.last, p.h, p.u, p.q0, p.len - p.shift, {}};
                ws.lasts()[blockIdx.x] = p.last;
            }
            tc::fence_before();
        }
        if (lane == 0) bulk_wait_all();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        Reader reader;
        if (warp == kKeyWarp || warp == kValueWarp) {
            // ---- keys or values, a tile at a time, page by page; the ring has them in turn ----
            const bool values = warp == kValueWarp;
            const CUtensorMap* map = values ? &v_map : &k_map;
            uint32_t stage = values, parity = 1;
            bool fine = true;
            const int boxes = kTile / a.box;
            uint32_t used = 0, on_raw = 0, last_parity = 0, raw_parity = 0;  // a bit for each stage: its last copy, for the way out
            int t0, t1, a0[2], a1[2], lo, hi, all_lo, all_hi, h;
            const int32_t* table;
            while (fine && reader.next(s_piece, bar, err, lane, [&](const Piece& p) {
                t0 = p.t0, t1 = p.t1, lo = p.lo, hi = p.hi, all_lo = p.all_lo, all_hi = p.all_hi, h = p.h;
                a0[0] = p.a0[0], a0[1] = p.a0[1], a1[0] = p.a1[0], a1[1] = p.a1[1];
                table = a.page_table + (int64_t)p.b * a.max_pages;
            })) {
#pragma unroll 1
                for (int t = t0; t < t1; ++t) {
                    if (!((t >= a0[0] && t < a1[0]) || (t >= a0[1] && t < a1[1]))) continue;
                    // lane i: box i of the tile
                    const int tok = t * kTile + lane * a.box;
                    const bool want = lane < boxes && tok < hi && tok + a.box > lo;
                    const int entry = a.page_shift >= 0 ? tok >> a.page_shift : tok / a.page_size, in_page = tok - entry * a.page_size;
                    const int page = want ? table[entry] : 0;
                    const bool bad = want && (page < 0 || page >= a.n_pages);
                    const unsigned good = __ballot_sync(0xffffffffu, want && !bad), zero = __ballot_sync(0xffffffffu, bad);
                    const uint32_t bytes = (uint32_t)__popc(good) * (uint32_t)a.box * (kTile * 2);
                    fine = wait_for(&bar.empty[stage], parity, err);
                    if (!fine) break;
                    uint8_t* dst = ring + stage * kStageBytes;
                    if (zero != 0) {  // keys and values of pages outside the cache count as zeros
                        if (lane == 0) atomicOr(&g_prompt_page_error, 1u);
                        for (unsigned z = zero; z != 0; z &= z - 1) {
                            const int r0 = (__ffs(z) - 1) * a.box;
#pragma unroll 1
                            for (int i = lane; i < a.box * 16; i += 32)
                                *reinterpret_cast<uint4*>(dst + (i & 1) * kSpan + r0 * kTile + (i >> 1) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async();
                        __syncwarp();
                    }
                    // values that some row may not see go through the edge warp
                    const bool edge = values && (t * kTile < all_lo || (t + 1) * kTile > all_hi);
                    uint64_t* b = edge ? &bar.raw[stage] : &bar.full[stage];
                    if (lane == 0) {
                        if (bytes > 0) mbar_expect_tx(b, bytes);
                        else mbar_arrive(b);
                    }
                    __syncwarp();
                    if (want && !bad) {
                        uint8_t* d = dst + lane * a.box * kTile;
                        tma_load4(d, map, 0, in_page, h, page, b);
                        tma_load4(d + kSpan, map, 64, in_page, h, page, b);
                    }
                    __syncwarp();
                    const uint32_t bit = 1u << stage;
                    used |= bit;
                    on_raw = edge ? on_raw | bit : on_raw & ~bit;
                    last_parity = (last_parity & ~bit) | (edge ? raw_parity & bit : parity != 0 ? 0u : bit);
                    if (edge) raw_parity ^= bit;
                    stage += 2;
                    if (stage >= kStages) stage -= kStages, parity ^= 1;
                }
            }
            // No copy and no arrival is on its way when the CTA leaves: the ring's stages behind the last tile, in their
            // order, are every other one for the keys and the ones between for the values.
#pragma unroll 1
            for (int i = values; fine && i < kStages; i += 2) {
                fine = wait_for(&bar.empty[stage], parity, err);
                stage += 2;
                if (stage >= kStages) stage -= kStages, parity ^= 1;
            }
            if (!fine)
#pragma unroll 1
                for (int i = 0; i < kStages; ++i)
                    if (used >> i & 1) drain(on_raw >> i & 1 ? &bar.raw[i] : &bar.full[i], last_parity >> i & 1);
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ---- products of a half: while this warp waits for its half's softmax the other half's run ----
            // An MMA's operands are uniform registers.  With one thread in a branch of its own, and operands that the
            // compiler does not know to be uniform, a warp issued an MMA every 115 to 130 cycles; with elect and
            // operands from lane 0 every 67 (64 is the tensor core's own time).
            const int half = uniform(warp) - kMmaWarp;
            uint32_t stage = 0, parity = 0, q_parity = 0, p_parity = 0, turn_parity = half == 0;  // half 0 goes first
            const uint32_t ring_addr = uniform(smem_addr(ring)), q_addr = uniform(smem_addr(rows_smem)) + half * kRowBytes;
            const uint32_t t_s = uniform(tmem) + kColS + half * kTile, t_o = uniform(tmem) + kColO + half * kTile;
            const uint64_t q_desc = tc::smem_desc_sw128(q_addr, 16, 1024);
            const uint64_t k_desc = tc::smem_desc_sw128(ring_addr, 16, 1024), v_desc = tc::smem_desc_sw128(ring_addr, kSpan, 1024);
            bool fine = true;
            int t, t1, a0, a1, b0, b1;  // tiles of the piece, of this half and of the other
            while (fine && reader.next(s_piece, bar, err, lane, [&](const Piece& p) {
                t = p.t0, t1 = p.t1, a0 = p.a0[half], a1 = p.a1[half], b0 = p.a0[half ^ 1], b1 = p.a1[half ^ 1];
            })) {
                auto pass = [&](uint32_t& st, uint32_t& par) {
                    if (++st == kStages) st = 0, par ^= 1;
                };
                auto my_turn = [&]() {
                    const bool got = lane_wait_for(&bar.turn[half], turn_parity, err);
                    turn_parity ^= 1;
                    return got;
                };
                auto scores = [&](uint32_t st) {  // by the elected lane
                    const uint64_t kd = k_desc + st * (kStageBytes >> 4);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t off = ((k >> 2) * kSpan + (k & 3) * 32) >> 4;
                        tc::mma_f16_ss(t_s, q_desc + off, kd + off, kIdescS, k > 0);
                    }
                    tc::commit(&bar.s_full[half]);
                };
#pragma unroll 1
                for (; t < t1; ++t) {
                    if (!(t >= a0 && t < a1)) {
                        if (!(t >= b0 && t < b1)) continue;
                        // a tile that only the other half takes
#pragma unroll 1
                        for (int i = 0; fine && i < 2; ++i) {
                            fine = __all_sync(0xffffffffu, lane_wait_for(&bar.full[stage], parity, err));
                            if (lane == 0) mbar_arrive(&bar.empty[stage]);
                            pass(stage, parity);
                        }
                        fine = __all_sync(0xffffffffu, fine && my_turn());
                        if (!fine) break;
                        if (lane == 0) mbar_arrive(&bar.turn[half ^ 1]);
                        continue;
                    }
                    if (t == a0) {
                        fine = lane_wait_for(&bar.full[stage], parity, err) && lane_wait_for(&bar.q_full[half], q_parity, err);
                        q_parity ^= 1;
                        if (!__all_sync(0xffffffffu, fine)) break;
                        tc::fence_after();
                        const uint32_t st = uniform(stage), last = uniform(a0 + 1 == a1);
                        if (tc::elect()) {
                            scores(st);
                            tc::commit(&bar.empty[st]);
                            if (last) tc::commit(&bar.q_free[half]);
                        }
                        __syncwarp();
                        pass(stage, parity);
                    }
                    // this tile's values, the next one's keys, this half's probabilities, and the other half's products done
                    uint32_t k_stage = stage, k_parity = parity;
                    pass(k_stage, k_parity);
                    const uint32_t vs = uniform(stage), ks = uniform(k_stage), more = uniform(t > a0), left = uniform(a1 - t - 1);
                    const uint64_t vd = v_desc + vs * (kStageBytes >> 4);
                    fine = lane_wait_for(&bar.full[stage], parity, err) && (left == 0 || lane_wait_for(&bar.full[k_stage], k_parity, err)) &&
                           lane_wait_for(&bar.p_full[half], p_parity, err) && my_turn();
                    p_parity ^= 1;
                    if (!__all_sync(0xffffffffu, fine)) break;
                    tc::fence_after();
                    if (tc::elect()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) tc::mma_f16_ts(t_o, t_s + 8 * k, vd + k * (2048 >> 4), kIdescO, k > 0 ? 1u : more);
                        if (left > 0) {
                            scores(ks);
                            tc::commit(&bar.empty[ks]);
                            if (left == 1) tc::commit(&bar.q_free[half]);
                        } else {
                            tc::commit(&bar.o_full[half]);
                        }
                        tc::commit(&bar.empty[vs]);
                        mbar_arrive(&bar.turn[half ^ 1]);
                    }
                    __syncwarp();
                    pass(stage, parity);
                    if (left > 0) pass(stage, parity);
                }
            }
            if (!fine) {
                if (tc::elect()) tc::commit(&bar.gave_up);
                __syncwarp();
                drain(&bar.gave_up, 0);
            }
        } else if (warp == kRowWarp || warp == kRowWarp + 1) {
            // ---- queries of a half: rows of 256 bytes, gathered, chunk i of a row at i ^ (row mod 8) ----
            const int half = warp - kRowWarp;
            uint32_t free_parity = 1;
            bool fine = true;
            const int chunk = lane & 15;
            const uint32_t dst = smem_addr(rows_smem + half * kRowBytes) + (chunk >> 3) * kSpan + (lane >> 4) * kTile;
            const uint32_t key = (uint32_t)(chunk & 7) ^ (uint32_t)(lane >> 4);
            const T* const base = static_cast<const T*>(a.q) + 8 * chunk;
            int rows, h, q0;
            unsigned f0;
            bool some;
            while (fine && reader.next(s_piece, bar, err, lane, [&](const Piece& p) {
                some = p.a0[half] < p.a1[half];
                f0 = (unsigned)p.f0 + half * kHalf, h = p.h, q0 = p.q0, rows = p.half_rows(half);
            })) {
                if (!some) continue;
                fine = wait_unit(&bar.q_free[half], free_parity, err);
                if (!fine) break;
                free_parity ^= 1;
                if (a.tiled_rows) {
                    // whole tokens' heads; rows behind the unit's last are those of the next tokens and are not used
                    if (lane < 2) {
                        if (lane == 0) mbar_expect_tx(&bar.q_full[half], kRowBytes);
                        __syncwarp(3);
                        tma_load3(rows_smem + half * kRowBytes + lane * kSpan, &q_map, 64 * lane, h * a.group, q0 + (int)token_of(a, f0), &bar.q_full[half]);
                    }
                    __syncwarp();
                    continue;
                }
#pragma unroll 1
                for (int r0 = 0; r0 < kHalf; r0 += 32) {
                    // each lane finds one row's place, then all copy two rows at a time
                    const unsigned f = f0 + min(r0 + lane, rows - 1), token = token_of(a, f);
                    const int64_t at = (int64_t)(q0 + (int)token) * a.q_token_stride +
                                       (int64_t)(h * a.group + (int)(f - token * a.group)) * a.q_head_stride;
#pragma unroll 4
                    for (int r = 0; r < 32; r += 2) {
                        const T* src = base + __shfl_sync(0xffffffffu, at, r + (lane >> 4));
                        cp_async16(dst + (r0 + r) * kTile + ((key ^ (r & 6)) << 4), src, r0 + r + (lane >> 4) < rows);
                    }
                }
                cp_async_commit();
                cp_async_wait<0>();
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.q_full[half]);
            }
            if (fine) wait_unit(&bar.q_free[half], free_parity, err);
        } else {
            // ---- the plan: the share's begin, and by the edge warp its end ----
            Walk walk;
            walk.units = 0;
            plan(a, walk, warp - kPlanWarp, s_cost, lane);
            if (warp > kPlanWarp && lane == 0) s_end = walk.at;
            fence_proxy_async();  // s_cost lies where the copies go, which wait for the plan
            pair_sync();
            walk.end = s_end;
            if (warp == kPlanWarp) {
                uint32_t slot = 0, parity = 1, n = 0;
                for (bool more = true; more; ++n) {
                    Piece p;
                    more = walk.next(a, p, lane);
                    if (!more) p.t0 = 1, p.t1 = 0;
                    if (!wait_unit(&bar.piece_empty[slot], parity, err)) break;
                    if (lane == 0) {
                        s_odd[n % (2 * kPieces)] = make_int2(0x7fffffff, -1);
                        s_piece[slot] = p;
                        mbar_arrive(&bar.piece_full[slot]);
                    }
                    __syncwarp();
                    if (++slot == kPieces) slot = 0, parity ^= 1;
                }
            } else {
                // ---- values that not every row of the unit sees: those outside what any sees become zeros, and so do infinities
                // and NaNs (a probability of 0 would not keep them out); rows that do see one get it in their epilogue ----
                constexpr uint32_t kOdd = kIsHalf ? 0x7c007c00u : 0x7f807f80u;  // exponents of such values
                uint32_t stage = 1, raw_parity = 0;  // the values' stage; a bit for each
                bool fine = true;
                int t0, t1, a0[2], a1[2], lo, hi, all_lo, all_hi;
                while (fine && reader.next(s_piece, bar, err, lane, [&](const Piece& p) {
                    t0 = p.t0, t1 = p.t1, lo = p.lo, hi = p.hi, all_lo = p.all_lo, all_hi = p.all_hi;
                    a0[0] = p.a0[0], a0[1] = p.a0[1], a1[0] = p.a1[0], a1[1] = p.a1[1];
                })) {
#pragma unroll 1
                    for (int t = t0; t < t1; ++t) {
                        if (!((t >= a0[0] && t < a1[0]) || (t >= a0[1] && t < a1[1]))) continue;
                        if (t * kTile < all_lo || (t + 1) * kTile > all_hi) {
                            fine = wait_unit(&bar.raw[stage], (raw_parity >> stage) & 1, err);
                            if (!fine) break;
                            raw_parity ^= 1u << stage;
                            uint8_t* v = ring + stage * kStageBytes;
                            const int lo_in = max(lo - t * kTile, 0), hi_in = min(hi - t * kTile, kTile);
                            // a lane takes a 16-byte chunk of every other row
                            uint8_t* const own = v + ((lane >> 3) & 1) * kSpan + (lane >> 4) * kTile + (lane & 7) * 16;
#pragma unroll 1
                            for (int r = lane >> 4; r < lo_in; r += 2) *reinterpret_cast<uint4*>(own + (r - (lane >> 4)) * kTile) = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                            for (int r = hi_in + ((hi_in ^ (lane >> 4)) & 1); r < kTile; r += 2)
                                *reinterpret_cast<uint4*>(own + (r - (lane >> 4)) * kTile) = make_uint4(0, 0, 0, 0);
                            uint32_t sum[2] = {0, 0};  // of 0 x: a NaN where some x is no number
                            if (max(lo, t * kTile) < all_lo || min(hi, (t + 1) * kTile) > all_hi) {  // not only at the unit's own edges
                                __syncwarp();
#pragma unroll 1
                                for (int r = 0; r < kTile; r += 16) {
                                    uint4 w[8];
#pragma unroll
                                    for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint4*>(own + (r + 2 * i) * kTile);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        sum[0] = add_zero_times(w[i].x, sum[0], T()), sum[1] = add_zero_times(w[i].y, sum[1], T());
                                        sum[0] = add_zero_times(w[i].z, sum[0], T()), sum[1] = add_zero_times(w[i].w, sum[1], T());
                                    }
                                }
                            }
                            if (__any_sync(0xffffffffu, ((sum[0] | sum[1]) & 0x7fff7fffu) != 0)) {
#pragma unroll 1
                                for (int i = lane; i < kTile * 16 * 4; i += 32) {
                                    uint32_t* at = reinterpret_cast<uint32_t*>(v) + i;
                                    *at &= ~__vcmpgeu2(*at & 0x7fff7fffu, kOdd);
                                }
                                if (lane == 0) {
                                    int2& odd = s_odd[(reader.n - 1) % (2 * kPieces)];
                                    odd = make_int2(min(odd.x, t), t);
                                }
                            }
                            fence_proxy_async();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar.full[stage]);
                        }
                        stage += 2;
                        if (stage >= kStages) stage -= kStages;
                    }
                }
            }
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) tc::dealloc(tmem, kCols);
}

// Parts of the units that several CTAs share, joined: CTA (c, y) takes kJoinRows rows of the unit that begins in the
// split's CTA c and goes on after it, and those gridDim.y times as far on, a thread four channels of a row, kJoinAhead
// parts of it at once.
// DIRECT: a CTA takes kJoinRows rows of the unit that one CTA of the split left.  Where that makes more than kJoinGrid rows
// of CTAs, of which most would have nothing to do, each looks up all units first and takes its share of their rows: 128
// sequences behind one prefix 105.8 us (with 32 direct rows 109.3), 8 drafts behind 100 keys, with nothing to join, 12.9 (20
// direct rows: 14.1; kJoinGrid 4: 12.0, but 24 packed prompts then 252.9 instead of 251.1); 4 sequences, 2 direct rows: 21.5
// (looked up 22.1).
__host__ __device__ constexpr int join_blocks(int slot_rows) { return (slot_rows + kJoinRows - 1) / kJoinRows; }
template <typename T, bool OWN, bool DIRECT>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(PromptArgs a) {
    static_assert(kJoinThreads == kJoinRows * kTile / 4, "a thread for each four channels");
    const int tid = threadIdx.x, in = tid % kJoinRows, g = tid / kJoinRows;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Workspace ws = {static_cast<float*>(a.workspace), slot_floats(a.slot_rows), a.ctas};
    if (OWN) {  // rows outside the groups have their own part only
        const int first = min(max(a.cu[0], 0), a.T), past = min(max(a.cu[a.B], first), a.T);
        const int64_t n = (int64_t)(a.T - (past - first)) * a.Hq * (kTile / 4);
        const int64_t step = (int64_t)gridDim.x * gridDim.y * kJoinThreads;
        for (int64_t i = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * kJoinThreads + tid; i < n; i += step) {
            const int64_t skip = (int64_t)first * a.Hq * (kTile / 4), at = i < skip ? i : i + (int64_t)(past - first) * a.Hq * (kTile / 4);
            const float4 v = reinterpret_cast<const float4*>(a.own_out)[at];
            reinterpret_cast<uint2*>(a.out)[at] = make_uint2(pack2(v.x, v.y, T()), pack2(v.z, v.w, T()));
            if (a.lse != nullptr && at % (kTile / 4) == 0) a.lse[at / (kTile / 4)] = a.own_lse[at / (kTile / 4)];
        }
    }
    auto join = [&](const Join& jn, int c0, int block) {
        const int r = block * kJoinRows + in;
        const unsigned f0 = (unsigned)jn.u * kUnit;
        if (r >= (int)(min(f0 + kUnit, (unsigned)jn.n * (unsigned)a.group) - f0)) return;
        const unsigned f = f0 + r, token = token_of(a, f);
        const int64_t row = (int64_t)(jn.q0 + (int)token) * a.Hq + jn.h * a.group + (int)(f - token * a.group);
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        float own_lse = 0.f;
        if (OWN) w = *reinterpret_cast<const float4*>(a.own_out + row * kTile + 4 * g), own_lse = a.own_lse[row];
        float m = -CUDART_INF_F, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0; c <= jn.last; c += kJoinAhead) {
            float4 po[kJoinAhead];
            float pm[kJoinAhead], pl[kJoinAhead];
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) {
                if (c + i > jn.last) break;
                const float* slot = ws.slot(c + i, c + i == c0 ? 1 : 0);
                po[i] = reinterpret_cast<const float4*>(slot)[(size_t)g * a.slot_rows + r];
                pm[i] = slot[a.slot_rows * kTile + r], pl[i] = slot[a.slot_rows * kTile + a.slot_rows + r];
            }
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) {
                if (c + i > jn.last) break;
                const float top = fmaxf(m, pm[i]), ref = top == -CUDART_INF_F ? 0.f : top;
                const float x = exp2f((m - ref) * a.join_scale), y = exp2f((pm[i] - ref) * a.join_scale);
                m = top;
                l = fmaf(y, pl[i], x * l);
                o.x = fmaf(y, po[i].x, x * o.x), o.y = fmaf(y, po[i].y, x * o.y);
                o.z = fmaf(y, po[i].z, x * o.z), o.w = fmaf(y, po[i].w, x * o.w);
            }
        }
        float inv = l != 0.f ? 1.f / l : 0.f, own = 0.f;
        float lse = l != 0.f ? (m * a.join_scale + (log2f(l) - (std::is_same<T, __half>::value ? kHalfLift : 0.f))) * kLn2 : -CUDART_INF_F;
        if (OWN) {
            float share;
            lse = join_lse(lse, own_lse, share, own);
            inv *= share;
        }
        o = l != 0.f ? make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (OWN) o = make_float4(fmaf(own, w.x, o.x), fmaf(own, w.y, o.y), fmaf(own, w.z, o.z), fmaf(own, w.w, o.w));
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * kTile + 4 * g) = make_uint2(pack2(o.x, o.y, T()), pack2(o.z, o.w, T()));
        if (g == 0 && a.lse != nullptr) a.lse[row] = lse;
    };
    if constexpr (DIRECT) {
        const int c0 = blockIdx.x;
        const Join jn = ws.joins()[c0];
        if (jn.last >= 0) join(jn, c0, blockIdx.y);
    } else {
        // the CTAs that left a unit, in the same order for all
        __shared__ int s_cta[kMaxCtas], s_n[kJoinThreads / 32];
        static_assert(kJoinThreads >= kMaxCtas, "a thread for each CTA of the split");
        const bool mine = tid < a.ctas && ws.lasts()[tid] >= 0;
        const unsigned found = __ballot_sync(0xffffffffu, mine);
        if (tid % 32 == 0) s_n[tid / 32] = __popc(found);
        __syncthreads();
        int joins = 0, at = __popc(found & bits_below(tid % 32));
#pragma unroll
        for (int i = 0; i < kJoinThreads / 32; ++i) {
            if (i < tid / 32) at += s_n[i];
            joins += s_n[i];
        }
        if (mine) s_cta[at] = tid;
        __syncthreads();
        const int items = joins * join_blocks(a.slot_rows);
#pragma unroll 1
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const int block = item / joins, c0 = s_cta[item - block * joins];
            const Join jn = ws.joins()[c0];
            join(jn, c0, block);
        }
    }
}

struct Kernels {
    void (*split)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, PromptArgs);
    void (*join)(PromptArgs);
};
template <typename T, bool OWN>
Kernels pick(bool general, bool capped, bool direct) {
    return {capped ? prompt_split_kernel<T, OWN, true, true> : general ? prompt_split_kernel<T, OWN, true, false> : prompt_split_kernel<T, OWN, false, false>,
            direct ? prompt_join_kernel<T, OWN, true> : prompt_join_kernel<T, OWN, false>};
}
template <typename T>
Kernels pick(bool general, bool capped, bool own, bool direct) {
    return own ? pick<T, true>(general, capped, direct) : pick<T, false>(general, capped, direct);
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

// Rows of queries or outputs as channels x heads x tokens, in boxes of 64 channels of `rows` rows: of a kv head's query
// heads and as many tokens as that makes, or of some of the heads.
cudaError_t rows_map(CUtensorMap* map, const PromptArgs& a, int dtype, const void* base, int64_t token_stride, int64_t head_stride,
                     int rows) {
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t sizes[3] = {kTile, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {a.Hq > 1 ? (cuuint64_t)head_stride * 2 : 256, a.T > 1 ? (cuuint64_t)token_stride * 2 : 256};
    const int heads = a.group < rows ? a.group : rows;
    const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)(rows / heads)}, step[3] = {1, 1, 1};
    const CUresult r = encode(map, dtype == KVARN_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                              const_cast<void*>(base), sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int slot_rows(int64_t T, int Hq, int Hkv) {
    const int64_t rows = T * (Hq / Hkv);
    return (int)(rows < 1 ? 1 : rows < kUnit ? rows : kUnit);
}

}  // namespace

size_t prompt_attention_workspace_bytes(int64_t T, int Hq, int Hkv) {
    const size_t bytes = 2 * kMaxCtas * slot_floats(slot_rows(T, Hq, Hkv)) * sizeof(float) + kMaxCtas * (sizeof(Join) + sizeof(int));
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
    // f / group = (f * mul) >> (32 + shift) for f < 2^31: mul = floor(2^(31 + s) / group) + 1, s = ceil(log2 group), is
    // off by less than 2^s / 2^31 of its quotient's last place times f
    int log2_group = 0;
    while ((1 << log2_group) < a.group) ++log2_group;
    a.group_shift = log2_group > 0 ? log2_group - 1 : 0;
    a.group_mul = (uint32_t)((1ull << (31 + log2_group)) / (unsigned)a.group + 1);
    // Scores are taken in the log2 domain.  Factors are kept finite (infinity times a score of 0 would be NaN), and twice
    // the cap too: one past 1.17e38 counts as that, which a score notices only if it is nearly as large.
    const auto finite = [](double x, double most) { return (float)(x > most ? most : x < -most ? -most : x); };
    const double scale = (double)a.scale * (double)kLog2e;
    a.score_scale = finite(scale, FLT_MAX);
    if (a.softcap > 0.f) {
        constexpr double kTanh[4] = {1.0, -0.333332400882, 0.133242366306, -0.0514300288342};  // 1 + z P(z) of cap_near
        a.cap = finite((double)a.softcap * (double)kLog2e, FLT_MAX / 2);
        a.cap_scale = finite(scale / (double)a.cap, FLT_MAX);
        for (int i = 0; i < 4; ++i) a.near[i] = finite(scale * kTanh[i], FLT_MAX);
    }
    a.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz((unsigned)a.page_size) : -1;
    a.box = a.page_size % 128 == 0 ? 128 : a.page_size % 64 == 0 ? 64 : a.page_size % 32 == 0 ? 32 : 16;
    const float c = a.scale * kLog2e;
    const bool general = a.softcap > 0.f || a.slopes != nullptr || !(c >= 1e-30f && c <= 1e30f);
    a.join_scale = general ? 1.f : c;
    const bool own = a.own_out != nullptr;
    const bool direct = join_blocks(a.slot_rows) <= kJoinGrid;
    const Kernels k = dtype == KVARN_DTYPE_FP16 ? pick<__half>(general, a.softcap > 0.f, own, direct) : pick<__nv_bfloat16>(general, a.softcap > 0.f, own, direct);
    CUtensorMap k_map, v_map, q_map = {}, o_map = {};
    // rows come by tiled copies where 128 of them are whole tokens and the strides are ones that the encoding takes
    a.tiled_rows = kHalf % a.group == 0 && (a.Hq == 1 || (a.q_head_stride > 0 && a.q_head_stride < (1ll << 38))) &&
                   (a.T == 1 || (a.q_token_stride > 0 && a.q_token_stride < (1ll << 38)));
    e = cache_map(&k_map, a, dtype, a.k_cache);
    if (e == cudaSuccess) e = cache_map(&v_map, a, dtype, a.v_cache);
    a.tiled_out = e == cudaSuccess && kHalf % a.group == 0 && rows_map(&o_map, a, dtype, a.out, (int64_t)a.Hq * kTile, kTile, 32) == cudaSuccess;
    if (e == cudaSuccess && a.tiled_rows)
        a.tiled_rows = rows_map(&q_map, a, dtype, a.q, a.q_token_stride, a.q_head_stride, kHalf) == cudaSuccess;
    if (e == cudaSuccess) e = set_smem_limit_once(k.split, kSmem, false, dev);
    if (e != cudaSuccess) return e;
    // no more CTAs than parts of kMinPart tiles that the call can have
    const int64_t units = (int64_t)a.Hkv * (((int64_t)a.T * a.group + kUnit - 1) / kUnit + a.B);
    const int64_t parts = units * (((int64_t)a.max_len + 2 * kTile - 1) / kTile);
    const int most = sms < kMaxCtas ? sms : kMaxCtas;
    const int ctas = (int)(parts < 1 ? 1 : parts < most ? parts : most);
    a.grid_mul = ~0ull / (unsigned)ctas + 1;
    a.ctas = ctas;
    e = launch_pdl(k.split, dim3(ctas), dim3(kThreads), kSmem, stream, k_map, v_map, q_map, o_map, a);
    if (e != cudaSuccess) return e;
    if (direct) return launch_pdl(k.join, dim3(ctas, join_blocks(a.slot_rows)), dim3(kJoinThreads), 0, stream, a);
    return launch_pdl(k.join, dim3(ctas * kJoinGrid), dim3(kJoinThreads), 0, stream, a);
}

}  // namespace kvarn
