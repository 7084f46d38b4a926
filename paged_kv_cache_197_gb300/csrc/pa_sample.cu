// From logits to tokens or to filtered probabilities (pa_sample.h).
//
// No row is sorted.  The tokens that top-k and top-p leave are those down to a border in the
// order (falling logit, rising index), and the border is searched: the tokens are counted in
// cells of a grid over the logits, which gives the cell of the border (exactly for top-k; for
// top-p as far as cells' mean weights tell); a second pass sums the weights before that cell and
// gathers the cell's tokens, whose sorted list has the border.  Cells with more than kList tokens
// are split on, over their logits and over the indices of equal logits.  A token is then
// drawn by the sums of runs of the vocabulary, which the same pass left, narrowed down to a run, a
// thread's piece of it and an entry; or the row is written.
//
// Weights and sums.  A logit is a grid point and a part of a cell, x = x_k + y, exactly;
// its weight exp(x / T) is exp(x_k / T), one of 4095 entries of a table in whole numbers of 2^-44
// made once a row to 2^-33, plus a correction of at most a 125th of it, w (1 - exp(-y / T)), which
// fp32 and the hardware's exp2 give to 2^-28.5 of w (2^-25 of the smallest).  The whole numbers are summed
// exactly, the corrections of a lane in fp32: 2^-32 of the sum for rows of real and of peaked logits, 2^-28 where a few
// tokens have most of it, and where a vocabulary's small weights are all equal their roundings to the unit
// add up (V half units).  So a border or draw comes out as it does in 64 bits unless two numbers agree to that:
// in 336000 rows of all kinds of logits and filters 79 did not, all of them so.  (fp32 weights and sums
// carry 2^-21: beside a vocabulary's tens of thousands of small weights, one row in a few hundred would
// be cut or drawn elsewhere.  Weights as pairs of fp32 took 45 instructions each, three times as many;
// GB300 has two fp64 lanes per SM and clock.)
//
// Bounds: not the bytes.  A row is a chain of dependent steps (the largest logit, the cells, the border's cell, the sums and the cell's
// tokens, their list, the draw or the row), each of them a pass of instructions or a meeting of the cluster.
// 64 rows of 131072 with top-p take 102 us where their bytes take 5; temperature alone 42; 384 rows of
// probabilities 557 (60).
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "pa_internal.cuh"
#include "pa_sample.h"

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kCells = 4096;  // of the grid; the last one holds all logits whose weight is 0
constexpr int kGroups = 64;   // of 64 cells
constexpr int kSplit = 512;   // bins of a cell that is split
constexpr int kList = 512;    // tokens that are listed (at most one a thread)
// top-k up to which its tokens are listed at once, from the largest logits of the row's parts: half as many as there are parts, so
// that few tokens are not below the k-th of these.  top-k 64 of 64 rows of 131072 takes 47 us so and 66 by the grid; 100 would take
// 60 and 69, 128 101 and 69.
constexpr int kFew = 64;
// Tokens up to a border's cell that are listed instead of summed: a list ends the call without the sums of runs, but ranking it takes
// as many comparisons as its square.  20 mixed rows of 50021 take 90 us with 512, 56 with 128 or 32; one row of 4000 25, 19 and 19.
constexpr int kWhole = 128;
constexpr int kMaxima = 128;  // largest logits of equal parts of a row
constexpr int kUnit = 44;     // a weight of 1 is 2^44
// Bits of a weight that are summed in 32 bits: a CTA has up to 131200 entries (2^20 in 128 runs, rounded up to 8), so 14 are the most.
// The rest is at most 1.01 * 2^16 with 32896 entries a CTA (2^18 a row), and half of that for twice as many: below 2^32 as well.
constexpr int kLimb = 14;
constexpr uint32_t kNone = 0xffffffffu;

struct SampleArgs {
    const void *x;
    int64_t x_stride;
    int32_t *tokens;
    float *token_probs;
    void *probs;
    int64_t p_stride;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int *err_flag;
    int V;
    int cluster;  // CTAs per row
    int run;      // entries of a warp's run (a multiple of 8)
    int drop;     // low bits that weights are short of, so that V of them stay below 2^63
};

// ------------------------------------------------------------------------------ weights
// 2^(j / 1024) = coarse[j / 32] fine[j % 32]; series of exp, in units of 2^-63 and 2^-62.
constexpr double exp_series(double y) {
    double term = 1.0, sum = 1.0;
    for (int n = 1; n < 24; ++n) {
        term *= y / n;
        sum += term;
    }
    return sum;
}
struct Powers {
    uint64_t coarse[32], fine[32];
    constexpr Powers() : coarse(), fine() {
        constexpr double kLn2 = 0.693147180559945309417;
        for (int i = 0; i < 32; ++i) {
            coarse[i] = (uint64_t)(exp_series(i / 32.0 * kLn2) * 9223372036854775808.0);
            fine[i] = (uint64_t)(exp_series(i / 1024.0 * kLn2) * 4611686018427387904.0);
        }
    }
};
__device__ const Powers kPowers = Powers();

// 2^-(turns 2^-56) as a number of 62 bits, in units of 2^-62, and its octaves: 2^-octaves 2^(j / 1024) (1 + q) / 2.
struct Power {
    uint64_t w;
    int octaves;
};
__device__ __forceinline__ Power power(uint64_t turns) {
    constexpr uint64_t kOne = 1ull << 56;
    const uint64_t left = kOne - (turns & (kOne - 1));  // up to the next octave
    uint64_t w = 1ull << 62;
    if (left < kOne) {
        const int j = (int)(left >> 46);
        const float r = (float)(uint32_t)((left >> 22) & 0xffffffu) * 5.8207660913467407e-11f;  // 2^-34
        const float q = r * __fmaf_rn(r, __fmaf_rn(r, 0.0555041087f, 0.240226507f), 0.693147181f);
        w = __umul64hi(kPowers.coarse[j / 32], kPowers.fine[j % 32]);
        w += __umul64hi(w, (uint64_t)__float2uint_rn(q * 2199023255552.f) << 23);  // q in units of 2^-41
    }
    return Power{w, (int)(turns >> 56)};
}

// A row's grid: steps g, a power of two from T / 125.5 on, so that 4095 of them span the 47 octaves in which
// weights are not 0.
struct Grid {
    float base;        // taken off all logits: 0, or the largest where it is far from 0 (exact for all that count)
    float low, high;   // what is left is cut to cells 0 .. kCells - 1
    float magic;       // 1.5 * 2^23 steps: a sum with it is rounded to a grid point
    float point;       // the grid point of the largest logit
    float c, over;     // log2(e) / T and 1 / T
    float unit;        // 2^(kUnit - drop)
    int zero;          // bits of point + magic

    // The cell of a logit (0: the largest one's), what is left of it without the base, and its part of a cell.
    __device__ __forceinline__ int cell(float x, float &y, float &part) const {
        y = fminf(fmaxf(__fsub_rn(x, base), low), high);  // (NaN: low)
        const float s = __fadd_rn(y, magic);
        part = __fsub_rn(y, __fsub_rn(s, magic));
        return (zero - __float_as_int(s)) & (kCells - 1);
    }
    __device__ __forceinline__ int cell(float x) const {
        return (zero - __float_as_int(__fadd_rn(fminf(fmaxf(__fsub_rn(x, base), low), high), magic))) & (kCells - 1);
    }
    // What is to be added to the weight of a part's grid point: the hardware's exp2, to 2^-22, of the whole weight, times
    // 1 - exp(-part / T), |part / T| < 1 / 125: 2^-28.5 of the weight, and 2^-30.5 more for each octave that it is below 1, which the
    // rounding of the exponent costs (2^-25 for the smallest, in which a unit is more).  The unit multiplies the power: in the
    // exponent it would round all of them to 2^-19, 2^-26.5 of the weight.
    __device__ __forceinline__ float rest(float y, float part) const {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(__fsub_rn(y, point), c)));
        const float z = part * over;
        return e * unit * (z * __fmaf_rn(z, __fmaf_rn(z, __fmaf_rn(z, -1.f / 24.f, 1.f / 6.f), -0.5f), 1.f));
    }
};

// The sum of a lane's weights.  It is 0 if and only if all of them are: corrections of weights that
// are 0 do not count.
struct Sum {
    uint64_t whole = 0;
    float rest = 0.f;
    __device__ __forceinline__ uint64_t total() const { return whole ? (uint64_t)max((long long)whole + __float2ll_rn(rest), 1ll) : 0; }
};

// ---------------------------------------------------------------------------- the order
// Keys rise with logits; -0 and 0 are equal, NaN is -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(fmaxf(x, -INFINITY) + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key); }

// A token's place in the order as one number: falling logit, rising index.
__device__ __forceinline__ uint64_t place_of(uint32_t key, int v) { return (uint64_t)~key << 32 | (uint32_t)v; }
__device__ __forceinline__ float logit_at(uint64_t place) { return logit_of(~(uint32_t)(place >> 32)); }

// The lowest key in [lo, hi] of which `holds` is true; it is false below some key, true above,
// and true at hi.  All lanes of a warp, 32 keys at a time.
template <typename F>
__device__ __forceinline__ uint32_t first_key(uint32_t lo, uint32_t hi, int lane, F holds) {
    while (lo < hi) {
        const uint32_t step = (hi - lo) / 32 + 1;
        const uint64_t mine = (uint64_t)lo + (uint64_t)lane * step;
        const unsigned yes = __ballot_sync(0xffffffffu, mine >= hi || holds((uint32_t)mine));
        if (!yes) {  // behind the last of them
            lo += 31 * step + 1;
        } else {
            const int at = __ffs(yes) - 1;
            const uint64_t upper = (uint64_t)lo + (uint64_t)at * step;
            hi = (uint32_t)min((uint64_t)hi, upper);
            if (at == 0) return hi;
            lo += (at - 1) * step + 1;
        }
    }
    return hi;
}

// -------------------------------------------------------------------------------- sums
__device__ __forceinline__ uint64_t warp_sum(uint64_t s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t s, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
    }
    return s;
}

// n f for f in [0, 1), rounded down (f in 64 bits behind the point: exact down to 2^-40), and
// whether something was cut off.
__device__ __forceinline__ uint64_t fraction_of(uint64_t n, float f, bool &cut) {
    const float scaled = f * 4294967296.f, whole = truncf(scaled);
    const uint64_t fixed = (uint64_t)(uint32_t)whole << 32 | (uint32_t)((scaled - whole) * 4294967296.f);
    cut = n * fixed != 0;
    return __umul64hi(n, fixed);
}
// The sum of weights that top-p keeps: tokens stay while the sum before them is below it.
__device__ __forceinline__ uint64_t top_p_goal(uint64_t whole, float top_p) {
    bool cut;
    const uint64_t n = fraction_of(whole, fmaxf(top_p, 0.f), cut);
    return max((uint64_t)1, n + cut);
}
// The running sum that a draw has to exceed (numbers outside [0, 1) give the first or last token).
__device__ __forceinline__ uint64_t draw_goal(uint64_t sum, float u) {
    bool cut;
    return u < 1.f ? fraction_of(sum, fmaxf(u, 0.f), cut) : sum - 1;
}

struct alignas(16) Part {  // a CTA's sums
    uint64_t mass, count, cell_mass, all_mass;
};
// What the CTAs of a cluster tell each other; a place of its own for each step.
enum { kFewSums, kCellBorder, kBins, kRuns, kExchanges };
struct alignas(16) Group {  // of cells: their tokens, and the weights of these at their grid points
    uint64_t mass, count;
};
struct alignas(16) Entry {  // of the list
    uint64_t place, weight;
};
struct alignas(16) Border {
    uint64_t mass_above, count_above, bin, count, mass, unused;
};

struct alignas(16) Shared {
    uint64_t table[kCells];
    uint32_t cells[kCells];      // tokens in each
    uint32_t hist[4][kSplit];    // of a cell that is split: counts, and sums of the weights' lowest kLimb bits, the next kLimb and the rest
    uint64_t own[kList];         // places gathered here
    Entry list[kList];           // all CTAs'
    uint64_t before_mass[kThreads];
    uint32_t before_count[kThreads];
    uint32_t maxima[kMaxima];    // keys
    Group mine[kGroups], groups[kMaxCluster][kGroups];  // this CTA's, and all CTAs'
    Power steps[2][kGroups];     // of the table: exp of 64 steps, and of one
    Part part[kExchanges][kMaxCluster];
    Border border;
    uint64_t warp_mass[kWarps], warp_count[kWarps];
    uint64_t run_mass[kWarps];   // of the runs' tokens before the cell of the border
    uint64_t added[kMaxCluster]; // of the list's tokens that stay, by CTA
    uint64_t cut[2], cut_mass[2];
    uint32_t n_own;
    uint32_t first;              // temperature 0
    uint32_t least;              // a key that top-k's tokens are not below
    Grid grid;
};
extern __shared__ __align__(16) char shared_bytes[];
__device__ __forceinline__ Shared &shared() { return *reinterpret_cast<Shared *>(shared_bytes); }

// ------------------------------------------------------------------- the cluster of a row
// Another CTA's copy of a number in shared memory.  A CTA's own is never reached through the cluster's window: accesses through it
// are ordered by the cluster's barriers, and a cluster of one has block barriers alone.
__device__ __forceinline__ uint32_t remote(const void *p, int rank) {
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
    return a;
}
__device__ __forceinline__ void put(uint64_t *p, uint64_t a, uint64_t b, int to, int rank) {
    if (to == rank) {
        p[0] = a;
        p[1] = b;
    } else {
        asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(remote(p, to)), "l"(a), "l"(b) : "memory");
    }
}
__device__ __forceinline__ void put(uint32_t *p, uint32_t a, int to, int rank) {
    if (to == rank)
        *p = a;
    else
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(p, to)), "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t get(const uint32_t *p, int from, int rank) {
    if (from == rank) return *p;
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, from)) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t get(const uint64_t *p, int from, int rank) {
    if (from == rank) return *p;
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, from)) : "memory");
    return v;
}

// ---------------------------------------------------------------------- a row's entries
// Entries of one 16-byte load; a row is walked in aligned units of them, the first and last
// of which may hang over its ends (those entries read as -inf, and are not loaded).
template <typename T>
constexpr int kVec = 16 / sizeof(T);

__device__ __forceinline__ void unpack(const uint4 &w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(const uint4 &w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float entry(const float *p) { return __ldg(p); }
__device__ __forceinline__ float entry(const uint16_t *p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }
__device__ __forceinline__ uint32_t bits_of(const float *p) { return __float_as_uint(__ldg(p)); }
__device__ __forceinline__ uint32_t bits_of(const uint16_t *p) { return __ldg(p); }

template <typename T>
struct Row {
    const T *base;  // of padded entry 0, 16-byte aligned; entry v is padded entry v + pad
    int pad, end;   // padded entries pad .. end - 1 are the row's

    __device__ __forceinline__ uint4 load(int at) const {
        if (at >= pad && at + kVec<T> <= end) return __ldg(reinterpret_cast<const uint4 *>(base + at));
        uint32_t w[4];
        constexpr int kWord = 4 / (int)sizeof(T);
        constexpr uint32_t kLow = sizeof(T) == 4 ? 0xff800000u : 0xff80u;  // -inf
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = 0;
#pragma unroll
            for (int j = 0; j < kWord; ++j) {
                const int p = at + i * kWord + j;
                w[i] |= (p >= pad && p < end ? bits_of(base + p) : kLow) << (16 * j);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float at(int p) const { return p >= pad && p < end ? entry(base + p) : -INFINITY; }
    // f(entries, padded index of the first) for the units of a warp's run [begin, stop), both multiples of 8
    template <typename F>
    __device__ __forceinline__ void units(int begin, int stop, int lane, F f) const {
        constexpr int N = kVec<T>;
        int p = begin + lane * N;
        uint4 next = make_uint4(0, 0, 0, 0);
        if (p < stop) next = load(p);
#pragma unroll 1
        for (; p < stop; p += 32 * N) {
            const uint4 raw = next;
            if (p + 32 * N < stop) next = load(p + 32 * N);
            float x[N];
            unpack(raw, x);
            f(x, p);
        }
    }
    // f(entry, padded index)
    template <typename F>
    __device__ __forceinline__ void each(int begin, int stop, int lane, F f) const {
        units(begin, stop, lane, [&](const float (&x)[kVec<T>], int p) {
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) f(x[i], p + i);
        });
    }
};

// One logit's weight.
__device__ __forceinline__ uint64_t weight_of(const Grid &grid, float x) {
    float y, part;
    const uint64_t w = shared().table[grid.cell(x, y, part)];
    return w + (uint64_t)__float2ll_rn(grid.rest(y, part));
}

// The same without a table, to 2^-35: the exponent as a pair of fp32, then in 64 bits.
__device__ __forceinline__ uint64_t weight_of(float2 scale, float top, int drop, float x) {
    if (x == top) return 1ull << (kUnit - drop);
    x = fmaxf(x, -INFINITY);
    const float d = __fsub_rn(x, top), b = __fsub_rn(d, x);
    const float e = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(top, b));
    const float t = __fmul_rn(d, scale.x);
    if (!(t > -62.f)) return 0;  // (-inf beside an infinity)
    const float low = __fmaf_rn(e, scale.x, __fmaf_rn(d, scale.y, __fmaf_rn(d, scale.x, -t)));
    const long long turns = __float2ll_rn(-t * 72057594037927936.f) - __float2ll_rn(low * 72057594037927936.f);
    const Power p = power((uint64_t)max(turns, 0ll));
    const int shift = 62 - kUnit + p.octaves + drop;
    return shift > 62 ? 0 : (p.w + (1ull << (shift - 1))) >> shift;
}

// ------------------------------------------------------------------------ steps of a CTA
// The steps are functions of their own (not inlined): each has the registers to itself, what a row's CTAs agree on
// lies in shared memory between them.

// Where a CTA stands: its row's cluster, and a warp's run.
struct Here {
    int C, rank, begin, stop;
};

// (Both halves of a cluster's barrier take whole warps: lanes that parted before one meet first.)
__device__ __forceinline__ void cluster_arrive(int C) {
    __syncwarp();
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait(int C) {
    __syncwarp();
    if (C > 1)
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
        __syncthreads();
}
__device__ __forceinline__ void meet(int C) {
    cluster_arrive(C);
    cluster_wait(C);
}

// The CTAs' sums: every CTA writes its own into all of them, and they meet.  `mine`: the same in the first warp's
// lanes.
__device__ __forceinline__ void exchange(const Here &h, int step, const Part &mine) {
    Part &to = shared().part[step][h.rank];
    if (threadIdx.x < h.C) {
        put(&to.mass, mine.mass, mine.count, threadIdx.x, h.rank);
        put(&to.cell_mass, mine.cell_mass, mine.all_mass, threadIdx.x, h.rank);
    }
    meet(h.C);
}

// Inclusive sums by thread; the warps' sums are left in warp_mass.
__device__ __forceinline__ uint64_t block_scan(uint64_t mass) {
    Shared &sh = shared();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    mass = warp_scan(mass, lane);
    __syncthreads();
    if (lane == 31) sh.warp_mass[warp] = mass;
    __syncthreads();
    const uint64_t m = warp_scan(lane < kWarps ? sh.warp_mass[lane] : 0, lane);
    const uint64_t before = __shfl_sync(0xffffffffu, m, max(warp - 1, 0));
    return warp > 0 ? mass + before : mass;
}
// The sum of a number that each warp has left in an array.
__device__ __forceinline__ uint64_t over_warps(const uint64_t *of) {
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < kWarps ? of[lane] : 0);
}

// What comes before each of the list's n tokens (thread t: entry t) in their order, or by index among the places up to
// `last`: weights and tokens.  All threads share the n^2 comparisons: 64 tokens take a few hundred clocks, a third of what
// sorting them takes, 300 about 10000 with two CTAs per SM, where sorting takes about the same.
template <bool BY_INDEX>
__device__ __noinline__ Entry rank_list(int n, uint64_t last) {
    Shared &sh = shared();
    const int tid = threadIdx.x;
    const int size = n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : kList, parts = kThreads / size;
    const uint64_t place = sh.list[tid & (size - 1)].place, mine = BY_INDEX ? (uint32_t)place : place;
    uint64_t mass = 0;
    uint32_t count = 0;
#pragma unroll 4
    for (int j = tid / size; j < n; j += parts) {
        const Entry e = sh.list[j];
        const bool before = (BY_INDEX ? (uint32_t)e.place : e.place) < mine && (!BY_INDEX || e.place <= last);
        mass += before ? e.weight : 0;
        count += before;
    }
    sh.before_mass[tid] = mass;
    sh.before_count[tid] = count;
    __syncthreads();
    mass = count = 0;
    if (tid < n)
        for (int i = tid; i < kThreads; i += size) {
            mass += sh.before_mass[i];
            count += sh.before_count[i];
        }
    __syncthreads();
    return Entry{mass, count};  // (place: the weights)
}

// The key of a row's largest logit, and the largest keys of kMaxima equal parts of the row: of groups of 4 C lanes.
template <typename T>
__device__ __noinline__ uint32_t find_top(Row<T> row, Here h) {
    Shared &sh = shared();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float m = -INFINITY;
    row.each(h.begin, h.stop, lane, [&](float x, int) { m = fmaxf(m, x); });
    for (int o = 2 * h.C; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int groups = 8 / h.C, share = kMaxima / h.C;  // of a warp, of a CTA
    if (lane % (4 * h.C) == 0) sh.before_count[warp * groups + lane / (4 * h.C)] = key_of(m);
    __syncthreads();
    cluster_wait(h.C);
    if (tid < kMaxima) put(&sh.maxima[h.rank * share + tid % share], sh.before_count[tid % share], tid / share, h.rank);
    meet(h.C);
    const uint32_t a = max(max(sh.maxima[lane], sh.maxima[lane + 32]), max(sh.maxima[lane + 64], sh.maxima[lane + 96]));
    return __reduce_max_sync(0xffffffffu, a);
}

// Temperature 0: the first place of the largest logit.
template <typename T>
__device__ __noinline__ int find_first(Row<T> row, Here h, float top) {
    Shared &sh = shared();
    const int lane = threadIdx.x & 31;
    uint32_t first = kNone;
    row.each(h.begin, h.stop, lane, [&](float x, int p) {
        if (x == top) first = min(first, (uint32_t)p);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) atomicMin(&sh.first, first);
    __syncthreads();
    exchange(h, kRuns, Part{sh.first, 0, 0, 0});
    for (int c = 0; c < h.C; ++c) first = min(first, (uint32_t)sh.part[kRuns][c].mass);
    return (int)first;
}

// log2(e) / T as a pair: the remainder of the division is exact.  T is cut to 2^-60 .. 2^80.
__device__ __forceinline__ float2 scale_of(float temperature) {
    const float t = fminf(fmaxf(temperature, 8.6736174e-19f), 1.2089258e24f);
    constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;
    const float hi = __fdiv_rn(kHi, t);
    return make_float2(hi, __fdiv_rn(__fadd_rn(__fmaf_rn(-hi, t, kHi), kLo), t));
}

__device__ __forceinline__ float step_of(float temperature) {
    const float t = fminf(fmaxf(temperature, 8.6736174e-19f), 1.2089258e24f);
    return __uint_as_float((__float_as_uint(t * (1.f / 125.5f)) + 0x7fffffu) & 0xff800000u);
}

// A row's table, in units of 2^-(kUnit - drop): entry 64 i + j as a product of exp(-64 i g / T) and exp(-j g / T).
__device__ __noinline__ void make_table(float temperature, int drop) {
    Shared &sh = shared();
    const int tid = threadIdx.x;
    const float2 scale = scale_of(temperature);
    const float step = step_of(temperature);
    if (tid < 2 * kGroups) {
        const uint64_t turns = (uint64_t)(scale.x * step * 72057594037927936.f) + (uint64_t)(int64_t)(scale.y * step * 72057594037927936.f);
        sh.steps[tid / kGroups][tid % kGroups] = power(turns * (tid < kGroups ? 64 * tid : tid - kGroups));
    }
    __syncthreads();
#pragma unroll 1
    for (int k = tid; k < kCells; k += kThreads) {
        const Power a = sh.steps[0][k / 64], b = sh.steps[1][k % 64];
        const uint64_t w = __umul64hi(a.w, b.w);  // units of 2^-60
        const int shift = 60 - kUnit + a.octaves + b.octaves + drop;
        sh.table[k] = shift > 61 || k == kCells - 1 ? 0 : (w + (1ull << (shift - 1))) >> shift;
    }
    __syncthreads();
}

// A row's grid.
__device__ __forceinline__ Grid make_grid(float top, float temperature, int drop) {
    const float t = fminf(fmaxf(temperature, 8.6736174e-19f), 1.2089258e24f), step = step_of(temperature);
    Grid g;
    if (top < INFINITY) {
        g.base = fabsf(top) > step * 1048576.f ? top : 0.f;
        g.high = __fsub_rn(top, g.base);
    } else {  // beside an infinity all numbers have weight 0: they are cut to the last cell, infinities to the first
        g.base = 3.402823466e38f;
        g.high = step * (kCells - 1);
    }
    g.magic = step * 12582912.f;
    const float s = __fadd_rn(g.high, g.magic);
    g.zero = __float_as_int(s);
    g.point = __fsub_rn(s, g.magic);
    g.low = g.point - step * (kCells - 1);
    g.c = scale_of(temperature).x;
    g.over = __fdiv_rn(1.f, t);
    g.unit = (float)(1ull << (kUnit - drop));
    return g;
}

// The tokens in the cells, in groups of 64 summed up for all CTAs.
template <typename T>
__device__ __noinline__ void count_cells(Row<T> row, Here h) {
    Shared &sh = shared();
    const int tid = threadIdx.x, lane = tid & 31;
    const Grid grid = sh.grid;
    row.units(h.begin, h.stop, lane, [&](const float (&x)[kVec<T>], int) {
        int k[kVec<T>];
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) k[i] = grid.cell(x[i]);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (k[i] < kCells - 1) atomicAdd(&sh.cells[k[i]], 1u);
    });
    __syncthreads();
    constexpr int kEach = kCells / kThreads;
    uint64_t mass = 0;
    uint32_t count = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const uint32_t n = sh.cells[tid * kEach + e];
        count += n;
        mass += n * sh.table[tid * kEach + e];
    }
#pragma unroll
    for (int o = 64 / kEach / 2; o > 0; o >>= 1) {
        mass += __shfl_xor_sync(0xffffffffu, mass, o);
        count += __shfl_xor_sync(0xffffffffu, count, o);
    }
    if (tid % (64 / kEach) == 0) sh.mine[tid / (64 / kEach)] = Group{mass, count};
    __syncthreads();
    if (tid / kGroups < h.C) {
        const Group g = sh.mine[tid % kGroups];
        put(&sh.groups[h.rank][tid % kGroups].mass, g.mass, g.count, tid / kGroups, h.rank);
    }
    meet(h.C);
}

// The cell of a border, left in `border` with the tokens before it and in it and their weights at their grid points: the first
// whose tokens (counting), or whose tokens' weights at their grid points, reach `want` together with those before; want 0: top_p of
// all weights.  It is cut to low .. high.  The first warp narrows it down to a group, and among the group's cells; two of them a lane.
__device__ __noinline__ void find_cell(Here h, bool counting, uint64_t want, float top_p, int low, int high, int V) {
    Shared &sh = shared();
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        uint64_t mass[2] = {0, 0}, count[2] = {0, 0};
        for (int c = 0; c < h.C; ++c) {
            const Group a = sh.groups[c][2 * lane], b = sh.groups[c][2 * lane + 1];
            mass[0] += a.mass;
            count[0] += a.count;
            mass[1] += b.mass;
            count[1] += b.count;
        }
        uint64_t upto_mass = warp_scan(mass[0] + mass[1], lane), upto_count = warp_scan(count[0] + count[1], lane);
        const uint64_t all_mass = __shfl_sync(0xffffffffu, upto_mass, 31), all_count = __shfl_sync(0xffffffffu, upto_count, 31);
        const uint64_t goal = want ? want : top_p_goal(all_mass, top_p);
        auto first = [&] {  // of the 64 that reaches the goal; 64: none
            const uint64_t upto = counting ? upto_count : upto_mass, second = counting ? count[1] : mass[1];
            const unsigned yes = __ballot_sync(0xffffffffu, upto >= goal);
            const int at = max(__ffs(yes) - 1, 0), late = __shfl_sync(0xffffffffu, (int)(upto - second < goal), at);
            return yes ? 2 * at + late : 64;
        };
        uint64_t before_mass = 0, before_count = 0, in_mass = 0, in_count = 0;
        auto look = [&](int of) {  // at one of the 64: what comes before it, and what is in it
            const bool late = of & 1;
            const uint64_t m = upto_mass - mass[1] - (late ? 0 : mass[0]), c = upto_count - count[1] - (late ? 0 : count[0]);
            before_mass = __shfl_sync(0xffffffffu, m, of / 2);
            before_count = __shfl_sync(0xffffffffu, c, of / 2);
            in_mass = __shfl_sync(0xffffffffu, late ? mass[1] : mass[0], of / 2);
            in_count = __shfl_sync(0xffffffffu, late ? count[1] : count[0], of / 2);
        };
        const int group = min(max(first(), low / 64), high / 64);
        look(group);
        uint64_t both[kMaxCluster];  // two cells' tokens
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
            both[c] = c < h.C ? get(reinterpret_cast<const uint64_t *>(&sh.cells[64 * group + 2 * lane]), c, h.rank) : 0;
        count[0] = count[1] = 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            count[0] += (uint32_t)both[c];
            count[1] += both[c] >> 32;
        }
        mass[0] = count[0] * sh.table[64 * group + 2 * lane];
        mass[1] = count[1] * sh.table[64 * group + 2 * lane + 1];
        upto_mass = before_mass + warp_scan(mass[0] + mass[1], lane);
        upto_count = before_count + warp_scan(count[0] + count[1], lane);
        const int cell = min(max(64 * group + first(), low), high);
        look(cell & 63);
        if (cell == kCells - 1) in_count = V - all_count;  // beyond all weights
        if (lane == 0) sh.border = Border{before_mass, before_count, (uint64_t)cell, in_count, in_mass, 0};
    }
    __syncthreads();
}

// The sums before cell `b` (left by run in run_mass, by CTA in part[kCellBorder]) and its tokens, gathered in own; all_up_to: instead
// all tokens up to the cell; all_wanted: the sum of all weights as well.  Tokens behind `last` in the order do not count.
template <typename T>
__device__ __noinline__ void sum_and_gather(Row<T> row, Here h, int b, bool all_up_to, bool all_wanted, uint64_t last) {
    Shared &sh = shared();
    const Grid grid = sh.grid;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sum before, all;
    uint64_t inside = 0;
    uint32_t n_inside = 0;
    const int summed = all_up_to ? 0 : b;
    // (Entry by entry, each with its own branches: a vector's entries summed at once and listed in a loop of their own need more
    // registers than there are, 64 rows with top-p 127 instead of 102 us.)
    row.each(h.begin, h.stop, lane, [&](float x, int p) {
        float y, part;
        const int k = grid.cell(x, y, part);
        if (k == b || (all_up_to && k < b)) {
            const uint64_t place = place_of(key_of(x), p);
            if (place <= last && p >= row.pad && p < row.end) {
                const uint32_t at = atomicAdd(&sh.n_own, 1u);
                if (at < kList) sh.own[at] = place;
                inside += weight_of(grid, x);
                ++n_inside;
            }
        }
        if (all_wanted || k < summed) {
            const uint64_t w = sh.table[k];
            const float rest = grid.rest(y, part);
            all.whole += w;
            all.rest += rest;
            if (k < summed) {
                before.whole += w;
                before.rest += rest;
            }
        }
    });
    const uint64_t run = warp_sum(before.total()), in = warp_sum(inside), total = warp_sum(all.total());
    n_inside = __reduce_add_sync(0xffffffffu, n_inside);
    __syncthreads();
    if (lane == 0) {
        sh.run_mass[warp] = run;
        sh.warp_mass[warp] = in;
        sh.warp_count[warp] = total;
        sh.before_mass[warp] = n_inside;
    }
    __syncthreads();
    exchange(h, kCellBorder, Part{over_warps(sh.run_mass), over_warps(sh.before_mass), over_warps(sh.warp_mass), over_warps(sh.warp_count)});
}

// The lowest key of the cells up to `b`.
__device__ __noinline__ uint32_t lowest_key(int b, uint32_t top_key) {
    const Grid grid = shared().grid;
    return first_key(key_of(-INFINITY), top_key, threadIdx.x & 31, [&](uint32_t key) { return grid.cell(logit_of(key)) <= b; });
}

// A cell of more than kList tokens, split on over their keys, and over the indices of equal keys, until a bin of the border has
// no more: its tokens are gathered in own, what comes before them is left in border.
template <typename T>
__device__ __noinline__ void split_cell(Row<T> row, Here h, int b, bool counting, uint64_t want, uint64_t base_mass, uint64_t base_count,
                                        uint32_t top_key, uint64_t last) {
    Shared &sh = shared();
    const Grid grid = sh.grid;
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t lo = lowest_key(b, top_key), hi = b > 0 ? lowest_key(b - 1, top_key) - 1 : top_key;
    int first = row.pad, final = row.end - 1;
#pragma unroll 1
    for (;;) {
        const bool single = lo == hi;
        const uint32_t width = single ? (uint32_t)(final - first) : hi - lo;
        const int shift = max(0, 32 - __clz(width) - 9);
        __syncthreads();
        for (int i = tid; i < 4 * kSplit; i += kThreads) (&sh.hist[0][0])[i] = 0;
        if (tid == 0) {
            sh.n_own = 0;
            sh.border = Border{base_mass, base_count, kSplit - 1, 0, 0, 0};
        }
        __syncthreads();
        auto bin_of = [&](uint32_t key, int p) {  // -1: none
            if (key < lo || key > hi || p < first || p > final) return -1;
            return (int)(((single ? (uint32_t)(p - first) : hi - key) >> shift) & (kSplit - 1));
        };
        row.each(h.begin, h.stop, lane, [&](float x, int p) {
            const uint32_t key = key_of(x);
            const int at = bin_of(key, p);
            if (at < 0 || place_of(key, p) > last) return;
            const uint64_t w = weight_of(grid, x);
            atomicAdd(&sh.hist[0][at], 1u);
            constexpr uint32_t kLow = (1u << kLimb) - 1;
            atomicAdd(&sh.hist[1][at], (uint32_t)w & kLow);
            atomicAdd(&sh.hist[2][at], (uint32_t)(w >> kLimb) & kLow);
            atomicAdd(&sh.hist[3][at], (uint32_t)(w >> 2 * kLimb));
        });
        meet(h.C);
        const int share = kSplit / h.C, mine = h.rank * share + tid;
        uint64_t mass = 0, count = 0;
        if (tid < share)
            for (int c = 0; c < h.C; ++c) {
                count += get(&sh.hist[0][mine], c, h.rank);
                mass += get(&sh.hist[1][mine], c, h.rank) + ((uint64_t)get(&sh.hist[2][mine], c, h.rank) << kLimb) +
                        ((uint64_t)get(&sh.hist[3][mine], c, h.rank) << 2 * kLimb);
            }
        uint64_t before_mass = block_scan(mass) - mass;
        const uint64_t sum_mass = over_warps(sh.warp_mass);
        uint64_t before_count = block_scan(count) - count;
        exchange(h, kBins, Part{sum_mass, over_warps(sh.warp_mass), 0, 0});
        before_mass += base_mass;
        before_count += base_count;
        for (int c = 0; c < h.rank; ++c) {
            before_mass += sh.part[kBins][c].mass;
            before_count += sh.part[kBins][c].count;
        }
        const uint64_t before = counting ? before_count : before_mass;
        if (tid < share && before < want && before + (counting ? count : mass) >= want)
            for (int c = 0; c < h.C; ++c) {
                put(&sh.border.mass_above, before_mass, before_count, c, h.rank);
                put(&sh.border.bin, mine, count, c, h.rank);
            }
        meet(h.C);
        const int bin = (int)sh.border.bin;
        base_mass = sh.border.mass_above;
        base_count = sh.border.count_above;
        if (sh.border.count <= kList) {
            row.each(h.begin, h.stop, lane, [&](float x, int p) {
                const uint32_t key = key_of(x);
                if (bin_of(key, p) != bin) return;
                const uint64_t place = place_of(key, p);
                if (place > last) return;
                const uint32_t i = atomicAdd(&sh.n_own, 1u);
                if (i < kList) sh.own[i] = place;
            });
            meet(h.C);
            return;
        }
        if (!single) {
            hi -= (uint32_t)bin << shift;
            lo = max(lo, hi - (uint32_t)((1ull << shift) - 1));
        } else {
            first += bin << shift;
            final = min(final, first + (int)((1ull << shift) - 1));
        }
    }
}

// All CTAs' gathered places in the list of every CTA, and their weights by `weight`; how many.
template <typename F>
__device__ __forceinline__ int join_lists(Here h, F weight) {
    Shared &sh = shared();
    const int tid = threadIdx.x, lane = tid & 31;
    // how many each CTA has; a thread's place in the joined list is a CTA's and one in its own
    const uint32_t has = lane < h.C ? min(get(&sh.n_own, lane, h.rank), (uint32_t)kList) : 0;
    uint32_t upto = has;
#pragma unroll
    for (int o = 1; o < kMaxCluster; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    int n = (int)__shfl_sync(0xffffffffu, upto, kMaxCluster - 1), from = 0, at = tid;
#pragma unroll
    for (int c = 0; c < kMaxCluster - 1; ++c) {
        const int end = (int)__shfl_sync(0xffffffffu, upto, c);
        if (tid >= end) {
            from = c + 1;
            at = tid - end;
        }
    }
    uint64_t mine = ~0ull;
    if (tid < n && at < kList) mine = get(&sh.own[at], from, h.rank);
    n = min(n, kList);
    cluster_arrive(h.C);  // has read the others' lists
    sh.list[tid] = Entry{mine, tid < n ? weight(logit_at(mine)) : 0};
    cluster_wait(h.C);
    __syncthreads();
    if (tid == 0) sh.n_own = 0;
    return n;
}

// What is found of top-k and top-p.
struct Kept {
    uint64_t last;      // the last place that stays
    uint64_t mass;      // of what stays; 0: not known
    int n;              // tokens in the list
    bool complete;      // the list has all that stays
    bool runs;          // run_mass, part[kCellBorder] and the list give the sums of what stays
};

// The borders of top-k (the want-th token, want 0: none) and top-p in a list of n tokens that follow base_count tokens
// with weights base_mass.  In a list of top-k's border, that of top-p may be before it: false.
__device__ __noinline__ bool cut_list(Kept &kept, int n, bool counting, uint64_t want, bool by_mass, float top_p, uint64_t base_mass,
                                      uint64_t base_count) {
    Shared &sh = shared();
    const int tid = threadIdx.x;
    const Entry before = rank_list<false>(n, 0);
    const Entry mine = sh.list[tid];
    const uint64_t upto = base_mass + before.place + mine.weight;
    const bool real = tid < n;
    kept.n = n;
    if (counting) {
        if (real && base_count + before.weight + 1 == want) {
            sh.cut[0] = mine.place;
            sh.cut_mass[0] = upto;
        }
        __syncthreads();
        kept.last = sh.cut[0];
        kept.mass = sh.cut_mass[0];
        if (!by_mass) return true;
        want = top_p_goal(kept.mass, top_p);
        if (want <= base_mass) return false;
    }
    const bool here = real && upto >= want && upto - mine.weight < want, any = __syncthreads_or(here);
    if (here || (!any && real && before.weight + 1 == n)) {  // (else the last of them)
        sh.cut[1] = mine.place;
        sh.cut_mass[1] = upto;
    }
    __syncthreads();
    kept.last = sh.cut[1];
    kept.mass = sh.cut_mass[1];
    return true;
}

// Top-k of few tokens: the k-th largest of the parts' largest logits is not above the k-th largest logit, and few tokens are not
// below it.  They are listed, and both borders are in the list; false if they are too many (equal or masked logits).
template <typename T>
__device__ __noinline__ bool find_few(Kept &kept, Row<T> row, Here h, int top_k, bool by_mass, float top_p, float top, float temperature,
                                      int drop) {
    Shared &sh = shared();
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < kMaxima) {
        const uint32_t mine = sh.maxima[tid];
        int before = 0;
#pragma unroll 8
        for (int j = 0; j < kMaxima; ++j) {
            const uint32_t key = sh.maxima[j];
            before += key > mine || (key == mine && j < tid);
        }
        if (before == top_k - 1) sh.least = mine;
    }
    __syncthreads();
    const float least = logit_of(sh.least);
    constexpr int N = kVec<T>;
    row.units(h.begin, h.stop, lane, [&](const float (&x)[N], int p) {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
        if (!(m >= least)) return;
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
            float one = x[0];
#pragma unroll
            for (int j = 1; j < N; ++j) one = i == j ? x[j] : one;
            if (!(one >= least) || p + i < row.pad || p + i >= row.end) continue;
            const uint32_t at = atomicAdd(&sh.n_own, 1u);
            if (at < kList) sh.own[at] = place_of(key_of(one), p + i);
        }
    });
    __syncthreads();
    exchange(h, kFewSums, Part{0, sh.n_own, 0, 0});
    uint64_t n_all = 0;
    for (int c = 0; c < h.C; ++c) n_all += sh.part[kFewSums][c].count;
    if (n_all > kList || n_all < top_k) {  // (fewer: NaN among the parts)
        __syncthreads();
        if (tid == 0) sh.n_own = 0;
        __syncthreads();
        return false;
    }
    const float2 scale = scale_of(temperature);
    const int n = join_lists(h, [&](float x) { return weight_of(scale, top, drop, x); });
    cut_list(kept, n, true, top_k, by_mass, top_p, 0, 0);
    kept.complete = true;
    return true;
}

template <typename T>
__device__ __noinline__ Kept find_borders(Row<T> row, Here h, bool by_count, bool by_mass, int top_k, float top_p, int V, uint32_t top_key) {
    Shared &sh = shared();
    const Grid grid = sh.grid;
    const int tid = threadIdx.x;
    Kept kept{~0ull, 0, 0, false, false};
    count_cells(row, h);
    int limit = by_count ? kCells - 1 : kCells - 2;  // the last cell that a border can be in
#pragma unroll 1
    for (int round = by_count ? 0 : 1; round < (by_mass ? 2 : 1); ++round) {
        const bool counting = round == 0, all_wanted = !counting && kept.mass == 0;
        uint64_t want = counting ? (uint64_t)top_k : all_wanted ? 0 : top_p_goal(kept.mass, top_p);
        // Counts give the cell; weights at the grid points may miss it, most often by what heavy tokens' weights are off, which is
        // the same for its neighbours: the next two tries take that off.  What is known of the border is kept, and from the third
        // try on what is open is halved, so that 12 more end it whatever the weights.  One to three passes for rows of real
        // and of peaked logits.
        int before = -1, behind = limit + 1, tries = 0;  // cells before and behind the border
        uint64_t low = 1, high = ~0ull;                  // sums at the grid points that lie between these
        bool settled = counting, all_up_to;
        find_cell(h, counting, want, top_p, 0, limit, V);
        int b;
        uint64_t above, cell_mass, n_cell, cells_before;
#pragma unroll 1
        for (;;) {
            b = (int)sh.border.bin;
            cells_before = sh.border.count_above;
            const uint64_t grid_before = sh.border.mass_above, grid_up_to = grid_before + sh.border.mass;
            all_up_to = cells_before + sh.border.count <= kWhole;
            sum_and_gather(row, h, b, all_up_to, all_wanted, kept.last);
            uint64_t all_mass = 0;
            above = cell_mass = n_cell = 0;
            for (int c = 0; c < h.C; ++c) {
                const Part p = sh.part[kCellBorder][c];
                above += p.mass;
                n_cell += p.count;
                cell_mass += p.cell_mass;
                all_mass += p.all_mass;
            }
            if (all_wanted) want = top_p_goal(all_mass, top_p);
            if (settled || (want > above && want <= above + cell_mass)) break;
            uint64_t goal;
            if (want > above) {
                before = b;
                low = grid_up_to + 1;
                goal = grid_up_to + (want - above - cell_mass);
            } else {
                behind = b;
                high = grid_before;
                goal = grid_before - min(grid_before, above - want);
            }
            // Nothing between the two: the end of the first (a sum's rounding must not send the border to and fro).
            settled = behind - before <= 1 || low > high;
            if (settled && before == b) break;
            __syncthreads();
            if (tid == 0) sh.n_own = 0;
            meet(h.C);
            const int middle = settled ? max(before, 0) : (before + behind) / 2;
            const bool guess = !settled && tries++ < 2;
            find_cell(h, false, min(max(goal, low), high), top_p, guess ? before + 1 : middle, guess ? behind - 1 : middle, V);
        }
        if (!counting) want = min(max(want, above + 1), above + cell_mass);
        uint64_t base_mass = above, base_count = all_up_to ? 0 : cells_before;
        const bool split = n_cell > kList;
        if (split) {
            split_cell(row, h, b, counting, want, base_mass, base_count, top_key, kept.last);
            base_mass = sh.border.mass_above;
            base_count = sh.border.count_above;
        }
        const int n = join_lists(h, [&](float x) { return weight_of(grid, x); });
        if (counting) limit = min(b, kCells - 2);
        if (n == 0) {  // the goal is beyond all weights by a sum's rounding: all tokens up to the cell
            kept.last = min(kept.last, place_of(lowest_key(b, top_key), 0x7fffffff));
            kept.mass = 0;
            kept.complete = kept.runs = false;
            break;
        }
        const bool found = cut_list(kept, n, counting, want, by_mass, top_p, base_mass, base_count);
        if (by_mass && found) round = 1;
        kept.complete = all_up_to && found;
        kept.runs = !split && !all_up_to && found;
    }
    return kept;
}

// The lowest key whose weight is enough.
__device__ __noinline__ uint32_t find_min_key(uint64_t least, uint32_t top_key) {
    const Grid grid = shared().grid;
    return first_key(key_of(-INFINITY), top_key, threadIdx.x & 31, [&](uint32_t key) { return weight_of(grid, logit_of(key)) >= least; });
}

// The sums of what stays: by run in warp_mass, by CTA in added; all of it.
template <typename T>
__device__ __noinline__ uint64_t sum_runs(Row<T> row, Here h, Kept kept, int run) {
    Shared &sh = shared();
    const Grid grid = sh.grid;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t own = 0;
    if (kept.runs) {
        // before the border's cell they are known; the list's tokens are added, run by run and CTA by CTA
        uint64_t cta = 0;
        for (int base = 0; base < kept.n; base += 32) {
            const Entry e = sh.list[base + lane];
            const uint64_t w = e.place <= kept.last ? e.weight : 0;
            const int of = (int)((uint32_t)e.place & 0x7fffffffu) / run;
            if (of == h.rank * kWarps + warp) own += w;
            if (of / kWarps == warp) cta += w;
        }
        own = sh.run_mass[warp] + warp_sum(own);
        cta = warp_sum(cta);
        if (lane == 0 && warp < h.C) sh.added[warp] = sh.part[kCellBorder][warp].mass + cta;
        __syncthreads();
        if (lane == 0) sh.warp_mass[warp] = own;
        __syncthreads();
    } else {
        Sum s;
        constexpr int N = kVec<T>;
        const bool all = kept.last == ~0ull;
        row.units(h.begin, h.stop, lane, [&](const float (&x)[N], int p) {
            bool stays[N], any = false;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                stays[i] = all || place_of(key_of(x[i]), p + i) <= kept.last;
                any |= stays[i];
            }
            if (!any) return;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float y, part;
                const uint64_t w = sh.table[grid.cell(x[i], y, part)];
                const float rest = grid.rest(y, part);
                s.whole += stays[i] ? w : 0;
                s.rest += stays[i] ? rest : 0.f;
            }
        });
        own = warp_sum(s.total());
        __syncthreads();
        if (lane == 0) sh.warp_mass[warp] = own;
        __syncthreads();
        exchange(h, kRuns, Part{over_warps(sh.warp_mass), 0, 0, 0});
        if (threadIdx.x < h.C) sh.added[threadIdx.x] = sh.part[kRuns][threadIdx.x].mass;
        __syncthreads();
    }
    uint64_t sum = 0;
    for (int c = 0; c < h.C; ++c) sum += sh.added[c];
    return sum;
}

// A token, and the sum that it was drawn from.
struct Drawn {
    int p;  // padded index, -1: not in this thread
    uint64_t sum;
};

// The draw from a list that has all that stays.
__device__ __noinline__ Drawn draw_from_list(Kept kept, float u) {
    Shared &sh = shared();
    const int tid = threadIdx.x;
    const uint64_t before = rank_list<true>(kept.n, kept.last).place;
    const Entry mine = sh.list[tid];
    const uint64_t w = tid < kept.n && mine.place <= kept.last ? mine.weight : 0;
    block_scan(w);
    const uint64_t sum = over_warps(sh.warp_mass), goal = draw_goal(sum, u);
    return Drawn{w > 0 && before <= goal && goal - before < w ? (int)(uint32_t)mine.place : -1, sum};
}

// The draw from the runs: the CTA and run that hold its place, a thread's piece of the run, an entry.
template <typename T>
__device__ __noinline__ Drawn draw_from_runs(Row<T> row, Here h, Kept kept, uint64_t sum, float u, int run) {
    Shared &sh = shared();
    const Grid grid = sh.grid;
    const int tid = threadIdx.x, lane = tid & 31;
    const uint64_t goal = draw_goal(sum, u);
    uint64_t before = 0;
    for (int c = 0; c < h.rank; ++c) before += sh.added[c];
    Drawn drawn{-1, sum};
    if (goal < before || goal - before >= sh.added[h.rank]) return drawn;
    const uint64_t upto = before + warp_scan(lane < kWarps ? sh.warp_mass[lane] : 0, lane);
    const int of = min(max(__ffs(__ballot_sync(0xffffffffu, upto > goal)) - 1, 0), kWarps - 1);
    const uint64_t up = __shfl_sync(0xffffffffu, upto, max(of - 1, 0));
    if (of > 0) before = up;
    const int from = (h.rank * kWarps + of) * run, each = (run + kThreads - 1) / kThreads;
    const int b = from + tid * each, e = min(min(b + each, from + run), row.end);
    auto entry_weight = [&](int p) {
        const float x = row.at(p);
        return place_of(key_of(x), p) <= kept.last ? weight_of(grid, x) : 0;
    };
    uint64_t piece = 0;
    for (int p = b; p < e; ++p) piece += entry_weight(p);
    const uint64_t place = block_scan(piece);
    // (single weights may add up to a little less than the run's sum)
    const uint64_t left = min(goal - before, over_warps(sh.warp_mass) - 1);
    if (place > left && place - piece <= left) {
        uint64_t at = place - piece;
        for (int p = b; p < e; ++p) {
            at += entry_weight(p);
            if (at > left) {
                drawn.p = p;
                break;
            }
        }
    }
    return drawn;
}

// The probability of a logit that stays, in fp32: that of the largest one times 2^t, t = (x - top) / T log2(e) as a pair.  (Whole numbers
// of 2^-44 would be too coarse for rare tokens.)
struct Probability {
    float2 scale;
    float top, largest;
    __device__ __forceinline__ float operator()(float x) const {
        if (x == top) return largest;
        x = fmaxf(x, -INFINITY);
        const float d = __fsub_rn(x, top), b = __fsub_rn(d, x);
        const float e = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(top, b));
        const float t = __fmul_rn(d, scale.x);
        const float low = __fmaf_rn(e, scale.x, __fmaf_rn(d, scale.y, __fmaf_rn(d, scale.x, -t)));
        return t >= -200.f ? exp2f(t) * __fmaf_rn(low, 0.693147181f, 1.f) * largest : 0.f;
    }
};
__device__ __forceinline__ Probability probability_of(float temperature, float top, uint64_t most, uint64_t sum) {
    return Probability{scale_of(temperature), top, __fdiv_rn((float)most, (float)sum)};
}

// ------------------------------------------------------------------------------ the kernel
enum { kDraw = 0, kProbsF32 = 1, kProbsBf16 = 2 };

// A row's probabilities, probability(x, padded index), written by runs.
template <typename T, int OUT, typename F>
__device__ __forceinline__ void write_row(const SampleArgs &a, const Row<T> &row, const Here &h, int64_t r, F probability) {
    constexpr int N = kVec<T>, kSize = OUT == kProbsF32 ? 4 : 2;
    char *out_row = static_cast<char *>(a.probs) + (r * a.p_stride - row.pad) * kSize;  // of padded entry 0
    const bool vector = ((uintptr_t)out_row & (N * kSize - 1) & 15) == 0;
    for (int p = h.begin + (threadIdx.x & 31) * N; p < h.stop; p += 32 * N) {
        float x[N], y[N];
        unpack(row.load(p), x);
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = probability(x[i], p + i);
        const bool whole = vector && p >= row.pad && p + N <= row.end;
        if constexpr (OUT == kProbsF32) {
            float *to = reinterpret_cast<float *>(out_row) + p;
            if (whole) {
#pragma unroll
                for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(to + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (p + i >= row.pad && p + i < row.end) to[i] = y[i];
            }
        } else {
            uint32_t w[N / 2];
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const __nv_bfloat162 two = __floats2bfloat162_rn(y[i], y[i + 1]);
                w[i / 2] = *reinterpret_cast<const uint32_t *>(&two);
            }
            uint16_t *to = reinterpret_cast<uint16_t *>(out_row) + p;
            if (whole) {
                if constexpr (N == 8)
                    *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                else
                    *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (p + i >= row.pad && p + i < row.end) to[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
            }
        }
    }
}

template <typename T, int OUT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
    Shared &sh = shared();
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x / a.cluster;
    Here h;
    h.C = a.cluster;
    h.rank = (int)(blockIdx.x % a.cluster);
    cluster_arrive(h.C);  // another CTA's shared memory may be written once it runs
    for (int i = tid; i < kCells; i += kThreads) sh.cells[i] = 0;
    if (tid == 0) {
        sh.n_own = 0;
        sh.first = kNone;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const float temperature = a.temperature ? a.temperature[r] : 1.f;
    const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    Row<T> row;
    {
        const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
        row.pad = (int)(((uintptr_t)x & 15) / sizeof(T));
        row.base = x - row.pad;
        row.end = row.pad + a.V;
    }
    h.begin = (h.rank * kWarps + (tid >> 5)) * a.run;
    h.stop = min((row.end + 7) / 8 * 8, h.begin + a.run);
    auto give = [&](int p, float probability) {  // one thread of the cluster
        a.tokens[r] = p - row.pad;
        if (a.token_probs) a.token_probs[r] = probability;
    };
    auto refuse = [&](int flag) {  // every CTA of the cluster alike
        if (h.rank == 0 && tid == 0) {
            if (a.err_flag) atomicOr(a.err_flag, flag);
            if (OUT == kDraw) give(row.pad - 1, 0.f);
        }
        if constexpr (OUT != kDraw) write_row<T, OUT>(a, row, h, r, [](float, int) { return 0.f; });
    };
    if (!(temperature >= 0.f && temperature <= 3.402823466e38f) || top_p != top_p || min_p != min_p) {
        cluster_wait(h.C);
        refuse(PA_FLAG_SAMPLING);
        return;
    }
    const uint32_t top_key = find_top(row, h);
    if (top_key == key_of(-INFINITY)) {
        refuse(PA_FLAG_PROBABILITY);
        return;
    }
    if (temperature == 0.f) {
        const int first = find_first(row, h, logit_of(top_key));
        if constexpr (OUT != kDraw)
            write_row<T, OUT>(a, row, h, r, [&](float, int p) { return p == first ? 1.f : 0.f; });
        else if (h.rank == 0 && tid == 0)
            give(first, 1.f);
        return;
    }
    const float top = logit_of(top_key);
    const bool by_count = top_k > 0 && top_k < a.V, by_mass = top_p < 1.f;
    Kept kept{~0ull, 0, 0, false, false};
    uint64_t most;  // the largest weight
    if (by_count && top_k <= kFew && find_few(kept, row, h, top_k, by_mass, top_p, top, temperature, a.drop)) {
        most = 1ull << (kUnit - a.drop);
    } else {
        if (tid == 0) sh.grid = make_grid(top, temperature, a.drop);
        make_table(temperature, a.drop);
        most = weight_of(sh.grid, top);
        if (by_count || by_mass) kept = find_borders(row, h, by_count, by_mass, top_k, top_p, a.V, top_key);
    }
    if (min_p > 0.f) {
        bool cut = false;
        const uint64_t least = min_p < 1.f ? max((uint64_t)1, fraction_of(most, min_p, cut) + cut) : most;
        if (kept.complete) {
            // Tokens with enough weight come first in the order, but for the roundings of two weights beside `least`: what stays ends
            // with the last of them.
            const Entry mine = sh.list[tid];
            const bool stays = tid < kept.n && mine.place <= kept.last && mine.weight >= least;
            __syncthreads();  // the cut has been read by all
            if (tid == 0) sh.cut[0] = 0;
            const Entry before = rank_list<false>(kept.n, 0);  // (its barriers part the line above from the next)
            if (stays) atomicMax(reinterpret_cast<unsigned long long *>(&sh.cut[0]), (unsigned long long)mine.place);
            __syncthreads();
            kept.last = sh.cut[0];
            if (stays && mine.place == kept.last) sh.cut_mass[0] = before.place + mine.weight;
            __syncthreads();
            kept.mass = sh.cut_mass[0];
        } else {
            const uint64_t place = place_of(find_min_key(least, top_key), 0x7fffffff);
            if (place < kept.last) {
                kept.last = place;
                kept.mass = 0;
                kept.runs = false;
            }
        }
    }
    if constexpr (OUT == kDraw) {
        Drawn drawn;
        if (kept.complete) {
            if (h.rank != 0) return;
            drawn = draw_from_list(kept, a.u[r]);
        } else {
            drawn = draw_from_runs(row, h, kept, sum_runs(row, h, kept, a.run), a.u[r], a.run);
        }
        if (drawn.p >= 0) give(drawn.p, probability_of(temperature, top, most, drawn.sum)(row.at(drawn.p)));
    } else {
        if (kept.mass == 0) kept.mass = sum_runs(row, h, kept, a.run);
        const Probability probability = probability_of(temperature, top, most, kept.mass);
        write_row<T, OUT>(a, row, h, r, [&](float x, int p) { return place_of(key_of(x), p) > kept.last ? 0.f : probability(x); });
    }
}

template <typename T, int OUT>
cudaError_t launch_sample(const SampleArgs &a, int R, cudaStream_t stream) {
    static std::atomic<bool> configured[64];  // per device: the shared-memory attribute is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(sample_kernel<T, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)R * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T, OUT>, a);
}

// The status of a launch.
pa_status launched(const char *fn, cudaError_t err) {
    const pa_status st = check_launch(fn);
    return st != PA_OK || err == cudaSuccess ? st : fail(PA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(err));
}

// The checks and the plan that both calls share.
pa_status plan_sample(const char *fn, SampleArgs &a, const void *logits, int64_t logit_stride, int logit_dtype, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p, int R, int V, int *err_flag) {
    if (R < 0) return fail(PA_ERR_INVALID_ARG, "%s: R = %d is negative", fn, R);
    if (logit_dtype != PA_PROB_F32 && logit_dtype != PA_PROB_BF16)
        return fail(PA_ERR_UNSUPPORTED, "%s: logit type %d not supported", fn, logit_dtype);
    if (V < 1) return fail(PA_ERR_INVALID_ARG, "%s: V = %d must be positive", fn, V);
    if (V > PA_SAMPLE_MAX_VOCABULARY) return fail(PA_ERR_UNSUPPORTED, "%s: V = %d (at most %d)", fn, V, PA_SAMPLE_MAX_VOCABULARY);
    if (R > 1 << 20) return fail(PA_ERR_UNSUPPORTED, "%s: at most 2^20 rows per call (got %d)", fn, R);
    constexpr int64_t kMost = (int64_t)1 << 40;
    if (logit_stride < V || logit_stride > kMost) return fail(PA_ERR_INVALID_ARG, "%s: row strides must be at least V", fn);
    if (R == 0) return PA_OK;
    if (!logits) return fail(PA_ERR_INVALID_ARG, "%s: null pointer", fn);
    if ((uintptr_t)logits & (logit_dtype == PA_PROB_F32 ? 3u : 1u))
        return fail(PA_ERR_INVALID_ARG, "%s: logits must be aligned to their type", fn);
    a.x = logits;
    a.x_stride = logit_stride;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.err_flag = err_flag;
    a.V = V;
    // One CTA or eight a row.  A single row gains from eight beyond 6000 entries (top-p, one and eight CTAs: 4000 entries 17.5 and 19.2
    // us, 6000 19.1 and 19.2, 8000 20.6 and 19.5, 16000 25.0 and 19.6); batches of 64 rows do not up to 16000 at least (33.9 and 52.8),
    // as their clusters no longer run at once.  The rule is for single rows; it does not look at R.
    a.cluster = V > 4000 ? kMaxCluster : 1;
    const int runs = a.cluster * kWarps;
    a.run = (int)align_up((size_t)((V + 7 + runs - 1) / runs), 8);  // (a row may start up to 7 entries into its first unit)
    while (V > 1 << (62 - kUnit + a.drop)) ++a.drop;  // V weights of 1 sum to 2^62 at most
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_sample_tokens(int32_t *tokens_out, float *probs_out, const void *logits, int64_t logit_stride, int logit_dtype,
                           const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                           const float *uniforms, int R, int V, int *err_flag, void *stream) {
    const char *fn = "pa_sample_tokens";
    clear_error();
    SampleArgs a{};
    const pa_status st = plan_sample(fn, a, logits, logit_stride, logit_dtype, temperature, top_k, top_p, min_p, R, V, err_flag);
    if (st != PA_OK || R == 0) return st;
    if (!tokens_out || !uniforms) return fail(PA_ERR_INVALID_ARG, "%s: null pointer", fn);
    a.tokens = tokens_out;
    a.token_probs = probs_out;
    a.u = uniforms;
    const cudaError_t err = logit_dtype == PA_PROB_F32 ? launch_sample<float, kDraw>(a, R, (cudaStream_t)stream)
                                                       : launch_sample<uint16_t, kDraw>(a, R, (cudaStream_t)stream);
    return launched(fn, err);
}

pa_status pa_sampling_probs(void *probs_out, int64_t prob_stride, int prob_dtype, const void *logits, int64_t logit_stride,
                            int logit_dtype, const float *temperature, const int32_t *top_k, const float *top_p,
                            const float *min_p, int R, int V, int *err_flag, void *stream) {
    const char *fn = "pa_sampling_probs";
    clear_error();
    SampleArgs a{};
    const pa_status st = plan_sample(fn, a, logits, logit_stride, logit_dtype, temperature, top_k, top_p, min_p, R, V, err_flag);
    if (st != PA_OK) return st;
    if (prob_dtype != PA_PROB_F32 && prob_dtype != PA_PROB_BF16)
        return fail(PA_ERR_UNSUPPORTED, "%s: probability type %d not supported", fn, prob_dtype);
    if (prob_stride < V || prob_stride > (int64_t)1 << 40) return fail(PA_ERR_INVALID_ARG, "%s: row strides must be at least V", fn);
    if (R == 0) return PA_OK;
    if (!probs_out) return fail(PA_ERR_INVALID_ARG, "%s: null pointer", fn);
    const int64_t in = logit_dtype == PA_PROB_F32 ? 4 : 2, out = prob_dtype == PA_PROB_F32 ? 4 : 2;
    if ((uintptr_t)probs_out & (out - 1)) return fail(PA_ERR_INVALID_ARG, "%s: probabilities must be aligned to their type", fn);
    const uintptr_t x = (uintptr_t)logits, y = (uintptr_t)probs_out;
    const uintptr_t xn = (uintptr_t)(((R - 1) * logit_stride + V) * in), yn = (uintptr_t)(((R - 1) * prob_stride + V) * out);
    if (x < y + yn && y < x + xn) return fail(PA_ERR_INVALID_ARG, "%s: probs_out overlaps logits", fn);
    a.probs = probs_out;
    a.p_stride = prob_stride;
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t err =
        logit_dtype == PA_PROB_F32
            ? (prob_dtype == PA_PROB_F32 ? launch_sample<float, kProbsF32>(a, R, s) : launch_sample<float, kProbsBf16>(a, R, s))
            : (prob_dtype == PA_PROB_F32 ? launch_sample<uint16_t, kProbsF32>(a, R, s) : launch_sample<uint16_t, kProbsBf16>(a, R, s));
    return launched(fn, err);
}

}  // extern "C"
