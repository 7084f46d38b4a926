// From logits to tokens or to filtered probabilities (pa_sample.h).
//
// Nothing is sorted.  The tokens that top-k and top-p leave are those down to a border in the
// order (falling logit, rising index), and the border is searched: the tokens are counted, and
// their weights summed, in 1024 bins over the logits; the bin that the border falls into is known
// exactly, and it is split further (over its logits, and over the indices of equal logits)
// until at most kList tokens are in question, which are gathered and sorted.  Then a token
// is drawn by sums over runs of the vocabulary, narrowed down to the run, a thread's piece of it
// and an entry; or the row is written.
//
// Weights are whole numbers: 2^45 exp((x - m) / T), rounded.  Their sums are exact and do not
// depend on the order, so every CTA of a row's cluster decides alike, bins may be filled by
// atomics, and a border is where it is in exact arithmetic unless two numbers agree to about
// 2^-36.  (fp32 weights carry 2^-23 each: with the vocabulary's tens of thousands of small
// weights near a border, one row in a hundred would be cut elsewhere.  GB300 has two fp64 lanes
// per SM and clock, so fp64 weights would take several times longer than the loads.)
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "pa_internal.cuh"
#include "pa_sample.h"

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;
constexpr int kBinsPerOctave = 32;  // of the first split: weights of a bin within 2.2 %
constexpr int kList = 512;          // tokens that are sorted (at most one a thread)
constexpr int kUnit = 45;           // a weight of 1 is 2^45
constexpr int kSteps = 1024;        // table steps an octave
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
// 2^(j / 1024) = kCoarse[j / 32] * kFine[j % 32]; series of exp, in units of 2^-63 and 2^-62.
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

// How a row's logits become weights: t = (x - top) / T log2(e), a pair of fp32.
struct Scale {
    float top, hi, lo;  // hi + lo = log2(e) / T
    int drop;
    const uint64_t *table;  // 2^(j / 1024) in units of 2^-46

    // -1024 t rounded (0 .. 4000 * 1024, rising as x falls), the remainder of t and its low part.
    __device__ __forceinline__ int steps(float x, float &rest, float &low) const {
        // x - top and its rounding error, then the product with its own
        const float d = __fsub_rn(x, top), b = __fsub_rn(d, x);
        const float e = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(top, b));
        const float h = __fmul_rn(d, hi);
        low = __fmaf_rn(e, hi, __fmaf_rn(d, lo, __fmaf_rn(d, hi, -h)));
        const float c = fmaxf(h, -4000.f);
        // the sum with 1.5 x 2^13 rounds to 2^-10 and leaves the whole number in the low bits
        const float t = __fadd_rn(c, 12288.f);
        rest = __fsub_rn(c, __fsub_rn(t, 12288.f));
        return __float_as_int(12288.f) - __float_as_int(t);
    }
    // 2^45 2^t, rounded to a multiple of 2^drop and over it.  2^t = 2^-whole 2^(j / 1024) (1 + q):
    // |rest| <= 2^-11, so q's fp32 rounding is 2^-36 of the weight.
    __device__ __forceinline__ uint64_t weight(int step, float rest, float low) const {
        constexpr float k1 = (float)(0.693147180559945309 * (1ull << 42)), k2 = (float)(0.240226506959100712 * (1ull << 42)),
                        k3 = (float)(0.0555041086648215800 * (1ull << 42));
        const float q = __fmaf_rn(rest, __fmaf_rn(rest, __fmaf_rn(rest, k3, k2), k1), low * k1);
        const int qi = __float2int_rn(q);  // units of 2^-42
        const uint64_t w = table[-step & (kSteps - 1)];
        const uint64_t full = w + (uint64_t)((int64_t)__mulhi((int)(w >> 16), qi) * 64);
        const int shift = (step + kSteps - 1) / kSteps + drop;
        return shift > kUnit + 1 ? 0 : ((full >> shift) + 1) >> 1;
    }
    __device__ __forceinline__ uint64_t weight(float x) const {
        float rest, low;
        const int step = steps(x, rest, low);
        return weight(step, rest, low);
    }
    // 2^t in fp32, for the probabilities that are written
    __device__ __forceinline__ float value(float x) const {
        const float d = __fsub_rn(x, top), b = __fsub_rn(d, x);
        const float e = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(top, b));
        const float h = __fmul_rn(d, hi);
        const float low = __fmaf_rn(e, hi, __fmaf_rn(d, lo, __fmaf_rn(d, hi, -h)));
        return h < -200.f ? 0.f : exp2f(h) * __fmaf_rn(low, 0.693147181f, 1.f);
    }
    __device__ __forceinline__ int bin(int step) const { return min(step / (kSteps / kBinsPerOctave), kBins - 1); }
};

// ---------------------------------------------------------------------------- the order
// Keys rise with logits; -0 and 0 are equal.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key); }

// A token's place in the order as one number: falling logit, rising index.
__device__ __forceinline__ uint64_t place_of(uint32_t key, int v) { return (uint64_t)~key << 32 | (uint32_t)v; }

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

struct alignas(16) Part {
    uint64_t mass, count;
};
struct alignas(16) Border {
    uint64_t mass_above, count_above;
    uint32_t bin, count;
};

struct alignas(16) Shared {
    uint64_t table[kSteps];
    uint32_t hist[4][kBins];  // counts, and sums of the weights' lowest 15 bits, the next 15 and the rest
    uint64_t own[kList];      // places gathered here, and of all CTAs
    uint64_t all[kList];
    Part part[2][kMaxCluster];
    Border border;
    uint64_t warp_mass[kWarps], warp_count[kWarps];
    uint64_t cut[2], cut_mass[2];
    uint32_t n_own;
    uint32_t first;           // temperature 0
};

// ------------------------------------------------------------------- the cluster of a row
__device__ __forceinline__ uint32_t remote(const void *p, int rank) {
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
    return a;
}
__device__ __forceinline__ void put(uint32_t to, uint64_t a, uint64_t b) {
    asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(to), "l"(a), "l"(b) : "memory");
}
__device__ __forceinline__ uint32_t get32(uint32_t from) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(from) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t get64(uint32_t from) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(from) : "memory");
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
    bool only_inf;  // the largest logit is +inf: the others do not count

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
    __device__ __forceinline__ float clean(float x) const {
        x = fmaxf(x, -INFINITY);  // NaN
        return only_inf ? (x == INFINITY ? 0.f : -INFINITY) : x;
    }
    __device__ __forceinline__ float at(int p) const {
        return p >= pad && p < end ? clean(entry(base + p)) : -INFINITY;
    }
    // f(x, padded index) for the entries of a warp's run [begin, stop), both multiples of 8
    template <typename F>
    __device__ __forceinline__ void each(int begin, int stop, int lane, F f) const {
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
#pragma unroll
            for (int i = 0; i < N; ++i) f(clean(x[i]), p + i);
        }
    }
};

enum { kDraw = 0, kProbsF32 = 1, kProbsBf16 = 2 };

template <typename T, int OUT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
    __shared__ Shared sh;
    const int C = a.cluster;
    auto cluster_arrive = [&] {
        __syncwarp();
        if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    };
    auto cluster_wait = [&] {
        if (C > 1)
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        else
            __syncthreads();
    };
    auto meet = [&] {
        cluster_arrive();
        cluster_wait();
    };
    cluster_arrive();  // another CTA's shared memory may be written once it runs
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = blockIdx.x / C, rank = blockIdx.x % C;
    for (int j = tid; j < kSteps; j += kThreads)
        // units of 2^-61 from the product's upper half, then of 2^-46
        sh.table[j] = (__umul64hi(kPowers.coarse[j / 32], kPowers.fine[j % 32]) + (1ull << 14)) >> 15;
    auto clear_bins = [&] {
        for (int i = tid; i < 4 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
    };
    clear_bins();
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
        row.only_inf = false;
    }
    const int begin = (rank * kWarps + warp) * a.run, stop = min((row.end + 7) / 8 * 8, begin + a.run);
    // a row's outputs: probability p of padded entry `at`
    char *out_row = nullptr;
    int out_size = 0;
    bool out_vector = false;
    if (OUT != kDraw) {
        out_size = OUT == kProbsF32 ? 4 : 2;
        out_row = static_cast<char *>(a.probs) + (r * a.p_stride - row.pad) * out_size;
        out_vector = ((uintptr_t)out_row & (kVec<T> * out_size - 1) & 15) == 0;
    }
    auto write_row = [&](auto probability) {
        constexpr int N = kVec<T>;
        for (int p = begin + lane * N; p < stop; p += 32 * N) {
            float x[N], y[N];
            unpack(row.load(p), x);
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = probability(row.clean(x[i]), p + i);
            if (OUT == kProbsF32) {
                float *to = reinterpret_cast<float *>(out_row) + p;
                if (out_vector && p >= row.pad && p + N <= row.end) {
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
                if (out_vector && p >= row.pad && p + N <= row.end) {
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
    };
    auto give = [&](int v, float p) {  // one thread of the cluster
        if (OUT == kDraw) {
            a.tokens[r] = v;
            if (a.token_probs) a.token_probs[r] = p;
        }
    };
    auto refuse = [&](int flag) {  // every CTA of the cluster alike
        if (rank == 0 && tid == 0) {
            if (a.err_flag) atomicOr(a.err_flag, flag);
            give(-1, 0.f);
        }
        if (OUT != kDraw) write_row([](float, int) { return 0.f; });
    };
    if (!(temperature >= 0.f && temperature <= 3.402823466e38f) || top_p != top_p || min_p != min_p) {
        cluster_wait();
        refuse(PA_FLAG_SAMPLING);
        return;
    }

    // The CTAs' sums of two numbers: every CTA writes its own into all of them, and they meet.
    int turn = 0;
    auto exchange = [&](uint64_t mass, uint64_t count) {  // in the first warp; then part[turn ^ 1]
        if (warp == 0 && lane < C) put(remote(&sh.part[turn][rank], lane), mass, count);
        meet();
        turn ^= 1;
    };
    auto sum_and_exchange = [&](uint64_t mass) {
        mass = warp_sum(mass);
        if (lane == 0) sh.warp_mass[warp] = mass;
        __syncthreads();
        exchange(warp_sum(warp == 0 && lane < kWarps ? sh.warp_mass[lane] : 0), 0);
    };
    auto block_scan = [&](uint64_t &mass, uint64_t &count) {  // inclusive, by thread
        mass = warp_scan(mass, lane);
        count = warp_scan(count, lane);
        __syncthreads();
        if (lane == 31) {
            sh.warp_mass[warp] = mass;
            sh.warp_count[warp] = count;
        }
        __syncthreads();
        const uint64_t m = warp_scan(lane < kWarps ? sh.warp_mass[lane] : 0, lane), c = warp_scan(lane < kWarps ? sh.warp_count[lane] : 0, lane);
        const uint64_t mb = __shfl_sync(0xffffffffu, m, max(warp - 1, 0)), cb = __shfl_sync(0xffffffffu, c, max(warp - 1, 0));
        if (warp > 0) {
            mass += mb;
            count += cb;
        }
    };

    // ---- the largest logit
    uint32_t top_key = 0;
    {
        float m = -INFINITY;
        row.each(begin, stop, lane, [&](float x, int) { m = fmaxf(m, x); });
        const uint32_t k = __reduce_max_sync(0xffffffffu, key_of(m));
        if (lane == 0) sh.warp_mass[warp] = k;
        if (tid == 0) {
            sh.n_own = 0;
            sh.first = kNone;
        }
        __syncthreads();
        cluster_wait();
        exchange(__reduce_max_sync(0xffffffffu, lane < kWarps ? (uint32_t)sh.warp_mass[lane] : 0), 0);
        for (int c = 0; c < C; ++c) top_key = max(top_key, (uint32_t)sh.part[turn ^ 1][c].mass);
    }
    float top = logit_of(top_key);
    if (top == -INFINITY) {
        refuse(PA_FLAG_PROBABILITY);
        return;
    }
    if (top == INFINITY) {
        row.only_inf = true;
        top = 0.f;
        top_key = key_of(0.f);
    }
    // What stays: places up to `last` in the order.
    uint64_t last = place_of(top_key, 0);
    auto stays = [&](float x, int p) { return place_of(key_of(x), p) <= last; };

    if (temperature == 0.f) {
        uint32_t first = kNone;
        row.each(begin, stop, lane, [&](float x, int p) {
            if (x == top) first = min(first, (uint32_t)p);
        });
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) atomicMin(&sh.first, first);
        __syncthreads();
        exchange(sh.first, 0);
        for (int c = 0; c < C; ++c) first = min(first, (uint32_t)sh.part[turn ^ 1][c].mass);
        if (OUT == kDraw) {
            if (rank == 0 && tid == 0) give((int)first - row.pad, 1.f);
        } else {
            write_row([&](float, int p) { return p == (int)first ? 1.f : 0.f; });
        }
        return;
    }

    Scale scale;
    scale.top = top;
    scale.table = sh.table;
    scale.drop = a.drop;
    {
        // log2(e) / T as a pair: the remainder of the division is exact
        constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;
        const float h = fminf(__fdiv_rn(kHi, temperature), 8.5e37f);
        scale.hi = h;
        scale.lo = h < 8.5e37f ? __fdiv_rn(__fadd_rn(__fmaf_rn(-h, temperature, kHi), kLo), temperature) : 0.f;
    }
    const uint64_t one = 1ull << (kUnit - a.drop);
    const bool by_count = top_k > 0 && top_k < a.V, by_mass = top_p < 1.f;
    last = ~0ull;
    uint64_t kept_mass = 0;   // of what stays, 0: not known
    bool complete = false;    // all that stays is in `all`, sorted: n_all of it
    int n_all = 0;
    uint64_t min_weight = 0;  // min-p
    if (min_p > 0.f) min_weight = max((uint64_t)1, min(one, (uint64_t)ceilf(__fmul_rn(fminf(min_p, 1.f), (float)one))));

    // ---- the borders of top-k and top-p
#pragma unroll 1
    for (int round = by_count ? 0 : 1; round < (by_mass ? 2 : 1); ++round) {
        const bool counting = round == 0;
        // Undecided: keys lo .. hi; of a single key, indices first .. final.  level 0: everything.
        uint32_t lo = 0, hi = kNone;
        int first = 0, final = row.end, shift = 0;
        uint64_t mass_above = 0, count_above = 0, want = top_k;
#pragma unroll 1
        for (int level = 0;; ++level) {
            const bool single = level > 0 && lo == hi;
            // the bin of an entry; -1 before all of them in the order, kBins behind
            auto bin_of = [&](int step, uint32_t key, int p) {
                if (level == 0) return scale.bin(step);
                if (key > hi) return -1;
                if (key < lo) return kBins;
                if (!single) return (int)((hi - key) >> shift);
                return p < first ? -1 : p > final ? kBins : (p - first) >> shift;
            };
            if (level > 0) {
                const uint32_t width = single ? (uint32_t)(final - first) : hi - lo;
                shift = max(0, 32 - __clz(width) - 10);
                clear_bins();
                __syncthreads();
            }
            row.each(begin, stop, lane, [&](float x, int p) {
                if (!stays(x, p)) return;
                float rest, low;
                const int step = scale.steps(x, rest, low);
                const int b = bin_of(step, key_of(x), p);
                if (b < 0 || b >= kBins) return;
                atomicAdd(&sh.hist[0][b], 1u);
                if (by_mass) {
                    const uint64_t w = scale.weight(step, rest, low);
                    atomicAdd(&sh.hist[1][b], (uint32_t)w & 0x7fffu);
                    atomicAdd(&sh.hist[2][b], (uint32_t)(w >> 15) & 0x7fffu);
                    atomicAdd(&sh.hist[3][b], (uint32_t)(w >> 30));
                }
            });
            meet();
            // this CTA's share of the bins, kEach of them a thread
            const int share = kBins / C, each = max(1, share / kThreads);
            uint64_t mass[2] = {0, 0}, count[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (e >= each || tid * each >= share) break;
                const int b = rank * share + tid * each + e;
                for (int c = 0; c < C; ++c) {
                    const uint32_t from = remote(&sh.hist[0][b], c);
                    count[e] += get32(from);
                    if (by_mass)
                        mass[e] += get32(from + 4 * kBins) + ((uint64_t)get32(from + 8 * kBins) << 15) +
                                   ((uint64_t)get32(from + 12 * kBins) << 30);
                }
            }
            uint64_t upto_mass = mass[0] + mass[1], upto_count = count[0] + count[1];
            block_scan(upto_mass, upto_count);
            exchange(__shfl_sync(0xffffffffu, warp_sum(lane < kWarps ? sh.warp_mass[lane] : 0), 0),
                     warp_sum(lane < kWarps ? sh.warp_count[lane] : 0));
            uint64_t before_mass = mass_above, before_count = count_above, all_mass = 0;
            for (int c = 0; c < C; ++c) {
                const Part p = sh.part[turn ^ 1][c];
                all_mass += p.mass;
                if (c < rank) {
                    before_mass += p.mass;
                    before_count += p.count;
                }
            }
            if (!counting && level == 0) {
                // entries stay while the sum before them is below top_p times the whole
                const uint64_t whole = kept_mass ? kept_mass : all_mass;
                want = top_p_goal(whole, top_p);
            }
            before_mass += upto_mass - mass[0] - mass[1];
            before_count += upto_count - count[0] - count[1];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (e >= each || tid * each >= share) break;
                const uint64_t before = counting ? before_count : before_mass;
                if (before < want && before + (counting ? count[e] : mass[e]) >= want)
                    for (int c = 0; c < C; ++c) {
                        const uint32_t to = remote(&sh.border, c);
                        put(to, before_mass, before_count);
                        asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(to + 16), "r"(rank * share + tid * each + e),
                                     "r"((uint32_t)count[e]) : "memory");
                    }
                before_mass += mass[e];
                before_count += count[e];
            }
            meet();
            const Border border = sh.border;
            const int b = (int)border.bin;
            const bool whole_list = border.count_above + border.count <= kList;
            if (whole_list || border.count <= kList) {
                // ---- few enough: gather them, all CTAs' in every CTA, and sort them
                row.each(begin, stop, lane, [&](float x, int p) {
                    if (!stays(x, p)) return;
                    float rest, low;
                    const int step = level == 0 ? scale.steps(x, rest, low) : 0;
                    const uint32_t key = key_of(x);
                    const int at = bin_of(step, key, p);
                    if (at == b || (whole_list && at < b)) {
                        const uint32_t i = atomicAdd(&sh.n_own, 1u);
                        if (i < kList) sh.own[i] = place_of(key, p);
                    }
                });
                meet();
                int n = 0;
                uint64_t mine = ~0ull;
                for (int c = 0; c < C; ++c) {
                    const int m = (int)min(get32(remote(&sh.n_own, c)), (uint32_t)kList);
                    if (tid >= n && tid < n + m) mine = get64(remote(&sh.own[tid - n], c));
                    n += m;
                }
                cluster_arrive();  // has read the others' lists
                int size = 32;
                while (size < n) size *= 2;
#pragma unroll 1
                for (int k = 2; k <= size; k *= 2) {
#pragma unroll 1
                    for (int j = k / 2; j > 0; j /= 2) {
                        uint64_t other;
                        if (j >= 32) {
                            __syncthreads();
                            sh.all[tid] = mine;
                            __syncthreads();
                            other = sh.all[tid ^ j];
                        } else {
                            other = __shfl_xor_sync(0xffffffffu, mine, j);
                        }
                        const bool lower = ((tid & j) == 0) == ((tid & k) == 0);
                        mine = lower ? min(mine, other) : max(mine, other);
                    }
                }
                __syncthreads();
                sh.all[tid] = mine;
                const bool real = tid < n;
                const uint64_t w = real ? scale.weight(logit_of(~(uint32_t)(mine >> 32))) : 0;
                uint64_t upto = w, unused = 0;
                block_scan(upto, unused);
                const uint64_t base_mass = whole_list ? 0 : border.mass_above, base_count = whole_list ? 0 : border.count_above;
                upto += base_mass;
                if (counting && real && base_count + tid + 1 == want) {
                    sh.cut[0] = mine;
                    sh.cut_mass[0] = upto;
                }
                __syncthreads();
                uint64_t goal = want;
                bool found = true;
                if (counting) {
                    last = sh.cut[0];
                    kept_mass = by_mass ? sh.cut_mass[0] : 0;
                    if (by_mass) {
                        goal = top_p_goal(kept_mass, top_p);
                        found = goal > base_mass;  // else the border of top-p is above this bin
                    }
                }
                if (by_mass && found) {
                    if (real && upto >= goal && upto - w < goal) {
                        sh.cut[1] = mine;
                        sh.cut_mass[1] = upto;
                    }
                    __syncthreads();
                    last = sh.cut[1];
                    kept_mass = sh.cut_mass[1];
                    round = 1;
                }
                complete = whole_list && found;
                n_all = n;
                cluster_wait();
                if (tid == 0) sh.n_own = 0;
                clear_bins();
                __syncthreads();
                break;
            }
            mass_above = border.mass_above;
            count_above = border.count_above;
            if (level == 0) {
                // the keys of the bin
                float rest, low;
                auto in = [&](int most) {
                    return first_key(key_of(-INFINITY), top_key, lane, [&](uint32_t key) { return scale.bin(scale.steps(logit_of(key), rest, low)) <= most; });
                };
                lo = in(b);
                hi = b > 0 ? in(b - 1) - 1 : top_key;
            } else if (!single) {
                hi -= (uint32_t)b << shift;
                lo = max(lo, hi - (uint32_t)((1ull << shift) - 1));
            } else {
                first += b << shift;
                final = min(final, first + (int)((1ull << shift) - 1));
            }
        }
    }
    // ---- min-p: the lowest key whose weight is enough
    if (min_weight > 0) {
        const uint32_t lowest = first_key(key_of(-INFINITY), top_key, lane, [&](uint32_t key) { return scale.weight(logit_of(key)) >= min_weight; });
        const uint64_t place = place_of(lowest, 0x7fffffff);
        if (place < last) {
            last = place;
            kept_mass = 0;
        }
    }

    if (complete) {
        // ---- all that stays is in the list
        uint64_t mine = sh.all[tid];
        bool real = tid < n_all && mine <= last;
        uint64_t w = real ? scale.weight(logit_of(~(uint32_t)(mine >> 32))) : 0;
        if (OUT == kDraw) {
            if (rank != 0) return;
            // by index
            const int n = __syncthreads_count(real);
            mine = real ? mine << 32 | mine >> 32 : ~0ull;
            int size = 32;
            while (size < n) size *= 2;
#pragma unroll 1
            for (int k = 2; k <= size; k *= 2) {
#pragma unroll 1
                for (int j = k / 2; j > 0; j /= 2) {
                    uint64_t other;
                    if (j >= 32) {
                        __syncthreads();
                        sh.all[tid] = mine;
                        __syncthreads();
                        other = sh.all[tid ^ j];
                    } else {
                        other = __shfl_xor_sync(0xffffffffu, mine, j);
                    }
                    const bool lower = ((tid & j) == 0) == ((tid & k) == 0);
                    mine = lower ? min(mine, other) : max(mine, other);
                }
            }
            w = tid < n ? scale.weight(logit_of(~(uint32_t)mine)) : 0;
            uint64_t upto = w, unused = 0;
            block_scan(upto, unused);
            const uint64_t sum = warp_sum(lane < kWarps ? sh.warp_mass[lane] : 0);
            const uint64_t target = draw_goal(sum, a.u[r]);
            if (w > 0 && upto > target && upto - w <= target) give((int)(mine >> 32) - row.pad, __fdiv_rn((float)w, (float)sum));
            return;
        }
        uint64_t upto = w, unused = 0;
        block_scan(upto, unused);
        kept_mass = warp_sum(lane < kWarps ? sh.warp_mass[lane] : 0);
    } else if (OUT == kDraw || kept_mass == 0) {
        // ---- the sums of the runs
        uint64_t s = 0;
        row.each(begin, stop, lane, [&](float x, int p) {
            if (stays(x, p)) s += scale.weight(x);
        });
        sum_and_exchange(s);
        uint64_t before = 0, sum = 0;
        for (int c = 0; c < C; ++c) {
            const uint64_t m = sh.part[turn ^ 1][c].mass;
            sum += m;
            if (c < rank) before += m;
        }
        kept_mass = sum;
        if (OUT == kDraw) {
            const uint64_t target = draw_goal(sum, a.u[r]);
            if (target < before || target >= before + sh.part[turn ^ 1][rank].mass) return;
            // the run, and a thread's piece of it
            const uint64_t upto = warp_scan(lane < kWarps ? sh.warp_mass[lane] : 0, lane) + before;
            const int w = __ffs(__ballot_sync(0xffffffffu, upto > target)) - 1;
            const uint64_t up = __shfl_sync(0xffffffffu, upto, max(w - 1, 0));
            if (w > 0) before = up;
            const int from = (rank * kWarps + w) * a.run, each = (a.run + kThreads - 1) / kThreads;
            const int b = from + tid * each, e = min(min(b + each, from + a.run), row.end);
            uint64_t piece = 0, unused = 0;
            for (int p = b; p < e; ++p) {
                const float x = row.at(p);
                if (stays(x, p)) piece += scale.weight(x);
            }
            uint64_t place = piece;
            block_scan(place, unused);
            place += before;
            if (place > target && place - piece <= target) {
                place -= piece;
                for (int p = b; p < e; ++p) {
                    const float x = row.at(p);
                    const uint64_t entry = stays(x, p) ? scale.weight(x) : 0;
                    place += entry;
                    if (place > target) {
                        give(p - row.pad, __fdiv_rn((float)entry, (float)sum));
                        break;
                    }
                }
            }
            return;
        }
    }
    if (OUT != kDraw) {
        const float over = __fdiv_rn((float)one, (float)kept_mass);
        write_row([&](float x, int p) { return stays(x, p) ? scale.value(x) * over : 0.f; });
    }
}

template <typename T, int OUT>
cudaError_t launch_sample(const SampleArgs &a, int R, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)R * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T, OUT>, a);
}

// The checks and the plan that both calls share; a.V = 0 where there is nothing to do.
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
    a.cluster = V > 4000 ? kMaxCluster : 1;
    const int runs = a.cluster * kWarps;
    a.run = (int)align_up((size_t)((V + 7 + runs - 1) / runs), 8);  // (a row may start up to 7 entries into its first unit)
    while (((int64_t)V << (kUnit - a.drop)) > ((int64_t)1 << 62)) ++a.drop;
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
    logit_dtype == PA_PROB_F32 ? launch_sample<float, kDraw>(a, R, (cudaStream_t)stream)
                               : launch_sample<uint16_t, kDraw>(a, R, (cudaStream_t)stream);
    return check_launch(fn);
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
    if (logit_dtype == PA_PROB_F32)
        prob_dtype == PA_PROB_F32 ? launch_sample<float, kProbsF32>(a, R, s) : launch_sample<float, kProbsBf16>(a, R, s);
    else
        prob_dtype == PA_PROB_F32 ? launch_sample<uint16_t, kProbsF32>(a, R, s) : launch_sample<uint16_t, kProbsBf16>(a, R, s);
    return check_launch(fn);
}

}  // extern "C"
