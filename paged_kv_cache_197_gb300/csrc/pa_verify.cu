// Verification of drafted tokens (pa_draft.h): which branch of the tree is kept, and the
// token drawn behind it.
//
// At a node with target distribution p and draft distribution q, rejecting a child replaces
// the residual R by max(R - Z q, 0), Z its sum.  Since q >= 0 the nested maxima collapse:
//   max(max(p - C q, 0) - Z q, 0) = max(p - (C + Z) q, 0),
// so the state of a node is one number C, a child's test needs p and q at its token alone,
// and a rejection costs one pass over the vocabulary for Z = sum_v max(p - C q, 0).
// The weights p - C q, their sums and the borders they are compared with are carried as
// unevaluated pairs of fp32 (two-term sums and products with their rounding errors): about 48
// bits at fp32 rates.  GB300 has two fp64 lanes per SM and clock: a pass would take several
// times longer than its loads, and one choice among 32 sums takes 1230 clocks in fp64.
//
// A cluster of CTAs serves a sequence, each CTA a slice of the vocabulary and each warp an
// equal run of it.  All CTAs walk the tree alike, from the tests' probabilities gathered for
// all rows at once, and meet only for the sum of a pass: every CTA writes its part into the
// others' shared memory (the same number to each), one cluster barrier, and each adds the parts
// in the same order, so all decide the same.  (Another CTA's shared memory may be written once that CTA runs: all
// arrive at a cluster barrier on entry and wait for it behind the first pass, so its latency
// lies behind the gather and the loads.)  The draw needs no further pass: the sums of the last
// one say which run holds the target's place.
// Bounds: the latency of steps that depend on one another.  64 chains over 131072 entries, 67 MB,
// take 19.3 us with the launch: 1.4 for the gather, 0.7 for the tests, 2 for the pass (4 where
// HBM is shared), 1.1 for the exchange, 3.4 for the draw.  (One CTA a sequence: 429 us; 256
// threads a CTA and the draw one warp's in fp64: 31.5.)
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "pa_draft.h"
#include "pa_internal.cuh"

namespace pa {
namespace {

// Threads of a CTA: 512 while two CTAs per SM hold the batch (a run is half as long, and so is
// a pass), else 256: four CTAs per SM at 64 registers hold 76 sequences.  16 trees over 50021 entries
// take 17.2 us with 512 and 23.3 with 256, 64 chains over 131072 27.3 and 18.6.
constexpr int kFew = 512, kMany = 256;
constexpr int kMaxWarps = kFew / 32;
constexpr int kMaxCluster = 8;

struct VerifyArgs {
    int32_t *tokens_out, *path, *n_out;
    int64_t *slots;
    const int32_t *tokens;
    const void *p, *q;
    int64_t p_stride, q_stride;
    const int32_t *query_start, *parents;
    const float *u, *u_final;
    const int32_t *block_tables, *context_lens;
    int *err_flag;
    int T, V, W, M, bs, N;  // W: columns of tokens_out and path
    int cluster, run;       // CTAs per sequence; vocabulary entries per warp (a multiple of 8)
    int vector;             // rows are 16-byte aligned
};

__device__ __forceinline__ void raise_flag(int *err_flag, int bit) {
    if (err_flag) atomicOr(err_flag, bit);
}

// A probability: negative and NaN entries count as 0.
__device__ __forceinline__ float prob(const float *row, int64_t v) { return fmaxf(__ldg(row + v), 0.f); }
__device__ __forceinline__ float prob(const uint16_t *row, int64_t v) {
    return fmaxf(__uint_as_float((uint32_t)__ldg(row + v) << 16), 0.f);
}

// Entries of one 16-byte load.
template <typename T>
constexpr int kVec = 16 / sizeof(T);
__device__ __forceinline__ void unpack(const uint4 &w, float (&x)[4]) {
    x[0] = fmaxf(__uint_as_float(w.x), 0.f);
    x[1] = fmaxf(__uint_as_float(w.y), 0.f);
    x[2] = fmaxf(__uint_as_float(w.z), 0.f);
    x[3] = fmaxf(__uint_as_float(w.w), 0.f);
}
__device__ __forceinline__ void unpack(const uint4 &w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = fmaxf(__uint_as_float(u[i] << 16), 0.f);
        x[2 * i + 1] = fmaxf(__uint_as_float(u[i] & 0xffff0000u), 0.f);
    }
}

// Four neighbouring entries (4 v aligned to them).
__device__ __forceinline__ void quad(const float *p, float *x) {
    const float4 w = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = fmaxf(w.x, 0.f);
    x[1] = fmaxf(w.y, 0.f);
    x[2] = fmaxf(w.z, 0.f);
    x[3] = fmaxf(w.w, 0.f);
}
__device__ __forceinline__ void quad(const uint16_t *p, float *x) {
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
    x[0] = fmaxf(__uint_as_float(w.x << 16), 0.f);
    x[1] = fmaxf(__uint_as_float(w.x & 0xffff0000u), 0.f);
    x[2] = fmaxf(__uint_as_float(w.y << 16), 0.f);
    x[3] = fmaxf(__uint_as_float(w.y & 0xffff0000u), 0.f);
}

// An unevaluated sum of two fp32, |lo| <= ulp(hi) / 2 up to a few roundings.
struct Pair {
    float hi, lo;
};

// max(p - C q, 0) as a pair.  C.hi q = h + e exactly (e the product's rounding error), p - h
// is a two-term difference with its error; C.lo q is below ulp(h) / 2.
__device__ __forceinline__ Pair residual(float p, float q, Pair C) {
    const float h = __fmul_rn(C.hi, q), e = __fmaf_rn(C.hi, q, -h);
    const float d = __fsub_rn(p, h), b = __fsub_rn(p, d);
    float lo = __fsub_rn(__fsub_rn(p, __fadd_rn(d, b)), __fsub_rn(h, b));
    lo = __fsub_rn(__fsub_rn(lo, e), __fmul_rn(C.lo, q));
    const float hi = __fadd_rn(d, lo);
    lo = __fsub_rn(lo, __fsub_rn(hi, d));
    const bool pos = hi > 0.f;
    return {pos ? hi : 0.f, pos ? lo : 0.f};
}

// The same for C = 1, a node's first rejection: p - q and its rounding error.
__device__ __forceinline__ Pair residual(float p, float q) {
    const float d = __fsub_rn(p, q), b = __fsub_rn(p, d);
    const float lo = __fsub_rn(__fsub_rn(p, __fadd_rn(d, b)), __fsub_rn(q, b));
    return {d > 0.f ? d : 0.f, d > 0.f ? lo : 0.f};
}

__device__ __forceinline__ void add(Pair &s, Pair x) {
    const float t = __fadd_rn(s.hi, x.hi), b = __fsub_rn(t, s.hi);
    const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(x.hi, b));
    s.lo = __fadd_rn(s.lo, __fadd_rn(e, x.lo));
    s.hi = t;
}

__device__ __forceinline__ Pair plus(Pair s, Pair x) {
    add(s, x);
    return s;
}

// x y for a single y, and whether a < b (the difference of the leading parts is exact where they
// are close).
__device__ __forceinline__ Pair times(Pair x, float y) {
    const float h = __fmul_rn(x.hi, y);
    return {h, __fmaf_rn(x.lo, y, __fmaf_rn(x.hi, y, -h))};
}
__device__ __forceinline__ bool less(Pair a, Pair b) { return __fadd_rn(__fsub_rn(a.hi, b.hi), __fsub_rn(a.lo, b.lo)) < 0.f; }

// The sum over the first `lanes` (a power of two) lanes' pairs, in each of them: the same hi, but lo
// differs between lanes by its roundings (add does not round alike with its operands exchanged).
__device__ __forceinline__ Pair lanes_sum(Pair s, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) {
        const Pair x{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)};
        add(s, x);
    }
    return s;
}

// Inclusive sums over the lanes.
__device__ __forceinline__ Pair lanes_scan(Pair s, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair x{__shfl_up_sync(0xffffffffu, s.hi, o), __shfl_up_sync(0xffffffffu, s.lo, o)};
        if (lane >= o) add(s, x);
    }
    return s;
}

// What the first warp asks of all: a pass over the node's residual, or nothing more.
struct Task {
    int cur, rejected;  // the node and its rejected children
    Pair c;
    int more;
    int n;              // rows on the path so far
};

struct Shared {
    Pair part[2][kMaxCluster];              // the CTAs' sums of a pass, by its parity
    Pair run[kMaxWarps];                    // the warps' sums of the last pass
    Pair piece[kMaxWarps];                  // the draw: the warps' sums of the run drawn from
    Task task;
    float tp[PA_TREE_MAX_NODES], tq[PA_TREE_MAX_NODES];  // p and q of each row's token at its parent
    int parent[PA_TREE_MAX_NODES], token[PA_TREE_MAX_NODES], place[PA_TREE_MAX_NODES];
    float u[PA_TREE_MAX_NODES];
    int block[PA_TREE_MAX_NODES];           // block of the sequence's slot at each place
    int gone[PA_TREE_MAX_NODES];            // the current node's rejected tokens (no drafter)
};

// A node's residual: its rows of p and q, C, and (no drafter) the tokens rejected.
template <typename T>
struct Residual {
    const T *p, *q;  // q null: R is p without the tokens gone
    Pair c;
    const int *gone;
    int n_gone;

    // R(v) from the entries x of p and y of q
    __device__ __forceinline__ Pair weight(int64_t v, float x, float y) const {
        if (q) return residual(x, y, c);
        for (int i = 0; i < n_gone; ++i)
            if (gone[i] == (int)v) return {0.f, 0.f};
        return {x, 0.f};
    }
};

// The sum of R over a warp's run [begin, end).  DRAFTED: 0 = p alone, 1 = p - q, 2 = p - C q.
template <typename T, int DRAFTED>
__device__ __forceinline__ Pair run_sum(const Residual<T> &R, int64_t begin, int64_t end, bool vector, int lane) {
    constexpr int N = kVec<T>;
    Pair s{0.f, 0.f};
    bool plain = true;  // no token of the run is gone
    if (!DRAFTED && R.n_gone > 0) {
        bool in = false;
        for (int i = lane; i < R.n_gone; i += 32) in |= R.gone[i] >= begin && R.gone[i] < end;
        plain = !__any_sync(0xffffffffu, in);
    }
    int64_t v = begin;
    if (vector && plain) {
        constexpr int U = 4;  // loads in flight per operand
        for (; v + 32 * N * U <= end; v += 32 * N * U) {
            uint4 a[U], b[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                a[i] = __ldg(reinterpret_cast<const uint4 *>(R.p + v + (i * 32 + lane) * N));
                if (DRAFTED) b[i] = __ldg(reinterpret_cast<const uint4 *>(R.q + v + (i * 32 + lane) * N));
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float x[N], y[N];
                unpack(a[i], x);
                if (DRAFTED) unpack(b[i], y);
#pragma unroll
                for (int e = 0; e < N; ++e)
                    add(s, DRAFTED == 2 ? residual(x[e], y[e], R.c) : DRAFTED == 1 ? residual(x[e], y[e]) : Pair{x[e], 0.f});
            }
        }
    }
    // what is left of the run, or all of it; entries behind the run count as 0
    constexpr int U = 8;
    for (; v < end; v += 32 * U) {
        float x[U], y[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t at = v + i * 32 + lane;
            x[i] = at < end ? prob(R.p, at) : 0.f;
            y[i] = DRAFTED && at < end ? prob(R.q, at) : 0.f;
        }
        if (plain) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                add(s, DRAFTED == 2 ? residual(x[i], y[i], R.c) : DRAFTED == 1 ? residual(x[i], y[i]) : Pair{x[i], 0.f});
        } else {
#pragma unroll 1
            for (int i = 0; i < U; ++i) {
                float xi = x[0];
#pragma unroll
                for (int k = 1; k < U; ++k) xi = i == k ? x[k] : xi;
                add(s, R.weight(v + i * 32 + lane, xi, 0.f));
            }
        }
    }
    return lanes_sum(s, 32);
}

// The sum of R over one lane's [b, e), eight entries at a time; vector: 16-byte loads (b a multiple
// of 4).
template <typename T>
__device__ __forceinline__ Pair piece_sum(const Residual<T> &R, int64_t b, int64_t e, bool vector) {
    Pair s{0.f, 0.f};
#pragma unroll 1
    for (int64_t v = b; v < e; v += 8) {
        float x[8], y[8];
        if (vector && v + 8 <= e) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                quad(R.p + v + i, x + i);
                if (R.q) quad(R.q + v + i, y + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = v + i < e ? prob(R.p, v + i) : 0.f;
                y[i] = R.q && v + i < e ? prob(R.q, v + i) : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) add(s, R.weight(v + i, x[i], y[i]));
    }
    return s;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
    constexpr int kWarps = kThreads / 32;
    __shared__ Shared sh;
    if (a.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    auto cluster_runs = [&] {  // every CTA of the cluster has started
        if (a.cluster > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int s = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = a.query_start[s], r1 = a.query_start[s + 1], L = r1 - r0;
    int32_t *tokens_out = a.tokens_out + (int64_t)s * a.W, *path = a.path + (int64_t)s * a.W;
    const bool offsets = r0 >= 0 && r1 <= a.T && L >= 0 && L <= a.W;
    const T *P = static_cast<const T *>(a.p), *Q = static_cast<const T *>(a.q);
    bool bad = false;
    if (offsets)
        for (int j = tid; j < L; j += kThreads) {
            const int p = a.parents[r0 + j], x = j ? a.tokens[r0 + j] : -1;
            bad |= p < -1 || p >= j;
            sh.parent[j] = p;
            sh.token[j] = x;
            sh.place[j] = j ? -1 : 0;
            sh.u[j] = j ? a.u[r0 + j] : 0.f;
            if (a.slots) {
                const int64_t at = ((int64_t)max(a.context_lens[s], 0) + j) / a.bs;
                sh.block[j] = at < a.M ? a.block_tables[(int64_t)s * a.M + at] : -1;
            }
            // every test needs p and q at the row's token, at its parent
            float tp = 0.f, tq = 0.f;
            if (p >= 0 && p < j && x >= 0 && x < a.V) {
                tp = prob(P + (r0 + p) * a.p_stride, x);
                tq = Q ? prob(Q + (r0 + p) * a.q_stride, x) : 1.f;
            }
            sh.tp[j] = tp;
            sh.tq[j] = tq;
        }
    bad = __syncthreads_or(bad);
    if (!offsets || bad || L == 0) {  // every CTA of the cluster alike
        cluster_runs();
        if (rank == 0) {
            for (int j = tid; j < a.W; j += kThreads) tokens_out[j] = path[j] = -1;
            if (offsets && a.slots)
                for (int j = tid; j < L; j += kThreads) a.slots[r0 + j] = -1;
            if (tid == 0) {
                a.n_out[s] = 0;
                if (!offsets) raise_flag(a.err_flag, PA_FLAG_QUERY_OUT_OF_RANGE);
                if (bad) raise_flag(a.err_flag, PA_FLAG_TREE_PARENT);
            }
        }
        return;
    }
    const int64_t begin = min((int64_t)a.V, ((int64_t)rank * kWarps + warp) * a.run), end = min((int64_t)a.V, begin + a.run);
    // ---- the walk, in the first warp; the others join it for the passes.  A row is tested
    // after its parent and its older siblings.
    int cur = 0, n = 1, rejected = 0, j = 1, pass = 0;
    Pair C{0.f, 0.f}, Z{1.f, 0.f}, total{0.f, 0.f};
    bool fresh = false;  // `total` is of the current residual
    Task task;
    auto left_at = [&](const Task &t) {
        return Residual<T>{P + (r0 + t.cur) * a.p_stride, Q && t.rejected > 0 ? Q + (r0 + t.cur) * a.q_stride : nullptr, t.c,
                           sh.gone, Q ? 0 : t.rejected};
    };
    for (;;) {
        if (warp == 0) {
            bool need = false;
            if (pass > 0) {  // back from a pass
                total = lanes_sum(lane < a.cluster ? sh.part[(pass - 1) & 1][lane] : Pair{0.f, 0.f}, kMaxCluster);
                total = {__shfl_sync(0xffffffffu, total.hi, 0), __shfl_sync(0xffffffffu, total.lo, 0)};
                if (rejected) Z = total;
                fresh = true;
            }
            while (!need && j < L) {
                // the next child of cur from row j on
                int at = L;
                for (int base = j & ~31; base < L; base += 32) {
                    const int i = base + lane;
                    const unsigned m = __ballot_sync(0xffffffffu, i >= j && i < L && sh.parent[i] == cur);
                    if (m) {
                        at = base + __ffs(m) - 1;
                        break;
                    }
                }
                j = at + 1;
                if (at >= L) break;
                const int x = sh.token[at];
                const float q = sh.tq[at];
                Pair R{sh.tp[at], 0.f};
                bool again = false;  // no drafter: the token was rejected before
                if (Q) {
                    if (rejected) R = residual(R.hi, q, C);
                } else {
                    for (int i = 0; i < rejected; ++i) again |= sh.gone[i] == x;
                    if (again) R.hi = 0.f;
                }
                // u Z q: the product of u and q is a pair, so a first child's test is exact
                const Pair uq = times(Pair{sh.u[at], 0.f}, q), uzq = plus(times(Z, uq.hi), Pair{__fmul_rn(Z.hi, uq.lo), 0.f});
                const bool inside = x >= 0 && x < a.V;
                if (!inside && rank == 0 && lane == 0) raise_flag(a.err_flag, PA_FLAG_TOKEN_OUT_OF_RANGE);
                if (inside && less(uzq, R)) {
                    cur = at;
                    C = {0.f, 0.f};
                    Z = {1.f, 0.f};
                    rejected = 0;
                    fresh = false;
                    if (lane == 0) sh.place[at] = n;
                    ++n;
                    continue;
                }
                add(C, Z);
                __syncwarp();
                if (!Q && lane == 0) sh.gone[rejected] = x;
                __syncwarp();
                ++rejected;
                // Without a drafter the mass after the first rejection falls by what is
                // rejected: no pass while the difference keeps its digits.
                const Pair rest = plus(Z, Pair{-R.hi, 0.f});
                if (!Q && rejected > 1 && rest.hi > 1e-6f) {
                    Z = rest;
                    fresh = again && fresh;
                } else {
                    need = true;
                }
            }
            if (!need && !fresh) need = true;  // the draw needs the sums
            if (!need && rejected && !(total.hi > 0.f)) {
                // nothing left: the target's own row
                rejected = 0;
                C = {0.f, 0.f};
                need = true;
            }
            if (lane == 0) sh.task = Task{cur, rejected, C, need, n};
        }
        __syncthreads();
        task = sh.task;
        if (!task.more) break;
        const Residual<T> R = left_at(task);
        const Pair d = !R.q ? run_sum<T, 0>(R, begin, end, a.vector != 0, lane)
                       : R.c.hi == 1.f && R.c.lo == 0.f ? run_sum<T, 1>(R, begin, end, a.vector != 0, lane)
                                                        : run_sum<T, 2>(R, begin, end, a.vector != 0, lane);
        if (lane == 0) sh.run[warp] = d;
        __syncthreads();
        if (pass == 0) cluster_runs();
        if (warp == 0) {
            Pair mine = lanes_sum(lane < kWarps ? sh.run[lane] : Pair{0.f, 0.f}, kWarps);
            // lane 0's, so that every CTA gets the same number
            mine = {__shfl_sync(0xffffffffu, mine.hi, 0), __shfl_sync(0xffffffffu, mine.lo, 0)};
            if (lane < a.cluster) {
                uint32_t to = (uint32_t)__cvta_generic_to_shared(&sh.part[pass & 1][rank]);
                asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(to) : "r"(lane));
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(mine.hi), "f"(mine.lo) : "memory");
            }
        }
        if (a.cluster > 1)
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else
            __syncthreads();
        ++pass;
    }
    // ---- the draw: the first v whose running sum of R exceeds u total; past all of them (numbers
    // of 1 or more, rounding) the last with weight.  It is narrowed down to a CTA, one of its runs,
    // a warp's and a lane's piece of that run (the CTA sums all of them at once), and parts of that
    // piece.  (One loop: most of a draw is latency and fetching its instructions, met once a
    // launch.  One warp that scanned the run, in fp64, took 12000 to 20000 clocks.)
    n = task.n;
    {
        const Residual<T> R = left_at(task);
        Pair before{0.f, 0.f}, target{0.f, 0.f}, own{0.f, 0.f};  // R's sum before what is left; its place; a thread's piece
        int64_t lo = 0, hi = a.V, threads_piece = 0;
#pragma unroll 1
        for (int level = 0;; ++level) {
            int64_t piece;
            Pair mine{0.f, 0.f};
            if (level == 0) {
                piece = (int64_t)a.run * kWarps;
                if (lane < a.cluster) mine = sh.part[(pass - 1) & 1][lane];
            } else if (level == 1) {
                piece = a.run;
                if (lane < kWarps) mine = sh.run[lane];
            } else if (level == 3) {
                piece = threads_piece;
                mine = own;
            } else {
                const int64_t len = hi - lo, parts = level == 2 ? kThreads : 32;
                const bool quads = a.vector && len >= 4 * parts;  // (lo stays a multiple of 4)
                piece = quads ? (len + 4 * parts - 1) / (4 * parts) * 4 : (len + parts - 1) / parts;
                const int64_t b = min(hi, lo + (level == 2 ? tid : lane) * piece);
                mine = piece_sum(R, b, min(hi, b + piece), quads);
                if (level == 2) {
                    own = mine;
                    threads_piece = piece;
                    piece *= 32;
                    mine = lanes_sum(mine, 32);
                    if (lane == 0) sh.piece[warp] = mine;
                    __syncthreads();
                    mine = lane < kWarps ? sh.piece[lane] : Pair{0.f, 0.f};
                }
            }
            const Pair upto = lanes_scan(mine, lane);
            if (level == 0) {
                const float all = __shfl_sync(0xffffffffu, upto.hi, 31);
                if (!(all > 0.f && all <= 3.402823466e38f)) {
                    if (rank == 0 && tid == 0) {
                        raise_flag(a.err_flag, PA_FLAG_PROBABILITY);
                        tokens_out[n - 1] = -1;
                    }
                    break;
                }
                target = times(Pair{all, __shfl_sync(0xffffffffu, upto.lo, 31)}, a.u_final[s]);
            }
            const unsigned any = __ballot_sync(0xffffffffu, mine.hi > 0.f);
            const unsigned hit = __ballot_sync(0xffffffffu, mine.hi > 0.f && less(target, plus(before, upto)));
            const int at = hit ? __ffs(hit) - 1 : 31 - __clz(any);
            if (at != (level == 0 ? rank : level == 2 ? warp : at)) break;
            const Pair up{__shfl_sync(0xffffffffu, upto.hi, max(at - 1, 0)), __shfl_sync(0xffffffffu, upto.lo, max(at - 1, 0))};
            if (at > 0) add(before, up);
            lo += at * piece;
            hi = min(hi, lo + piece);
            if (hi - lo <= 1 && level != 1) {
                if (lane == 0 && (level > 1 || warp == 0)) tokens_out[n - 1] = (int)lo;
                break;
            }
        }
    }
    // ---- the branch
    if (rank != 0) return;
    for (int j = n + tid; j < a.W; j += kThreads) tokens_out[j] = path[j] = -1;
    if (tid == 0) a.n_out[s] = n;
    for (int j = tid; j < L; j += kThreads) {
        const int place = sh.place[j];
        int64_t slot = -1;
        if (place >= 0) {
            path[place] = r0 + j;
            if (place > 0) tokens_out[place - 1] = sh.token[j];
            if (a.slots) {
                const int64_t pos = (int64_t)max(a.context_lens[s], 0) + place;
                const int b = sh.block[place];
                if (b >= 0 && b < a.N)
                    slot = (int64_t)b * a.bs + pos % a.bs;
                else
                    raise_flag(a.err_flag, PA_FLAG_BLOCK_OUT_OF_RANGE);
            }
        }
        if (a.slots) a.slots[r0 + j] = slot;
    }
}

template <typename T>
cudaError_t launch_verify(const VerifyArgs &a, int S, int threads, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S * a.cluster);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return threads == kFew ? cudaLaunchKernelEx(&cfg, verify_kernel<T, kFew>, a) : cudaLaunchKernelEx(&cfg, verify_kernel<T, kMany>, a);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_verify_tree(int32_t *tokens_out, int32_t *path, int32_t *n_out, int64_t *slot_mapping,
                                    const int32_t *draft_tokens, const void *target_probs, int64_t target_stride,
                                    const void *draft_probs, int64_t draft_stride, int prob_dtype,
                                    const int32_t *query_start, const int32_t *parents, const float *uniforms,
                                    const float *final_uniforms, int S, int T, int V, int max_query_len,
                                    const int32_t *block_tables, int M, const int32_t *context_lens, int bs, int N,
                                    int *err_flag, void *stream) {
    const char *fn = "pa_verify_tree";
    clear_error();
    if (S < 0 || T < 0) return fail(PA_ERR_INVALID_ARG, "%s: S = %d, T = %d", fn, S, T);
    if (S == 0) return PA_OK;
    if (prob_dtype != PA_PROB_F32 && prob_dtype != PA_PROB_BF16)
        return fail(PA_ERR_UNSUPPORTED, "%s: probability type %d not supported", fn, prob_dtype);
    if (V < 1 || V > (1 << 30)) return fail(PA_ERR_INVALID_ARG, "%s: V = %d (1 .. 2^30)", fn, V);
    if (T == 0 || max_query_len < 1 || max_query_len > T || max_query_len > PA_TREE_MAX_NODES)
        return fail(PA_ERR_INVALID_ARG, "%s: max_query_len = %d (1 .. min(T, %d))", fn, max_query_len, PA_TREE_MAX_NODES);
    if (S > 65535) return fail(PA_ERR_UNSUPPORTED, "%s: at most 65535 sequences per call (got %d)", fn, S);
    constexpr int64_t kMost = (int64_t)1 << 40;
    if (target_stride < V || target_stride > kMost || (draft_probs && (draft_stride < V || draft_stride > kMost)))
        return fail(PA_ERR_INVALID_ARG, "%s: row strides must be at least V", fn);
    if (!tokens_out || !path || !n_out || !draft_tokens || !target_probs || !query_start || !parents || !uniforms ||
        !final_uniforms)
        return fail(PA_ERR_INVALID_ARG, "%s: null pointer", fn);
    const unsigned grain = prob_dtype == PA_PROB_F32 ? 3u : 1u;
    if (((uintptr_t)target_probs & grain) || ((uintptr_t)draft_probs & grain))
        return fail(PA_ERR_INVALID_ARG, "%s: probabilities must be aligned to their type", fn);
    if (slot_mapping) {
        if (!block_tables || !context_lens) return fail(PA_ERR_INVALID_ARG, "%s: null pointer (slot_mapping)", fn);
        if (M <= 0 || N <= 0) return fail(PA_ERR_INVALID_ARG, "%s: N = %d, M = %d must be positive", fn, N, M);
        if (bs != 16 && bs != 32) return fail(PA_ERR_UNSUPPORTED, "%s: block size %d not supported (16 or 32)", fn, bs);
    }
    VerifyArgs a{};
    a.tokens_out = tokens_out;
    a.path = path;
    a.n_out = n_out;
    a.slots = slot_mapping;
    a.tokens = draft_tokens;
    a.p = target_probs;
    a.q = draft_probs;
    a.p_stride = target_stride;
    a.q_stride = draft_stride;
    a.query_start = query_start;
    a.parents = parents;
    a.u = uniforms;
    a.u_final = final_uniforms;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.err_flag = err_flag;
    a.T = T;
    a.V = V;
    a.W = max_query_len;
    a.M = M;
    a.bs = bs;
    a.N = N;
    // small vocabularies: one CTA, whose sums need no cluster barrier (16 trees of 20 to 48 rows, one
    // CTA / eight: 13.5 / 14.8 us at 4000 entries, 15.0 / 14.0 at 8000, 51.3 / 17.2 at 50021; other counts
    // between one and eight, and batches that take several waves of clusters, are not measured)
    a.cluster = V > 6000 ? kMaxCluster : 1;
    const int threads = (int64_t)S * a.cluster <= 2 * device_sms() ? kFew : kMany;
    const int64_t runs = (int64_t)a.cluster * (threads / 32);
    a.run = (int)align_up((size_t)((V + runs - 1) / runs), 8);
    const int64_t elem = prob_dtype == PA_PROB_F32 ? 4 : 2;
    auto rows16 = [&](const void *p, int64_t stride) { return aligned16(p) && stride * elem % 16 == 0; };
    a.vector = rows16(target_probs, target_stride) && (!draft_probs || rows16(draft_probs, draft_stride));
    prob_dtype == PA_PROB_F32 ? launch_verify<float>(a, S, threads, (cudaStream_t)stream)
                              : launch_verify<uint16_t>(a, S, threads, (cudaStream_t)stream);
    return check_launch(fn);
}
