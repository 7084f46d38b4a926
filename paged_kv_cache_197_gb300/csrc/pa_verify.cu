// Verification of drafted tokens (pa_draft.h): which branch of the tree is kept, and the
// token drawn behind it.
//
// At a node with target distribution p and draft distribution q, rejecting a child replaces
// the residual R by max(R - Z q, 0), Z its sum.  Since q >= 0 the nested maxima collapse:
//   max(max(p - C q, 0) - Z q, 0) = max(p - (C + Z) q, 0),
// so the state of a node is one number C, a child's test needs p and q at its token alone,
// and a rejection costs one pass over the vocabulary for Z = sum_v max(p - C q, 0).
// The weights p - C q and their sums are carried as unevaluated pairs of fp32 (two-term
// sums and products with their rounding errors): about 48 bits at fp32 rates, where GB300's
// fp64 lanes (two per SM and clock) would take several times longer than the loads.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "pa_draft.h"
#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

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
};

__device__ __forceinline__ void raise_flag(int *err_flag, int bit) {
    if (err_flag) atomicOr(err_flag, bit);
}

// A probability: negative and NaN entries count as 0.
template <typename T>
__device__ __forceinline__ float prob(const T *row, int64_t v) {
    float x;
    if constexpr (sizeof(T) == 4)
        x = row[v];
    else
        x = __uint_as_float((uint32_t)row[v] << 16);
    return x > 0.f ? x : 0.f;
}

// An unevaluated sum of two fp32, |lo| <= ulp(hi) / 2 up to a few roundings.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair split(double x) {
    const float hi = (float)x;
    return {hi, (float)(x - (double)hi)};
}

// max(p - C q, 0) as a pair.  C q = h + e exactly (e the product's rounding error), p - h is
// a two-term difference with its error; C.lo q is below ulp(h) / 2.
__device__ __forceinline__ Pair residual(float p, float q, Pair C) {
    const float h = __fmul_rn(C.hi, q), e = __fmaf_rn(C.hi, q, -h);
    const float d = __fsub_rn(p, h), b = __fsub_rn(p, d);
    float lo = __fadd_rn(__fsub_rn(__fsub_rn(p, __fadd_rn(d, b)), __fsub_rn(h, b)), 0.f);
    lo = __fsub_rn(__fsub_rn(lo, e), __fmul_rn(C.lo, q));
    const float hi = __fadd_rn(d, lo);
    lo = __fsub_rn(lo, __fsub_rn(hi, d));
    const bool pos = hi > 0.f;
    return {pos ? hi : 0.f, pos ? lo : 0.f};
}

__device__ __forceinline__ void add(Pair &s, Pair x) {
    const float t = __fadd_rn(s.hi, x.hi), b = __fsub_rn(t, s.hi);
    const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(x.hi, b));
    s.lo = __fadd_rn(s.lo, __fadd_rn(e, x.lo));
    s.hi = t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ double s_sum[kWarps];
    __shared__ int s_parent[PA_TREE_MAX_NODES], s_place[PA_TREE_MAX_NODES];
    __shared__ int s_next;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = a.query_start[s], r1 = a.query_start[s + 1], L = r1 - r0;
    for (int j = tid; j < a.W; j += kThreads) a.tokens_out[(int64_t)s * a.W + j] = a.path[(int64_t)s * a.W + j] = -1;
    const bool offsets = r0 >= 0 && r1 <= a.T && L >= 0 && L <= a.W;
    bool bad = false;
    if (offsets)
        for (int j = tid; j < L; j += kThreads) {
            s_parent[j] = a.parents[r0 + j];
            s_place[j] = -1;
            bad |= s_parent[j] < -1 || s_parent[j] >= j;
        }
    bad = __syncthreads_or(bad);
    if (!offsets || bad || L == 0) {
        if (tid == 0) {
            a.n_out[s] = 0;
            if (!offsets) raise_flag(a.err_flag, PA_FLAG_QUERY_OUT_OF_RANGE);
            if (bad) raise_flag(a.err_flag, PA_FLAG_TREE_PARENT);
        }
        if (offsets && a.slots)
            for (int j = tid; j < L; j += kThreads) a.slots[r0 + j] = -1;
        return;
    }
    const T *P = static_cast<const T *>(a.p), *Q = static_cast<const T *>(a.q);
    int cur = 0, n = 1, rejected = 0;  // rejected children of cur
    double C = 0.0, Z = 1.0;
    // the mass of R = max(p - C q, 0), or of p without the rejected children of cur
    auto weight = [&](const T *pr, const T *qr, Pair c, int v) -> Pair {
        const float p = prob(pr, v);
        if (qr) return residual(p, prob(qr, v), c);
        return {p, 0.f};
    };
    auto is_rejected = [&](int v, int before) {  // one-hot drafts: v a child of cur tried before row `before`
        for (int j = cur + 1; j < before; ++j)
            if (s_parent[j] == cur && a.tokens[r0 + j] == v) return true;
        return false;
    };
    auto mass = [&](int before) -> double {
        const T *pr = P + (r0 + cur) * a.p_stride, *qr = Q && rejected ? Q + (r0 + cur) * a.q_stride : nullptr;
        const Pair c = split(C);
        Pair sum{0.f, 0.f};
        for (int v = tid; v < a.V; v += kThreads) {
            if (!Q && rejected && is_rejected(v, before)) continue;
            add(sum, weight(pr, qr, c, v));
        }
        double d = (double)sum.hi + (double)sum.lo;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        __syncthreads();
        if (lane == 0) s_sum[warp] = d;
        __syncthreads();
        d = 0.0;
        for (int w = 0; w < kWarps; ++w) d += s_sum[w];
        return d;
    };
    if (tid == 0) s_place[0] = 0;
    for (int j = 1; j < L; ++j) {  // children come after their parent, and in the order they are tried
        if (s_parent[j] != cur) continue;
        const int x = a.tokens[r0 + j];
        bool yes = false;
        if (x < 0 || x >= a.V) {
            if (tid == 0) raise_flag(a.err_flag, PA_FLAG_TOKEN_OUT_OF_RANGE);
        } else {
            const double p = prob(P + (r0 + cur) * a.p_stride, x);
            const double q = Q ? prob(Q + (r0 + cur) * a.q_stride, x) : 1.0;
            const double R = Q ? fmax(p - C * q, 0.0) : (rejected && is_rejected(x, j) ? 0.0 : p);
            yes = (double)a.u[r0 + j] * Z * q < R;
        }
        if (yes) {
            cur = j;
            C = 0.0;
            Z = 1.0;
            rejected = 0;
            if (tid == 0) s_place[j] = n;
            ++n;
        } else {
            ++rejected;
            C += Z;
            Z = mass(j + 1);
        }
    }
    // the next token: the first v whose running sum of R exceeds u Z
    double total = rejected ? Z : mass(0);
    if (rejected && !(total > 0.0)) {  // nothing left: the target's own row
        rejected = 0;
        C = 0.0;
        total = mass(0);
    }
    int next = -1;
    if (total > 0.0 && total <= 1.7e308) {
        const T *pr = P + (r0 + cur) * a.p_stride, *qr = Q && rejected ? Q + (r0 + cur) * a.q_stride : nullptr;
        const Pair c = split(C);
        const double target = (double)a.u_final[s] * total;
        // each warp sums an equal run of the vocabulary; the run that passes the target is
        // scanned by its warp
        const int run = (a.V + kWarps - 1) / kWarps, begin = min(a.V, warp * run), end = min(a.V, begin + run);
        auto weigh = [&](int v) -> double {
            if (!Q && rejected && is_rejected(v, L)) return 0.0;
            const Pair w = weight(pr, qr, c, v);
            return (double)w.hi + (double)w.lo;
        };
        double d = 0.0;
        int last = -1;  // the last v with any weight
        for (int v = begin + lane; v < end; v += 32) {
            const double w = weigh(v);
            d += w;
            if (w > 0.0) last = v;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            d += __shfl_xor_sync(0xffffffffu, d, o);
            last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
        }
        __syncthreads();
        if (lane == 0) s_sum[warp] = d;
        if (tid == 0) s_next = -1;
        __syncthreads();
        double before = 0.0;
        for (int w = 0; w < warp; ++w) before += s_sum[w];
        if (last >= 0) atomicMax(&s_next, last);
        __syncthreads();
        const int fallback = s_next;
        __syncthreads();
        if (tid == 0) s_next = 0x7fffffff;
        __syncthreads();
        if (before <= target && before + d > target) {
            double at = before;
            for (int v0 = begin; v0 < end; v0 += 32) {
                const int v = v0 + lane;
                double w = v < end ? weigh(v) : 0.0, scan = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, scan, o);
                    if (lane >= o) scan += y;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, w > 0.0 && at + scan > target);
                if (hit) {
                    if (lane == 0) atomicMin(&s_next, v0 + __ffs(hit) - 1);
                    break;
                }
                at += __shfl_sync(0xffffffffu, scan, 31);
            }
        }
        __syncthreads();
        next = s_next == 0x7fffffff ? fallback : s_next;
    } else if (tid == 0) {
        raise_flag(a.err_flag, PA_FLAG_PROBABILITY);
    }
    __syncthreads();
    if (tid == 0) a.n_out[s] = n;
    for (int j = tid; j < L; j += kThreads) {
        const int place = s_place[j];
        int64_t slot = -1;
        if (place >= 0) {
            a.path[(int64_t)s * a.W + place] = r0 + j;
            if (place > 0) a.tokens_out[(int64_t)s * a.W + place - 1] = a.tokens[r0 + j];
            if (place == n - 1) a.tokens_out[(int64_t)s * a.W + place] = next;
            if (a.slots) {
                const int64_t pos = (int64_t)max(a.context_lens[s], 0) + place;
                const int b = pos / a.bs < a.M ? a.block_tables[(int64_t)s * a.M + pos / a.bs] : -1;
                if (b >= 0 && b < a.N)
                    slot = (int64_t)b * a.bs + pos % a.bs;
                else
                    raise_flag(a.err_flag, PA_FLAG_BLOCK_OUT_OF_RANGE);
            }
        }
        if (a.slots) a.slots[r0 + j] = slot;
    }
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
    launch_dependent(prob_dtype == PA_PROB_F32 ? verify_kernel<float> : verify_kernel<uint16_t>, dim3(S), dim3(kThreads), 0,
                     (cudaStream_t)stream, a);
    return check_launch(fn);
}
