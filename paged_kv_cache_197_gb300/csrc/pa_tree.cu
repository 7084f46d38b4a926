// Attention of a tree of drafted tokens over the paged cache (pa_draft.h).
//
// Row i of a sequence attends all C cached tokens and, among its sequence's own rows, its
// ancestors and itself.  With the keys split into those two sets, and (m, l, o) the
// maximum, sum and weighted values of a set's softmax in the exp2 domain,
//   out = (2^(m1 - m) o1 + 2^(m2 - m) o2) / (2^(m1 - m) l1 + 2^(m2 - m) l2),  m = max(m1, m2):
// the context needs no mask at all and streams like a prompt every row shares, and the
// tree's own rows, a few hundred at most, are joined afterwards.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "pa_mma.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

using tiled::bf16x2;
using tiled::ex2;

struct TreeArgs {
    uint16_t *out;
    const uint16_t *q, *k, *v;  // [T][Hq][D]; rows' own keys and values
    int64_t k_stride, v_stride;
    const int32_t *parents, *query_start, *context_lens;
    int *err_flag;
    int S, T, Hq, Hkv, G;
    int chunks;                 // groups of query heads a warp takes at once
    int max_context_len, max_query_len;
    float scale_log2;
    // the context's partials: per partition of part_tokens tokens ...
    const float *ws_acc, *ws_ml;  // [T][Hq][max_parts][D], [T][Hq][max_parts][2]
    int part_tokens, max_parts;
    // ... or, with tiles.prefix, as the tcgen05 kernel leaves them
    TreeContext tiles;
};

// Rows of a CTA: with 8 the ragged batch of 33 to 64 nodes takes 0.6 us more (coarser last waves),
// with 2, which stage the sequence's rows for fewer of their own, 9.3 us.
constexpr int kJoinWarps = 4;
// Rows of a sequence kept in shared memory: of 512 bytes at head_dim 128, 45 KB with the
// parents, four CTAs an SM, and below the 48 KB a launch may have unasked.
constexpr int kStagedRows = 88;
static_assert(kStagedRows * 512 + PA_TREE_MAX_NODES * 4 <= 48 * 1024, "shared memory of a join without an attribute");

// The sums over the warp of HEADS values; lane i ends with that of value i % HEADS.  Halving
// exchanges while there is more than one value to a lane, then plain sums: 6 shuffles for
// four values instead of 20.
template <int HEADS>
__device__ __forceinline__ float sums(float (&x)[HEADS], int lane) {
#pragma unroll
    for (int o = 1, n = HEADS / 2; n >= 1; o <<= 1, n >>= 1) {
        const bool odd = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = odd ? x[2 * i] : x[2 * i + 1], keep = odd ? x[2 * i + 1] : x[2 * i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float s = x[0];
#pragma unroll
    for (int o = HEADS; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// One warp per (row, kv head, up to HEADS of its query heads); a CTA takes four rows of a
// sequence, and a lane D / 32 dims of every head.  The softmax scalars of head h are kept by
// the lanes i with i % HEADS = h, and spread when a row is added up.  First the row's
// ancestors, from the row up, in fp32, the sequence's keys and values for the kv head
// staged in shared memory (longer trees read them from L2); then the context's partials.
// Launched as a programmatic dependent: the first part, which the context's kernel does not
// touch, runs before the wait.  The first CTA waits even where it has nothing to join (a sequence
// left out): the context's kernel has then ended when this one has, and what comes next on
// the stream, another call with this workspace perhaps, waits for this one alone.
template <int D, int HEADS, bool STAGED>
__global__ void __launch_bounds__(kJoinWarps * 32, 32 / kJoinWarps) tree_join_kernel(const __grid_constant__ TreeArgs a) {
    constexpr int PER = D / 32;
    extern __shared__ __align__(16) unsigned char rows[];  // [rows][K D, V D] bf16
    __shared__ int s_parent[PA_TREE_MAX_NODES];
    const int tid = threadIdx.x, lane = tid & 31, s = blockIdx.z;
    const int kvh = blockIdx.y / a.chunks, h0 = blockIdx.y % a.chunks * HEADS;
    const int i = blockIdx.x * kJoinWarps + (tid >> 5);
    const int r0 = a.query_start[s], r1 = a.query_start[s + 1], L = r1 - r0;
    auto depart = [] {
        if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    };
    if (!(r0 >= 0 && r1 <= a.T && L >= 0 && L <= a.max_query_len)) return depart();  // flagged by the context's kernel
    const int top = min(L, ((int)blockIdx.x + 1) * kJoinWarps);  // ancestors are above their rows
    if ((int)blockIdx.x * kJoinWarps >= L && blockIdx.x > 0) return;
    if constexpr (STAGED) {
        constexpr int CH = D / 8;  // 16-byte pieces of a key or value
        for (int x = tid; x < top * 2 * CH; x += kJoinWarps * 32) {
            const int r = x / (2 * CH), c = x % (2 * CH);
            const uint16_t *src = c < CH ? a.k + (r0 + r) * a.k_stride + kvh * D + c * 8
                                         : a.v + (r0 + r) * a.v_stride + kvh * D + (c - CH) * 8;
            tiled::cp_async16(tiled::smem_u32(rows + x * 16), src, 16);
        }
        tiled::cp_async_commit();
    }
    bool bad = false;
    for (int j = tid; j < L; j += kJoinWarps * 32) {
        const int p = a.parents[r0 + j];
        s_parent[j] = p;
        bad |= p < -1 || p >= j;
    }
    const int ctx = min(max(a.context_lens[s], 0), a.max_context_len);
    const int heads = min(HEADS, a.G - h0);
    const int64_t pair = (int64_t)(r0 + i) * a.Hq + kvh * a.G + h0;  // row of the first head
    auto load = [&](const uint16_t *p, float (&x)[PER]) {
#pragma unroll
        for (int e = 0; e < PER; e += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(p + e);
            x[e] = __uint_as_float(w << 16);
            x[e + 1] = __uint_as_float(w & 0xffff0000u);
        }
    };
    float q[HEADS][PER], acc[HEADS][PER], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        if (i < L) load(a.q + (pair + (h < heads ? h : 0)) * D + lane * PER, q[h]);
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[h][e] = 0.f;
    }
    if constexpr (STAGED) tiled::cp_async_wait<0>();
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && a.err_flag) atomicOr(a.err_flag, PA_FLAG_TREE_PARENT);
        return depart();
    }
    if (i >= L) return depart();
    const int mine = lane % HEADS;  // the head whose scalars this lane keeps
    // acc = acc f + w x, with head h's f and w from the lane that keeps them
    auto add = [&](float f, float w, auto row) {
        if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                const float fh = __shfl_sync(0xffffffffu, f, h);
#pragma unroll
                for (int e = 0; e < PER; ++e) acc[h][e] *= fh;
            }
        }
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            const float wh = __shfl_sync(0xffffffffu, w, h);
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[h][e] = fmaf(wh, row(h, e), acc[h][e]);
        }
    };
    for (int at = i; at >= 0; at = s_parent[at]) {  // strictly decreasing: at most L steps
        float k[PER], v[PER], x[HEADS];
        if constexpr (STAGED) {
            const uint16_t *row = reinterpret_cast<const uint16_t *>(rows) + at * 2 * D + lane * PER;
            load(row, k);
            load(row + D, v);
        } else {
            load(a.k + (r0 + at) * a.k_stride + kvh * D + lane * PER, k);
            load(a.v + (r0 + at) * a.v_stride + kvh * D + lane * PER, v);
        }
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            x[h] = 0.f;
#pragma unroll
            for (int e = 0; e < PER; ++e) x[h] = fmaf(q[h][e], k[e], x[h]);
        }
        const float y = sums(x, lane) * a.scale_log2, mn = fmaxf(m, y), base = mn == -INFINITY ? 0.f : mn;
        const float f = m == mn ? 1.f : ex2(m - base), w = ex2(y - base);
        m = mn;
        l = l * f + w;
        add(f, w, [&](int, int e) { return v[e]; });
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // where the partials lie: lane h < HEADS keeps head h's first row and the step to its next
    const float *acc_in = a.ws_acc, *ml_in = a.ws_ml;
    int64_t row = (pair + mine) * a.max_parts, step = 1, later = 0;  // later: row of the second partial
    int n;
    if (a.tiles.prefix == nullptr) {
        n = (ctx + a.part_tokens - 1) / a.part_tokens;
        later = row + 1;
    } else {
        const TreeContext &c = a.tiles;
        const int64_t tiles = (ctx + kTreeTile - 1) / kTreeTile, total = c.prefix[a.S];
        n = 0;
        if (tiles > 0) {
            const int64_t first = c.prefix[s] + kvh * tree_unit_len(tiles, c.cols) + tree_pad(c.cols), groups = min((int64_t)c.groups, total);
            const int64_t g0 = tree_group_of(first, total, groups), g1 = tree_group_of(first + tiles - 1, total, groups);
            n = (int)(g1 - g0) + 1;
            if (n == 1) {
                acc_in = c.whole_acc;
                ml_in = c.whole_ml;
                row = pair + mine;
            } else {
                acc_in = c.cut_acc;
                ml_in = c.cut_ml;
                const int col = i * a.G + h0 + mine, member = col / c.cols, in = col % c.cols;
                const int64_t cta = g0 * c.members + member;
                row = (cta * 2 + 1) * c.cols + in;
                later = (cta + c.members) * 2 * c.cols + in;
                step = (int64_t)c.members * 2 * c.cols;
            }
        }
    }
    for (int p = 0; p < n; ++p) {
        float x[HEADS][PER];
        float2 ml = make_float2(-INFINITY, 0.f);
        if (mine < heads) ml = *reinterpret_cast<const float2 *>(ml_in + row * 2);
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            const int64_t r = __shfl_sync(0xffffffffu, row, h < heads ? h : 0);
            const float *src = acc_in + r * D + lane * PER;
            if constexpr (PER == 4) {
                const float4 w = *reinterpret_cast<const float4 *>(src);
                x[h][0] = w.x;
                x[h][1] = w.y;
                x[h][2] = w.z;
                x[h][3] = w.w;
            } else {
                const float2 w = *reinterpret_cast<const float2 *>(src);
                x[h][0] = w.x;
                x[h][1] = w.y;
            }
        }
        row = p == 0 ? later : row + step;
        const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.f : mn;
        const float f = m == mn ? 1.f : ex2(m - base), w = ex2(ml.x - base);
        m = mn;
        l = l * f + w * ml.y;
        add(f, w, [&](int h, int e) { return x[h][e]; });
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        const float ih = __shfl_sync(0xffffffffu, inv, h);
        if (h >= heads) continue;
        uint16_t *dst = a.out + (pair + h) * D + lane * PER;
        uint32_t w[PER / 2];
#pragma unroll
        for (int e = 0; e < PER; e += 2) w[e / 2] = bf16x2(acc[h][e] * ih, acc[h][e + 1] * ih);
        if constexpr (PER == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(dst) = w[0];
    }
}

template <int D, int HEADS>
cudaError_t launch_join(TreeArgs a, cudaStream_t stream) {
    a.chunks = (a.G + HEADS - 1) / HEADS;
    const dim3 grid((a.max_query_len + kJoinWarps - 1) / kJoinWarps, a.Hkv * a.chunks, a.S);
    if (a.max_query_len <= kStagedRows)
        return launch_dependent(tree_join_kernel<D, HEADS, true>, grid, dim3(kJoinWarps * 32), (size_t)a.max_query_len * 4 * D,
                                stream, a);
    return launch_dependent(tree_join_kernel<D, HEADS, false>, grid, dim3(kJoinWarps * 32), 0, stream, a);
}

// Up to four heads a warp (eight: 126.5 against 123.1 us for the 70B-shaped batch, 105 registers and
// half the warps per SM; two: 125.8).
template <int D>
cudaError_t launch_join_heads(const TreeArgs &a, cudaStream_t stream) {
    return a.G == 1 ? launch_join<D, 1>(a, stream) : a.G == 2 ? launch_join<D, 2>(a, stream)
           : launch_join<D, 4>(a, stream);
}

// Partitions of the contexts and the workspace: as for the multi-token calls, n balanced
// partitions of the longest context scored by (last-wave fill) x len / (len + 512), with at
// least two waves of two CTAs per SM.
struct TreePlan {
    int CB, part_tokens, max_parts;
    // tcgen05: members and groups of CTAs, columns per CTA, and where the cut partials and
    // the sequences' first tiles lie
    int members, groups, cols;
    size_t ml_off, cut_off, cut_ml_off, prefix_off, bytes;
};

TreePlan plan_tree(int S, int T, int Hq, int Hkv, int D, int kv_dtype, int max_context_len, int max_query_len) {
    TreePlan p{};
    const int G = Hq / Hkv, ctx = std::max(max_context_len, 1), sms = device_sms();
    if (tree_tc_eligible(D, kv_dtype)) {
        const int64_t columns = (int64_t)max_query_len * G;
        p.cols = columns <= 128 ? 128 : 256;
        p.members = (int)((columns + p.cols - 1) / p.cols);
        p.groups = std::max(1, sms / p.members);
        const size_t whole = (size_t)T * Hq, cut = (size_t)p.groups * p.members * 2 * p.cols;
        p.ml_off = align_up(whole * D * sizeof(float), 256);
        p.cut_off = align_up(p.ml_off + whole * 2 * sizeof(float), 256);
        p.cut_ml_off = align_up(p.cut_off + cut * D * sizeof(float), 256);
        p.prefix_off = align_up(p.cut_ml_off + cut * 2 * sizeof(float), 256);
        p.bytes = align_up(p.prefix_off + (size_t)(S + 1) * sizeof(int64_t), 256);
        return p;
    }
    p.CB = std::max(1, (int)(((int64_t)max_query_len * G + multi_cols_per_cta() - 1) / multi_cols_per_cta()));
    const double units = (double)S * Hkv * p.CB, slots = (double)sms * 2;
    p.part_tokens = 256;
    double best = -1.0;
    for (int n = 1; n <= (ctx + 255) / 256; ++n) {
        const int cand = std::min(4096, std::max(256, (int)align_up((size_t)((ctx + n - 1) / n), 64)));
        const int parts = (ctx + cand - 1) / cand;
        if (parts != n) continue;
        const double waves = units * parts / slots;
        if (waves < 2.0 && cand != 256) continue;
        const double len = (double)std::min(cand, ctx), score = waves / std::ceil(waves) * len / (len + 512.0);
        if (score > best + 1e-9) {
            best = score;
            p.part_tokens = cand;
        }
    }
    p.max_parts = (ctx + p.part_tokens - 1) / p.part_tokens;
    const size_t rows = (size_t)T * Hq * p.max_parts;
    p.ml_off = align_up(rows * D * sizeof(float), 256);
    p.bytes = align_up(p.ml_off + rows * 2 * sizeof(float), 256);
    return p;
}

pa_status check_tree_args(const char *fn, int S, int T, int Hq, int Hkv, int D, int bs, int kv_dtype,
                          int max_context_len, int max_query_len) {
    const pa_status st = check_decode_shape(fn, S, Hq, Hkv, D, bs, kv_dtype, max_context_len);
    if (st != PA_OK) return st;
    if (T < 0) return fail(PA_ERR_INVALID_ARG, "%s: T = %d", fn, T);
    if (max_query_len < 1 || max_query_len > T || max_query_len > PA_TREE_MAX_NODES)
        return fail(PA_ERR_INVALID_ARG, "%s: max_query_len = %d (1 .. min(T, %d))", fn, max_query_len, PA_TREE_MAX_NODES);
    const int64_t cb = ((int64_t)max_query_len * (Hq / Hkv) + multi_cols_per_cta() - 1) / multi_cols_per_cta();
    if ((int64_t)Hkv * cb > 65535 || (int64_t)Hkv * ((Hq / Hkv + 3) / 4) > 65535)
        return fail(PA_ERR_UNSUPPORTED, "%s: too many rows and heads", fn);
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_tree_workspace_size(int S, int T, int Hq, int Hkv, int D, int bs, int kv_dtype, int max_context_len,
                              int max_query_len) {
    if (check_tree_args("pa_tree_workspace_size", S, T, Hq, Hkv, D, bs, kv_dtype, max_context_len, max_query_len) != PA_OK)
        return 0;
    return plan_tree(S, T, Hq, Hkv, D, kv_dtype, max_context_len, max_query_len).bytes;
}

pa_status pa_tree_attention(pa_bf16 *out, const pa_bf16 *query, const pa_bf16 *key, int64_t key_stride,
                            const pa_bf16 *value, int64_t value_stride, const void *k_cache, const void *v_cache,
                            const float *k_scale, const float *v_scale, int kv_dtype, const int32_t *block_tables,
                            int M, const int32_t *context_lens, const int32_t *query_start, const int32_t *parents,
                            int S, int T, int Hq, int Hkv, int D, int bs, int N, float scale, int max_context_len,
                            int max_query_len, void *workspace, size_t workspace_bytes, int *err_flag,
                            void *stream) {
    const char *fn = "pa_tree_attention";
    clear_error();
    if (S == 0 || T == 0) return PA_OK;
    const pa_status st = check_tree_args(fn, S, T, Hq, Hkv, D, bs, kv_dtype, max_context_len, max_query_len);
    if (st != PA_OK) return st;
    if (N <= 0 || M <= 0) return fail(PA_ERR_INVALID_ARG, "%s: N = %d, M = %d must be positive", fn, N, M);
    if ((int64_t)max_context_len > (int64_t)M * bs)
        return fail(PA_ERR_OUT_OF_RANGE, "%s: max_context_len %d exceeds M * bs = %lld", fn, max_context_len,
                    (long long)M * bs);
    if (!out || !query || !key || !value || !k_cache || !v_cache || !block_tables || !context_lens || !query_start ||
        !parents)
        return fail(PA_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (kv_dtype != PA_KV_BF16 && (!k_scale || !v_scale))
        return fail(PA_ERR_INVALID_ARG, "%s: an int8 or fp8 cache needs k_scale and v_scale", fn);
    if (!aligned16(out) || !aligned16(query) || !aligned16(key) || !aligned16(value) || !aligned16(k_cache) ||
        !aligned16(v_cache) || (kv_dtype != PA_KV_BF16 && (!aligned16(k_scale) || !aligned16(v_scale))))
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    const int64_t kw = (int64_t)Hkv * D;
    constexpr int64_t kMost = (int64_t)1 << 36;
    if (key_stride < kw || value_stride < kw || key_stride % 8 != 0 || value_stride % 8 != 0 || key_stride > kMost ||
        value_stride > kMost)
        return fail(PA_ERR_INVALID_ARG, "%s: row strides must be multiples of 8, at least heads * head_dim", fn);
    if (!(scale == scale) || scale == __builtin_inff() || scale == -__builtin_inff())
        return fail(PA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    const TreePlan plan = plan_tree(S, T, Hq, Hkv, D, kv_dtype, max_context_len, max_query_len);
    if (!workspace || workspace_bytes < plan.bytes)
        return fail(PA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", fn, plan.bytes,
                    workspace ? workspace_bytes : (size_t)0);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(PA_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    char *ws = static_cast<char *>(workspace);
    const int G = Hq / Hkv, g_shift = (G & (G - 1)) == 0 ? __builtin_ctz((unsigned)G) : -1;
    TreeArgs t{};
    t.out = out;
    t.q = query;
    t.k = key;
    t.v = value;
    t.k_stride = key_stride;
    t.v_stride = value_stride;
    t.parents = parents;
    t.query_start = query_start;
    t.context_lens = context_lens;
    t.err_flag = err_flag;
    t.S = S;
    t.T = T;
    t.Hq = Hq;
    t.Hkv = Hkv;
    t.G = G;
    t.max_context_len = max_context_len;
    t.max_query_len = max_query_len;
    t.scale_log2 = scale * 1.4426950408889634f;
    cudaError_t err;
    if (plan.cols > 0) {
        TreeContext c{};
        c.q = query;
        c.k_cache = k_cache;
        c.v_cache = v_cache;
        c.k_scale = k_scale;
        c.v_scale = v_scale;
        c.block_tables = block_tables;
        c.context_lens = context_lens;
        c.query_start = query_start;
        c.whole_acc = (float *)ws;
        c.whole_ml = (float *)(ws + plan.ml_off);
        c.cut_acc = (float *)(ws + plan.cut_off);
        c.cut_ml = (float *)(ws + plan.cut_ml_off);
        c.prefix = (int64_t *)(ws + plan.prefix_off);
        c.err_flag = err_flag;
        c.M = M;
        c.S = S;
        c.T = T;
        c.Hq = Hq;
        c.Hkv = Hkv;
        c.G = G;
        c.N = N;
        c.g_shift = g_shift;
        c.members = plan.members;
        c.groups = plan.groups;
        c.cols = plan.cols;
        c.max_context_len = max_context_len;
        c.max_query_len = max_query_len;
        c.scale_log2 = t.scale_log2;
        err = launch_tree_tc(c, bs, kv_dtype, (cudaStream_t)stream);
        t.tiles = c;
    } else {
        MultiArgs c{};
        c.out = out;
        c.q = query;
        c.k_cache = k_cache;
        c.v_cache = v_cache;
        c.k_scale = k_scale;
        c.v_scale = v_scale;
        c.block_tables = block_tables;
        c.context_lens = context_lens;
        c.query_start = query_start;
        c.ws_acc = (float *)ws;
        c.ws_ml = (float *)(ws + plan.ml_off);
        c.err_flag = err_flag;
        c.M = M;
        c.S = S;
        c.T = T;
        c.Hq = Hq;
        c.Hkv = Hkv;
        c.G = G;
        c.g_shift = g_shift;
        c.N = N;
        c.CB = plan.CB;
        c.part_tokens = plan.part_tokens;
        c.max_parts = plan.max_parts;
        c.max_context_len = max_context_len;
        c.max_query_len = max_query_len;
        c.scale_log2 = t.scale_log2;
        err = launch_multi_context(c, D, bs, kv_dtype, (cudaStream_t)stream);
        t.ws_acc = c.ws_acc;
        t.ws_ml = c.ws_ml;
        t.part_tokens = plan.part_tokens;
        t.max_parts = plan.max_parts;
    }
    if (err != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(err));
    }
    err = D == 128 ? launch_join_heads<128>(t, (cudaStream_t)stream) : launch_join_heads<64>(t, (cudaStream_t)stream);
    if (err != cudaSuccess) {
        cudaGetLastError();
        return fail(PA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(err));
    }
    return check_launch(fn);
}

}  // extern "C"
