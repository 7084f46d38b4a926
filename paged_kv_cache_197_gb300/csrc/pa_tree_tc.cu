// The context's part of tree attention on the fifth-generation tensor cores (head_dim 128).
//
// Every (row, query head) column of a sequence and kv head attends every cached token: one
// softmax over the context without a mask, S = Q K^T, P = 2^(S - m), O = P V, with the
// running maximum m and sum l of each column in registers and O in tensor memory.
//
// One CTA per SM (224 KB of shared memory, all 512 tensor-memory columns) works through its
// share of all tiles of the batch (pa_tree.cuh): 128 tokens of K and V at a time, staged by
// TMA into a ring of five 32 KB stages that runs on across units.  Ten warps with fixed
// roles, coupled by mbarriers:
//   * warps 0-3 and 4-7 are two lanes of 128 columns, a thread per column.  With more than
//     128 columns the lanes take the two halves of 256 columns and share every staged
//     tile; with at most 128 they take the same columns and alternate tiles, and are
//     joined at the end of a unit.  Either way one lane's exponentials run while the
//     tensor cores work for the other;
//   * warp 8 copies K and V tiles; warp 9 issues the products.
// Tensor memory: S of the lanes at columns 0 and 128 (overwritten by P as bf16 pairs, the A
// operand of P V), O at 256 and 384.
// Bounds: up to 128 columns, or 256 shared ones, the 64 KB of a K and V tile take 2800 SM
// clocks at the measured HBM rate and the products 1024 / 2048, so HBM bounds; more columns
// reread the tiles through L2 and the products bound.
// Every wait is bounded; a wait that gives up stops the CTA (PA_FLAG_TIMEOUT).
#include <math.h>

#include <atomic>

#include "pa_stages.h"
#include "pa_tc.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

using namespace tc;

constexpr int kTile = kTreeTile;
constexpr int kD = 128;
constexpr int kLaneCols = 128;
constexpr int kTileBytes = kTile * kD * 2;   // 32 KB: two 64-dim halves of 128 rows of 128 B
constexpr int kHalf = kTile * 128;
constexpr int kStages = 5;
constexpr int kOffQ = 0, kOffRing = 2 * kTileBytes, kOffShared = kOffRing + kStages * kTileBytes;
constexpr int kThreads = 320;
constexpr uint32_t kTmemS = 0, kTmemO = 256;  // + 128 per lane
constexpr float kRescaleLog2 = 8.0f;

struct Shared {
    float2 ml[2][kLaneCols];                    // lanes joined: each one's (max, sum) per column
    uint64_t full[kStages], free[kStages];      // ring stages: landed / consumed
    uint64_t sfull[2], pfull[2], odone[2];      // per lane: S written, P written, P V done
    uint64_t qfull[2];                          // per lane: the unit's queries are staged
    uint64_t mlready, oread;                    // lanes joined: both (max, sum) and O in / read
    uint64_t drain;
    int64_t total, first_tile;                  // of all tiles; of the first sequence
    int first_seq;
    int wsum[kThreads / 32];
    uint32_t taddr;
    int abort;
};
constexpr int kSmem = kOffShared + (int)sizeof(Shared);
static_assert(kSmem <= 232448, "shared memory of one CTA per SM");

__device__ __forceinline__ void raise_flag(int *err_flag, int bit) {
    if (err_flag) atomicOr(err_flag, bit);
}

// A bounded wait that also ends when another role gave up.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, int *abort) {
    const uint32_t b = tc_smem(bar);
    unsigned long long t0 = 0;
    for (int it = 0;; ++it) {
        uint32_t done;
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(b), "r"(parity)
            : "memory");
        if (done) return true;
        if (*(volatile int *)abort) return false;
        if (it == 0)
            t0 = tc_now();
        else if (tc_now() - t0 > kTcWaitNs) {
            atomicOr(abort, 1);
            return false;
        }
    }
}

// Byte offset of the 16-byte chunk ch of row r in a 128-row tile with the 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_chunk(int r, int ch) {
    return (ch >> 3) * kHalf + (r >> 3) * 1024 + (r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// The next range of tiles of one (sequence, kv head) in a CTA's share.
struct Walk {
    int64_t pos, end, before;  // tiles: here, end of the share, before sequence s
    int s, tiles;              // sequence and its tiles per kv head (-1: not read yet)
    int kvh, t0, n, ctx, r0, ncols;

    __device__ __forceinline__ bool next(const TreeContext &a) {
        if (pos >= end) return false;
        for (;;) {
            if (tiles < 0) {
                const int r1 = a.query_start[s + 1];
                r0 = a.query_start[s];
                ctx = min(max(a.context_lens[s], 0), a.max_context_len);  // at most M * bs
                const int L = r1 - r0;
                ncols = L * a.G;
                tiles = r0 >= 0 && r1 <= a.T && L >= 1 && L <= a.max_query_len ? (ctx + kTile - 1) / kTile : 0;
            }
            if (pos < before + (int64_t)tiles * a.Hkv) break;
            before += (int64_t)tiles * a.Hkv;
            ++s;
            tiles = -1;
        }
        const int64_t in = pos - before;
        kvh = (int)(in / tiles);
        t0 = (int)(in % tiles);
        n = (int)min((int64_t)(tiles - t0), end - pos);
        pos += n;
        return true;
    }
};

template <int BS, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const __grid_constant__ TreeContext a, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) unsigned char smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem + kOffShared);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((tc_smem(smem) & 1023) != 0) {  // the swizzled tiles need their alignment
        if (tid == 0) raise_flag(a.err_flag, PA_FLAG_TIMEOUT);
        return;
    }
    const int group = blockIdx.x / a.members, member = blockIdx.x % a.members;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(tc_smem(&sh.full[i]));
            mbar_init(tc_smem(&sh.free[i]));
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(tc_smem(&sh.sfull[w]));
            mbar_init(tc_smem(&sh.odone[w]));
            mbar_init_n(tc_smem(&sh.pfull[w]), kLaneCols);
            mbar_init_n(tc_smem(&sh.qfull[w]), kLaneCols);
        }
        mbar_init_n(tc_smem(&sh.mlready), 2 * kLaneCols);
        mbar_init_n(tc_smem(&sh.oread), 2 * kLaneCols);
        mbar_init(tc_smem(&sh.drain));
        sh.abort = 0;
        sh.first_seq = 0;
        sh.first_tile = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc_smem(&sh.taddr))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the batch's tiles: their number, then the sequence this share begins in
    auto tiles_of = [&](int s, bool report) -> int {
        const int lim = a.max_context_len;
        const int ctx = a.context_lens[s], r0 = a.query_start[s], r1 = a.query_start[s + 1], L = r1 - r0;
        const bool ok = r0 >= 0 && r1 <= a.T && L >= 0 && L <= a.max_query_len;
        if (report && (ctx < 0 || ctx > lim)) raise_flag(a.err_flag, PA_FLAG_CONTEXT_OUT_OF_RANGE);
        if (report && !ok) raise_flag(a.err_flag, PA_FLAG_QUERY_OUT_OF_RANGE);
        return ok && L > 0 ? (min(max(ctx, 0), lim) + kTile - 1) / kTile : 0;
    };
    int64_t sum = 0;
    for (int s = tid; s < a.S; s += kThreads) sum += tiles_of(s, blockIdx.x == 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (tid == 0) sh.total = 0;
    __syncthreads();
    if (lane == 0 && sum) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.total), (unsigned long long)sum);
    __syncthreads();
    const int64_t total = sh.total * a.Hkv;
    const int64_t groups = min((int64_t)a.groups, total);  // no share is empty: a cut unit's are consecutive
    const int64_t begin = group < groups ? group * total / groups : total;
    const int64_t end = group < groups ? (group + 1) * total / groups : total;
    int64_t carry = 0;
    for (int base = 0; base < a.S; base += kThreads) {
        const int s = base + tid, n = s < a.S ? tiles_of(s, false) : 0;
        int v = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        if (lane == 31) sh.wsum[warp] = v;
        __syncthreads();
        int64_t mine = carry + v - n;
        for (int w = 0; w < kThreads / 32; ++w) {
            mine += w < warp ? sh.wsum[w] : 0;
            carry += sh.wsum[w];
        }
        const int64_t first = mine * a.Hkv;
        if (s < a.S && blockIdx.x == 0) a.prefix[s] = first;
        if (s < a.S && begin >= first && begin < first + (int64_t)n * a.Hkv) {
            sh.first_seq = s;
            sh.first_tile = first;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) a.prefix[a.S] = total;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.taddr;
    Walk w{begin, end, sh.first_tile, sh.first_seq, -1};
    int *abort = &sh.abort;

    // lane 1 has work: its half of the columns, or (lanes on the same columns) a second tile
    auto second = [&](const Walk &u) { return SPLIT ? u.n > 1 : u.ncols - member * a.cols > kLaneCols; };
    // the member has columns of this sequence at all
    auto mine = [&](const Walk &u) { return u.ncols > member * a.cols; };
    // Ring positions of tile t's K and V within a unit of n tiles, in the order they are used:
    // K0 V0 K1 V1 .. (shared tiles), K0 K1 V0 K2 V1 .. (alternating lanes).
    auto k_at = [&](int t, int n) { return SPLIT ? (t == 0 ? 0 : 2 * t - 1) : 2 * t; };
    auto v_at = [&](int t, int n) { return SPLIT ? (t < n - 1 ? 2 * t + 2 : 2 * n - 1) : 2 * t + 1; };

    if (warp == 8) {
        // ---- copies
        const int oob_row = a.N * a.Hkv * BS;  // a row past the pool: the copy fills zeros
        constexpr int kBoxes = kTile / BS * 2;  // two 64-dim boxes per block
        int issued = 0;
        bool ok = true;
        while (ok && w.next(a)) {
            if (!mine(w)) continue;
            const int nblk = (w.ctx + BS - 1) / BS;
            auto fill = [&](bool is_k, int t) {
                const int st = issued % kStages, use = issued / kStages;
                int y = oob_row;
                const int idx = (w.t0 + t) * (kTile / BS) + lane / 2;
                if (lane < kBoxes && idx < nblk) {
                    const int b = __ldg(a.block_tables + (int64_t)w.s * a.M + idx);
                    if (b >= 0 && b < a.N)
                        y = (b * a.Hkv + w.kvh) * BS;
                    else if (is_k && member == 0)
                        raise_flag(a.err_flag, PA_FLAG_BLOCK_OUT_OF_RANGE);
                }
                if (use > 0) ok = wait_for(&sh.free[st], (use - 1) & 1, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                const uint32_t bar = tc_smem(&sh.full[st]);
                if (lane == 0) mbar_expect(bar, kTileBytes);
                __syncwarp();
                if (lane < kBoxes)
                    tma_load(tc_smem(smem + kOffRing + st * kTileBytes) + (lane & 1) * kHalf + (lane / 2) * BS * 128,
                             is_k ? &kmap : &vmap, (lane & 1) * 64, y, bar);
                __syncwarp();
                ++issued;
            };
            fill(true, 0);
            for (int t = 0; ok && t < w.n; ++t) {
                if (SPLIT && t + 1 < w.n) fill(true, t + 1);
                if (ok) fill(false, t);
                if (!SPLIT && ok && t + 1 < w.n) fill(true, t + 1);
            }
        }
        if (!ok) {
            // stopping early: copies already issued may still be landing in shared memory
            for (int st = 0; st < kStages; ++st) {
                const StageFill f = last_fill(issued, kStages, st);
                if (f.any) mbar_wait(tc_smem(&sh.full[st]), f.parity);
            }
        }
    } else if (warp == 9) {
        // ---- products: the whole warp waits, lane 0 issues
        int ring = 0, pv[2] = {0, 0}, qs[2] = {0, 0};
        bool ok = true;
        auto stage_addr = [&](int at) { return tc_smem(smem + kOffRing + ((ring + at) % kStages) * kTileBytes); };
        auto landed = [&](int at) { return wait_for(&sh.full[(ring + at) % kStages], ((ring + at) / kStages) & 1, abort); };
        while (ok && w.next(a)) {
            if (!mine(w)) continue;
            const bool two = second(w);
            // S of lane l, tile t; `last`: no other lane uses this K after it
            auto scores = [&](int l, int t, bool first, bool last) {
                const int at = k_at(t, w.n);
                if (first) ok = wait_for(&sh.qfull[l], qs[l]++ & 1, abort);
                // S overwrites P: the lane's last P V is done (this also orders O for its rows)
                if (ok && pv[l] > 0) ok = wait_for(&sh.odone[l], (pv[l] - 1) & 1, abort);
                if (ok) ok = landed(at);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t qb = tc_smem(smem + kOffQ + l * kTileBytes), kb = stage_addr(at);
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                        umma(tmem + kTmemS + l * 128, sw128_desc(qb + off, 16, 1024), sw128_desc(kb + off, 16, 1024),
                             bf16_idesc(128, kTile, 0), kk > 0);
                    }
                    umma_commit(tc_smem(&sh.sfull[l]));
                    if (last) umma_commit(tc_smem(&sh.free[(ring + at) % kStages]));
                }
                __syncwarp();
            };
            auto weighted = [&](int l, int t, bool first, bool last) {
                const int at = v_at(t, w.n);
                ok = wait_for(&sh.pfull[l], pv[l] & 1, abort);
                if (ok) ok = landed(at);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t vb = stage_addr(at);
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        umma_ts(tmem + kTmemO + l * 128, tmem + kTmemS + l * 128 + kk * 8,
                                sw128_desc(vb + kk * 2048, kHalf, 1024), bf16_idesc(128, kD, 1), !first || kk > 0);
                    umma_commit(tc_smem(&sh.odone[l]));
                    if (last) umma_commit(tc_smem(&sh.free[(ring + at) % kStages]));
                }
                __syncwarp();
                ++pv[l];
            };
            if constexpr (SPLIT) {
                scores(0, 0, true, true);
                if (ok && two) scores(1, 1, true, true);
                for (int t = 0; ok && t < w.n; ++t) {
                    weighted(t & 1, t, t < 2, true);
                    if (ok && t + 2 < w.n) scores(t & 1, t + 2, false, true);
                }
            } else {
                scores(0, 0, true, !two);
                if (ok && two) scores(1, 0, true, true);
                for (int t = 0; ok && t < w.n; ++t) {
                    weighted(0, t, t == 0, !two);
                    if (ok && t + 1 < w.n) scores(0, t + 1, false, !two);
                    if (ok && two) weighted(1, t, t == 0, true);
                    if (ok && two && t + 1 < w.n) scores(1, t + 1, false, true);
                }
            }
            ring += 2 * w.n;
        }
        if (!ok) {
            // stopping early: every product already issued finishes before tensor memory is released
            if (lane == 0) umma_commit(tc_smem(&sh.drain));
            __syncwarp();
            mbar_wait(tc_smem(&sh.drain), 0);
        }
    } else {
        // ---- a lane's columns: thread = column = tensor-memory lane
        const int l = warp >> 2, row = tid & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_off + kTmemS + l * 128, t_o = tmem + lane_off + kTmemO + l * 128;
        unsigned char *qbuf = smem + kOffQ + l * kTileBytes;
        int done = 0, ring = 0, joins = 0;  // tiles of this lane; ring position; units joined
        bool ok = true;
        while (ok && w.next(a)) {
            if (!mine(w)) continue;
            const bool two = second(w);
            const bool active = l == 0 || two;
            if (!SPLIT && !active) {
                ring += 2 * w.n;
                continue;
            }
            const int c = member * a.cols + (SPLIT ? 0 : l * kLaneCols) + row;
            const bool col = c < w.ncols;
            const int tok = a.g_shift >= 0 ? c >> a.g_shift : c / a.G, head = c - tok * a.G;
            const int64_t pair = (int64_t)(w.r0 + tok) * a.Hq + w.kvh * a.G + head;
            float m = -INFINITY, sum_l = 0.f;
            if (active) {
                // the unit's queries (this lane's products with the last unit's are done)
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + pair * kD);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (col) x = __ldg(src + i);
                    *reinterpret_cast<uint4 *>(qbuf + tile_chunk(row, i)) = x;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(tc_smem(&sh.qfull[l]));
            }
            // a warp none of whose columns is real keeps step without computing
            const bool idle = member * a.cols + (SPLIT ? 0 : l * kLaneCols) + (warp & 3) * 32 >= w.ncols;
            for (int t = SPLIT ? l : 0; t < w.n; t += SPLIT ? 2 : 1) {
                ok = wait_for(&sh.sfull[l], done & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                const int k0 = (w.t0 + t) * kTile;
                if (!idle) {
                    float sv[kTile];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(t_s + 32 * q, sv + 32 * q);
                    tmem_wait_ld();
                    if (k0 + kTile > w.ctx) {
#pragma unroll
                        for (int k = 0; k < kTile; ++k)
                            if (k0 + k >= w.ctx) sv[k] = -INFINITY;
                    }
                    float mx[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) mx[i] = sv[i];
#pragma unroll
                    for (int k = 8; k < kTile; ++k) mx[k & 7] = fmaxf(mx[k & 7], sv[k]);
                    const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                            fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) *
                                      a.scale_log2;
                    // the running maximum is raised only by more than 2^8; then l and O shrink
                    float f = 1.f;
                    bool shrink = false;
                    if (top > m + kRescaleLog2) {
                        if (m != -INFINITY) {
                            f = tc_exp2(m - top);
                            sum_l *= f;
                            shrink = true;
                        }
                        m = top;
                    }
                    if (__any_sync(0xffffffffu, shrink)) {
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            float ov[32];
                            tmem_ld32(t_o + 32 * q, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) ov[i] *= f;
                            tmem_st32(t_o + 32 * q, ov);
                        }
                    }
                    const float base = m == -INFINITY ? 0.f : m;
                    float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float pw[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int k = 64 * q + 2 * i;
                            const float p0 = tc_exp2(fmaf(sv[k], a.scale_log2, -base));
                            const float p1 = tc_exp2(fmaf(sv[k + 1], a.scale_log2, -base));
                            ls[i & 3] += p0 + p1;
                            pw[i] = __uint_as_float(tc_bf16x2(p0, p1));
                        }
                        tmem_st32(t_s + 32 * q, pw);
                    }
                    sum_l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                    tmem_wait_st();
                }
                // rows past the context inside its last block may hold anything, and a zero
                // weight times a NaN is a NaN: zero them in the V stage
                if (k0 + kTile > w.ctx && w.ctx % BS != 0 && (SPLIT || l == 0)) {
                    const int at = ring + v_at(t, w.n), st = at % kStages;
                    ok = wait_for(&sh.full[st], (at / kStages) & 1, abort);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const int lo = w.ctx - k0, hi = min(kTile, (w.ctx + BS - 1) / BS * BS - k0);
                    unsigned char *vst = smem + kOffRing + st * kTileBytes;
                    for (int i = row; i < (hi - lo) * 16; i += kLaneCols)
                        *reinterpret_cast<uint4 *>(vst + tile_chunk(lo + i / 16, i % 16)) = make_uint4(0u, 0u, 0u, 0u);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                tc_fence_before();
                mbar_arrive(tc_smem(&sh.pfull[l]));
                ++done;
            }
            ring += 2 * w.n;
            if (!ok) break;
            // ---- the columns' partials
            const bool all = w.t0 == 0 && w.n == w.tiles;
            const int64_t at = all ? pair : ((int64_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * a.cols + (c - member * a.cols);
            float *acc = (all ? a.whole_acc : a.cut_acc) + at * kD;
            float2 *ml = reinterpret_cast<float2 *>(all ? a.whole_ml : a.cut_ml) + at;
            if (active) ok = wait_for(&sh.odone[l], (done - 1) & 1, abort);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            if constexpr (!SPLIT) {
#pragma unroll 1
                for (int q = 0; q < 4 && !idle; ++q) {
                    float ov[32];
                    tmem_ld32(t_o + 32 * q, ov);
                    tmem_wait_ld();
                    if (!col) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<float4 *>(acc)[8 * q + i] =
                            make_float4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
                }
                if (col) *ml = make_float2(m, sum_l);
            } else {
                // both lanes hold a part of the same columns: each joins half of the dims
                sh.ml[l][row] = make_float2(m, sum_l);
                tc_fence_before();
                mbar_arrive(tc_smem(&sh.mlready));
                ok = wait_for(&sh.mlready, joins & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                const float2 x = sh.ml[0][row], y = sh.ml[1][row];
                const float top = fmaxf(x.x, y.x), base = top == -INFINITY ? 0.f : top;
                const float fx = tc_exp2(x.x - base), fy = tc_exp2(y.x - base);
#pragma unroll 1
                for (int q = 2 * l; q < 2 * l + 2 && !idle; ++q) {
                    float ov[32];
                    tmem_ld32(tmem + lane_off + kTmemO + 32 * q, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) ov[i] *= fx;
                    if (two) {
                        float other[32];
                        tmem_ld32(tmem + lane_off + kTmemO + 128 + 32 * q, other);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] = fmaf(other[i], fy, ov[i]);
                    }
                    if (!col) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<float4 *>(acc)[8 * q + i] =
                            make_float4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
                }
                if (col && l == 0) *ml = make_float2(top, x.y * fx + y.y * fy);
                // O may be overwritten, and ml, once both lanes have read them
                tc_fence_before();
                mbar_arrive(tc_smem(&sh.oread));
                ok = wait_for(&sh.oread, joins & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                ++joins;
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sh.abort) raise_flag(a.err_flag, PA_FLAG_TIMEOUT);
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// A cache pool [N][Hkv][bs][128] bf16 as rows of 128 values, copied in boxes of 64 values x
// bs rows with the 128-byte swizzle.
bool pool_map(CUtensorMap *map, const void *pool, int rows, int bs) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)kD * 2};
    const cuuint32_t box[2] = {64u, (cuuint32_t)bs};
    const cuuint32_t estr[2] = {1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BS, bool SPLIT>
cudaError_t launch_typed(const TreeContext &a, cudaStream_t stream) {
    CUtensorMap kmap, vmap;
    if ((int64_t)a.N * a.Hkv * BS >= (int64_t)INT32_MAX) return cudaErrorInvalidValue;  // TMA row coordinates
    const int rows = a.N * a.Hkv * BS;
    if (!pool_map(&kmap, a.k_cache, rows, BS) || !pool_map(&vmap, a.v_cache, rows, BS)) return cudaErrorInvalidValue;
    static std::atomic<bool> configured[64];  // per device: the shared-memory attribute is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(tree_tc_kernel<BS, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    return launch_dependent(tree_tc_kernel<BS, SPLIT>, dim3(a.groups * a.members), dim3(kThreads), kSmem, stream, a, kmap,
                            vmap);
}

}  // namespace

bool tree_tc_eligible(int D, int kv_dtype) { return D == kD && kv_dtype == PA_KV_BF16; }

cudaError_t launch_tree_tc(const TreeContext &a, int bs, int kv_dtype, cudaStream_t stream) {
    if (kv_dtype != PA_KV_BF16) return cudaErrorInvalidValue;
    if (a.cols == kLaneCols) return bs == 16 ? launch_typed<16, true>(a, stream) : launch_typed<32, true>(a, stream);
    return bs == 16 ? launch_typed<16, false>(a, stream) : launch_typed<32, false>(a, stream);
}

}  // namespace pa
