// The context's part of tree attention on the fifth-generation tensor cores (head_dim 128).
//
// Every (row, query head) column of a sequence and kv head attends every cached token: one
// softmax over the context without a mask, S = Q K^T, P = 2^(S - m), O = P V, with the
// running maximum m and sum l of each column in registers and O in tensor memory.
//
// One CTA per SM (224 KB of shared memory, all 512 tensor-memory columns) works through its
// share of all tiles of the batch (pa_tree.cuh): 128 tokens of K and V at a time, staged by
// TMA into a ring of five 32 KB stages that runs on across units.  Warps with fixed roles,
// coupled by mbarriers:
//   * warps 0-3 and 4-7 are two lanes of 128 columns, a thread per column.  With more than
//     128 columns the lanes take the two halves of 256 columns and share every staged
//     tile; with at most 128 they take the same columns and alternate tiles, and are
//     joined at the end of a unit.  Either way one lane's exponentials run while the
//     tensor cores work for the other;
//   * warp 8 copies K and V tiles; one thread each of warps 9 and 10 issues a lane's products.
//     (Warp 11 fills the warpgroup, whose spare registers go to the columns.)
// Tensor memory: S of the lanes at columns 0 and 128 (overwritten by P as bf16 pairs, the A
// operand of P V), O at 256 and 384.
// Bounds: up to 128 columns, or 256 shared ones, the 64 KB of a K and V tile take 2800 SM
// clocks at the measured HBM rate and the products 1024 / 2048, so HBM bounds; more columns
// reread the tiles through L2 and the products bound.
// Every wait is bounded; a wait that gives up stops the CTA (PA_FLAG_TIMEOUT).
#include <math.h>

#include <atomic>

#include "pa_tc.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

using namespace tc;

constexpr int kTile = kTreeTile;
constexpr int kD = 128;
constexpr int kLaneCols = 128;
constexpr int kTileBytes = kTile * kD * 2;   // 32 KB
// A staged tile: groups of 8 rows, each as two 64-dim halves of 8 x 128 B (one swizzle atom
// each).  A cache block is then one copy of bs x 256 contiguous bytes, and the atoms of a
// half lie a constant 2 KB apart, as the matrix descriptors need.
constexpr int kHalf = 1024, kGroup = 2048;
constexpr int kStages = 5;
// Ring position p lands in stage p % kStages and completes barrier p % kFull.  With
// alternating lanes a lane sees only its own positions, up to three apart, and copies land
// in any order, so a stage's own barrier could still be at the other lane's copy of
// position p - 5 when position p is asked for, and that phase has the parity of p's
// predecessor's predecessor.  With two barriers a stage the predecessor is p - 10, and a
// copy past p - 5 is only issued once p - 10 was consumed.
constexpr int kFull = 2 * kStages;
constexpr int kOffQ = 0, kOffRing = 2 * kTileBytes, kOffShared = kOffRing + kStages * kTileBytes;
constexpr int kThreads = 384;  // three warpgroups: two lanes of columns; copies and products
constexpr int kRegsColumns = 192, kRegsOther = 120;  // 2 x 128 x 192 + 128 x 120 = 384 x 168 at launch
constexpr uint32_t kTmemS = 0, kTmemO = 256;  // + 128 per lane
constexpr float kRescaleLog2 = 8.0f;

struct Shared {
    float2 ml[2][kLaneCols];                    // lanes joined: each one's (max, sum) per column
    uint64_t full[kFull], free[kStages];        // ring positions landed / stages consumed
    uint64_t sfull[2], pfull[2], odone[2];      // per lane: S written, P written, P V done
    uint64_t qfull[2];                          // per lane: the unit's queries are staged
    uint64_t mlready, oread;                    // lanes joined: both (max, sum) and O in / read
    uint64_t turn[2];                           // shared tiles: the lane may issue its next products
    uint64_t drain[2];
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

// Byte offset of the 16-byte chunk ch of row r in a tile (128-byte swizzle).
__device__ __forceinline__ uint32_t tile_chunk(int r, int ch) {
    return (r >> 3) * kGroup + (ch >> 3) * kHalf + (r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// One block of a pool, [bs / 8][2][8][64] in the order of a staged tile.
__device__ __forceinline__ void tma_block(uint32_t dst, const CUtensorMap *map, int group, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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
        for (int i = 0; i < kFull; ++i) mbar_init(tc_smem(&sh.full[i]));
        for (int i = 0; i < kStages; ++i) {
            mbar_init_n(tc_smem(&sh.free[i]), SPLIT ? 1 : 2);  // lanes that read a stage
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(tc_smem(&sh.sfull[w]));
            mbar_init(tc_smem(&sh.odone[w]));
            mbar_init_n(tc_smem(&sh.pfull[w]), kLaneCols);
            mbar_init_n(tc_smem(&sh.qfull[w]), kLaneCols);
        }
        mbar_init_n(tc_smem(&sh.mlready), 2 * kLaneCols);
        mbar_init_n(tc_smem(&sh.oread), 2 * kLaneCols);
        mbar_init(tc_smem(&sh.turn[0]));
        mbar_init(tc_smem(&sh.turn[1]));
        mbar_init(tc_smem(&sh.drain[0]));
        mbar_init(tc_smem(&sh.drain[1]));
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
    const int n_first = tid < a.S ? tiles_of(tid, blockIdx.x == 0) : 0;
    int64_t sum = n_first;
    for (int s = tid + kThreads; s < a.S; s += kThreads) sum += tiles_of(s, blockIdx.x == 0);
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
        const int s = base + tid, n = base == 0 ? n_first : s < a.S ? tiles_of(s, false) : 0;
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
    auto k_at = [](int t, int n) { return SPLIT ? (t == 0 ? 0 : 2 * t - 1) : 2 * t; };
    auto v_at = [](int t, int n) { return SPLIT ? (t < n - 1 ? 2 * t + 2 : 2 * n - 1) : 2 * t + 1; };

    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
        // ---- copies: lane i takes block i of a tile
        constexpr int kBlocks = kTile / BS, kGroups = BS / 8;  // 8-row groups of a block and kv head
        const int oob = a.N * a.Hkv * kGroups;  // past the pool: the copy fills zeros
        const uint32_t box = tc_smem(smem + kOffRing) + lane * BS * 256;
        int st = 0;
        uint32_t phase = 0;   // of the stage's next wait for `free`
        int issued = 0;
        bool ok = true, first = true;
        auto fill = [&](const CUtensorMap *map, int y) {
            if (issued >= kStages) ok = wait_for(&sh.free[st], phase ^ 1, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            const uint32_t bar = tc_smem(&sh.full[issued % kFull]);
            if (lane == 0) mbar_expect(bar, kTileBytes);
            __syncwarp();
            if (lane < kBlocks) tma_block(box + st * kTileBytes, map, y, bar);
            ++issued;
            if (++st == kStages) {
                st = 0;
                phase ^= 1;
            }
        };
        while (ok && w.next(a)) {
            if (!mine(w)) continue;
            const int nblk = (w.ctx + BS - 1) / BS;
            const int32_t *table = a.block_tables + (int64_t)w.s * a.M;
            // the raw table entry of this lane's block of tile t; -2 for blocks past the context
            auto entry = [&](int t) {
                const int idx = (w.t0 + t) * kBlocks + lane;
                return t < w.n && lane < kBlocks && idx < nblk ? __ldg(table + idx) : -2;
            };
            auto row_of = [&](int t, int b) {
                if (b >= 0 && b < a.N) return (b * a.Hkv + w.kvh) * kGroups;
                const int idx = (w.t0 + t) * kBlocks + lane;
                if (t < w.n && lane < kBlocks && idx < nblk && member == 0) raise_flag(a.err_flag, PA_FLAG_BLOCK_OUT_OF_RANGE);
                return oob;
            };
            // With the ring's copies of all SMs queued up, a load that misses L2 takes several
            // microseconds: the unit's table entries are fetched into L2 at its start (32 to a
            // line) and loaded two tiles ahead of their copies, and the first unit's queries
            // go before all copies but one.
            for (int i = lane * 32; i < w.n * kBlocks; i += 32 * 32) prefetch_l2(table + min(w.t0 * kBlocks + i, nblk - 1));
            int y = row_of(0, entry(0)), e1 = entry(1), e2 = entry(2);
            fill(&kmap, y);
            if (first) {
                first = false;
                ok = wait_for(&sh.qfull[0], 0, abort);
                if (second(w) && ok) ok = wait_for(&sh.qfull[1], 0, abort);
                ok = __all_sync(0xffffffffu, ok);
            }
            for (int t = 0; ok && t < w.n; ++t) {
                const int yn = row_of(t + 1, e1);
                e1 = e2;
                e2 = entry(t + 3);
                if (SPLIT && t + 1 < w.n) fill(&kmap, yn);
                if (ok) fill(&vmap, y);
                if (!SPLIT && ok && t + 1 < w.n) fill(&kmap, yn);
                y = yn;
            }
        }
        if (!ok) {
            // stopping early: copies already issued may still be landing in shared memory
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait(tc_smem(&sh.full[i % kFull]), (i / kFull) & 1);
        }
    } else if (warp < 11) {
        // ---- products of lane l: one thread waits and issues (a thread per lane, so that one
        // lane's waits do not hold up the other's products)
        if (lane == 0) {
            const int l = warp - 9;
            int ring = 0;
            uint32_t pv = 0, qs = 0, taken = 0;
            bool ok = true;
            const uint32_t t_s = tmem + kTmemS + l * 128, t_o = tmem + kTmemO + l * 128;
            const uint64_t qd = sw128_desc(tc_smem(smem + kOffQ + l * kTileBytes), 16, kGroup);
            const uint64_t kd = sw128_desc(tc_smem(smem + kOffRing), 16, kGroup);
            const uint64_t vd = sw128_desc(tc_smem(smem + kOffRing), kHalf, kGroup);
            const uint32_t sfull = tc_smem(&sh.sfull[l]), odone = tc_smem(&sh.odone[l]);
            while (ok && w.next(a)) {
                if (!mine(w)) continue;
                if (l == 1 && !second(w)) {
                    // the other lane reads these tiles alone
                    if constexpr (!SPLIT)
                        for (int at = ring; ok && at < ring + 2 * w.n; ++at) {
                            ok = wait_for(&sh.full[at % kFull], (at / kFull) & 1, abort);
                            if (ok) mbar_arrive(tc_smem(&sh.free[at % kStages]));
                        }
                    ring += 2 * w.n;
                    continue;
                }
                auto landed = [&](int at) { return wait_for(&sh.full[at % kFull], (at / kFull) & 1, abort); };
                auto scores = [&](int at) {
                    tc_fence_after();
                    const uint64_t k0 = kd + (uint64_t)(at % kStages * (kTileBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk) {
                        const uint64_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        umma(t_s, qd + off, k0 + off, bf16_idesc(128, kTile, 0), kk > 0);
                    }
                    umma_commit(sfull);
                };
                auto weighted = [&](int at, bool first) {
                    tc_fence_after();
                    const uint64_t v0 = vd + (uint64_t)(at % kStages * (kTileBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        umma_ts(t_o, t_s + kk * 8, v0 + (kk * 2 * kGroup >> 4), bf16_idesc(128, kD, 1), !first || kk > 0);
                    umma_commit(odone);
                    ++pv;
                };
                constexpr int kStep = SPLIT ? 2 : 1;
                const int t_first = SPLIT ? l : 0;
                // Lanes that share their tiles take turns at the tensor cores, P V and the next
                // S at a time: left alone they fall into step, both computing exponentials and
                // then both waiting for products.  What a turn needs is waited for before it.
                const bool turns = !SPLIT && second(w);
                int k_pos = ring + k_at(t_first, w.n);
                // (the queries first: their lane has seen every earlier unit's end)
                ok = wait_for(&sh.qfull[l], qs++ & 1, abort) && landed(k_pos);
                if (ok) {
                    scores(k_pos);
                    umma_commit(tc_smem(&sh.free[k_pos % kStages]));
                }
                for (int t = t_first; ok && t < w.n; t += kStep) {
                    const bool more = t + kStep < w.n;
                    const int v_pos = ring + v_at(t, w.n);
                    k_pos = ring + k_at(t + kStep, w.n);
                    ok = landed(v_pos) && (SPLIT || !more || landed(k_pos)) && wait_for(&sh.pfull[l], pv & 1, abort);
                    if (ok && turns && (l == 1 || taken > 0)) ok = wait_for(&sh.turn[l], (l == 1 ? taken : taken - 1) & 1, abort);
                    if (!ok) break;
                    weighted(v_pos, t == t_first);
                    // S overwrites P: P V is done first (this also orders O for its rows)
                    if (more) {
                        ok = wait_for(&sh.odone[l], (pv - 1) & 1, abort) && (!SPLIT || landed(k_pos));
                        if (!ok) break;
                        scores(k_pos);
                    }
                    if (turns) {
                        mbar_arrive(tc_smem(&sh.turn[l ^ 1]));
                        ++taken;
                    }
                    umma_commit(tc_smem(&sh.free[v_pos % kStages]));
                    if (more) umma_commit(tc_smem(&sh.free[k_pos % kStages]));
                }
                ring += 2 * w.n;
            }
            if (!ok) {
                // stopping early: every product already issued finishes before tensor memory is released
                umma_commit(tc_smem(&sh.drain[l]));
                mbar_wait(tc_smem(&sh.drain[l]), 0);
            }
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsColumns));
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
                // the unit's queries (this lane's products with the last unit's are done): a
                // row at a time by half a warp
                uint4 x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = 2 * i + (lane >> 4);
                    const int64_t from = __shfl_sync(0xffffffffu, col ? pair : -1, r);
                    x[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (from >= 0) x[i] = __ldg(reinterpret_cast<const uint4 *>(a.q + from * kD) + (lane & 15));
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    *reinterpret_cast<uint4 *>(qbuf + tile_chunk((warp & 3) * 32 + 2 * i + (lane >> 4), lane & 15)) = x[i];
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(tc_smem(&sh.qfull[l]));
            }
            // the next unit's queries into L2, long before they are loaded
            {
                Walk u = w;
                if (u.next(a) && mine(u) && (SPLIT || l == 0 || second(u)) && c < u.ncols) {
                    const uint16_t *src = a.q + ((int64_t)(u.r0 + tok) * a.Hq + u.kvh * a.G + head) * kD;
                    prefetch_l2(src);
                    prefetch_l2(src + 64);
                }
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
                if (k0 + kTile > w.ctx && w.ctx % BS != 0) {
                    const int at = ring + v_at(t, w.n), st = at % kStages;
                    ok = wait_for(&sh.full[at % kFull], (at / kFull) & 1, abort);
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
            // ---- the columns' partials, 32 dims at a time through the query buffer (the unit's
            // products with it are done): rows by threads in, 128-byte pieces of rows out
            const bool all = w.t0 == 0 && w.n == w.tiles;
            const int64_t at = all ? pair : ((int64_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * a.cols + (c - member * a.cols);
            float *acc = all ? a.whole_acc : a.cut_acc;
            float2 *ml = reinterpret_cast<float2 *>(all ? a.whole_ml : a.cut_ml) + at;
            constexpr int kPitch = 144;  // of a staged row of 128 bytes: no bank conflicts
            unsigned char *stage = qbuf + (warp & 3) * 32 * kPitch;
            auto put = [&](const float (&ov)[32], int q) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4 *>(stage + lane * kPitch + i * 16) =
                        make_float4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 4 * i + (lane >> 3);
                    const int64_t to = __shfl_sync(0xffffffffu, col ? at : -1, r);
                    const float4 x = *reinterpret_cast<const float4 *>(stage + r * kPitch + (lane & 7) * 16);
                    if (to >= 0) *reinterpret_cast<float4 *>(acc + to * kD + 32 * q + (lane & 7) * 4) = x;
                }
            };
            if (active) ok = wait_for(&sh.odone[l], (done - 1) & 1, abort);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            if constexpr (!SPLIT) {
#pragma unroll 1
                for (int q = 0; q < 4 && !idle; ++q) {
                    float ov[32];
                    tmem_ld32(t_o + 32 * q, ov);
                    tmem_wait_ld();
                    put(ov, q);
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
                    put(ov, q);
                }
                if (col && l == 0) *ml = make_float2(top, x.y * fx + y.y * fy);
                // O may be overwritten, and ml, once both lanes have read them
                tc_fence_before();
                mbar_arrive(tc_smem(&sh.oread));
                ok = wait_for(&sh.oread, joins & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                ++joins;
            }
            __syncwarp();
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sh.abort) raise_flag(a.err_flag, PA_FLAG_TIMEOUT);
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// A cache pool [N][Hkv][bs][128] bf16 as [8-row group][64-dim half][8 rows][64], copied a
// block at a time with the 128-byte swizzle.
bool pool_map(CUtensorMap *map, const void *pool, int groups, int bs) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, 8, 2, (cuuint64_t)groups};
    const cuuint64_t strides[3] = {kD * 2, 128, 8 * kD * 2};
    const cuuint32_t box[4] = {64u, 8u, 2u, (cuuint32_t)(bs / 8)};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BS, bool SPLIT>
cudaError_t launch_typed(const TreeContext &a, cudaStream_t stream) {
    CUtensorMap kmap, vmap;
    if ((int64_t)a.N * a.Hkv * BS >= (int64_t)INT32_MAX) return cudaErrorInvalidValue;  // TMA coordinates
    const int groups = a.N * a.Hkv * (BS / 8);
    if (!pool_map(&kmap, a.k_cache, groups, BS) || !pool_map(&vmap, a.v_cache, groups, BS)) return cudaErrorInvalidValue;
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
