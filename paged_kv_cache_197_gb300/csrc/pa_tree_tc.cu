// The context's part of tree attention on the fifth-generation tensor cores (head_dim 128).
//
// Every (row, query head) column of a sequence and kv head attends every cached token: one
// softmax over the context without a mask, S = Q K^T, P = 2^(S - m), O = P V, with the
// running base m and sum l of each column in registers and O in tensor memory.
//
// One CTA per SM (224 KB of shared memory, all 512 tensor-memory columns) works through its
// share of all tiles of the batch (pa_tree.cuh), 128 tokens of K and V at a time, in a ring
// of 32 KB stages that runs on across units.  Warps with fixed roles, coupled by mbarriers:
//   * warps 0-3 and 4-7 are two lanes of 128 columns, a thread per column.  With more than
//     128 columns the lanes take the two halves of 256 columns and share every staged
//     tile; with at most 128 they take the same columns and alternate tiles, and are
//     joined at the end of a unit.  Either way one lane's exponentials run while the
//     tensor cores work for the other;
//     The columns' threads also stage their lane's queries: the next unit's are copied
//     asynchronously once the last S of a unit is in, behind its last exponentials and the
//     write of its partials;
//   * warp 8 copies K and V tiles (TMA); one thread each of warps 9 and 10 issues a lane's
//     products (warp 11 fills the warpgroup, whose spare registers go to the columns);
//   * 8-bit caches: warp 8 copies codes and scales into a ring of 16 KB stages; warps 12-15
//     turn those of K, warps 16-19 those of V into fp16 in the stages the products read.
// Tensor memory: S of the lanes at columns 0 and 128 (overwritten by P as 16-bit pairs, the A
// operand of P V), O at 256 and 384.
// 8-bit caches: K's codes are exact in fp16, and a score is multiplied by its token's scale in
// fp32 (fp16 of code x scale would put scores of a few hundred off by a tenth and more; it
// saved 5 us of 132 for the fp8 batch).  A value is code x scale in fp16, in units of a power
// of two per tile (2^e, the tile's largest scale below 2^7 of them, so entries below 448 x 128),
// the scale rounded to fp16 and the product once more (2^-11 each; scales to 2^-20 of the tile's
// largest keep all their bits, and what is below 2^-31 of it is lost).  The query rows are fp16
// scaled by a power of two each (exact), which the columns take into their score factor; and
// they keep the base m above the scores plus the values' e: a weight p 2^e stays below 2^8
// whatever the scales.
// Weights are rounded to V's 16-bit type, as the two operands of a product have one type; their
// sum l takes them unrounded.  Against 64 bits the bf16 outputs are off by 0.0023 relative,
// where fp32 weights leave the output's own rounding, 0.0017; with fp16 weights it is 0.0017 too.
// Bounds: with up to 128 columns the 64 KB of a bf16 K and V tile take 2800 SM clocks at the
// measured HBM rate and the products 1024, so HBM bounds.  129 to 256 columns take 2048 clocks of
// products, and a lane's chain of S, exponentials, P V and the next S 3700 to 3800 by clock
// stamps, which bounds them, although every tile is fetched once for all the columns.  More
// columns reread the tiles through L2, a CTA for every 256.  Measured with the join: 20 trees of 16
// nodes over 8000 tokens (64/8 heads, 668 MB) 121 us, 5.5 TB/s; 16 trees of 33 to 64 nodes over 700
// to 8191 tokens (32/8 heads: 132 to 256 columns) 89.9 us, with the copies alone 74; 64 trees of 9
// to 16 nodes over 128 to 4096 tokens of an fp8 cache 133 us, the copies and changes of unit 93, the
// conversion 12 (int8 132).
// Every wait is bounded; a wait that gives up stops the CTA (PA_FLAG_TIMEOUT).
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "pa_mma.cuh"
#include "pa_tc.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

using namespace tc;

constexpr int kTile = kTreeTile;
constexpr int kD = 128;
constexpr int kLaneCols = 128;
constexpr int kTileBytes = kTile * kD * 2;   // 32 KB
constexpr int kRawBytes = kTile * kD;        // 16 KB of 8-bit codes
// A staged tile: groups of 8 rows, each as two 64-dim halves of 8 x 128 B (one swizzle atom
// each).  A cache block is then one copy of bs x 256 contiguous bytes, and the atoms of a
// half lie a constant 2 KB apart, as the matrix descriptors need.
constexpr int kHalf = 1024, kGroup = 2048;
constexpr uint32_t kTmemS = 0, kTmemO = 256;  // + 128 per lane
constexpr float kRescaleLog2 = 8.0f;
constexpr int kScaleSlots = 4;

// Shared memory and threads of a kernel.  Ring position p lands in stage p % kStages and
// completes barriers p % kFull, of its landing and of its consumption.  With alternating
// lanes a lane sees only its own positions, up to three apart, and copies land in any
// order, so a stage's own barrier could still be at the other lane's copy of the stage's
// previous position when p is asked for, and that phase has the parity of the one p waits
// for.  With two barriers a stage the predecessor on a barrier is two uses of the stage
// back, and a copy after that is only issued once it was consumed.  (The two groups that
// convert codes see every other position as well.)
template <typename KV, bool SPLIT>
struct Geo {
    static constexpr bool kQuant = sizeof(KV) == 1;
    static constexpr int kStages = kQuant ? 3 : 5, kFull = 2 * kStages;  // stages, barriers
    // query buffers: one per lane, or one for both lanes where they have the same columns and
    // codes need the room
    static constexpr int kQueries = kQuant && SPLIT ? 1 : 2;
    static constexpr bool kShared = kQueries == 1;
    static constexpr int kRaw = !kQuant ? 0 : SPLIT ? 5 : 3;  // stages of codes
    static constexpr int kOffRing = kQueries * kTileBytes, kOffRaw = kOffRing + kStages * kTileBytes;
    static constexpr int kOffShared = kOffRaw + kRaw * kRawBytes;
    static constexpr int kRawFull = 2 * kRaw;                 // their barriers, as for the ring
    static constexpr int kThreads = kQuant ? 640 : 384;
    // registers a thread: the columns' warps take what the others leave of the launch's
    // 3 x 168 or 5 x 96
    static constexpr int kRegsColumns = kQuant ? 128 : 200, kRegsOther = kQuant ? 72 : 104;
};

template <typename G>
struct Shared {
    float2 ml[2][kLaneCols];                    // lanes joined: each one's (base, sum) per column
    float raw_scale[G::kQuant ? G::kRaw : 1][G::kQuant ? kTile : 4];  // scales of the codes' stages
    float unit[kScaleSlots];                    // tiles' powers of two for V, as exponents
    float k_scale[G::kQuant ? kScaleSlots : 1][G::kQuant ? kTile : 4];  // tiles' scales of K
    float rs[2][G::kQuant ? kLaneCols : 1];     // columns' score factors, by query buffer
    uint64_t full[G::kFull], free[G::kFull];    // ring positions landed / consumed
    uint64_t raw_full[G::kQuant ? G::kRawFull : 1], raw_free[G::kQuant ? G::kRaw : 1];
    uint64_t units[2 * kScaleSlots], units_free[kScaleSlots];  // of unit and k_scale: both in / read
    uint64_t sfull[2], pfull[2], odone[2];      // per lane: S written, P written, P V done
    uint64_t qfull[2];                          // query buffers staged
    uint64_t mlready, oread;                    // lanes joined: both (base, sum) and O in / read
    uint64_t turn[2];                           // shared tiles: the lane may issue its next products
    uint64_t drain[2];
    int64_t total, first_tile;                  // of all positions; of the first sequence
    int first_seq;
    int wsum[20];
    uint32_t taddr;
    int abort;
};

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

// One block of a bf16 pool, [bs / 8][2][8][64] in the order of a staged tile.
__device__ __forceinline__ void tma_block(uint32_t dst, const CUtensorMap *map, int group, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(bar)
        : "memory");
}

// Eight floats, one 32-byte sector.
__device__ __forceinline__ void store8(float *p, const float *v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A range of tiles of one (sequence, kv head).
struct Unit {
    int s, kvh, t0, n, tiles, ctx, r0, ncols;
};

// The units of a CTA's share, in order; COLS columns to a CTA.
template <int COLS>
struct Walk {
    int64_t pos, end, before;  // positions: here, end of the share, before sequence s
    int s, tiles;              // sequence and its tiles per kv head (-1: not read yet)
    int ctx, r0, ncols;

    __device__ __forceinline__ bool next(const TreeContext &a, Unit &u) {
        while (pos < end) {
            if (tiles < 0) {
                const int r1 = a.query_start[s + 1];
                r0 = a.query_start[s];
                ctx = min(max(a.context_lens[s], 0), a.max_context_len);  // at most M * bs
                const int L = r1 - r0;
                ncols = L * a.G;
                tiles = r0 >= 0 && r1 <= a.T && L >= 1 && L <= a.max_query_len ? (ctx + kTile - 1) / kTile : 0;
            }
            const int64_t len = tree_unit_len(tiles, COLS);
            if (pos >= before + len * a.Hkv) {
                before += len * a.Hkv;
                ++s;
                tiles = -1;
                continue;
            }
            const int64_t in = pos - before;
            if (len * a.Hkv <= 0x7fffffff)
                u.kvh = (int)((uint32_t)in / (uint32_t)len);
            else
                u.kvh = (int)(in / len);
            const int off = (int)(in - u.kvh * len);
            const int64_t step = min(len - off, end - pos);
            pos += step;
            u.s = s;
            u.t0 = max(0, off - tree_pad(COLS));
            u.n = (int)(off + step) - tree_pad(COLS) - u.t0;
            u.tiles = tiles;
            u.ctx = ctx;
            u.r0 = r0;
            u.ncols = ncols;
            if (u.n > 0) return true;  // else only the unit's head start
        }
        return false;
    }
};

// Sixteen codes of one row, times a scale if scaled, as sixteen fp16 (two 16-byte words).
template <typename KV>
__device__ __forceinline__ void scaled_f16(const uint4 &c, bool scaled, __half2 scale, uint4 &lo, uint4 &hi) {
    if constexpr (sizeof(KV) == 1) {
        tiled::codes_to_f16_exact<KV>(c, lo, hi);
        if (!scaled) return;
        uint32_t *w[8] = {&lo.x, &lo.y, &lo.z, &lo.w, &hi.x, &hi.y, &hi.z, &hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(w[i]), scale);
            *w[i] = *reinterpret_cast<const uint32_t *>(&x);
        }
    }
}

constexpr float kTiny = 1.17549435e-38f;  // least score factor: 0 times a masked -inf is a NaN
constexpr int kScaleTop = 7;  // scales below 2^7 units: 448 x 2^7 is below fp16's 65504

// Two fp32 operations in one instruction (one at a time: 141.6 instead of 132.5 us for the fp8
// batch, 90.7 instead of 89.7 for the ragged one).
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b) {
    asm("{\n.reg .b64 p, q;\nmov.b64 p, {%0, %1};\nmov.b64 q, {%2, %3};\nmul.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}\n"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ void fma2(float &x, float &y, float a, float c) {
    asm("{\n.reg .b64 p, q, r;\nmov.b64 p, {%0, %1};\nmov.b64 q, {%2, %2};\nmov.b64 r, {%3, %3};\nfma.rn.f32x2 p, p, q, r;\n"
        "mov.b64 {%0, %1}, p;\n}\n"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(c));
}
__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {
    asm("{\n.reg .b64 p, q;\nmov.b64 p, {%0, %1};\nmov.b64 q, {%2, %3};\nadd.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}\n"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}

// Exponent e with |x| < 2^e for the bits of a positive x, kept in -100 .. 100.
__device__ __forceinline__ int exponent_over(uint32_t bits) {
    return min(max((int)((bits >> 23) & 0xffu) - 126, -100), 100);
}

template <typename KV, int BS, bool SPLIT>
__global__ void __launch_bounds__(Geo<KV, SPLIT>::kThreads, 1)
tree_tc_kernel(const __grid_constant__ TreeContext a, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
    using G = Geo<KV, SPLIT>;
    constexpr bool QUANT = G::kQuant;
    constexpr int kCols = SPLIT ? kLaneCols : 2 * kLaneCols;
    constexpr int kThreads = G::kThreads, kStages = G::kStages, kFull = G::kFull;
    static_assert(G::kOffShared + sizeof(Shared<G>) <= 232448, "shared memory of one CTA per SM");
    extern __shared__ __align__(1024) unsigned char smem[];
    Shared<G> &sh = *reinterpret_cast<Shared<G> *>(smem + G::kOffShared);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((tc_smem(smem) & 1023) != 0) {  // the swizzled tiles need their alignment
        if (tid == 0) raise_flag(a.err_flag, PA_FLAG_TIMEOUT);
        return;
    }
    const int group = blockIdx.x / a.members, member = blockIdx.x % a.members;
    if (warp == 1) {
        for (int i = lane; i < kFull; i += 32) mbar_init_n(tc_smem(&sh.full[i]), QUANT ? 128 : 1);
        for (int i = lane; i < kFull; i += 32) mbar_init_n(tc_smem(&sh.free[i]), SPLIT ? 1 : 2);  // lanes that read a stage
        for (int i = lane; i < G::kRawFull; i += 32) mbar_init_n(tc_smem(&sh.raw_full[i]), 33);  // codes, each lane's scales
        for (int i = lane; i < G::kRaw; i += 32) mbar_init_n(tc_smem(&sh.raw_free[i]), 128);
        if (QUANT && lane < 2 * kScaleSlots) mbar_init_n(tc_smem(&sh.units[lane]), 129);  // K's group, V's first thread
        if (QUANT && lane < kScaleSlots) mbar_init_n(tc_smem(&sh.units_free[lane]), SPLIT ? kLaneCols : 2 * kLaneCols);
        if (lane < 2) {
            mbar_init(tc_smem(&sh.sfull[lane]));
            mbar_init(tc_smem(&sh.odone[lane]));
            mbar_init_n(tc_smem(&sh.pfull[lane]), kLaneCols);
            mbar_init_n(tc_smem(&sh.qfull[lane]), G::kShared ? 2 * kLaneCols : kLaneCols);
            mbar_init(tc_smem(&sh.turn[lane]));
            mbar_init(tc_smem(&sh.drain[lane]));
            mbar_init_n(tc_smem(lane ? &sh.mlready : &sh.oread), 2 * kLaneCols + (lane && G::kShared ? 1 : 0));
        }
        if (lane == 0) {
            sh.abort = 0;
            sh.first_seq = 0;
            sh.first_tile = 0;
            sh.total = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc_smem(&sh.taddr))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the batch's positions: their number, then the sequence this share begins in
    auto len_of = [&](int s, bool report) -> int {
        const int lim = a.max_context_len;
        const int ctx = a.context_lens[s], r0 = a.query_start[s], r1 = a.query_start[s + 1], L = r1 - r0;
        const bool ok = r0 >= 0 && r1 <= a.T && L >= 0 && L <= a.max_query_len;
        if (report && (ctx < 0 || ctx > lim)) raise_flag(a.err_flag, PA_FLAG_CONTEXT_OUT_OF_RANGE);
        if (report && !ok) raise_flag(a.err_flag, PA_FLAG_QUERY_OUT_OF_RANGE);
        return ok && L > 0 ? (int)tree_unit_len((min(max(ctx, 0), lim) + kTile - 1) / kTile, kCols) : 0;
    };
    const int n_first = tid < a.S ? len_of(tid, blockIdx.x == 0) : 0;
    int64_t sum = n_first;
    for (int s = tid + kThreads; s < a.S; s += kThreads) sum += len_of(s, blockIdx.x == 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0 && sum) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.total), (unsigned long long)sum);
    __syncthreads();
    const int64_t total = sh.total * a.Hkv;
    const int64_t groups = min((int64_t)a.groups, total);
    const int64_t begin = group < groups ? group * total / groups : total;
    const int64_t end = group < groups ? (group + 1) * total / groups : total;
    int64_t carry = 0;
    for (int base = 0; base < a.S; base += kThreads) {
        const int s = base + tid, n = base == 0 ? n_first : s < a.S ? len_of(s, false) : 0;
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
    Walk<kCols> w{begin, end, sh.first_tile, sh.first_seq, -1, 0, 0, 0};
    int *abort = &sh.abort;

    // lane 1 has work: its half of the columns, or (lanes on the same columns) a second tile
    auto second = [&](const Unit &u) { return SPLIT ? u.n > 1 : u.ncols - member * a.cols > kLaneCols; };
    // the member's next unit with columns
    auto next_unit = [&](Unit &u) {
        while (w.next(a, u))
            if (u.ncols > member * a.cols) return true;
        return false;
    };
    // Ring positions of tile t's K and V within a unit of n tiles, in the order they are used:
    // K0 V0 K1 V1 .. (shared tiles), K0 K1 V0 K2 V1 .. (alternating lanes).
    auto k_at = [](int t, int n) { return SPLIT ? (t == 0 ? 0 : 2 * t - 1) : 2 * t; };
    auto v_at = [](int t, int n) { return SPLIT ? (t < n - 1 ? 2 * t + 2 : 2 * n - 1) : 2 * t + 1; };

    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kRegsOther));
    if (warp == 8) {
        // ---- copies: lane i takes block i of a tile
        constexpr int kBlocks = kTile / BS, kGroups = BS / 8;  // 8-row groups of a block and kv head
        constexpr int kSlots = QUANT ? G::kRaw : kStages;
        const int oob = QUANT ? a.N * a.Hkv * BS : a.N * a.Hkv * kGroups;  // past the pool: the copy fills zeros
        const uint32_t box = tc_smem(smem + (QUANT ? G::kOffRaw : G::kOffRing)) + lane * BS * (QUANT ? kD : 2 * kD);
        int st = 0, issued = 0;            // stage, ring position
        bool ok = true, first = true;
        Unit u{}, nu;
        bool have = next_unit(nu);
        // K (map, y) or V of this lane's block; 8-bit: the block's scales too, none where b < 0
        auto fill = [&](bool is_k, int y, int b) {
            const int last = issued - kSlots;  // the stage's last position
            if (last >= 0)
                ok = QUANT ? wait_for(&sh.raw_free[st], (last / kSlots) & 1, abort)
                           : wait_for(&sh.free[last % kFull], (last / kFull) & 1, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            const CUtensorMap *map = is_k ? &kmap : &vmap;
            if constexpr (QUANT) {
                const uint32_t bar = tc_smem(&sh.raw_full[issued % (QUANT ? G::kRawFull : 1)]);
                if (lane == 0) mbar_expect(bar, kRawBytes);
                __syncwarp();
                if (lane < kBlocks) tma_load(box + st * kRawBytes, map, 0, y, bar);
                __syncwarp();
                // the scales, four tokens a lane in one instruction (a bulk copy per block
                // took the fp8 batch 0.6 us longer)
                const int from = __shfl_sync(0xffffffffu, b, 4 * lane / BS);
                const float *scale = (is_k ? a.k_scale : a.v_scale) + ((int64_t)max(from, 0) * a.Hkv + u.kvh) * BS + 4 * lane % BS;
                tiled::cp_async16(tc_smem(sh.raw_scale[st] + 4 * lane), scale, from >= 0 ? 16 : 0);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
            } else {
                const uint32_t bar = tc_smem(&sh.full[issued % kFull]);
                if (lane == 0) mbar_expect(bar, kTileBytes);
                __syncwarp();
                if (lane < kBlocks) tma_block(box + st * kTileBytes, map, y, bar);
            }
            ++issued;
            if (++st == kSlots) st = 0;
        };
        while (ok && have) {
            u = nu;
            const int nblk = (u.ctx + BS - 1) / BS;
            const int32_t *table = a.block_tables + (int64_t)u.s * a.M;
            // the raw table entry of this lane's block of tile t; -2 for blocks past the context
            auto entry = [&](int t) {
                const int idx = (u.t0 + t) * kBlocks + lane;
                return t < u.n && lane < kBlocks && idx < nblk ? __ldg(table + idx) : -2;
            };
            auto checked = [&](int t, int b) {  // -1 where nothing is read
                if (b >= 0 && b < a.N) return b;
                const int idx = (u.t0 + t) * kBlocks + lane;
                if (t < u.n && lane < kBlocks && idx < nblk && member == 0) raise_flag(a.err_flag, PA_FLAG_BLOCK_OUT_OF_RANGE);
                return -1;
            };
            auto row_of = [&](int b) { return b >= 0 ? (b * a.Hkv + u.kvh) * (QUANT ? BS : kGroups) : oob; };
            // With the ring's copies of all SMs queued up, a load that misses L2 takes several
            // microseconds: the unit's table entries are fetched into L2 at its start (32 to a
            // line) and loaded two tiles ahead of their copies, and the first unit's queries
            // go before all copies but one.
            for (int i = lane * 32; i < u.n * kBlocks; i += 32 * 32) prefetch_l2(table + min(u.t0 * kBlocks + i, nblk - 1));
            int b = checked(0, entry(0)), e1 = entry(1), e2 = entry(2);
            fill(true, row_of(b), b);
            if (first) {
                first = false;  // (their barrier's next phase needs this unit's other tiles)
                if (ok) ok = wait_for(&sh.qfull[0], 0, abort);
                ok = __all_sync(0xffffffffu, ok);
            }
            have = next_unit(nu);
            for (int t = 0; ok && t < u.n; ++t) {
                const int bn = checked(t + 1, e1);
                e1 = e2;
                e2 = entry(t + 3);
                if (SPLIT && t + 1 < u.n) fill(true, row_of(bn), bn);
                if (ok) fill(false, row_of(b), b);
                if (!SPLIT && ok && t + 1 < u.n) fill(true, row_of(bn), bn);
                b = bn;
            }
        }
        if (!ok) {
            // stopping early: copies already issued may still be landing in shared memory
            for (int i = max(0, issued - kSlots); i < issued; ++i) {
                if constexpr (QUANT)
                    mbar_wait(tc_smem(&sh.raw_full[i % G::kRawFull]), (i / G::kRawFull) & 1);
                else
                    mbar_wait(tc_smem(&sh.full[i % kFull]), (i / kFull) & 1);
            }
        }
    } else if (warp < 11) {
        // ---- products of lane l: one thread waits and issues (a thread per lane, so that one
        // lane's waits do not hold up the other's products)
        if (lane == 0) {
            const int l = warp - 9;
            int ring = 0;
            uint32_t pv = 0, staged = 0, taken = 0;
            bool ok = true;
            const uint32_t t_s = tmem + kTmemS + l * 128, t_o = tmem + kTmemO + l * 128;
            const uint64_t qd = sw128_desc(tc_smem(smem), 16, kGroup);
            const uint64_t kd = sw128_desc(tc_smem(smem + G::kOffRing), 16, kGroup);
            const uint64_t vd = sw128_desc(tc_smem(smem + G::kOffRing), kHalf, kGroup);
            // fp16 operands (8-bit caches) have type code 0 where bf16 has 1
            constexpr uint32_t kType = QUANT ? (1u << 7) | (1u << 10) : 0u;
            constexpr uint32_t kScores = bf16_idesc(128, kTile, 0) ^ kType, kWeighted = bf16_idesc(128, kD, 1) ^ kType;
            const uint32_t sfull = tc_smem(&sh.sfull[l]), odone = tc_smem(&sh.odone[l]);
            Unit u, nu;
            bool have = next_unit(nu);
            while (ok && have) {
                u = nu;
                const bool two = second(u);
                const int qb = G::kShared ? 0 : l;
                if (l == 1 && !two) {
                    // shared queries are staged for every unit: the unit does not end before this
                    // thread has seen its own (a phase later the parity would say nothing)
                    if (G::kShared) {
                        ok = wait_for(&sh.qfull[0], staged++ & 1, abort);
                        if (ok) mbar_arrive(tc_smem(&sh.mlready));
                    }
                    // the other lane reads these tiles alone
                    for (int at = ring; !SPLIT && ok && at < ring + 2 * u.n; ++at) {
                        ok = wait_for(&sh.full[at % kFull], (at / kFull) & 1, abort);
                        if (ok) mbar_arrive(tc_smem(&sh.free[at % kFull]));
                    }
                    ring += 2 * u.n;
                    have = next_unit(nu);
                    continue;
                }
                auto landed = [&](int at) { return wait_for(&sh.full[at % kFull], (at / kFull) & 1, abort); };
                auto scores = [&](int at) {
                    tc_fence_after();
                    const uint64_t q0 = qd + (uint64_t)(qb * (kTileBytes >> 4)), k0 = kd + (uint64_t)(at % kStages * (kTileBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk) {
                        const uint64_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        umma(t_s, q0 + off, k0 + off, kScores, kk > 0);
                    }
                    umma_commit(sfull);
                };
                auto weighted = [&](int at, bool first) {
                    tc_fence_after();
                    const uint64_t v0 = vd + (uint64_t)(at % kStages * (kTileBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        umma_ts(t_o, t_s + kk * 8, v0 + (kk * 2 * kGroup >> 4), kWeighted, !first || kk > 0);
                    umma_commit(odone);
                    ++pv;
                };
                constexpr int kStep = SPLIT ? 2 : 1;
                const int t_first = SPLIT ? l : 0;
                // Lanes that share their tiles take turns at the tensor cores, P V and the next
                // S at a time: left alone they fall into step, both computing exponentials and
                // then both waiting for products.  What a turn needs is waited for before it.
                const bool turns = !SPLIT && two;
                int k_pos = ring + k_at(t_first, u.n);
                // the queries first: they are staged when the lane's last unit is done, which
                // bounds how far ahead of the ring a lane asks
                ok = wait_for(&sh.qfull[qb], staged++ & 1, abort);
                if (ok && G::kShared && l == 1) mbar_arrive(tc_smem(&sh.mlready));
                // S overwrites P: the lane's last P V is done
                if (ok && pv > 0) ok = wait_for(&sh.odone[l], (pv - 1) & 1, abort);
                if (ok) ok = landed(k_pos);
                if (ok) {
                    scores(k_pos);
                    umma_commit(tc_smem(&sh.free[k_pos % kFull]));
                }
                have = next_unit(nu);
                for (int t = t_first; ok && t < u.n; t += kStep) {
                    const bool more = t + kStep < u.n;
                    const int v_pos = ring + v_at(t, u.n);
                    k_pos = ring + k_at(t + kStep, u.n);
                    ok = landed(v_pos) && (SPLIT || !more || landed(k_pos)) && wait_for(&sh.pfull[l], pv & 1, abort);
                    if (ok && turns && (l == 1 || taken > 0)) ok = wait_for(&sh.turn[l], (l == 1 ? taken : taken - 1) & 1, abort);
                    if (!ok) break;
                    weighted(v_pos, t == t_first);
                    if (more) {
                        ok = wait_for(&sh.odone[l], (pv - 1) & 1, abort) && (!SPLIT || landed(k_pos));
                        if (!ok) break;
                        scores(k_pos);
                    }
                    if (turns) {
                        mbar_arrive(tc_smem(&sh.turn[l ^ 1]));
                        ++taken;
                    }
                    umma_commit(tc_smem(&sh.free[v_pos % kFull]));
                    if (more) umma_commit(tc_smem(&sh.free[k_pos % kFull]));
                }
                ring += 2 * u.n;
            }
            if (!ok) {
                // stopping early: every product already issued finishes before tensor memory is released
                umma_commit(tc_smem(&sh.drain[l]));
                mbar_wait(tc_smem(&sh.drain[l]), 0);
            }
        }
        __syncwarp();
    } else if (QUANT && warp >= 12) {
        // ---- 8-bit caches: codes of K, or of V, to fp16
        const bool is_k = warp < 16;
        const int me = tid & 127;
        int ring = 0, tile = 0;
        bool ok = true;
        Unit u;
        while (ok && next_unit(u)) {
            for (int t = 0; ok && t < u.n; ++t) {
                constexpr int kRaw = QUANT ? G::kRaw : 1, kRawFull = QUANT ? G::kRawFull : 1;
                const int at = ring + (is_k ? k_at(t, u.n) : v_at(t, u.n));
                const int rst = at % kRaw, st = at % kStages, j = tile + t;
                ok = wait_for(&sh.raw_full[at % kRawFull], (at / kRawFull) & 1, abort);
                if (ok && at >= kStages) ok = wait_for(&sh.free[(at - kStages) % kFull], ((at - kStages) / kFull) & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const int left = u.ctx - (u.t0 + t) * kTile;  // tokens of the context from the tile on
                // the tile's power of two (scales behind the context may hold anything)
                const float *scale = sh.raw_scale[rst];
                const float4 s4 = reinterpret_cast<const float4 *>(scale)[lane];
                const float top = fmaxf(fmaxf(4 * lane < left ? fabsf(s4.x) : 0.f, 4 * lane + 1 < left ? fabsf(s4.y) : 0.f),
                                        fmaxf(4 * lane + 2 < left ? fabsf(s4.z) : 0.f, 4 * lane + 3 < left ? fabsf(s4.w) : 0.f));
                const int e = exponent_over(__reduce_max_sync(0xffffffffu, __float_as_uint(top))) - kScaleTop;
                const float down = is_k ? 1.f : __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e
                if (is_k || me == 0) {
                    // the lanes have read this slot's last tile
                    if (j >= kScaleSlots) ok = wait_for(&sh.units_free[j % kScaleSlots], (j / kScaleSlots - 1) & 1, abort);
                    if (is_k)
                        sh.k_scale[j % kScaleSlots][me] = scale[me];
                    else
                        sh.unit[j % kScaleSlots] = (float)e;
                    mbar_arrive(tc_smem(&sh.units[j % (2 * kScaleSlots)]));
                }
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                // this thread's piece c of rows r0, r0 + 16, ..: two 8-value chunks each.  Eight
                // lanes take the same half of rows r and r ^ 5: both tiles are swizzled by the
                // row's low three bits, codes in pieces (the two rows' halves then lie apart: bit
                // 2) and values in chunks (every other one: bit 0), so neither the loads nor the
                // stores meet a bank twice.
                const int low = ((me >> 5) & 1) + ((me >> 3) & 2);  // rows 0 .. 3 of eight, with 5, 4, 7, 6
                const int r0 = (me >> 6) * 8 + ((me & 4) ? low ^ 5 : low), c = (me & 3) + ((me >> 1) & 4);
                const unsigned char *from = smem + G::kOffRaw + rst * kRawBytes + r0 * kD + ((c ^ (r0 & 7)) << 4);
                unsigned char *to = smem + G::kOffRing + st * kTileBytes;
                unsigned char *to0 = to + tile_chunk(r0, 2 * c), *to1 = to + tile_chunk(r0, 2 * c + 1);
                constexpr int kAtOnce = 2;
#pragma unroll 1
                for (int r = r0; r < kTile; r += 16 * kAtOnce, from += 16 * kAtOnce * kD, to0 += 2 * kAtOnce * kGroup, to1 += 2 * kAtOnce * kGroup) {
                    uint4 code[kAtOnce], lo, hi;
                    float sc[kAtOnce];
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        code[k] = *reinterpret_cast<const uint4 *>(from + k * 16 * kD);
                        sc[k] = scale[r + 16 * k] * down;
                    }
                    if (left < kTile) {  // codes and scales of no token
#pragma unroll
                        for (int k = 0; k < kAtOnce; ++k)
                            if (r + 16 * k >= left) {
                                code[k] = make_uint4(0u, 0u, 0u, 0u);
                                sc[k] = 0.f;
                            }
                    }
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        scaled_f16<KV>(code[k], !is_k, __float2half2_rn(sc[k]), lo, hi);
                        *reinterpret_cast<uint4 *>(to0 + k * 2 * kGroup) = lo;
                        *reinterpret_cast<uint4 *>(to1 + k * 2 * kGroup) = hi;
                    }
                }
                fence_async();
                mbar_arrive(tc_smem(&sh.full[at % kFull]));
                mbar_arrive(tc_smem(&sh.raw_free[rst]));
            }
            ring += 2 * u.n;
            tile += u.n;
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kRegsColumns));
        // ---- a lane's columns: thread = column = tensor-memory lane
        const int l = warp >> 2, row = tid & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_off + kTmemS + l * 128, t_o = tmem + lane_off + kTmemO + l * 128;
        int done = 0, ring = 0, joins = 0, tile = 0;  // tiles of this lane; ring position; units joined; tile
        bool ok = true;
        Unit u, nu;
        bool have = next_unit(nu);
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // the columns take |scale|
        // Staging the lane's queries of unit x: pieces of 16 bytes, a row by 16 threads, copied
        // asynchronously by `stage` and made ready by `staged`.
        constexpr int kRowsAtOnce = (G::kShared ? 256 : 128) / 16;
        const int me = G::kShared ? tid : row, piece = me & 15;
        unsigned char *qbuf = smem + (G::kShared ? 0 : l) * kTileBytes;
        const int lane_col = member * a.cols + (SPLIT ? 0 : l * kLaneCols);  // the lane's first column
        auto stage = [&](const Unit &x) {
#pragma unroll 4
            for (int r = me >> 4; r < kLaneCols; r += kRowsAtOnce) {
                const int cc = lane_col + r;
                const int tok = a.g_shift >= 0 ? cc >> a.g_shift : cc / a.G, head = cc - tok * a.G;
                const bool real = cc < x.ncols;
                const int64_t at = ((int64_t)(x.r0 + tok) * a.Hq + x.kvh * a.G + head) * kD + piece * 8;
                tiled::cp_async16(tc_smem(qbuf + tile_chunk(r, piece)), real ? a.q + at : a.q, real ? 16 : 0);
            }
        };
        auto staged = [&] {
            tiled::cp_async_wait_all();
            if (QUANT || flip) {
                // 8-bit caches: as fp16 scaled by 2^sig per row, sig putting the row's largest |q|
                // in [2^13, 2^14).  Each thread rewrites what it copied itself.
#pragma unroll 2
                for (int r = me >> 4; r < kLaneCols; r += kRowsAtOnce) {
                    uint4 *at = reinterpret_cast<uint4 *>(qbuf + tile_chunk(r, piece));
                    const uint4 x = *at;
                    uint32_t q[4] = {x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip};
                    if constexpr (QUANT) {
                        float f[8], amax = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            f[2 * e] = __uint_as_float(q[e] << 16);
                            f[2 * e + 1] = __uint_as_float(q[e] & 0xffff0000u);
                            amax = fmaxf(amax, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
                        }
#pragma unroll
                        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                        const int sig = amax > 0.f ? min(100, max(-100, 14 - tiled::exponent_above(amax))) : 0;
                        const float up = __uint_as_float((uint32_t)(127 + sig) << 23);  // 2^sig
#pragma unroll
                        for (int e = 0; e < 4; ++e) q[e] = tiled::f16x2(f[2 * e] * up, f[2 * e + 1] * up);
                        if (piece == 0) sh.rs[G::kShared ? 0 : l][r] = fabsf(a.scale_log2) * __uint_as_float((uint32_t)(127 - sig) << 23);
                    }
                    *at = make_uint4(q[0], q[1], q[2], q[3]);
                }
            }
            fence_async();
            mbar_arrive(tc_smem(&sh.qfull[G::kShared ? 0 : l]));
        };
        // whether this lane stages queries for unit x
        auto stages = [&](const Unit &x) { return G::kShared || l == 0 || second(x); };
        bool pending = have && stages(nu);
        if (pending) stage(nu);
        uint32_t units = 0;  // units whose queries this lane staged
        while (ok && have) {
            u = nu;
            const bool two = second(u);
            const bool active = l == 0 || two;
            if (pending) staged();
            pending = false;
            have = next_unit(nu);
            if (!SPLIT && !active) {
                if constexpr (QUANT) {  // the other lane reads these tiles' powers alone
                    for (int t = 0; ok && t < u.n; ++t) {
                        const int j = tile + t;
                        ok = wait_for(&sh.units[j % (2 * kScaleSlots)], j / (2 * kScaleSlots) & 1, abort);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        mbar_arrive(tc_smem(&sh.units_free[j % kScaleSlots]));
                    }
                }
                ring += 2 * u.n;
                tile += u.n;
                if (ok && have && stages(nu)) {
                    stage(nu);
                    pending = true;
                }
                continue;
            }
            const int c = lane_col + row;
            const bool col = c < u.ncols;
            float m = -INFINITY, sum_l = 0.f, rs = fabsf(a.scale_log2);
            if constexpr (QUANT) {
                ok = wait_for(&sh.qfull[G::kShared ? 0 : l], units & 1, abort);  // the factors of all the lane's rows
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                rs = sh.rs[G::kShared ? 0 : l][row];
            }
            ++units;
            // the lane's last tile
            const int t_last = SPLIT ? u.n - 1 - ((u.n - 1 - l) & 1) : u.n - 1;
            // a warp none of whose columns is real keeps step without computing
            const bool idle = lane_col + (warp & 3) * 32 >= u.ncols;
            for (int t = SPLIT ? l : 0; t < u.n; t += SPLIT ? 2 : 1) {
                const int j = tile + t;
                ok = wait_for(&sh.sfull[l], done & 1, abort);
                if (QUANT && ok) ok = wait_for(&sh.units[j % (2 * kScaleSlots)], j / (2 * kScaleSlots) & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                if (!G::kShared && t == t_last && have && stages(nu)) {
                    // the lane's products with this unit's queries are done
                    stage(nu);
                    pending = true;
                }
                const int k0 = (u.t0 + t) * kTile;
                if (!idle) {
                    const int left = u.ctx - k0;  // tokens of the context from the tile on
                    float factor = rs, over = 0.f;  // of the scores; exponent of the values' unit
                    if constexpr (QUANT) over = sh.unit[j % kScaleSlots];
                    // 8-bit caches: 32 scores of codes times their tokens' scales
                    auto scaled = [&](float (&x)[32], int q) {
                        if constexpr (QUANT) {
                            const float4 *ks = reinterpret_cast<const float4 *>(sh.k_scale[j % kScaleSlots]) + 8 * q;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float4 w = ks[k];
                                mul2(x[4 * k], x[4 * k + 1], w.x, w.y);
                                mul2(x[4 * k + 2], x[4 * k + 3], w.z, w.w);
                            }
                        }
                    };
                    if (left < kTile) factor = fmaxf(factor, kTiny);
                    // The scores are read twice, for the maximum and for the weights, 64 and 32 at a
                    // time, in loops that stay loops: all 128 in registers spilled, and code
                    // unrolled over the tile starved the roles of instructions.
                    float mx[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) mx[i] = -INFINITY;
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        float sv[32];
                        tmem_ld32(t_s + 32 * h, sv);
                        tmem_wait_ld();
                        scaled(sv, h);
                        if (left < kTile) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (32 * h + k >= left) sv[k] = -INFINITY;
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k) mx[k & 7] = fmaxf(mx[k & 7], sv[k]);
                    }
                    const float top = fmaf(fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                                 fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))),
                                           factor, over);
                    // the running base is raised only by more than 2^8; then l and O shrink
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
                    const float base = (m == -INFINITY ? 0.f : m) - over;  // weights come in units of 2^-over
                    float ls[4] = {0.f, 0.f, 0.f, 0.f};
                    // 32 scores into weights, over the columns of scores already read
                    auto weigh = [&](float (&x)[32], int q) {
                        if (left < kTile) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (32 * q + k >= left) x[k] = -INFINITY;
                        }
                        float pw[16];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float p[4];
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                fma2(x[2 * i + e], x[2 * i + e + 1], factor, -base);
                                p[e] = tc_exp2(x[2 * i + e]);
                                p[e + 1] = tc_exp2(x[2 * i + e + 1]);
                                add2(ls[e], ls[e + 1], p[e], p[e + 1]);
                            }
                            if constexpr (QUANT) {
                                pw[i] = __uint_as_float(tiled::f16x2(p[0], p[1]));
                                pw[i + 1] = __uint_as_float(tiled::f16x2(p[2], p[3]));
                            } else {
                                pw[i] = __uint_as_float(tc_bf16x2(p[0], p[1]));
                                pw[i + 1] = __uint_as_float(tc_bf16x2(p[2], p[3]));
                            }
                        }
                        tmem_st16(t_s + 16 * q, pw);
                    };
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        float x[32];
                        tmem_ld32(t_s + 32 * q, x);
                        tmem_wait_ld();
                        scaled(x, q);
                        weigh(x, q);
                    }
                    const float sum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
                    sum_l += QUANT ? sum * tc_exp2(-over) : sum;
                    tmem_wait_st();
                }
                if constexpr (QUANT) {
                    mbar_arrive(tc_smem(&sh.units_free[j % kScaleSlots]));
                } else if (k0 + kTile > u.ctx && u.ctx % BS != 0) {
                    // rows past the context inside its last block may hold anything, and a zero
                    // weight times a NaN is a NaN: zero them in the V stage
                    const int at = ring + v_at(t, u.n), st = at % kStages;
                    ok = wait_for(&sh.full[at % kFull], (at / kFull) & 1, abort);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const int lo = u.ctx - k0, hi = min(kTile, (u.ctx + BS - 1) / BS * BS - k0);
                    unsigned char *vst = smem + G::kOffRing + st * kTileBytes;
                    for (int i = row; i < (hi - lo) * 16; i += kLaneCols)
                        *reinterpret_cast<uint4 *>(vst + tile_chunk(lo + i / 16, i % 16)) = make_uint4(0u, 0u, 0u, 0u);
                    fence_async();
                }
                tc_fence_before();
                mbar_arrive(tc_smem(&sh.pfull[l]));
                ++done;
            }
            ring += 2 * u.n;
            tile += u.n;
            if (!ok) break;
            // ---- the columns' partials: a thread's row, a sector at a time
            const int tok = a.g_shift >= 0 ? c >> a.g_shift : c / a.G, head = c - tok * a.G;
            const int64_t pair = (int64_t)(u.r0 + tok) * a.Hq + u.kvh * a.G + head;
            const bool all = u.t0 == 0 && u.n == u.tiles;
            const int64_t at = all ? pair : ((int64_t)blockIdx.x * 2 + (u.t0 == 0 ? 1 : 0)) * a.cols + (c - member * a.cols);
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
                    if (col) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) store8(acc + 32 * q + 8 * i, ov + 8 * i);
                    }
                    __syncwarp();
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
                    if (col) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) store8(acc + 32 * q + 8 * i, ov + 8 * i);
                    }
                    __syncwarp();
                }
                if (col && l == 0) *ml = make_float2(top, x.y * fx + y.y * fy);
                // O may be overwritten, and ml, once both lanes have read them
                tc_fence_before();
                mbar_arrive(tc_smem(&sh.oread));
                ok = wait_for(&sh.oread, joins & 1, abort);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                ++joins;
                if (!pending && have && stages(nu)) {  // one buffer for both lanes, or no tile in this unit
                    stage(nu);
                    pending = true;
                }
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

// A bf16 pool [N][Hkv][bs][128] as [8-row group][64-dim half][8 rows][64], copied a block at
// a time with the 128-byte swizzle; a pool of 8-bit codes as rows of 128 bytes, copied a
// block at a time as they are.
bool pool_map(CUtensorMap *map, const void *pool, int rows, int bs, bool codes) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    if (codes) {
        const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)rows};
        const cuuint64_t strides[1] = {(cuuint64_t)kD};
        const cuuint32_t box[2] = {(cuuint32_t)kD, (cuuint32_t)bs};
        return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(pool), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    const cuuint64_t dims[4] = {64, 8, 2, (cuuint64_t)(rows / 8)};
    const cuuint64_t strides[3] = {kD * 2, 128, 8 * kD * 2};
    const cuuint32_t box[4] = {64u, 8u, 2u, (cuuint32_t)(bs / 8)};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename KV, int BS, bool SPLIT>
cudaError_t launch_typed(const TreeContext &a, cudaStream_t stream) {
    using G = Geo<KV, SPLIT>;
    constexpr int kSmem = G::kOffShared + (int)sizeof(Shared<G>);
    CUtensorMap kmap, vmap;
    if ((int64_t)a.N * a.Hkv * BS >= (int64_t)INT32_MAX) return cudaErrorInvalidValue;  // TMA coordinates
    const int rows = a.N * a.Hkv * BS;
    if (!pool_map(&kmap, a.k_cache, rows, BS, G::kQuant) || !pool_map(&vmap, a.v_cache, rows, BS, G::kQuant))
        return cudaErrorInvalidValue;
    static std::atomic<bool> configured[64];  // per device: the shared-memory attribute is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(tree_tc_kernel<KV, BS, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    return launch_dependent(tree_tc_kernel<KV, BS, SPLIT>, dim3(a.groups * a.members), dim3(G::kThreads), kSmem, stream, a,
                            kmap, vmap);
}

template <typename KV>
cudaError_t launch_kv(const TreeContext &a, int bs, cudaStream_t stream) {
    if (a.cols == kLaneCols)
        return bs == 16 ? launch_typed<KV, 16, true>(a, stream) : launch_typed<KV, 32, true>(a, stream);
    return bs == 16 ? launch_typed<KV, 16, false>(a, stream) : launch_typed<KV, 32, false>(a, stream);
}

}  // namespace

bool tree_tc_eligible(int D, int kv_dtype) {
    return D == kD && (kv_dtype == PA_KV_BF16 || kv_dtype == PA_KV_INT8 || kv_dtype == PA_KV_FP8);
}

cudaError_t launch_tree_tc(const TreeContext &a, int bs, int kv_dtype, cudaStream_t stream) {
    if (kv_dtype == PA_KV_INT8) return launch_kv<int8_t>(a, bs, stream);
    if (kv_dtype == PA_KV_FP8) return launch_kv<tiled::e4m3_tag>(a, bs, stream);
    return launch_kv<uint16_t>(a, bs, stream);
}

}  // namespace pa
