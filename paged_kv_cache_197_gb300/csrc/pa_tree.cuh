// Tree attention (pa_draft.h): what its kernels share.
#pragma once

#include "pa_draft.h"
#include "pa_internal.cuh"

namespace pa {

// The context's part on the tcgen05 kernel.  The contexts are cut into 128-token tiles and
// all (sequence, kv head) units laid end to end; group g of min(`groups`, total) takes positions
// [g * total / groups, (g + 1) * total / groups), whatever the lengths of the sequences, and
// the `members` CTAs of a group take `cols` (row, query head) columns each.  A unit that
// lies in one group leaves one partial per column in `whole`; a cut one leaves one in a slot
// of each CTA: slot 0 where the unit began before the CTA's range, slot 1 where it begins in
// it.
struct TreeContext {
    const uint16_t *q;
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *block_tables, *context_lens, *query_start;
    float *whole_acc, *whole_ml;  // [T][Hq][128], [T][Hq][2]
    float *cut_acc, *cut_ml;      // [CTA][2][cols][128], [CTA][2][cols][2]
    int64_t *prefix;              // [S + 1]: first position of each sequence (written by the kernel)
    int *err_flag;
    int M, S, T, Hq, Hkv, G, N, g_shift;
    int members, groups, cols;
    int max_context_len, max_query_len;
    float scale_log2;
};

constexpr int kTreeTile = 128;  // cached tokens per tile
// Each unit is laid out with a head start of positions before its tiles, about what changing over
// to it costs in tiles, so that shares of many short units are smaller: 3 where the lanes share
// their tiles, and a tile takes the products of both, else 4.  Batches of 128 to 8191 tokens a
// sequence, 2 / 3 / 4 / 5 positions: shared bf16 101.1 / 98.0 / 98.9 / 100.0 us, shared fp8 133.4 /
// 128.9 / 130.9 / 131.7; 3 / 4 / 5 / 6: up to 128 columns fp8 141.9 / 133.3 / 134.4 / -, bf16 110.0 /
// 110.7 / 111.1 / 112.6.
__host__ __device__ constexpr int tree_pad(int cols) { return cols > 128 ? 3 : 4; }
__host__ __device__ inline int64_t tree_unit_len(int64_t tiles, int cols) { return tiles > 0 ? tiles + tree_pad(cols) : 0; }

// Group whose range holds position x of `total`.
__host__ __device__ inline int64_t tree_group_of(int64_t x, int64_t total, int64_t groups) {
    return ((x + 1) * groups - 1) / total;
}

bool tree_tc_eligible(int D, int kv_dtype);
cudaError_t launch_tree_tc(const TreeContext &a, int bs, int kv_dtype, cudaStream_t stream);

}  // namespace pa
