// Cached rows read back into dense ones (pa.h): the inverse of the append.
//
// A lane takes eight entries of a row, 16 bytes of a bf16 cache or 8 of an 8-bit one, and
// writes 16 bytes; a warp's lanes are neighbours in the token's rows, so what it writes is one
// run of 512 bytes and what it reads whole rows of 64 to 256.  kBatch pieces are in flight in a
// thread.  Bound by HBM beyond a few thousand tokens: 131072 tokens of 8 heads take 138 us from an fp8 cache (815 MB, 5.9 TB/s,
// 0.88 of the measured copy rate), 139 from int8, 159 from bf16 (1.07 GB, 6.7 TB/s, the copy rate itself); 8192 from bf16 13.1.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;

struct GatherArgs {
    uint16_t *key, *value;
    int64_t key_stride, value_stride;
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int64_t *slots;
    int *err_flag;
    int T, Hkv, bs_shift;
    int64_t slots_end;
    int tokens;  // of a CTA
};

// Eight codes times their scale, rounded once.
template <int KV>
__device__ __forceinline__ uint4 dequantise(uint2 codes, float scale) {
    const uint32_t c[2] = {codes.x, codes.y};
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = c[i / 2] >> (16 * (i & 1));
        float2 x;
        if constexpr (KV == PA_KV_FP8) {
            x = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3)));
        } else {
            x = make_float2((float)(int8_t)two, (float)(int8_t)(two >> 8));
        }
        const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(x.x, scale), __fmul_rn(x.y, scale));
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, int KV>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ GatherArgs a) {
    constexpr int kPieces = D / 8;  // of a row
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int per_side = a.Hkv * kPieces, per_token = 2 * per_side;  // keys' pieces, then values'
    const int n = (int)min((int64_t)a.tokens, a.T - t0) * per_token;
    for (int base = threadIdx.x; base < n; base += kThreads * kBatch) {
        uint4 whole[kBatch];
        uint2 codes[kBatch];
        float scale[kBatch];
        uint16_t *to[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = base + b * kThreads;
            to[b] = nullptr;
            if (i >= n) continue;
            const int tt = i / per_token, in = i % per_token;
            const bool is_value = in >= per_side;
            const int piece = is_value ? in - per_side : in, h = piece / kPieces, c = piece % kPieces;
            const int64_t t = t0 + tt, slot = a.slots[t];
            if (slot < 0) continue;
            if (slot >= a.slots_end) {
                if (in == 0 && a.err_flag) atomicOr(a.err_flag, PA_FLAG_SLOT_OUT_OF_RANGE);
                continue;
            }
            const int64_t row = (((slot >> a.bs_shift) * a.Hkv + h) << a.bs_shift) + (slot & ((1 << a.bs_shift) - 1));
            const void *cache = is_value ? a.v_cache : a.k_cache;
            if constexpr (KV == PA_KV_BF16) {
                whole[b] = __ldg(static_cast<const uint4 *>(cache) + row * kPieces + c);
            } else {
                codes[b] = __ldg(static_cast<const uint2 *>(cache) + row * kPieces + c);
                scale[b] = __ldg((is_value ? a.v_scale : a.k_scale) + row);
            }
            to[b] = (is_value ? a.value + t * a.value_stride : a.key + t * a.key_stride) + piece * 8;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (!to[b]) continue;
            if constexpr (KV != PA_KV_BF16) whole[b] = dequantise<KV>(codes[b], scale[b]);
            *reinterpret_cast<uint4 *>(to[b]) = whole[b];
        }
    }
}

// Whether [a, a + n) and [b, b + m) bytes overlap.
bool overlap(const void *a, int64_t n, const void *b, int64_t m) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_gather_cache(pa_bf16 *key_out, int64_t key_stride, pa_bf16 *value_out, int64_t value_stride,
                                     const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                                     int kv_dtype, const int64_t *slot_mapping, int T, int Hkv, int D, int bs, int N,
                                     int *err_flag, void *stream) {
    const char *fn = "pa_gather_cache";
    clear_error();
    if (T < 0) return fail(PA_ERR_INVALID_ARG, "%s: T = %d is negative", fn, T);
    pa_status st = check_cache_shape(fn, Hkv, D, bs, N);
    if (st != PA_OK) return st;
    if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_INT8 && kv_dtype != PA_KV_FP8)
        return fail(PA_ERR_UNSUPPORTED, "%s: kv dtype %d not supported", fn, kv_dtype);
    if (Hkv > 65536) return fail(PA_ERR_UNSUPPORTED, "%s: too many heads", fn);
    const int64_t row = (int64_t)Hkv * D;
    constexpr int64_t kMost = (int64_t)1 << 40;
    if (key_stride < row || value_stride < row || key_stride % 8 != 0 || value_stride % 8 != 0 || key_stride > kMost ||
        value_stride > kMost)
        return fail(PA_ERR_INVALID_ARG, "%s: token strides must be multiples of 8, at least Hkv * head_dim", fn);
    if (T == 0) return PA_OK;
    const bool scaled = kv_dtype != PA_KV_BF16;
    if (!key_out || !value_out || !k_cache || !v_cache || !slot_mapping || (scaled && (!k_scale || !v_scale)))
        return fail(PA_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(key_out) || !aligned16(value_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (scaled && (!aligned16(k_scale) || !aligned16(v_scale))))
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    const int64_t kb = 2 * ((T - 1) * key_stride + row), vb = 2 * ((T - 1) * value_stride + row);
    const int64_t cache = (int64_t)N * bs * row * (scaled ? 1 : 2);
    for (const void *c : {k_cache, v_cache})
        if (overlap(key_out, kb, c, cache) || overlap(value_out, vb, c, cache))
            return fail(PA_ERR_INVALID_ARG, "%s: an output overlaps the cache", fn);
    // rows of keys and values may lie in turn (slices of one tensor), but not on one another
    if (overlap(key_out, kb, value_out, vb)) {
        const int64_t apart = (int64_t)((uintptr_t)value_out - (uintptr_t)key_out) / 2 % key_stride;  // of a key's row to the next value's
        const int64_t gap = apart < 0 ? apart + key_stride : apart;
        if (key_stride != value_stride || gap < row || key_stride - gap < row)
            return fail(PA_ERR_INVALID_ARG, "%s: key_out overlaps value_out", fn);
    }
    GatherArgs a{};
    a.key = key_out;
    a.value = value_out;
    a.key_stride = key_stride;
    a.value_stride = value_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.slots = slot_mapping;
    a.err_flag = err_flag;
    a.T = T;
    a.Hkv = Hkv;
    a.bs_shift = bs == 32 ? 5 : 4;
    a.slots_end = (int64_t)N * bs;
    // a full batch a thread, but fewer tokens a CTA while the grid is short of two CTAs per SM
    const int per_token = 2 * Hkv * (D / 8);
    const int fair = (int)std::max<int64_t>(1, T / (2 * device_sms()));
    a.tokens = std::max(1, std::min(kThreads * kBatch / per_token, fair));
    const dim3 grid((unsigned)((T + a.tokens - 1) / a.tokens));
    auto launch = [&](auto *kernel) { launch_dependent(kernel, grid, dim3(kThreads), 0, (cudaStream_t)stream, a); };
    if (kv_dtype == PA_KV_BF16)
        launch(D == 128 ? gather_kernel<128, PA_KV_BF16> : gather_kernel<64, PA_KV_BF16>);
    else if (kv_dtype == PA_KV_INT8)
        launch(D == 128 ? gather_kernel<128, PA_KV_INT8> : gather_kernel<64, PA_KV_INT8>);
    else
        launch(D == 128 ? gather_kernel<128, PA_KV_FP8> : gather_kernel<64, PA_KV_FP8>);
    return check_launch(fn);
}
