// Rotary positions fused with the cache append (pa_draft.h).
//
// A pair (x, x') of a head at position p is a complex number turned by the angle p f_j:
//   y = x cos - x' sin,  y' = x' cos + x sin.
// The frequency is held as a 64-bit fraction of a turn, F_j = f_j / 2 pi in units of
// 2^-64, so p F_j mod 2^64 is the angle with its whole turns removed exactly: one wide
// integer product instead of a 64-bit floating-point reduction (GB300 has two fp64 lanes
// per SM and clock), and no loss at far positions (the error is p 2^-65 turns; an fp32
// product p f_j is already 0.06 radians off at a million positions).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "pa_draft.h"
#include "pa_internal.cuh"

namespace pa {
namespace {

// Tokens per CTA; a thread has kBatch rows in flight, four or (layout 2) one: 8192 tokens take 56.3 us (4 tokens 59.4, 8
// tokens 69.8; 1 token 56.4; two rows in flight 56.8).
constexpr int kTokens = 2;
constexpr int kThreadsPerToken = 64;
constexpr int kThreads = kTokens * kThreadsPerToken;

struct RotaryArgs {
    uint16_t *q_out, *k_out;
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;
    const int64_t *slots, *positions;
    const uint64_t *table;
    int *err_flag;
    float factor;
    int rot, T, Hq, Hkv, bs, N;
    int rows;           // Hq + Hkv, + Hkv value rows when appending
    int rows_per_cta;   // a multiple of the rows a CTA takes at once
};

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight 8-bit codes of a row with this scale: the cache's rounding rules.
template <int KV>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
    uint32_t code[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float u = __fdiv_rn(x[e], scale), w = __fdiv_rn(x[e + 1], scale);
        uint32_t two;
        if constexpr (KV == PA_KV_FP8) {
            two = __nv_cvt_float2_to_fp8x2(make_float2(u, w), __NV_SATFINITE, __NV_E4M3);
        } else {
            // The sum with 1.5 x 2^23 rounds to an integer, ties to even, and leaves it in the low
            // bits (float-to-int conversions took 2.4 us more for 6000 tokens).
            const float i0 = __fadd_rn(fminf(fmaxf(u, -127.f), 127.f), 12582912.f), i1 = __fadd_rn(fminf(fmaxf(w, -127.f), 127.f), 12582912.f);
            two = (__float_as_uint(i0) & 0xffu) | ((__float_as_uint(i1) & 0xffu) << 8);
        }
        code[e / 4] |= two << (8 * (e & 2));
    }
    return make_uint2(code[0], code[1]);
}

// A CTA takes kTokens tokens, 64 threads each: D / 16 lanes per head row, a lane two 16-byte
// pieces of it, so that the partners of a pair meet in one lane, and the lane's cosines and
// sines serve all the rows it visits.
// LAYOUT: 0 = half (rot_dim / 2 a multiple of 8: pieces c and c + rot_dim / 16, the rest of
// the head in the other lanes), 1 = interleaved (neighbouring pieces), 2 = half with any
// other rot_dim (neighbouring pieces, partners read again from L1, by words where they align).
// Bounds: HBM beyond a few hundred tokens.  8192 tokens of 64 + 8 + 8 heads, 336 MB, 56.3 us:
// 5.97 TB/s, 0.88 of the measured copy rate; drafted rows, without a cache: 302 MB, 48.2 us.  (66.5 us
// with one piece a lane and partners through shuffles, when the instructions were most of the
// time.)  An fp8 cache takes longer for fewer bytes, 319 MB, 65.3 us, and the more so the more rows
// are quantised: 32 + 32 + 32 heads, 338 MB, 87.7 us.  Layout 2 is bound by its partners' loads:
// 6000 tokens of the first heads with rot_dim 20 take 59.4 us, interleaved 41.5 (two bytes at a time
// and two rows in flight, in more registers, 97.6).
template <int D, int KV, int LAYOUT>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    constexpr int LPR = D / 16;                      // lanes per row
    constexpr int SLOTS = kThreadsPerToken / LPR;    // rows of a token at once
    constexpr int kBatch = LAYOUT == 2 ? 1 : 4;
    __shared__ float2 s_cs[kTokens][D / 2];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, half = a.rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    for (int i = tid; i < kTokens * half; i += kThreads) {
        const int tt = i / half, j = i % half;
        if (t0 + tt >= a.T) break;
        const uint64_t phase = (uint64_t)a.positions[t0 + tt] * a.table[j];
        // the nearest quarter turn, and the signed rest in half turns: at most 1/4, so its fp32
        // rounding is 2^-27 of a half turn
        const uint32_t quarter = (uint32_t)((phase + 0x2000000000000000ull) >> 62);
        const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));
        float s, c;
        sincospif((float)rest * 1.0842021724855044e-19f, &s, &c);  // 2^-63
        const float cq = quarter & 1 ? -s : c, sq = quarter & 1 ? c : s;
        s_cs[tt][j] = make_float2((quarter & 2 ? -cq : cq) * a.factor, (quarter & 2 ? -sq : sq) * a.factor);
    }
    const int tt = tid / kThreadsPerToken, in = tid % kThreadsPerToken;
    const int64_t t = t0 + tt;
    const bool real = t < a.T;
    const bool append = a.k_cache != nullptr;
    const int64_t slot = append && real ? a.slots[t] : -1;
    __syncthreads();
    if (!real) return;
    const int c = in % LPR, slot0 = in / LPR;
    const unsigned gmask = ((1u << LPR) - 1u) << ((tid & 31) / LPR * LPR);
    // the lane's pieces (units of 8 elements), and whether pairs in them are turned
    const int rotated = a.rot / 16;  // LAYOUT 0: lanes with pairs
    const bool paired = LAYOUT != 0 || c < rotated;
    const int p0 = LAYOUT == 0 ? (paired ? c : 2 * c) : 2 * c, p1 = LAYOUT == 0 && paired ? c + rotated : p0 + 1;
    // cosines and sines: of pair e in both pieces (LAYOUT 0), of pairs 2e, 2e + 1 (1), or of
    // element e, signed (2; elements not turned: 1 and 0)
    constexpr int NC = LAYOUT == 2 ? 16 : 8;
    float cs[NC], sn[NC];
#pragma unroll
    for (int e = 0; e < NC; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
        if constexpr (LAYOUT == 2) {
            const int i = 16 * c + e;
            if (i < a.rot) {
                const float2 w = s_cs[tt][i < half ? i : i - half];
                cs[e] = w.x;
                sn[e] = i < half ? -w.y : w.y;
            }
        } else {
            const int j = LAYOUT == 0 ? 8 * p0 + e : 8 * c + e;
            if (paired && j < half) {
                const float2 w = s_cs[tt][j];
                cs[e] = w.x;
                sn[e] = w.y;
            }
        }
    }
    // 32-bit words of the two pieces that hold turned elements (bf16 words that do not keep
    // their bits, NaN payloads among them)
    const int words0 = LAYOUT == 0 ? (paired ? 4 : 0) : min(max((a.rot - 8 * p0) / 2, 0), 4);
    const int words1 = LAYOUT == 0 ? (paired ? 4 : 0) : min(max((a.rot - 8 * p1) / 2, 0), 4);
    const bool store = slot >= 0 && slot < (int64_t)a.N * a.bs;
    if (append && blockIdx.y == 0 && in == 0 && slot >= (int64_t)a.N * a.bs && a.err_flag)
        atomicOr(a.err_flag, PA_FLAG_SLOT_OUT_OF_RANGE);
    const int64_t blk = store ? slot / a.bs : 0;
    const int off = store ? (int)(slot % a.bs) : 0;

    auto rotate = [&](const uint4 &r0, const uint4 &r1, const float (&part)[LAYOUT == 2 ? 16 : 1], float (&x)[8], float (&y)[8]) {
        unpack8(r0, x);
        unpack8(r1, y);
        if constexpr (LAYOUT == 0) {
            if (paired) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = x[e], w = y[e];
                    x[e] = fmaf(-w, sn[e], u * cs[e]);
                    y[e] = fmaf(u, sn[e], w * cs[e]);
                }
            }
        } else if constexpr (LAYOUT == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e < words0) {
                    const float u = x[2 * e], w = x[2 * e + 1];
                    x[2 * e] = fmaf(-w, sn[e], u * cs[e]);
                    x[2 * e + 1] = fmaf(u, sn[e], w * cs[e]);
                }
                if (e < words1) {
                    const float u = y[2 * e], w = y[2 * e + 1];
                    y[2 * e] = fmaf(-w, sn[4 + e], u * cs[4 + e]);
                    y[2 * e + 1] = fmaf(u, sn[4 + e], w * cs[4 + e]);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (16 * c + e < a.rot) x[e] = fmaf(part[e], sn[e], x[e] * cs[e]);
                if (16 * c + 8 + e < a.rot) y[e] = fmaf(part[8 + e], sn[8 + e], y[e] * cs[8 + e]);
            }
        }
    };
    auto keep = [](const uint4 &raw, uint4 w, int words) {
        if (words < 1) w.x = raw.x;
        if (words < 2) w.y = raw.y;
        if (words < 3) w.z = raw.z;
        if (words < 4) w.w = raw.w;
        return w;
    };
    // KIND 0: query rows, 1: key rows, 2: value rows; head h of this token at src + h D
    auto rows = [&](auto kind, int begin, int end, const uint16_t *src, uint16_t *out, void *cache, float *scales) {
        constexpr int KIND = decltype(kind)::value;
        src += (int64_t)(begin + slot0) * D;
        if (out) out += (int64_t)(begin + slot0) * D;
        int64_t row = (blk * a.Hkv + begin + slot0) * a.bs + off;
        const int64_t row_step = (int64_t)SLOTS * a.bs;
        for (int h = begin + slot0; h < end; h += SLOTS * kBatch) {
            uint4 raw[kBatch][2];
            float part[LAYOUT == 2 && KIND < 2 ? kBatch : 1][LAYOUT == 2 ? 16 : 1];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (h + b * SLOTS >= end) break;
                raw[b][0] = *reinterpret_cast<const uint4 *>(src + b * SLOTS * D + 8 * p0);
                raw[b][1] = *reinterpret_cast<const uint4 *>(src + b * SLOTS * D + 8 * p1);
                if constexpr (LAYOUT == 2 && KIND < 2) {
                    if (half % 2 == 0) {  // two partners to a word
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const int i = 16 * c + e;
                            const uint32_t w = i < a.rot ? *reinterpret_cast<const uint32_t *>(src + b * SLOTS * D + (i < half ? i + half : i - half)) : 0u;
                            part[b][e] = __uint_as_float(w << 16);
                            part[b][e + 1] = __uint_as_float(w & 0xffff0000u);
                        }
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int i = 16 * c + e;
                        part[b][e] = i < a.rot ? __uint_as_float((uint32_t)src[b * SLOTS * D + (i < half ? i + half : i - half)] << 16) : 0.f;
                    }
                }
            }
            // a row may be rotated in place: all its lanes have read it before one writes
            if (LAYOUT == 2) __syncwarp(gmask);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (h + b * SLOTS >= end) break;
                float x[8], y[8];
                uint4 w0 = raw[b][0], w1 = raw[b][1];
                if constexpr (KIND < 2) {
                    rotate(raw[b][0], raw[b][1], part[LAYOUT == 2 ? b : 0], x, y);
                    w0 = keep(w0, pack8(x), words0);
                    w1 = keep(w1, pack8(y), words1);
                    if (KIND == 0 || out) {
                        *reinterpret_cast<uint4 *>(out + b * SLOTS * D + 8 * p0) = w0;
                        *reinterpret_cast<uint4 *>(out + b * SLOTS * D + 8 * p1) = w1;
                    }
                } else if constexpr (KV != PA_KV_BF16) {
                    unpack8(w0, x);
                    unpack8(w1, y);
                }
                if (KIND == 0 || !store) continue;
                const int64_t at = (row + b * row_step) * D;
                if constexpr (KV == PA_KV_BF16) {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(cache) + at + 8 * p0) = w0;
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(cache) + at + 8 * p1) = w1;
                } else {
                    float amax = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(x[e]), fabsf(y[e])));
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(gmask, amax, o));
                    const float scale = amax > 0.f ? __fdiv_rn(amax, KV == PA_KV_FP8 ? 448.f : 127.f) : 1.f;
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + at + 8 * p0) = codes8<KV>(x, scale);
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + at + 8 * p1) = codes8<KV>(y, scale);
                    if (c == 0) scales[row + b * row_step] = scale;
                }
            }
            src += SLOTS * kBatch * D;
            if (out) out += SLOTS * kBatch * D;
            row += row_step * kBatch;
        }
    };
    const int lo = blockIdx.y * a.rows_per_cta, hi = min(a.rows, lo + a.rows_per_cta);
    if (lo < a.Hq)
        rows(std::integral_constant<int, 0>(), lo, min(hi, a.Hq), a.q + t * a.q_stride, a.q_out + t * a.Hq * D, nullptr, nullptr);
    const int klo = max(lo - a.Hq, 0), khi = min(hi - a.Hq, a.Hkv);
    if (klo < khi)
        rows(std::integral_constant<int, 1>(), klo, khi, a.k + t * a.k_stride, a.k_out ? a.k_out + t * a.Hkv * D : nullptr, a.k_cache,
             a.k_scale);
    const int vlo = max(lo - a.Hq - a.Hkv, 0), vhi = hi - a.Hq - a.Hkv;
    if (vlo < vhi && store)
        rows(std::integral_constant<int, 2>(), vlo, vhi, a.v + t * a.v_stride, nullptr, a.v_cache, a.v_scale);
}

template <int D, int KV>
cudaError_t launch_rotary_typed(const RotaryArgs &a, int layout, dim3 grid, cudaStream_t stream) {
    auto *k = layout == 0 ? rotary_kernel<D, KV, 0> : layout == 1 ? rotary_kernel<D, KV, 1> : rotary_kernel<D, KV, 2>;
    return launch_dependent(k, grid, dim3(kThreads), 0, stream, a);
}

template <int D>
cudaError_t launch_rotary(const RotaryArgs &a, int kv_dtype, int layout, dim3 grid, cudaStream_t stream) {
    if (kv_dtype == PA_KV_INT8) return launch_rotary_typed<D, PA_KV_INT8>(a, layout, grid, stream);
    if (kv_dtype == PA_KV_FP8) return launch_rotary_typed<D, PA_KV_FP8>(a, layout, grid, stream);
    return launch_rotary_typed<D, PA_KV_BF16>(a, layout, grid, stream);
}

// Whether [a, a + n) and [b, b + m) bytes overlap.
bool overlap(const void *a, int64_t n, const void *b, int64_t m) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_rotary_frequencies(int rot_dim, double base, int scaling, double factor, double original_context,
                                double p0, double p1, double *inv_freq, double *attention_factor) {
    const char *fn = "pa_rotary_frequencies";
    clear_error();
    if (!inv_freq) return fail(PA_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (scaling < PA_ROTARY_PLAIN || scaling > PA_ROTARY_WAVELENGTH)
        return fail(PA_ERR_UNSUPPORTED, "%s: scaling %d not supported", fn, scaling);
    if (rot_dim < (scaling == PA_ROTARY_BASE ? 4 : 2) || rot_dim % 2 != 0)
        return fail(PA_ERR_INVALID_ARG, "%s: rot_dim = %d", fn, rot_dim);
    if (!(base > 1.0) || !std::isfinite(base)) return fail(PA_ERR_INVALID_ARG, "%s: base = %g", fn, base);
    if (scaling != PA_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return fail(PA_ERR_INVALID_ARG, "%s: factor = %g", fn, factor);
    const bool parts = scaling == PA_ROTARY_RAMP || scaling == PA_ROTARY_WAVELENGTH;
    if (parts && (!(original_context > 0.0) || !std::isfinite(original_context) || !std::isfinite(p0) || !std::isfinite(p1) ||
                  !(p0 > 0.0) || !(p1 > 0.0) || (scaling == PA_ROTARY_RAMP ? !(p0 > p1) : !(p1 > p0))))
        return fail(PA_ERR_INVALID_ARG, "%s: original_context = %g, p0 = %g, p1 = %g", fn, original_context, p0, p1);
    constexpr double kTwoPi = 6.283185307179586476925;
    const int n = rot_dim / 2;
    const double b = scaling == PA_ROTARY_BASE ? base * std::pow(factor, (double)rot_dim / (rot_dim - 2)) : base;
    // RAMP: the (fractional) pair index that turns `turns` times within original_context
    auto pair_of = [&](double turns) { return n * std::log(original_context / (turns * kTwoPi)) / std::log(b); };
    double low = 0.0, high = 0.0;
    if (scaling == PA_ROTARY_RAMP) {
        low = std::fmax(std::floor(pair_of(p0)), 0.0);
        high = std::fmin(std::ceil(pair_of(p1)), (double)(rot_dim - 1));
        if (!(high > low)) high = low + 1e-3;  // a step instead of a ramp
    }
    for (int j = 0; j < n; ++j) {
        const double f = std::pow(b, -(double)j / n);
        double g = f;
        if (scaling == PA_ROTARY_LINEAR) g = f / factor;
        if (scaling == PA_ROTARY_RAMP) {
            const double r = std::fmin(std::fmax((j - low) / (high - low), 0.0), 1.0);
            g = f / factor * r + f * (1.0 - r);
        }
        if (scaling == PA_ROTARY_WAVELENGTH) {
            const double turns = original_context * f / kTwoPi;  // original_context / wavelength
            const double r = std::fmin(std::fmax((turns - p0) / (p1 - p0), 0.0), 1.0);
            g = f / factor * (1.0 - r) + f * r;
        }
        inv_freq[j] = g;
    }
    if (attention_factor) *attention_factor = scaling == PA_ROTARY_RAMP ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return PA_OK;
}

pa_status pa_rotary_table(const double *inv_freq, int n, uint64_t *table) {
    const char *fn = "pa_rotary_table";
    clear_error();
    if (n < 0) return fail(PA_ERR_INVALID_ARG, "%s: n = %d", fn, n);
    if (n > 0 && (!inv_freq || !table)) return fail(PA_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (int j = 0; j < n; ++j)
        if (!std::isfinite(inv_freq[j])) return fail(PA_ERR_INVALID_ARG, "%s: inv_freq[%d] is not finite", fn, j);
    for (int j = 0; j < n; ++j) {
        // the size without its whole turns (exact), then the sign: modulo one turn
        double turns = std::fabs(inv_freq[j]) / 6.283185307179586476925;
        turns -= std::floor(turns);
        const double u = std::nearbyint(turns * 18446744073709551616.0);
        const uint64_t t = u >= 18446744073709551616.0 ? 0 : (uint64_t)u;
        table[j] = inv_freq[j] < 0.0 ? 0 - t : t;
    }
    return PA_OK;
}

pa_status pa_rotary_and_cache(pa_bf16 *query_out, pa_bf16 *key_out, const pa_bf16 *query, int64_t query_stride,
                              const pa_bf16 *key, int64_t key_stride, const pa_bf16 *value, int64_t value_stride,
                              void *k_cache, void *v_cache, float *k_scale, float *v_scale, int kv_dtype,
                              const int64_t *slot_mapping, const int64_t *positions, const uint64_t *table,
                              int rot_dim, int interleaved, float attention_factor, int T, int Hq, int Hkv, int D,
                              int bs, int N, int *err_flag, void *stream) {
    const char *fn = "pa_rotary_and_cache";
    clear_error();
    const bool append = k_cache != nullptr || v_cache != nullptr;
    if (T < 0) return fail(PA_ERR_INVALID_ARG, "%s: T = %d is negative", fn, T);
    if (Hq <= 0 || Hkv <= 0) return fail(PA_ERR_INVALID_ARG, "%s: Hq = %d, Hkv = %d", fn, Hq, Hkv);
    if (D != 64 && D != 128) return fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d not supported (64 or 128)", fn, D);
    if (Hq > 65536 || Hkv > 65536) return fail(PA_ERR_UNSUPPORTED, "%s: too many heads", fn);
    if (rot_dim < 2 || rot_dim > D || rot_dim % 2 != 0)
        return fail(PA_ERR_INVALID_ARG, "%s: rot_dim = %d (even, 2 .. head_dim)", fn, rot_dim);
    if (!std::isfinite(attention_factor)) return fail(PA_ERR_INVALID_ARG, "%s: attention_factor must be finite", fn);
    if (append) {
        pa_status st = check_cache_shape(fn, Hkv, D, bs, N);
        if (st != PA_OK) return st;
        if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_INT8 && kv_dtype != PA_KV_FP8)
            return fail(PA_ERR_UNSUPPORTED, "%s: kv dtype %d not supported", fn, kv_dtype);
    }
    const int64_t qw = (int64_t)Hq * D, kw = (int64_t)Hkv * D;
    constexpr int64_t kMost = (int64_t)1 << 40;
    if (query_stride < qw || key_stride < kw || query_stride % 8 != 0 || key_stride % 8 != 0 || query_stride > kMost ||
        key_stride > kMost)
        return fail(PA_ERR_INVALID_ARG, "%s: token strides must be multiples of 8, at least heads * head_dim", fn);
    if (append && (value_stride < kw || value_stride % 8 != 0 || value_stride > kMost))
        return fail(PA_ERR_INVALID_ARG, "%s: token strides must be multiples of 8, at least heads * head_dim", fn);
    if (T == 0) return PA_OK;
    if (!query_out || !query || !key || !positions || !table || (!append && !key_out))
        return fail(PA_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (append && (!k_cache || !v_cache || !value || !slot_mapping || (kv_dtype != PA_KV_BF16 && (!k_scale || !v_scale))))
        return fail(PA_ERR_INVALID_ARG, "%s: null pointer (appending)", fn);
    if (!aligned16(query_out) || !aligned16(key_out) || !aligned16(query) || !aligned16(key))
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    if (append && (!aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache) ||
                   (kv_dtype != PA_KV_BF16 && (!aligned16(k_scale) || !aligned16(v_scale)))))
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    // an output may be its own dense input; any other overlap would be read after it is written
    const int64_t qo = 2 * (int64_t)T * qw, ko = 2 * (int64_t)T * kw;
    const int64_t qi = 2 * ((T - 1) * query_stride + qw), ki = 2 * ((T - 1) * key_stride + kw);
    const int64_t vi = append ? 2 * ((T - 1) * value_stride + kw) : 0;
    const bool q_same = query_out == query && query_stride == qw, k_same = key_out == key && key_stride == kw;
    if ((!q_same && overlap(query_out, qo, query, qi)) || overlap(query_out, qo, key, ki) ||
        (!k_same && overlap(key_out, ko, key, ki)) || overlap(key_out, ko, query, qi) || overlap(query_out, qo, key_out, ko) ||
        (append && (overlap(query_out, qo, value, vi) || overlap(key_out, ko, value, vi))))
        return fail(PA_ERR_INVALID_ARG, "%s: an output overlaps an input (only whole dense tensors may be rotated in place)", fn);
    RotaryArgs a{};
    a.q_out = query_out;
    a.k_out = key_out;
    a.q = query;
    a.k = key;
    a.v = value;
    a.q_stride = query_stride;
    a.k_stride = key_stride;
    a.v_stride = value_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.slots = slot_mapping;
    a.positions = positions;
    a.table = table;
    a.err_flag = err_flag;
    a.factor = attention_factor;
    a.rot = rot_dim;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.bs = bs;
    a.N = N;
    a.rows = Hq + Hkv + (append ? Hkv : 0);
    // enough CTAs for one wave at two per SM, else all rows of a token in one CTA (its
    // cosines are computed once)
    const int step = kThreadsPerToken / (D / 16);  // rows of a token at once
    const int groups = (T + kTokens - 1) / kTokens;
    const int most = (a.rows + step - 1) / step;
    const int split = std::min(most, std::max(1, 304 / groups));
    a.rows_per_cta = (most + split - 1) / split * step;
    const dim3 grid(groups, (a.rows + a.rows_per_cta - 1) / a.rows_per_cta);
    const int layout = interleaved ? 1 : (rot_dim / 2) % 8 == 0 ? 0 : 2;
    if (!append) kv_dtype = PA_KV_BF16;
    D == 128 ? launch_rotary<128>(a, kv_dtype, layout, grid, (cudaStream_t)stream)
             : launch_rotary<64>(a, kv_dtype, layout, grid, (cudaStream_t)stream);
    return check_launch(fn);
}

}  // extern "C"
