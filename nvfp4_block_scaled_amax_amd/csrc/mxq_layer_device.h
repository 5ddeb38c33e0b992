// mxq_layer_device.h -- device helpers of the layer operators: exponentials,
// sums over wavefronts, typed element access.
#pragma once

#include "mxq_device.h"

namespace mxq {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr float LOG2E = 0x1.715476p+0f;           // fp32(log2 e)
constexpr float LOG2E_LO = 0x1.4ae0cp-26f;        // log2 e - LOG2E
constexpr float LN2 = 0x1.62e43p-1f;

// -inf as a bit test: logits and biases equal to it mark experts that are
// never selected.  NaN counts as -inf too.  The bits are hidden from the
// compiler as bits of a float: under -fno-honor-nans it may otherwise merge
// the test with a later comparison and lose the NaN.
__device__ __forceinline__ bool is_masked(float x)
{
    uint32_t u = f2u(x);
    asm("" : "+v"(u));
    return u == 0xFF800000u || (u & 0x7FFFFFFFu) > 0x7F800000u;
}

// e^x for finite x: v_exp_f32 (1 ulp) of the rounded x log2 e, corrected by
// the rounding error of that product, so the relative error does not grow
// with |x|.  Saturates at e^88.7 (the last finite value is e^88.72) and at 0.
__device__ __forceinline__ float exp_f32(float x)
{
    x = __builtin_amdgcn_fmed3f(x, -120.0f, 88.7f);
    const float t = x * LOG2E;
    const float err = __builtin_fmaf(x, LOG2E, -t) + x * LOG2E_LO;
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, err * LN2, e);
}

// e^(x - m) for finite x and m.  The difference is rounded to half a step of it,
// 2^-19 at 32 to 64, which the exponential would have as a relative error;
// what it leaves (exact, by the two sums' errors) joins the result.
__device__ __forceinline__ float exp_diff_f32(float x, float m)
{
    const float d = x - m, b = d - x;
    const float lost = (x - (d - b)) - (m + b);
    const float e = exp_f32(d);
    return d > -120.0f ? __builtin_fmaf(e, lost, e) : e;     // below, d may be infinite
}

// x sigmoid(x), the sigmoid from the exponential that does not overflow.
__device__ __forceinline__ float silu_f32(float x)
{
    const float e = exp_f32(x < 0.0f ? x : -x);
    return x * ((x < 0.0f ? e : 1.0f) / (1.0f + e));
}

// e^x in 64 bits: x = n ln 2 + r with |r| <= ln 2 / 2 (ln 2 split in two so
// that r is exact to 2^-60), Taylor's series to r^13 (the next term is below
// 2^-57), scaled by 2^n.
__device__ __forceinline__ double exp_f64(double x)
{
    x = x < -745.0 ? -745.0 : x > 709.0 ? 709.0 : x;
    const double n = __builtin_rint(x * 0x1.71547652b82fep+0);
    double r = __builtin_fma(n, -0x1.62e42fefa3800p-1, x);
    r = __builtin_fma(n, -0x1.ef35793c76730p-45, r);
    double p = 1.0 / 6227020800.0;
    p = __builtin_fma(p, r, 1.0 / 479001600.0);
    p = __builtin_fma(p, r, 1.0 / 39916800.0);
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// The value of another lane (any lane of the wavefront).
__device__ __forceinline__ uint32_t lane_get(uint32_t v, uint32_t src)
{
    return (uint32_t)__builtin_amdgcn_ds_bpermute((int)(src << 2), (int)v);
}
__device__ __forceinline__ int lane_get(int v, uint32_t src)
{
    return __builtin_amdgcn_ds_bpermute((int)(src << 2), v);
}
__device__ __forceinline__ float lane_get(float v, uint32_t src)
{
    return u2f(lane_get(f2u(v), src));
}
__device__ __forceinline__ double lane_get(double v, uint32_t src)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = lane_get((uint32_t)u, src), hi = lane_get((uint32_t)(u >> 32), src);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ float sum16_f32(float v)
{
    const uint2_t r = __builtin_amdgcn_permlane16_swap(f2u(v), f2u(v), false, false);
    return u2f(r[0]) + u2f(r[1]);
}
__device__ __forceinline__ float sum32_f32(float v)
{
    const uint2_t r = __builtin_amdgcn_permlane32_swap(f2u(v), f2u(v), false, false);
    return u2f(r[0]) + u2f(r[1]);
}
// Sum over the 16 lanes of a row, the same value in each of them: every step
// adds the two halves of a pair, and a + b = b + a.
__device__ __forceinline__ float row_sum_f32(float v)
{
    v += u2f(dpp<DPP_XOR1>(f2u(v)));
    v += u2f(dpp<DPP_XOR2>(f2u(v)));
    v += u2f(dpp<DPP_HALF_MIRROR>(f2u(v)));
    v += u2f(dpp<DPP_MIRROR>(f2u(v)));
    return v;
}
__device__ __forceinline__ float wave_sum_f32(float v)
{
    return sum32_f32(sum16_f32(row_sum_f32(v)));
}

// Element i of an array of BF16 or FP32 values.
template <bool BF16>
__device__ __forceinline__ float ld_elem(const void *p, int64_t i)
{
    if constexpr (BF16)
        return u2f((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16);
    else
        return reinterpret_cast<const float *>(p)[i];
}

// BF16 nearest-even of a finite value or an infinity.
__device__ __forceinline__ uint16_t bf16_rne(float f)
{
    const uint32_t u = f2u(f);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}
template <bool BF16>
__device__ __forceinline__ void st_elem(void *p, int64_t i, float v)
{
    if constexpr (BF16)
        reinterpret_cast<uint16_t *>(p)[i] = bf16_rne(v);
    else
        reinterpret_cast<float *>(p)[i] = v;
}

}  // namespace mxq
