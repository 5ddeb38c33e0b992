// mxq_matvec.hip -- products of few rows with NVFP4 weights: a decode step's
// projections (dense) and experts (expert-sorted rows, the gate/up pair with
// SwiGLU in the epilogue).  C[m][n] = s_x[m] s_b[n] sum_k x[m][k]
// dec(code[n][k]) dec(block scale[n][k/16]), fp32 accumulation.
#include "mxq_layer.h"
#include "mxq_layer_device.h"

namespace mxq {

namespace {

constexpr int MV_WAVES = 4;

// The 16 values of block b of activation row r (NVFP4: without its FP32
// scale).
template <int FMT>
__device__ __forceinline__ void act_block(float (&v)[16], const ActX &x, int64_t r, int64_t b,
                                          int64_t K)
{
    if constexpr (FMT == MXQ_X_BF16) {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(x.x) + r * K + 16 * b;
#pragma unroll
        for (int i = 0; i < 16; i++)
            v[i] = u2f((uint32_t)p[i] << 16);
    } else if constexpr (FMT == MXQ_X_F32) {
        const float *p = reinterpret_cast<const float *>(x.x) + r * K + 16 * b;
#pragma unroll
        for (int i = 0; i < 16; i++)
            v[i] = p[i];
    } else {
        const uint2 c = ld8(reinterpret_cast<const uint8_t *>(x.x) + r * (K >> 1) + 8 * b);
        const float d = e4m3_value(x.bs[r * (K >> 4) + b]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2_t p = e2m1_values(((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu);
            v[2 * i] = p[0] * d;
            v[2 * i + 1] = p[1] * d;
        }
    }
}

// Summed in 64 bits: partial sums neither overflow nor underflow where the
// scaled result does not.
template <int FMT>
__device__ __forceinline__ float row_product(const ActX &x, int64_t r, const WeightB &w,
                                             int64_t n, int64_t K, float scale)
{
    double sum = 0.0;
    for (int64_t b = lane_id(); b < K / 16; b += 64) {
        float v[16];
        act_block<FMT>(v, x, r, b, K);
        const uint2 c = ld8(w.codes + n * (K >> 1) + 8 * b);
        const float d = e4m3_value(w.bs[n * (K >> 4) + b]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2_t p = e2m1_values(((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu);
            sum = __builtin_fma((double)(p[0] * d), (double)v[2 * i], sum);
            sum = __builtin_fma((double)(p[1] * d), (double)v[2 * i + 1], sum);
        }
    }
    for (uint32_t m = 1; m < 64; m <<= 1)
        sum += lane_get(sum, lane_id() ^ m);
    return (float)(sum * (double)scale);
}

template <bool BF16_OUT, int FMT>
__global__ void __launch_bounds__(64 * MV_WAVES) nvfp4_matvec_kernel(
    ActX x, WeightB b, const float *scales, int64_t rows_per_scale, int64_t M, int64_t N,
    int64_t K, void *c)
{
    const int64_t n = (int64_t)wg_id() * MV_WAVES + wave_in_group();
    if (n >= N)
        return;
    const float sb = scales[n / rows_per_scale];
    for (int64_t m = 0; m < M; m++) {
        const float s = row_product<FMT>(x, m, b, n, K, FMT == MXQ_X_NVFP4 ? sb * x.s[m] : sb);
        if (lane_id() == 0)
            st_elem<BF16_OUT>(c, m * N + n, s);
    }
}

template <bool BF16_OUT, int FMT>
__global__ void __launch_bounds__(64 * MV_WAVES) nvfp4_expert_kernel(
    ActX x, int64_t n_tokens, const int64_t *row_tokens, const int64_t *seg_offsets,
    int64_t n_tiles, int64_t total_rows, WeightB w, WeightB up, const float *scales, int64_t N,
    int64_t K, void *c)
{
    const int64_t e = wg_id() / (uint32_t)n_tiles, tile = wg_id() % (uint32_t)n_tiles;
    const int64_t n = tile * MV_WAVES + wave_in_group();
    if (n >= N)
        return;
    int64_t r0 = seg_offsets[e], r1 = seg_offsets[e + 1];
    r0 = r0 < 0 ? 0 : r0;
    r1 = r1 > total_rows ? total_rows : r1;
    for (int64_t r = r0; r < r1; r++) {
        int64_t xr = r;
        if (row_tokens) {
            xr = row_tokens[r];
            xr = xr < 0 ? 0 : xr >= n_tokens ? n_tokens - 1 : xr;
        }
        const float s = (FMT == MXQ_X_NVFP4 ? x.s[xr] : 1.0f) * scales[e];
        float g = row_product<FMT>(x, xr, w, e * N + n, K, s);
        if (up.codes) {
            const float u = row_product<FMT>(x, xr, up, e * N + n, K, s);
            g = silu_f32(g) * u;
        }
        if (lane_id() == 0)
            st_elem<BF16_OUT>(c, r * N + n, g);
    }
}

}  // namespace

#define MV_DISPATCH(KERNEL, ...)                                                                  \
    do {                                                                                          \
        if (bf16_out) {                                                                           \
            if (x.fmt == MXQ_X_BF16)                                                              \
                hipLaunchKernelGGL((KERNEL<true, MXQ_X_BF16>), __VA_ARGS__);                      \
            else if (x.fmt == MXQ_X_F32)                                                          \
                hipLaunchKernelGGL((KERNEL<true, MXQ_X_F32>), __VA_ARGS__);                       \
            else                                                                                  \
                hipLaunchKernelGGL((KERNEL<true, MXQ_X_NVFP4>), __VA_ARGS__);                     \
        } else {                                                                                  \
            if (x.fmt == MXQ_X_BF16)                                                              \
                hipLaunchKernelGGL((KERNEL<false, MXQ_X_BF16>), __VA_ARGS__);                     \
            else if (x.fmt == MXQ_X_F32)                                                          \
                hipLaunchKernelGGL((KERNEL<false, MXQ_X_F32>), __VA_ARGS__);                      \
            else                                                                                  \
                hipLaunchKernelGGL((KERNEL<false, MXQ_X_NVFP4>), __VA_ARGS__);                    \
        }                                                                                         \
    } while (0)

hipError_t launch_nvfp4_matvec(const ActX &x, const WeightB &b, const float *scales,
                               int64_t rows_per_scale, int64_t M, int64_t N, int64_t K,
                               bool bf16_out, void *c, hipStream_t stream)
{
    const dim3 grid((unsigned)((N + MV_WAVES - 1) / MV_WAVES)), block(64 * MV_WAVES);
    MV_DISPATCH(nvfp4_matvec_kernel, grid, block, 0, stream, x, b, scales, rows_per_scale, M, N,
                K, c);
    return hipGetLastError();
}

bool expert_grid_ok(int64_t n_groups, int64_t, int64_t N)
{
    return n_groups * ((N + MV_WAVES - 1) / MV_WAVES) < ((int64_t)1 << 24);
}

hipError_t launch_nvfp4_expert_matvec(const ActX &x, int64_t n_tokens, const int64_t *row_tokens,
                                      const int64_t *seg_offsets, int64_t n_groups,
                                      int64_t total_rows, const WeightB &w, const WeightB &up,
                                      const float *scales, int64_t N, int64_t K, bool bf16_out,
                                      void *c, hipStream_t stream)
{
    const int64_t n_tiles = (N + MV_WAVES - 1) / MV_WAVES;
    const dim3 grid((unsigned)(n_tiles * n_groups)), block(64 * MV_WAVES);
    MV_DISPATCH(nvfp4_expert_kernel, grid, block, 0, stream, x, n_tokens, row_tokens, seg_offsets,
                n_tiles, total_rows, w, up, scales, N, K, c);
    return hipGetLastError();
}

}  // namespace mxq
