// mxq_moe.hip -- routing tokens to experts and bringing expert rows back.
//
// Route: each token's top_k experts under softmax or sigmoid scores (with an
// optional balance bias and expert groups), their weights, and the index
// maps of the expert-sorted layout.  The selection is that of the exact
// scores: the order is decided in 64 bits.
#include "mxq_layer.h"
#include "mxq_layer_device.h"

namespace mxq {

namespace {

constexpr int ROUTE_WAVES = 4;                    // tokens per workgroup, one per wavefront
// Tokens per tile of the map kernels: 64-token words of a bit per (token,
// expert), WORDS of them per tile.
constexpr int MAP_WORDS = 4, MAP_TOKENS = 64 * MAP_WORDS;
constexpr int MAP_THREADS = 256;

struct RouteArgs {
    const void *logits;
    const float *bias;
    int64_t n_tokens;
    int n_experts, top_k, n_groups, topk_groups, group_topk;
    bool sigmoid, renorm;
    float scale;
    float *weights;
    int64_t *experts;
};

// The larger key, of equal keys the lower index; key -inf loses to nothing
// but another -inf.
__device__ __forceinline__ void argmax_step(double &v, int &i, double ov, int oi)
{
    if (ov > v || (ov == v && oi < i)) {
        v = ov;
        i = oi;
    }
}
__device__ __forceinline__ void wave_argmax(double &v, int &i, uint32_t lane)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        argmax_step(v, i, lane_get(v, lane ^ m), (int)lane_get((uint32_t)i, lane ^ m));
}
__device__ __forceinline__ double wave_sum_f64(double v, uint32_t lane)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        v += lane_get(v, lane ^ m);
    return v;
}

constexpr double NONE = -__builtin_inf();

// One wavefront routes one token; lane l holds experts l, l + 64, ...
template <bool BF16, int V>
__global__ void __launch_bounds__(64 * ROUTE_WAVES) moe_route_kernel(RouteArgs a)
{
    const uint32_t lane = lane_id();
    const int64_t t = (int64_t)wg_id() * ROUTE_WAVES + wave_in_group();
    if (t >= a.n_tokens)
        return;
    const int E = a.n_experts;
    double x[V], key[V];
    double m = NONE;
#pragma unroll
    for (int j = 0; j < V; j++) {
        const int e = 64 * j + (int)lane;
        float f = -__builtin_inff();
        if (e < E) {
            f = ld_elem<BF16>(a.logits, t * E + e);
            if (is_masked(f) || (a.bias && is_masked(a.bias[e])))
                f = -__builtin_inff();
            f = f < 3.402823466e+38f ? f : 3.402823466e+38f;
        }
        x[j] = (double)f;
        m = x[j] > m ? x[j] : m;
    }
    const bool by_logit = !a.bias && (a.n_groups == 1 || a.group_topk == 1);
    double denom = 1.0;
    if (!a.sigmoid) {
        int dummy = 0;
        wave_argmax(m, dummy, lane);
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < V; j++)
            s += x[j] == NONE ? 0.0 : exp_f64(x[j] - m);
        denom = wave_sum_f64(s, lane);
    }
    auto score = [&](double v) {
        return a.sigmoid ? 1.0 / (1.0 + exp_f64(-v)) : exp_f64(v - m) / denom;
    };
#pragma unroll
    for (int j = 0; j < V; j++) {
        const int e = 64 * j + (int)lane;
        key[j] = x[j];
        if (!by_logit && x[j] != NONE)
            key[j] = score(x[j]) + (a.bias ? (double)a.bias[e] : 0.0);
    }
    if (a.n_groups > 1) {
        // Lane g keeps group g's score: the sum of its best group_topk keys.
        const int per = E / a.n_groups;
        double gs = NONE;
        for (int g = 0; g < a.n_groups; g++) {
            double sum = 0.0;
            int first = -1;
            for (int r = 0; r < a.group_topk; r++) {
                double v = NONE;
                int i = E;
#pragma unroll
                for (int j = 0; j < V; j++) {
                    const int e = 64 * j + (int)lane;
                    if (e / per == g && e < E && e != first)
                        argmax_step(v, i, key[j], e);
                }
                wave_argmax(v, i, lane);
                if (v == NONE)
                    break;
                sum += v;
                if (r == 0)
                    first = i;
            }
            if ((int)lane == g)
                gs = first < 0 ? NONE : sum;
        }
        uint64_t keep = 0;
        for (int r = 0; r < a.topk_groups; r++) {
            double v = gs;
            int i = (int)lane;
            wave_argmax(v, i, lane);
            keep |= (uint64_t)1 << i;
            if ((int)lane == i)
                gs = NONE;
        }
#pragma unroll
        for (int j = 0; j < V; j++) {
            const int e = 64 * j + (int)lane;
            if (e < E && !((keep >> (e / per)) & 1))
                key[j] = NONE;
        }
    }
    // Lane c keeps the c-th choice.
    double sel = 0.0;
    int chosen = -1;
    for (int c = 0; c < a.top_k; c++) {
        double v = NONE;
        int i = 64 * V;
#pragma unroll
        for (int j = 0; j < V; j++)
            argmax_step(v, i, key[j], 64 * j + (int)lane);
        wave_argmax(v, i, lane);
        if (v == NONE)
            break;
        double xv = 0.0;
#pragma unroll
        for (int j = 0; j < V; j++)
            if (64 * j + (int)lane == i) {
                key[j] = NONE;
                xv = x[j];
            }
        xv = lane_get(xv, (uint32_t)i & 63);
        if ((int)lane == c) {
            chosen = i;
            sel = xv;
        }
    }
    // Renormalized weights depend on the scores' ratios alone: a softmax over
    // the selected logits, or sigmoids scaled by e^-top where the largest
    // selected logit, top, is negative, so that no sum underflows.
    if (chosen >= 0 && !a.renorm)
        sel = score(sel);
    if (a.renorm) {
        double top = chosen >= 0 ? sel : NONE;
        int dummy = 0;
        wave_argmax(top, dummy, lane);
        if (a.sigmoid && top > 0.0)
            top = 0.0;
        if (chosen < 0)
            sel = 0.0;
        else if (!a.sigmoid)
            sel = exp_f64(sel - top);
        else
            sel = sel >= 0.0 ? 1.0 / (1.0 + exp_f64(-sel))
                             : exp_f64(sel - top) / (1.0 + exp_f64(sel));
    }
    if (a.renorm) {
        const double s = wave_sum_f64(sel, lane);
        sel = s > 0.0 ? sel / s : 0.0;
    }
    if ((int)lane < a.top_k) {
        a.weights[t * a.top_k + lane] = (float)(sel * (double)a.scale);
        a.experts[t * a.top_k + lane] = chosen;
    }
}

// Bit t of mask[e][w]: token 64 w + t of the tile chose expert e.  Bits are
// set with LDS atomics (whose order cannot matter) and ranks are population
// counts, so the maps do not depend on any order of execution.
__device__ __forceinline__ void tile_masks(uint64_t *mask, const int64_t *experts, int64_t t0,
                                           int tokens, int top_k, int E)
{
    for (int i = (int)tid(); i < E * MAP_WORDS; i += MAP_THREADS)
        mask[i] = 0;
    __syncthreads();
    for (int i = (int)tid(); i < tokens * top_k; i += MAP_THREADS) {
        const int64_t e = experts[t0 * top_k + i];
        const int t = i / top_k;
        if (e >= 0)
            __hip_atomic_fetch_or(&mask[e * MAP_WORDS + (t >> 6)], (uint64_t)1 << (t & 63),
                                  __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
}
__device__ __forceinline__ int popc(uint64_t v) { return __builtin_popcountll(v); }

__global__ void __launch_bounds__(MAP_THREADS) moe_count_kernel(const int64_t *experts,
                                                                int64_t n_tokens, int top_k,
                                                                int E, int *hist)
{
    extern __shared__ uint64_t mask[];
    const int64_t t0 = (int64_t)wg_id() * MAP_TOKENS;
    const int tokens = (int)(n_tokens - t0 < MAP_TOKENS ? n_tokens - t0 : MAP_TOKENS);
    tile_masks(mask, experts, t0, tokens, top_k, E);
    for (int e = (int)tid(); e < E; e += MAP_THREADS) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < MAP_WORDS; w++)
            n += popc(mask[e * MAP_WORDS + w]);
        hist[(int64_t)wg_id() * E + e] = n;
    }
}

// Tile w's copies to their rows: the first row of expert e (the counts of
// the experts before it), the copies of earlier tiles, the earlier tokens
// of the tile.
__global__ void __launch_bounds__(MAP_THREADS) moe_maps_kernel(
    const int64_t *experts, int64_t n_tokens, int top_k, int E, int n_tiles, const int *hist,
    int64_t *token_rows, int64_t *row_tokens, int64_t *seg_offsets)
{
    extern __shared__ uint64_t mask[];
    int *base = reinterpret_cast<int *>(mask + E * MAP_WORDS);      // [E + 1]
    int *before = base + E + 1;                                     // [E]
    const int tile = (int)wg_id();
    const int64_t t0 = (int64_t)tile * MAP_TOKENS;
    const int tokens = (int)(n_tokens - t0 < MAP_TOKENS ? n_tokens - t0 : MAP_TOKENS);
    for (int e = (int)tid(); e < E; e += MAP_THREADS) {
        int n = 0, b = 0;
        for (int i = 0; i < n_tiles; i++) {
            if (i == tile)
                b = n;
            n += hist[(int64_t)i * E + e];
        }
        base[e + 1] = n;
        before[e] = b;
    }
    tile_masks(mask, experts, t0, tokens, top_k, E);
    if (tid() == 0) {
        int n = 0;
        base[0] = 0;
        for (int e = 0; e < E; e++) {
            n += base[e + 1];
            base[e + 1] = n;
        }
    }
    __syncthreads();
    for (int i = (int)tid(); i < tokens * top_k; i += MAP_THREADS) {
        const int64_t g = t0 * top_k + i;
        const int64_t e = experts[g];
        const int t = i / top_k;
        int64_t row = -1;
        if (e >= 0) {
            int r = base[e] + before[e];
            for (int w = 0; w < (t >> 6); w++)
                r += popc(mask[e * MAP_WORDS + w]);
            r += popc(mask[e * MAP_WORDS + (t >> 6)] & (((uint64_t)1 << (t & 63)) - 1));
            row = r;
            row_tokens[row] = t0 + t;
        }
        token_rows[g] = row;
    }
    // Dropped copies leave rows past the last segment; their token is -1.
    const int64_t total = n_tokens * top_k;
    for (int64_t r = base[E] + (int64_t)tile * MAP_THREADS + tid(); r < total;
         r += (int64_t)n_tiles * MAP_THREADS)
        row_tokens[r] = -1;
    if (tile == 0)
        for (int e = (int)tid(); e <= E; e += MAP_THREADS)
            seg_offsets[e] = base[e];
}

}  // namespace

static int64_t map_tiles(int64_t n_tokens) { return (n_tokens + MAP_TOKENS - 1) / MAP_TOKENS; }

int64_t moe_route_workspace(int64_t n_tokens, int64_t n_experts)
{
    return map_tiles(n_tokens) * n_experts * (int64_t)sizeof(int);
}

template <bool BF16>
static void route_launch(const RouteArgs &a, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.n_tokens + ROUTE_WAVES - 1) / ROUTE_WAVES)),
        block(64 * ROUTE_WAVES);
    const int v = (a.n_experts + 63) / 64;
    if (v <= 1)
        hipLaunchKernelGGL((moe_route_kernel<BF16, 1>), grid, block, 0, stream, a);
    else if (v <= 2)
        hipLaunchKernelGGL((moe_route_kernel<BF16, 2>), grid, block, 0, stream, a);
    else if (v <= 4)
        hipLaunchKernelGGL((moe_route_kernel<BF16, 4>), grid, block, 0, stream, a);
    else if (v <= 8)
        hipLaunchKernelGGL((moe_route_kernel<BF16, 8>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((moe_route_kernel<BF16, 16>), grid, block, 0, stream, a);
}

hipError_t launch_moe_route(bool bf16, const void *logits, const float *bias, int64_t n_tokens,
                            int64_t n_experts, const mxq_route_params &p, float *weights,
                            int64_t *experts, int64_t *token_rows, int64_t *row_tokens,
                            int64_t *seg_offsets, void *workspace, hipStream_t stream)
{
    RouteArgs a{logits, bias, n_tokens, (int)n_experts, (int)p.top_k, (int)p.n_groups,
                (int)p.topk_groups, (int)p.group_topk, p.scoring == MXQ_SCORE_SIGMOID,
                p.renormalize != 0, p.scale, weights, experts};
    if (bf16)
        route_launch<true>(a, stream);
    else
        route_launch<false>(a, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !token_rows)
        return e;
    const int E = (int)n_experts, tiles = (int)map_tiles(n_tokens);
    const size_t mask_bytes = (size_t)E * MAP_WORDS * 8;
    hipLaunchKernelGGL(moe_count_kernel, dim3(tiles), dim3(MAP_THREADS), mask_bytes, stream,
                       experts, n_tokens, (int)p.top_k, E, static_cast<int *>(workspace));
    e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(moe_maps_kernel, dim3(tiles), dim3(MAP_THREADS),
                       mask_bytes + (2 * (size_t)E + 1) * 4, stream, experts, n_tokens,
                       (int)p.top_k, E, tiles, static_cast<const int *>(workspace), token_rows,
                       row_tokens, seg_offsets);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Router gradient.  With s the scores, S the sum of the selected ones and
// g_i = scale dw_i: renormalized ds_i = (g_i - sum_j g_j s_j / S) / S,
// otherwise ds_i = g_i; then dx_e = s_e (1 - s_e) ds_e (sigmoid) or
// s_e (ds_e - sum_j ds_j s_j) (softmax), ds_e = 0 for unselected experts.
// ---------------------------------------------------------------------------
namespace {

struct RouteBwdArgs {
    const float *d_weights;
    const void *logits;
    const int64_t *experts;
    int64_t n_tokens;
    int n_experts, top_k;
    bool sigmoid, renorm;
    float scale;
    void *d_logits;
};

template <bool BF16, int V>
__global__ void __launch_bounds__(64 * ROUTE_WAVES) moe_route_backward_kernel(RouteBwdArgs a)
{
    const uint32_t lane = lane_id();
    const int64_t t = (int64_t)wg_id() * ROUTE_WAVES + wave_in_group();
    if (t >= a.n_tokens)
        return;
    const int E = a.n_experts;
    float s[V], ds[V];
    bool dead[V];
    float m = -3.402823466e+38f;
#pragma unroll
    for (int j = 0; j < V; j++) {
        const int e = 64 * j + (int)lane;
        float f = e < E ? ld_elem<BF16>(a.logits, t * E + e) : -__builtin_inff();
        dead[j] = is_masked(f);
        f = f < 3.402823466e+38f ? f : 3.402823466e+38f;
        s[j] = dead[j] ? -3.402823466e+38f : f;
        m = s[j] > m ? s[j] : m;
        ds[j] = 0.0f;
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const float o = lane_get(m, lane ^ k);
        m = o > m ? o : m;
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; j++) {
        if (a.sigmoid)
            s[j] = dead[j] ? 0.0f : 1.0f / (1.0f + exp_f32(-s[j]));
        else
            s[j] = dead[j] ? 0.0f : exp_f32(s[j] - m);
        sum += s[j];
    }
    if (!a.sigmoid) {
        sum = wave_sum_f32(sum);
        const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int j = 0; j < V; j++)
            s[j] *= r;
    }
    float S = 0.0f, gs = 0.0f;
    for (int c = 0; c < a.top_k; c++) {
        const int64_t e64 = a.experts[t * a.top_k + c];
        if (e64 < 0 || e64 >= E)
            continue;
        const int e = (int)e64;
        const float g = a.d_weights[t * a.top_k + c] * a.scale;
#pragma unroll
        for (int j = 0; j < V; j++)
            if (64 * j + (int)lane == e) {
                ds[j] += g;
                S += s[j];
                gs += g * s[j];
            }
    }
    S = wave_sum_f32(S);
    gs = wave_sum_f32(gs);
    if (a.renorm) {
        const float r = S > 0.0f ? 1.0f / S : 0.0f;
        const float mean = gs * r;
        for (int c = 0; c < a.top_k; c++) {
            const int64_t e64 = a.experts[t * a.top_k + c];
            if (e64 < 0 || e64 >= E)
                continue;
#pragma unroll
            for (int j = 0; j < V; j++)
                if (64 * j + (int)lane == (int)e64)
                    ds[j] -= mean;
        }
#pragma unroll
        for (int j = 0; j < V; j++)
            ds[j] *= r;
        gs = 0.0f;      // sum_j ds_j s_j of renormalized weights
    }
#pragma unroll
    for (int j = 0; j < V; j++) {
        const int e = 64 * j + (int)lane;
        const float d = a.sigmoid ? ds[j] * s[j] * (1.0f - s[j]) : s[j] * (ds[j] - gs);
        if (e < E)
            st_elem<BF16>(a.d_logits, t * E + e, d);
    }
}

template <bool BF16>
void route_backward_launch(const RouteBwdArgs &a, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.n_tokens + ROUTE_WAVES - 1) / ROUTE_WAVES)),
        block(64 * ROUTE_WAVES);
    const int v = (a.n_experts + 63) / 64;
    if (v <= 1)
        hipLaunchKernelGGL((moe_route_backward_kernel<BF16, 1>), grid, block, 0, stream, a);
    else if (v <= 2)
        hipLaunchKernelGGL((moe_route_backward_kernel<BF16, 2>), grid, block, 0, stream, a);
    else if (v <= 4)
        hipLaunchKernelGGL((moe_route_backward_kernel<BF16, 4>), grid, block, 0, stream, a);
    else if (v <= 8)
        hipLaunchKernelGGL((moe_route_backward_kernel<BF16, 8>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((moe_route_backward_kernel<BF16, 16>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_moe_route_backward(bool bf16, const float *d_weights, const void *logits,
                                     const int64_t *experts, int64_t n_tokens, int64_t n_experts,
                                     int64_t top_k, bool sigmoid, bool renorm, float scale,
                                     void *d_logits, hipStream_t stream)
{
    const RouteBwdArgs a{d_weights, logits, experts, n_tokens, (int)n_experts, (int)top_k,
                         sigmoid, renorm, scale, d_logits};
    if (bf16)
        route_backward_launch<true>(a, stream);
    else
        route_backward_launch<false>(a, stream);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Combine: out[t] = sum_c w[t][c] rows[token_rows[t][c]], accumulated in
// fp32 in the order of c.
// ---------------------------------------------------------------------------
namespace {

constexpr int COMBINE_THREADS = 256;

// Eight values of a row (16 bytes of BF16, 32 of FP32).
template <bool BF16>
__device__ __forceinline__ void ld8v(float (&v)[8], const void *p, int64_t i)
{
    if constexpr (BF16) {
        const uint4 q = ld16(reinterpret_cast<const uint16_t *>(p) + i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            v[2 * k] = bf16_lo(w[k]);
            v[2 * k + 1] = bf16_hi(w[k]);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint4 q = ld16(reinterpret_cast<const float *>(p) + i + 4 * h);
            v[4 * h] = u2f(q.x);
            v[4 * h + 1] = u2f(q.y);
            v[4 * h + 2] = u2f(q.z);
            v[4 * h + 3] = u2f(q.w);
        }
    }
}
template <bool BF16>
__device__ __forceinline__ void st8v(void *p, int64_t i, const float (&v)[8])
{
    if constexpr (BF16) {
        u32x4_t q;
#pragma unroll
        for (int k = 0; k < 4; k++)
            q[k] = (uint32_t)bf16_rne(v[2 * k]) | (uint32_t)bf16_rne(v[2 * k + 1]) << 16;
        *reinterpret_cast<u32x4_t *>(reinterpret_cast<uint16_t *>(p) + i) = q;
    } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const u32x4_t q = {f2u(v[4 * h]), f2u(v[4 * h + 1]), f2u(v[4 * h + 2]),
                               f2u(v[4 * h + 3])};
            *reinterpret_cast<u32x4_t *>(reinterpret_cast<float *>(p) + i + 4 * h) = q;
        }
    }
}

template <bool BF16, bool BF16_OUT>
__global__ void __launch_bounds__(COMBINE_THREADS) moe_combine_kernel(
    const void *rows, int64_t total_rows, const int64_t *token_rows, const float *weights,
    int top_k, int64_t cols, void *out)
{
    const int64_t t = wg_id();
    for (int64_t c8 = 8 * (int64_t)tid(); c8 < cols; c8 += 8 * COMBINE_THREADS) {
        float acc[8] = {};
        for (int c = 0; c < top_k; c++) {
            const int64_t r = token_rows[t * top_k + c];
            if (r < 0 || r >= total_rows)
                continue;
            const float w = weights[t * top_k + c];
            float y[8];
            ld8v<BF16>(y, rows, r * cols + c8);
#pragma unroll
            for (int k = 0; k < 8; k++)
                acc[k] = __builtin_fmaf(w, y[k], acc[k]);
        }
        st8v<BF16_OUT>(out, t * cols + c8, acc);
    }
}

// d_rows[r] = w dout[t], d_weights = <dout[t], rows[r]>; workgroups past
// n_tokens zero the rows past the last segment.
template <bool BF16>
__global__ void __launch_bounds__(COMBINE_THREADS) moe_combine_backward_kernel(
    const void *d_out, const void *rows, int64_t total_rows, const int64_t *token_rows,
    const float *weights, const int64_t *seg_end, int64_t n_tokens, int top_k, int64_t cols,
    void *d_rows, float *d_weights, int64_t n_wgs)
{
    __shared__ float part[COMBINE_THREADS / 64];
    const int64_t t = wg_id();
    if (seg_end) {
        const float zero[8] = {};
        int64_t end = *seg_end;
        end = end < 0 ? 0 : end;
        for (int64_t r = end + t; r < total_rows; r += n_wgs)
            for (int64_t c8 = 8 * (int64_t)tid(); c8 < cols; c8 += 8 * COMBINE_THREADS)
                st8v<BF16>(d_rows, r * cols + c8, zero);
    }
    for (int c = 0; c < top_k; c++) {
        const int64_t r = token_rows[t * top_k + c];
        const bool live = r >= 0 && r < total_rows;
        const float w = weights[t * top_k + c];
        float dot = 0.0f;
        if (live)
            for (int64_t c8 = 8 * (int64_t)tid(); c8 < cols; c8 += 8 * COMBINE_THREADS) {
                float d[8], y[8];
                ld8v<BF16>(d, d_out, t * cols + c8);
                ld8v<BF16>(y, rows, r * cols + c8);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    dot = __builtin_fmaf(d[k], y[k], dot);
                    d[k] *= w;
                }
                st8v<BF16>(d_rows, r * cols + c8, d);
            }
        dot = wave_sum_f32(dot);
        if (lane_id() == 0)
            part[wave_in_group()] = dot;
        __syncthreads();
        if (tid() == 0)
            d_weights[t * top_k + c] = part[0] + part[1] + part[2] + part[3];
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_moe_combine(bool bf16, const void *rows, int64_t total_rows,
                              const int64_t *token_rows, const float *weights, int64_t n_tokens,
                              int64_t top_k, int64_t cols, bool bf16_out, void *out,
                              hipStream_t stream)
{
    const dim3 grid((unsigned)n_tokens), block(COMBINE_THREADS);
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, rows, total_rows, token_rows, weights,
                           (int)top_k, cols, out);
    };
    if (bf16)
        bf16_out ? launch(moe_combine_kernel<true, true>) : launch(moe_combine_kernel<true, false>);
    else
        bf16_out ? launch(moe_combine_kernel<false, true>)
                 : launch(moe_combine_kernel<false, false>);
    return hipGetLastError();
}

hipError_t launch_moe_combine_backward(bool bf16, const void *d_out, const void *rows,
                                       int64_t total_rows, const int64_t *token_rows,
                                       const float *weights, const int64_t *seg_offsets,
                                       int64_t n_groups, int64_t n_tokens, int64_t top_k,
                                       int64_t cols, void *d_rows, float *d_weights,
                                       hipStream_t stream)
{
    const dim3 grid((unsigned)n_tokens), block(COMBINE_THREADS);
    const int64_t *end = seg_offsets ? seg_offsets + n_groups : nullptr;
    if (bf16)
        hipLaunchKernelGGL(moe_combine_backward_kernel<true>, grid, block, 0, stream, d_out,
                           rows, total_rows, token_rows, weights, end, n_tokens, (int)top_k,
                           cols, d_rows, d_weights, n_tokens);
    else
        hipLaunchKernelGGL(moe_combine_backward_kernel<false>, grid, block, 0, stream, d_out,
                           rows, total_rows, token_rows, weights, end, n_tokens, (int)top_k,
                           cols, d_rows, d_weights, n_tokens);
    return hipGetLastError();
}

}  // namespace mxq
