// mxq_moe.hip -- routing tokens to experts and bringing expert rows back.
//
// Route: each token's top_k experts under softmax or sigmoid scores (with an
// optional balance bias and expert groups), their weights, and the index
// maps of the expert-sorted layout.
//
// A token is worked on by L lanes (16, or 64 for many experts or choices),
// each with V consecutive experts in registers; the next choice is a maximum
// over them by DPP, then the lowest index among those equal to it.  The
// selection is that of the exact scores: without a bias (and with groups
// ranked by their best expert) scores rise with the logits, so the logits
// themselves are compared; otherwise the keys are formed in fp32 with a bound
// on their error, and a wavefront that finds two neighbours of the order
// closer than the bound repeats its tokens in 64 bits.
//
// Maps: a tile is 64 tokens, and a 64-bit word per (tile, expert) marks the
// tokens that chose the expert.  Bits are set with atomics, whose order
// cannot matter, and a copy's rank is a population count, so the maps do
// not depend on any order of execution.  One tile: the routing workgroup
// writes them itself.  Few: a second kernel sums the tiles before its own.
// Many: a kernel between them forms those sums, one wavefront an expert.
//
// Bound by the selection's chain: 7 tokens x 256 experts in 8 groups take 9.0
// us, 32768 x 128 top-8 14.7 us, then 6.3 us for the sums and 4.7 us for the maps.
#include "mxq_layer.h"
#include "mxq_layer_device.h"

namespace mxq {

namespace {

constexpr int ROUTE_THREADS = 512;
constexpr int MAP_TOKENS = 64;                    // tokens of a tile
constexpr int MAP_SELF_TILES = 16;                // most tiles that sum up for themselves

struct RouteArgs {
    const void *logits;
    const float *bias;
    int64_t n_tokens;
    int n_experts, top_k, n_groups, topk_groups, group_topk, per_group;
    Div per_div;
    bool sigmoid, renorm;
    float scale;
    float *weights;
    int64_t *experts;
    int64_t *token_rows, *row_tokens, *seg_offsets;     // one tile: written here
    uint64_t *masks;                                    // [tile][expert], nullptr: no maps
};

template <typename T>
__device__ __forceinline__ T none();
template <>
__device__ __forceinline__ float none<float>() { return -__builtin_inff(); }
template <>
__device__ __forceinline__ double none<double>() { return -__builtin_inf(); }

template <int CTRL>
__device__ __forceinline__ float dpp_get(float v) { return u2f(dpp<CTRL>(f2u(v))); }
template <int CTRL>
__device__ __forceinline__ int dpp_get(int v) { return (int)dpp<CTRL>((uint32_t)v); }
template <int CTRL>
__device__ __forceinline__ double dpp_get(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 |
                                          dpp<CTRL>((uint32_t)u));
}
// v and its copy from lane ^ 16 or lane ^ 32 joined by f: a permlane swap of two
// copies of v leaves the pair's values in the two registers, in one order or
// the other, and f does not mind the order.
template <int STEP>
__device__ __forceinline__ uint2_t far_pair(uint32_t v)
{
    if constexpr (STEP == 16)
        return __builtin_amdgcn_permlane16_swap(v, v, false, false);
    else
        return __builtin_amdgcn_permlane32_swap(v, v, false, false);
}
template <int STEP, typename F>
__device__ __forceinline__ float join_far(float v, F f)
{
    const uint2_t r = far_pair<STEP>(f2u(v));
    return f(u2f(r[0]), u2f(r[1]));
}
template <int STEP, typename F>
__device__ __forceinline__ int join_far(int v, F f)
{
    const uint2_t r = far_pair<STEP>((uint32_t)v);
    return f((int)r[0], (int)r[1]);
}
template <int STEP, typename F>
__device__ __forceinline__ double join_far(double v, F f)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint2_t lo = far_pair<STEP>((uint32_t)u), hi = far_pair<STEP>((uint32_t)(u >> 32));
    return f(__builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]),
             __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]));
}
// f over the L lanes of a token, the same in each.
template <int L, typename T, typename F>
__device__ __forceinline__ T over_lanes(T v, F f)
{
    v = f(v, dpp_get<DPP_XOR1>(v));
    v = f(v, dpp_get<DPP_XOR2>(v));
    v = f(v, dpp_get<DPP_HALF_MIRROR>(v));
    v = f(v, dpp_get<DPP_MIRROR>(v));
    if constexpr (L == 64) {
        v = join_far<16>(v, f);
        v = join_far<32>(v, f);
    }
    return v;
}
struct MaxOf {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a > b ? a : b; }
};
struct MinOf {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a < b ? a : b; }
};
struct SumOf {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

__device__ __forceinline__ float exp_of(float x) { return exp_f32(x); }
__device__ __forceinline__ double exp_of(double x) { return exp_f64(x); }

// The largest of the lanes' keys and its index (the lowest of equals; any
// index if all keys are none).
template <int L, int V, typename T>
__device__ __forceinline__ T best_key(const T (&key)[V], int l, int *index)
{
    T m = key[0];
#pragma unroll
    for (int j = 1; j < V; j++)
        m = key[j] > m ? key[j] : m;
    m = over_lanes<L>(m, MaxOf{});
    int i = 1 << 20;
#pragma unroll
    for (int j = V - 1; j >= 0; j--)
        i = key[j] == m ? l * V + j : i;
    *index = over_lanes<L>(i, MinOf{});
    return m;
}

// Chooses the experts of a token from its logits x (none: never selected, a
// score of 0) and biases (none: never selected, its score a term of the
// softmax's sum like any other): lane c of its L lanes gets choice c, -1 where
// none is left.  lds: room for the keys of a token (groups).  Returns whether
// the keys' error leaves no doubt (always in 64 bits); den is the softmax's
// sum under the largest logit m.
template <bool BY_LOGIT, int L, int V, typename T>
__device__ __forceinline__ bool choose(const RouteArgs &a, const float (&x)[V],
                                       const float (&bias)[V], int l, T *lds, int *chosen,
                                       T *top, T *den)
{
    constexpr bool by_logit = BY_LOGIT;
    T key[V], m = none<T>(), sum = 0;
#pragma unroll
    for (int j = 0; j < V; j++) {
        key[j] = (T)x[j];
        m = key[j] > m ? key[j] : m;
    }
    T doubt = 0;
    if (!a.sigmoid && (!by_logit || !a.renorm)) {
        m = over_lanes<L>(m, MaxOf{});
#pragma unroll
        for (int j = 0; j < V; j++)
            sum += key[j] == none<T>() ? (T)0 : exp_of(key[j] - m);
        sum = over_lanes<L>(sum, SumOf{});
    }
    *top = m;
    *den = sum;
    if (!by_logit) {
        // fp32 scores are off by less than 2^-20 of the largest (exponential, sum of 1024
        // terms, quotient), keys by another 2^-24 of their size.
        doubt = (T)0x1p-18 * (a.sigmoid ? (T)1 : (T)1 / sum);
#pragma unroll
        for (int j = 0; j < V; j++)
            if (key[j] != none<T>())
                key[j] = (a.sigmoid ? (T)1 / ((T)1 + exp_of(-key[j])) : exp_of(key[j] - m) / sum) +
                         (T)bias[j];
    }
    bool sure = true;
    auto close_keys = [&](T hi, T lo, T doubt) {
        const T size = hi > -lo ? hi : -lo;
        return sizeof(T) == 4 && !by_logit && lo != none<T>() &&
               hi - lo <= doubt + (T)0x1p-20 * (size > (T)0 ? size : (T)0);
    };
    if (a.n_groups > 1) {
        // Lane g sums up groups g, g + L, ...: their best one or two keys.
#pragma unroll
        for (int j = 0; j < V; j++)
            lds[l * V + j] = key[j];
        constexpr int GS = 64 / L;
        // A sum of two keys is as uncertain as the keys are large, however small it is
        // itself (size: the most of any group).
        T gs[GS], size = 0;
#pragma unroll
        for (int i = 0; i < GS; i++) {
            const int g = l + L * i;
            T m1 = none<T>(), m2 = none<T>();
            if (g < a.n_groups)
                for (int k0 = 0; k0 < a.per_group; k0 += 8) {
                    T v[8];
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const int i = k0 + k < a.per_group ? k0 + k : a.per_group - 1;
                        v[k] = lds[g * a.per_group + i];
                    }
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const T vk = k0 + k < a.per_group ? v[k] : none<T>();
                        const T lo = vk > m1 ? m1 : vk;
                        m1 = vk > m1 ? vk : m1;
                        m2 = lo > m2 ? lo : m2;
                    }
                }
            const bool two = a.group_topk == 2 && m2 != none<T>();
            gs[i] = two ? m1 + m2 : m1;
            const T sz = (m1 < 0 ? -m1 : m1) + (m2 < 0 ? -m2 : m2);
            size = two && sz > size ? sz : size;
        }
        T group_doubt = doubt;
        if constexpr (sizeof(T) == 4 && !by_logit)
            if (a.group_topk == 2)
                group_doubt = 2 * doubt + (T)0x1p-20 * over_lanes<L>(size, MaxOf{});
        uint64_t keep = 0;
        T last = none<T>();
        for (int r = 0; r <= a.topk_groups; r++) {
            T v = gs[0];
#pragma unroll
            for (int i = 1; i < GS; i++)
                v = gs[i] > v ? gs[i] : v;
            v = over_lanes<L>(v, MaxOf{});
            if (r == a.topk_groups) {             // the best group left out
                sure = sure && !close_keys(last, v, group_doubt);
                break;
            }
            int g = 1 << 20;
#pragma unroll
            for (int i = GS - 1; i >= 0; i--)
                g = gs[i] == v ? l + L * i : g;
            g = over_lanes<L>(g, MinOf{});
            if (v != none<T>())
                keep |= (uint64_t)1 << g;
#pragma unroll
            for (int i = 0; i < GS; i++)
                gs[i] = l + L * i == g ? none<T>() : gs[i];
            last = v;
        }
#pragma unroll
        for (int j = 0; j < V; j++) {
            const uint32_t e = (uint32_t)(l * V + j);
            const uint32_t g = udiv(e, a.per_div);
            key[j] = g < 64 && ((keep >> g) & 1) ? key[j] : none<T>();
        }
    }
    *chosen = -1;
    T last = none<T>();
    for (int c = 0; c <= a.top_k; c++) {
        if (c == a.top_k && by_logit)
            break;
        int i;
        const T v = best_key<L, V, T>(key, l, &i);
        if (c > 0)
            sure = sure && !close_keys(last, v, doubt);
        if (c == a.top_k)
            break;
        const bool some = v != none<T>();
        if (l == c)
            *chosen = some ? i : -1;
#pragma unroll
        for (int j = 0; j < V; j++)
            key[j] = l * V + j == i ? none<T>() : key[j];
        last = v;
    }
    return sure;
}

// A choice's part of the sum of the selected scores, x its logit.  It depends on
// the scores' ratios alone: a softmax over the selected logits, or sigmoids
// scaled by e^-h where the largest selected logit, h, is negative, so that no
// sum underflows.
template <int L>
__device__ __forceinline__ float share_of(bool sigmoid, bool mine, float x)
{
    float h = over_lanes<L>(mine ? x : -__builtin_inff(), MaxOf{}), w = 0.0f;
    h = sigmoid && h > 0.0f ? 0.0f : h;
    if (mine)
        w = sigmoid && x >= 0.0f ? 1.0f / (1.0f + exp_f32(-x))
                                 : exp_diff_f32(x, h) / (sigmoid ? 1.0f + exp_f32(x) : 1.0f);
    const float s = over_lanes<L>(w, SumOf{});
    return s > 0.0f ? w / s : 0.0f;
}

__device__ __forceinline__ int popc(uint64_t v) { return __builtin_popcountll(v); }

// Inclusive sum over the 64 lanes: shifts within rows of 16, then the last lane
// of a row to the next row, and of the lower half to the upper.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_rows(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v)
{
    v += dpp_rows<0x111, 0xF>(v);
    v += dpp_rows<0x112, 0xF>(v);
    v += dpp_rows<0x114, 0xF>(v);
    v += dpp_rows<0x118, 0xF>(v);
    v += dpp_rows<0x142, 0xA>(v);
    v += dpp_rows<0x143, 0xC>(v);
    return v;
}
// base[e] = sum of n[0 .. e) for e <= E, by the first wavefront of a workgroup.
__device__ __forceinline__ void expert_bases(int *base, const int *n, int E)
{
    if (wave_in_group() == 0) {
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + (int)lane_id();
            const int v = e < E ? n[e] : 0, s = wave_scan(v);
            if (e < E)
                base[e] = carry + s - v;
            carry += __builtin_amdgcn_readlane(s, 63);
        }
        if (lane_id() == 0)
            base[E] = carry;
    }
}
// The copies of tile t0 .. to their rows: the first row of (tile, expert) and
// the tokens of the tile before.
__device__ __forceinline__ void write_rows(const uint64_t *mask, const int *first,
                                           const int64_t *experts, int64_t t0, int tokens,
                                           int top_k, int64_t *token_rows, int64_t *row_tokens)
{
    for (int i = (int)tid(); i < tokens * top_k; i += ROUTE_THREADS) {
        const int64_t g = t0 * top_k + i, e = experts[g];
        const int t = (int)((uint32_t)i / (uint32_t)top_k);
        int64_t row = -1;
        if (e >= 0) {
            row = first[e] + popc(mask[e] & (((uint64_t)1 << t) - 1));
            row_tokens[row] = t0 + t;
        }
        token_rows[g] = row;
    }
}
// Dropped copies leave rows past the last segment; their token is -1.
__device__ __forceinline__ void write_tail(int64_t used, int64_t total, int wg, int wgs,
                                           int64_t *row_tokens)
{
    for (int64_t r = used + (int64_t)wg * ROUTE_THREADS + tid(); r < total;
         r += (int64_t)wgs * ROUTE_THREADS)
        row_tokens[r] = -1;
}

template <bool BY_LOGIT, bool BF16, int L, int V>
__global__ void __launch_bounds__(ROUTE_THREADS) moe_route_kernel(RouteArgs a)
{
    constexpr int SLOTS = ROUTE_THREADS / L;      // tokens at once
    extern __shared__ __attribute__((aligned(16))) uint8_t shared[];
    // Keys of every slot's token (groups), then the tile's masks and first rows (maps).
    double *keys = reinterpret_cast<double *>(shared);
    uint64_t *mask = reinterpret_cast<uint64_t *>(shared + (a.n_groups > 1 ? SLOTS * L * V * 8 : 0));
    const int E = a.n_experts, l = (int)tid() % L, slot = (int)tid() / L;
    const int64_t t0 = (int64_t)wg_id() * MAP_TOKENS;
    const int tokens = (int)(a.n_tokens - t0 < MAP_TOKENS ? a.n_tokens - t0 : MAP_TOKENS);
    if (a.masks) {
        for (int e = (int)tid(); e < E; e += ROUTE_THREADS)
            mask[e] = 0;
        __syncthreads();
    }
    for (int i = 0; i < tokens; i += SLOTS) {
        // Slots past the last token repeat it and write nothing.
        const int i0 = i + slot < tokens ? i + slot : tokens - 1;
        const int64_t t = t0 + i0;
        const bool live = i + slot < tokens;
        float x[V], bias[V];
#pragma unroll
        for (int j = 0; j < V; j++) {
            const int e = l * V + j;
            float f = -__builtin_inff();
            bias[j] = 0.0f;
            if (e < E) {
                f = ld_elem<BF16>(a.logits, t * E + e);
                f = is_masked(f) ? -__builtin_inff() : f;
                if (a.bias) {
                    bias[j] = a.bias[e];
                    bias[j] = is_masked(bias[j]) ? -__builtin_inff() : bias[j];
                }
                f = f < 3.402823466e+38f ? f : 3.402823466e+38f;
            }
            x[j] = f;
        }
        int chosen;
        float top, den;
        const bool sure = choose<BY_LOGIT, L, V, float>(
            a, x, bias, l, reinterpret_cast<float *>(keys + slot * L * V), &chosen, &top, &den);
        if constexpr (!BY_LOGIT)
            if (__builtin_amdgcn_ballot_w64(!sure) != 0) {
                double top64, den64;
                (void)choose<false, L, V, double>(a, x, bias, l, keys + slot * L * V, &chosen,
                                                  &top64, &den64);
            }
        const bool mine = l < a.top_k && chosen >= 0;
        float xv = mine ? ld_elem<BF16>(a.logits, t * E + chosen) : -__builtin_inff();
        xv = xv < 3.402823466e+38f ? xv : 3.402823466e+38f;
        float w = 0.0f;
        if (a.renorm) {
            w = share_of<L>(a.sigmoid, mine, xv);
        } else if (mine) {
            w = a.sigmoid ? 1.0f / (1.0f + exp_f32(-xv)) : exp_diff_f32(xv, top) / den;
        }
        if (live && l < a.top_k) {
            a.weights[t * a.top_k + l] = w * a.scale;
            a.experts[t * a.top_k + l] = chosen;
            if (a.masks && chosen >= 0)
                __hip_atomic_fetch_or(&mask[chosen], (uint64_t)1 << i0, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_WORKGROUP);
        }
    }
    if (!a.masks)
        return;
    __syncthreads();
    if (a.token_rows) {                           // the only tile
        int *base = reinterpret_cast<int *>(mask + E), *n = base + E + 1;
        for (int e = (int)tid(); e < E; e += ROUTE_THREADS)
            n[e] = popc(mask[e]);
        __syncthreads();
        expert_bases(base, n, E);
        __syncthreads();
        write_rows(mask, base, a.experts, t0, tokens, a.top_k, a.token_rows, a.row_tokens);
        write_tail(base[E], (int64_t)tokens * a.top_k, 0, 1, a.row_tokens);
        for (int e = (int)tid(); e <= E; e += ROUTE_THREADS)
            a.seg_offsets[e] = base[e];
        return;
    }
    for (int e = (int)tid(); e < E; e += ROUTE_THREADS)
        a.masks[(int64_t)wg_id() * E + e] = mask[e];
}

// before[tile][e] = expert e's copies in earlier tiles, total[e] all of them.
// A workgroup takes 16 experts (whose masks are a line in memory) and splits
// the tiles into 64 runs.
constexpr int SUM_EXPERTS = 16, SUM_RUNS = 64;
__global__ void __launch_bounds__(SUM_EXPERTS *SUM_RUNS) moe_sum_kernel(const uint64_t *masks,
                                                                        int E, int n_tiles,
                                                                        int *before, int *total)
{
    __shared__ int part[2][SUM_RUNS][SUM_EXPERTS];
    const int k = (int)tid() % SUM_EXPERTS, run = (int)tid() / SUM_EXPERTS;
    const int e = (int)wg_id() * SUM_EXPERTS + k;
    const int each = (n_tiles + SUM_RUNS - 1) / SUM_RUNS, i0 = run * each;
    const int i1 = i0 + each < n_tiles ? i0 + each : n_tiles;
    const bool in = e < E;
    int n = 0;
    for (int i = i0; i < i1; i++)
        n += in ? popc(masks[(int64_t)i * E + e]) : 0;
    // Inclusive sums over the runs, doubling the distance.
    int b = n, buf = 0;
    part[0][run][k] = b;
    for (int d = 1; d < SUM_RUNS; d *= 2, buf ^= 1) {
        __syncthreads();
        b += run >= d ? part[buf][run - d][k] : 0;
        part[buf ^ 1][run][k] = b;
    }
    b -= n;
    if (in) {
        for (int i = i0; i < i1; i++) {
            before[(int64_t)i * E + e] = b;
            b += popc(masks[(int64_t)i * E + e]);
        }
        if (run == SUM_RUNS - 1)
            total[e] = b;
    }
}

// One tile a workgroup.  total == nullptr: the sums over tiles are formed here.
__global__ void __launch_bounds__(ROUTE_THREADS) moe_maps_kernel(
    const int64_t *experts, int64_t n_tokens, int top_k, int E, int n_tiles,
    const uint64_t *masks, const int *before, const int *total, int64_t *token_rows,
    int64_t *row_tokens, int64_t *seg_offsets)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t shared[];
    uint64_t *mask = reinterpret_cast<uint64_t *>(shared);          // [E]
    int *n = reinterpret_cast<int *>(mask + E), *base = n + E;       // [E], [E + 1]
    int *first = base + E + 1;                                       // [E]
    const int tile = (int)wg_id();
    const int64_t t0 = (int64_t)tile * MAP_TOKENS;
    const int tokens = (int)(n_tokens - t0 < MAP_TOKENS ? n_tokens - t0 : MAP_TOKENS);
    for (int e = (int)tid(); e < E; e += ROUTE_THREADS) {
        mask[e] = masks[(int64_t)tile * E + e];
        if (total) {
            n[e] = total[e];
            first[e] = before[(int64_t)tile * E + e];
        } else {
            int all = 0, b = 0;
            for (int i = 0; i < n_tiles; i++) {
                b = i == tile ? all : b;
                all += popc(masks[(int64_t)i * E + e]);
            }
            n[e] = all;
            first[e] = b;
        }
    }
    __syncthreads();
    expert_bases(base, n, E);
    __syncthreads();
    for (int e = (int)tid(); e < E; e += ROUTE_THREADS)
        first[e] += base[e];
    __syncthreads();
    write_rows(mask, first, experts, t0, tokens, top_k, token_rows, row_tokens);
    write_tail(base[E], n_tokens * top_k, tile, n_tiles, row_tokens);
    if (tile == 0)
        for (int e = (int)tid(); e <= E; e += ROUTE_THREADS)
            seg_offsets[e] = base[e];
}

}  // namespace

static int64_t map_tiles(int64_t n_tokens) { return (n_tokens + MAP_TOKENS - 1) / MAP_TOKENS; }

// Masks, sums before a tile, totals.
int64_t moe_route_workspace(int64_t n_tokens, int64_t n_experts)
{
    return (map_tiles(n_tokens) * (8 + 4) + 4) * n_experts;
}

// L lanes a token and V experts a lane.
template <bool BY_LOGIT, bool BF16>
static void route_launch(const RouteArgs &a, hipStream_t stream)
{
    const dim3 grid((unsigned)map_tiles(a.n_tokens)), block(ROUTE_THREADS);
    // Few tokens: as many lanes on each as there are, for the shorter chain.
    const bool narrow = a.n_experts <= 256 && a.top_k <= 16 && a.n_tokens > 32;
    const int lanes = narrow ? 16 : 64, v = (a.n_experts + lanes - 1) / lanes;
    int vp = 1;
    while (vp < v)
        vp *= 2;
    const size_t lds = (a.n_groups > 1 ? (size_t)ROUTE_THREADS * vp * 8 : 0) +
                       (a.masks ? (size_t)a.n_experts * 16 + 8 : 0);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, lds, stream, a); };
    if (narrow)
        vp == 1   ? go(moe_route_kernel<BY_LOGIT, BF16, 16, 1>)
        : vp == 2 ? go(moe_route_kernel<BY_LOGIT, BF16, 16, 2>)
        : vp == 4 ? go(moe_route_kernel<BY_LOGIT, BF16, 16, 4>)
        : vp == 8 ? go(moe_route_kernel<BY_LOGIT, BF16, 16, 8>)
                  : go(moe_route_kernel<BY_LOGIT, BF16, 16, 16>);
    else
        vp == 1   ? go(moe_route_kernel<BY_LOGIT, BF16, 64, 1>)
        : vp == 2 ? go(moe_route_kernel<BY_LOGIT, BF16, 64, 2>)
        : vp == 4 ? go(moe_route_kernel<BY_LOGIT, BF16, 64, 4>)
        : vp == 8 ? go(moe_route_kernel<BY_LOGIT, BF16, 64, 8>)
                  : go(moe_route_kernel<BY_LOGIT, BF16, 64, 16>);
}

hipError_t launch_moe_route(bool bf16, const void *logits, const float *bias, int64_t n_tokens,
                            int64_t n_experts, const mxq_route_params &p, float *weights,
                            int64_t *experts, int64_t *token_rows, int64_t *row_tokens,
                            int64_t *seg_offsets, void *workspace, hipStream_t stream)
{
    const int E = (int)n_experts, tiles = (int)map_tiles(n_tokens);
    const bool one = tiles == 1;
    uint64_t *masks = token_rows ? static_cast<uint64_t *>(workspace) : nullptr;
    const int per = E / (int)p.n_groups;
    const RouteArgs a{logits, bias, n_tokens, E, (int)p.top_k, (int)p.n_groups,
                      (int)p.topk_groups, (int)p.group_topk, per, make_div((uint32_t)per),
                      p.scoring == MXQ_SCORE_SIGMOID, p.renormalize != 0, p.scale, weights,
                      experts, one ? token_rows : nullptr, row_tokens, seg_offsets, masks};
    // Scores rise with the logits: without a bias, and where groups are ranked by their
    // best expert, the logits decide.
    if (!bias && (p.n_groups == 1 || p.group_topk == 1))
        bf16 ? route_launch<true, true>(a, stream) : route_launch<true, false>(a, stream);
    else
        bf16 ? route_launch<false, true>(a, stream) : route_launch<false, false>(a, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !token_rows || one)
        return e;
    int *before = reinterpret_cast<int *>(masks + (int64_t)tiles * E);
    int *total = before + (int64_t)tiles * E;
    const bool sums = tiles > MAP_SELF_TILES;
    if (sums) {
        hipLaunchKernelGGL(moe_sum_kernel, dim3((E + SUM_EXPERTS - 1) / SUM_EXPERTS),
                           dim3(SUM_EXPERTS * SUM_RUNS), 0, stream, masks, E, tiles, before,
                           total);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(moe_maps_kernel, dim3(tiles), dim3(ROUTE_THREADS), (size_t)E * 20 + 4,
                       stream, experts, n_tokens, (int)p.top_k, E, tiles, masks, before,
                       sums ? total : nullptr, token_rows, row_tokens, seg_offsets);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Router gradient.  With s the scores and g_i = scale dw_i, in forms that lose
// nothing where scores are near 0 or 1, and in which equal g_i of renormalized
// weights, and a single choice, give exactly 0:
//   renormalized, w_i = s_i / sum of the selected s (as the forward forms it):
//     dx_i = w_i sum_j (g_i - g_j) w_j, times 1 - s_i = sigmoid(-x_i) for sigmoids;
//   sigmoid: dx_i = g_i s_i (1 - s_i), s (1 - s) = e / (1 + e)^2 with e = e^-|x|;
//   softmax: dx_i = s_i (sum_j (g_i - g_j) s_j + g_i U) for a selected i, U the sum
//     of the other experts' scores, and -s_e sum_j g_j s_j for the others.
// Only the last needs the logits of the experts that were not selected.  One
// read of what is needed, one write of the gradient: 20011 x 160 top-6 FP32 take
// 7.4 us renormalized (12.8 MB written; 11.6 us with every logit read and every
// score formed), 10.5 us as a plain softmax, whose exponentials bound it.
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

// L lanes a token; lane l holds experts l, l + L, ... (coalesced), and choice l.
template <bool BF16, int L, int V>
__global__ void __launch_bounds__(ROUTE_THREADS) moe_route_backward_kernel(RouteBwdArgs a)
{
    const int l = (int)tid() % L;
    const int64_t t = (int64_t)wg_id() * (ROUTE_THREADS / L) + tid() / L;
    const bool live = t < a.n_tokens;
    const int64_t tt = live ? t : a.n_tokens - 1;
    const int E = a.n_experts;
    constexpr float LOW = -3.402823466e+38f;
    auto score_in = [&](float f) { return f < -LOW ? f : -LOW; };
    // Choice l of the token: its expert, gradient and logit.
    const int64_t e64 = l < a.top_k ? a.experts[tt * a.top_k + l] : -1;
    int ce = e64 >= 0 && e64 < E ? (int)e64 : -1;
    float cx = ce >= 0 ? ld_elem<BF16>(a.logits, tt * E + ce) : LOW;
    ce = is_masked(cx) ? -1 : ce;
    cx = score_in(cx);
    const float cg = ce >= 0 ? a.d_weights[tt * a.top_k + l] * a.scale : 0.0f;
    const float ce_abs = exp_f32(cx < 0.0f ? cx : -cx);              // e^-|x|
    const uint32_t lane0 = lane_id() & ~(uint32_t)(L - 1);
    float d[V] = {}, cd;
    if (!a.renorm && a.sigmoid) {
        cd = cg * ce_abs / ((1.0f + ce_abs) * (1.0f + ce_abs));
    } else {
        float q, s[V];
        if (a.renorm) {
            q = share_of<L>(a.sigmoid, ce >= 0, cx);
        } else {
            float m = LOW, sum = 0.0f;
            bool dead[V];
#pragma unroll
            for (int j = 0; j < V; j++) {
                const int e = L * j + l;
                const float f = e < E ? ld_elem<BF16>(a.logits, tt * E + e) : -__builtin_inff();
                dead[j] = is_masked(f);
                s[j] = dead[j] ? LOW : score_in(f);
                m = s[j] > m ? s[j] : m;
            }
            m = over_lanes<L>(m, MaxOf{});
#pragma unroll
            for (int j = 0; j < V; j++) {
                s[j] = dead[j] ? 0.0f : exp_f32(s[j] - m);
                sum += s[j];
            }
            sum = over_lanes<L>(sum, SumOf{});
            const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
            for (int j = 0; j < V; j++)
                s[j] *= r;
            q = ce >= 0 ? exp_diff_f32(cx, m) * r : 0.0f;
        }
        float u = 0.0f, gs = 0.0f, S = 0.0f;
        for (int c = 0; c < a.top_k; c++) {
            const float qc = lane_get(q, lane0 + c), gc = lane_get(cg, lane0 + c);
            u = __builtin_fmaf(cg - gc, qc, u);
            gs = __builtin_fmaf(gc, qc, gs);
            S += qc;
        }
        if (!a.renorm) {
            // U as 1 - S where that keeps its precision (10.4 us for 32768 x 128 top-8),
            // else summed (12.0 us).
            float others = 1.0f - S;
            if (__builtin_amdgcn_ballot_w64(S > 0.875f) != 0) {
                uint32_t selected = 0;            // of the lane's experts
                for (int c = 0; c < a.top_k; c++) {
                    const int ec = lane_get(ce, lane0 + c);
                    selected |= ec >= 0 && (ec & (L - 1)) == l ? 1u << (ec / L) : 0u;
                }
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < V; j++)
                    sum += (selected >> j) & 1 ? 0.0f : s[j];
                sum = over_lanes<L>(sum, SumOf{});
                others = S > 0.875f ? sum : others;
            }
            u = __builtin_fmaf(cg, others, u);
#pragma unroll
            for (int j = 0; j < V; j++)
                d[j] = -s[j] * gs;
        }
        cd = q * u;
        if (a.sigmoid)
            cd *= (cx < 0.0f ? 1.0f : ce_abs) / (1.0f + ce_abs);
    }
    // To the experts' lanes.
    for (int c = 0; c < a.top_k; c++) {
        const int ec = lane_get(ce, lane0 + c);
        const float dc = lane_get(cd, lane0 + c);
#pragma unroll
        for (int j = 0; j < V; j++)
            d[j] = L * j + l == ec ? dc : d[j];
    }
#pragma unroll
    for (int j = 0; j < V; j++) {
        const int e = L * j + l;
        if (live && e < E)
            st_elem<BF16>(a.d_logits, t * E + e, d[j]);
    }
}

template <bool BF16>
void route_backward_launch(const RouteBwdArgs &a, hipStream_t stream)
{
    const bool narrow = a.n_experts <= 256 && a.top_k <= 16;
    const int lanes = narrow ? 16 : 64, v = (a.n_experts + lanes - 1) / lanes;
    const int slots = ROUTE_THREADS / lanes;
    const dim3 grid((unsigned)((a.n_tokens + slots - 1) / slots)), block(ROUTE_THREADS);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    if (narrow)
        v <= 2    ? go(moe_route_backward_kernel<BF16, 16, 2>)
        : v <= 4  ? go(moe_route_backward_kernel<BF16, 16, 4>)
        : v <= 8  ? go(moe_route_backward_kernel<BF16, 16, 8>)
        : v <= 12 ? go(moe_route_backward_kernel<BF16, 16, 12>)
                  : go(moe_route_backward_kernel<BF16, 16, 16>);
    else
        v <= 2   ? go(moe_route_backward_kernel<BF16, 64, 2>)
        : v <= 8 ? go(moe_route_backward_kernel<BF16, 64, 8>)
                 : go(moe_route_backward_kernel<BF16, 64, 16>);
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

constexpr int COMBINE_THREADS = 256;              // at most; a thread takes 8 columns
constexpr int COMBINE_ROWS = 8;                   // rows of a token in flight

// Eight values of a row (16 bytes of BF16, 32 of FP32), as loaded.  Rows are
// read once and written once: accesses that do not stay in the caches.
template <bool BF16>
struct Raw8 {
    uint4 q[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *p, int64_t i)
    {
        if constexpr (BF16) {
            q[0] = ld_nt16(reinterpret_cast<const uint16_t *>(p) + i);
        } else {
            q[0] = ld_nt16(reinterpret_cast<const float *>(p) + i);
            q[1] = ld_nt16(reinterpret_cast<const float *>(p) + i + 4);
        }
    }
    __device__ __forceinline__ void zero()
    {
        for (auto &v : q)
            v = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ float operator[](int k) const
    {
        const uint4 &v = q[BF16 ? 0 : k / 4];
        const int c = BF16 ? k / 2 : k % 4;
        const uint32_t w = c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
        return !BF16 ? u2f(w) : (k & 1) ? bf16_hi(w) : bf16_lo(w);
    }
};
template <bool BF16>
__device__ __forceinline__ void st8v(void *p, int64_t i, const float (&v)[8])
{
    if constexpr (BF16) {
        u32x4_t q;
#pragma unroll
        for (int k = 0; k < 4; k++)
            q[k] = (uint32_t)bf16_rne(v[2 * k]) | (uint32_t)bf16_rne(v[2 * k + 1]) << 16;
        __builtin_nontemporal_store(
            q, reinterpret_cast<u32x4_t *>(reinterpret_cast<uint16_t *>(p) + i));
    } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const u32x4_t q = {f2u(v[4 * h]), f2u(v[4 * h + 1]), f2u(v[4 * h + 2]),
                               f2u(v[4 * h + 3])};
            __builtin_nontemporal_store(
                q, reinterpret_cast<u32x4_t *>(reinterpret_cast<float *>(p) + i + 4 * h));
        }
    }
}

// A workgroup per token (of as many threads as the columns want).  Bound by HBM:
// with inputs and outputs that are in no cache, 32768 tokens x 8 rows of 2048
// BF16 take 198 us (1.21 GB, 6.1 TB/s).  The rows of COMBINE_ROWS choices are
// loaded before the first is used: with a load and its sum in turn 261 us.
// Cached loads cost 213 us, cached stores 223 us, both 234 us.
template <bool BF16, bool BF16_OUT>
__global__ void __launch_bounds__(COMBINE_THREADS) moe_combine_kernel(
    const void *rows, int64_t total_rows, const int64_t *token_rows, const float *weights,
    int top_k, int64_t cols, int threads, void *out)
{
    const int64_t t = wg_id();
    for (int64_t c8 = 8 * (int64_t)tid(); c8 < cols; c8 += 8 * threads) {
        float acc[8] = {};
        for (int c0 = 0; c0 < top_k; c0 += COMBINE_ROWS) {
            Raw8<BF16> y[COMBINE_ROWS];
            float w[COMBINE_ROWS];
#pragma unroll
            for (int i = 0; i < COMBINE_ROWS; i++) {
                const int c = c0 + i < top_k ? c0 + i : top_k - 1;
                const int64_t r = token_rows[t * top_k + c];
                w[i] = weights[t * top_k + c];
                const bool live = c0 + i < top_k && r >= 0 && r < total_rows;
                y[i].zero();
                if (live)
                    y[i].load(rows, r * cols + c8);
                else
                    w[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < COMBINE_ROWS; i++)
#pragma unroll
                for (int k = 0; k < 8; k++)
                    acc[k] = __builtin_fmaf(w[i], y[i][k], acc[k]);
        }
        st8v<BF16_OUT>(out, t * cols + c8, acc);
    }
}

// d_rows[r] = w dout[t], d_weights = <dout[t], rows[r]>; the workgroups together
// zero the rows past the last segment.  9001 tokens x 8 rows of 2048 BF16, in no
// cache, take 114 us (598 MB, 5.2 TB/s; a copy of 300 MiB reaches 5.4): with
// cached loads 117 us, cached stores 124 us, with four rows in flight 122 us.
template <bool BF16>
__global__ void __launch_bounds__(COMBINE_THREADS) moe_combine_backward_kernel(
    const void *d_out, const void *rows, int64_t total_rows, const int64_t *token_rows,
    const float *weights, const int64_t *seg_end, int top_k, int64_t cols, int threads,
    void *d_rows, float *d_weights, int64_t n_wgs)
{
    __shared__ float part[COMBINE_ROWS][COMBINE_THREADS / 64];
    const int64_t t = wg_id();
    const int waves = threads / 64;
    if (seg_end) {
        const float zero[8] = {};
        int64_t end = *seg_end;
        end = end < 0 ? 0 : end;
        for (int64_t r = end + t; r < total_rows; r += n_wgs)
            for (int64_t c8 = 8 * (int64_t)tid(); c8 < cols; c8 += 8 * threads)
                st8v<BF16>(d_rows, r * cols + c8, zero);
    }
    for (int c0 = 0; c0 < top_k; c0 += COMBINE_ROWS) {
        float dot[COMBINE_ROWS] = {}, w[COMBINE_ROWS];
        int64_t r[COMBINE_ROWS];
#pragma unroll
        for (int i = 0; i < COMBINE_ROWS; i++) {
            const int c = c0 + i < top_k ? c0 + i : top_k - 1;
            r[i] = token_rows[t * top_k + c];
            w[i] = weights[t * top_k + c];
            if (c0 + i >= top_k || r[i] >= total_rows)
                r[i] = -1;
        }
        for (int64_t c8 = 8 * (int64_t)tid(); c8 < cols; c8 += 8 * threads) {
            Raw8<BF16> d, y[COMBINE_ROWS];
            d.load(d_out, t * cols + c8);
#pragma unroll
            for (int i = 0; i < COMBINE_ROWS; i++)
                if (r[i] >= 0)
                    y[i].load(rows, r[i] * cols + c8);
#pragma unroll
            for (int i = 0; i < COMBINE_ROWS; i++)
                if (r[i] >= 0) {
                    float g[8];
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        dot[i] = __builtin_fmaf(d[k], y[i][k], dot[i]);
                        g[k] = d[k] * w[i];
                    }
                    st8v<BF16>(d_rows, r[i] * cols + c8, g);
                }
        }
#pragma unroll
        for (int i = 0; i < COMBINE_ROWS; i++) {
            const float sum = wave_sum_f32(dot[i]);
            if (lane_id() == 0)
                part[i][wave_in_group()] = sum;
        }
        __syncthreads();
        const int i = (int)tid();
        if (i < COMBINE_ROWS && c0 + i < top_k) {
            float sum = 0.0f;
            for (int v = 0; v < waves; v++)
                sum += part[i][v];
            d_weights[t * top_k + c0 + i] = sum;
        }
        __syncthreads();
    }
}

// Threads of a token: 8 columns each, whole wavefronts.
int combine_threads(int64_t cols)
{
    const int64_t n = (cols / 8 + 63) / 64 * 64;
    return (int)(n < COMBINE_THREADS ? n : COMBINE_THREADS);
}

}  // namespace

hipError_t launch_moe_combine(bool bf16, const void *rows, int64_t total_rows,
                              const int64_t *token_rows, const float *weights, int64_t n_tokens,
                              int64_t top_k, int64_t cols, bool bf16_out, void *out,
                              hipStream_t stream)
{
    const int threads = combine_threads(cols);
    const dim3 grid((unsigned)n_tokens), block(threads);
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, rows, total_rows, token_rows, weights,
                           (int)top_k, cols, threads, out);
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
    const int threads = combine_threads(cols);
    const dim3 grid((unsigned)n_tokens), block(threads);
    const int64_t *end = seg_offsets ? seg_offsets + n_groups : nullptr;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, d_out, rows, total_rows, token_rows,
                           weights, end, (int)top_k, cols, threads, d_rows, d_weights, n_tokens);
    };
    bf16 ? launch(moe_combine_backward_kernel<true>) : launch(moe_combine_backward_kernel<false>);
    return hipGetLastError();
}

}  // namespace mxq
