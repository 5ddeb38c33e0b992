// mxq_attention.hip -- attention over a paged cache of NVFP4 keys and values
// (rows as the per-token quantizer writes them: codes, E4M3 block scales, one
// FP32 scale).  One wavefront per (sequence, query, head) walks the keys with
// the running maximum and sum of an online softmax.
#include "mxq_layer.h"
#include "mxq_layer_device.h"

namespace mxq {

namespace {

template <int D>
__global__ void __launch_bounds__(64) nvfp4_attention_kernel(AttnArgs a)
{
    constexpr int V = D / 64;                       // values per lane
    const uint32_t lane = lane_id();
    const int64_t id = wg_id();
    const int64_t head = id % a.n_heads, qi = id / a.n_heads % a.q_len,
                  b = id / a.n_heads / a.q_len;
    const int64_t kvh = head / (a.n_heads / a.n_kv_heads);
    int64_t len = a.seq_lens[b];
    const int64_t cap = a.max_pages * a.page_size;
    len = len < 0 ? 0 : len > cap ? cap : len;
    const int64_t pos = len - a.q_len + qi;
    const int64_t hi = a.causal ? pos + 1 : len;
    int64_t lo = a.window > 0 ? pos - a.window + 1 : 0;
    lo = lo < 0 ? 0 : lo;
    float q[V], o[V] = {};
#pragma unroll
    for (int j = 0; j < V; j++)
        q[j] = u2f((uint32_t)a.q[id * D + lane * V + j] << 16);
    float m = -3.0e38f, l = 0.0f;
    for (int64_t t = lo; t < hi; t++) {
        int64_t page = a.block_table[b * a.max_pages + t / a.page_size];
        page = page < 0 ? 0 : page >= a.n_pages ? a.n_pages - 1 : page;
        const int64_t row = (page * a.n_kv_heads + kvh) * a.page_size + t % a.page_size;
        auto value = [&](const uint8_t *codes, const uint8_t *bs, int j) {
            const int d = (int)lane * V + j;
            const uint32_t c = codes[row * (D / 2) + d / 2];
            return e2m1_values(c)[d & 1] * e4m3_value(bs[row * (D / 16) + d / 16]);
        };
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < V; j++)
            s = __builtin_fmaf(q[j], value(a.k, a.kbs, j), s);
        s = wave_sum_f32(s) * a.ks[row] * a.scale;
        const float mn = s > m ? s : m;
        const float al = exp_f32(m - mn), p = exp_f32(s - mn);
        m = mn;
        l = l * al + p;
        const float pv = p * a.vs[row];
#pragma unroll
        for (int j = 0; j < V; j++)
            o[j] = o[j] * al + pv * value(a.v, a.vbs, j);
    }
    const float r = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int j = 0; j < V; j++)
        a.out[id * D + lane * V + j] = bf16_rne(o[j] * r);
    if (a.lse && lane == 0)
        a.lse[id] = l > 0.0f ? m + __builtin_amdgcn_logf(l) * LN2 : -__builtin_inff();
}

}  // namespace

int64_t nvfp4_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t)
{
    return 0;
}

hipError_t launch_nvfp4_attention(const AttnArgs &a, void *, hipStream_t stream)
{
    const dim3 grid((unsigned)(a.n_seqs * a.q_len * a.n_heads)), block(64);
    if (a.head_dim == 64)
        hipLaunchKernelGGL(nvfp4_attention_kernel<64>, grid, block, 0, stream, a);
    else if (a.head_dim == 128)
        hipLaunchKernelGGL(nvfp4_attention_kernel<128>, grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL(nvfp4_attention_kernel<256>, grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxq
