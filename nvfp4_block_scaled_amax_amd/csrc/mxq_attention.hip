// mxq_attention.hip -- attention over a paged cache of NVFP4 keys and values
// (rows as the per-token quantizer writes them: codes, E4M3 block scales, one
// FP32 scale).
//
// Mathematics.  A wavefront keeps 16 RT query rows (the queries of one
// key/value head: q_len times the heads that share it) and walks keys 32 at a
// time.  S^T = K q^T and O^T += V^T P^T are 16x16x32 FP16 matrix instructions
// with the cache as their first operand, so that a query row is a lane
// column (lane % 16) throughout: the softmax's row maximum and sum are over a
// lane's own registers and the four lanes l, l + 16, l + 32, l + 48, and P
// leaves the first product's accumulators in the layout the second takes
// (its contraction index, the key, may come in any order that both operands
// share: slot j of lane group g is key 4g + j of the tile's first 16 keys
// for j < 4, of its second 16 otherwise).
//   dec(code) dec(block scale) is an exact FP16 value (6 significant bits).
// The FP32 scales stay out of the products: a key's scale multiplies its
// scores, a value's scale multiplies the softmax's numerators p, which are
// rounded to FP16 as p s_v 2^(14-E), with E the exponent of the running
// maximum of p s_v, tracked beside the running maximum of the scores: the
// largest numerator lands in [2^14, 2^15), and one within 2^-28 of it keeps
// all its 11 bits whatever the scales are.  A step with smaller ones (whose
// values may be all that an output element is made of, where the others'
// codes are 0) takes those in a second round of products under 2^29.  q is exact in FP16 under a
// power of two per row.
//   Operand order.  A lane reads the D/4 consecutive elements of a key that
// belong to its group (one 16-byte load at D = 128) and the queries are
// loaded in the same order.  Of a value row lane l reads elements D/16 l
// onwards; two keys' nibbles are merged byte-wise (even and odd elements),
// so that one conversion yields the pair (key t, key t + 1) of one element,
// which is what the second product's first operand holds.  Nothing of the
// cache passes through LDS.
//
// Split.  A workgroup of four wavefronts takes a chunk of the keys of one
// (sequence, key/value head, row tile), its wavefronts every fourth tile of
// it; they join through LDS.  The lengths are device data, so the chunks are
// planned on the device: every workgroup sums the lengths and derives the
// same chunk size, about ATT_TARGET equal chunks over the whole batch, so
// that long sequences take many workgroups and short ones one (with chunks
// planned on the host from the longest length, most workgroups of a ragged
// batch were empty, and those that were not sat on few XCDs: 221 us against
// 156 us with the XCDs evened out and XXX us planned here).  A sequence that
// is one chunk is written by its workgroup; otherwise partial results go to
// the workspace and a second kernel joins them.
#include "mxq_layer.h"
#include "mxq_layer_device.h"

namespace mxq {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int ATT_WAVES = 4, ATT_THREADS = 64 * ATT_WAVES;
constexpr int ATT_TILE = 32;                        // keys per step of a wavefront
constexpr int ATT_MIN_CHUNK = 2 * ATT_TILE * ATT_WAVES;
#ifndef ATT_T
#define ATT_T 1024
#endif
constexpr int ATT_TARGET = ATT_T;                   // chunks a launch aims at
constexpr float NO_MAX = -1.0e30f;                  // running maximum before the first key
constexpr float LOW = 0x1p-14f, LOW_UP = 0x1p29f;   // numerators of the second round

struct AttnK {
    const uint16_t *q;
    const uint8_t *k, *kbs;
    const float *ks;
    const uint8_t *v, *vbs;
    const float *vs;
    const int64_t *table, *lens;
    int64_t n_pages, max_pages;
    int q_len, n_heads, n_kv_heads, group, page_size, rows;   // rows = q_len * group
    Div page_div, group_div;
    float scale;                                     // softmax_scale * log2 e
    int causal, window;
    int n_seqs, row_tiles, tile_rows;                // tile_rows = 16 RT
    bool split;
    uint16_t *out;
    float *lse;
    float *part_ml, *part_o;                         // [unit][tile row][2], [..][D]
};

// Keys the rows of one row tile can see at most, over the tiles of sequence b
// (the plan's length of the sequence).
__device__ __forceinline__ int seq_len(const AttnK &a, int b)
{
    const int64_t cap = a.max_pages * a.page_size, n = a.lens[b];
    return (int)(n < 0 ? 0 : n > cap ? cap : n);
}
__device__ __forceinline__ int seq_span(const AttnK &a, int len)
{
    if (!a.causal || a.window == 0)
        return len;
    // The tile's first row reaches back window - 1 keys, rounded down to a tile.
    const int64_t w = (int64_t)a.window + a.tile_rows + ATT_TILE;
    return w < len ? (int)w : len;
}

__device__ __forceinline__ int wave_scan(int v, int lane)       // inclusive
{
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const int o = (int)lane_get((uint32_t)v, (uint32_t)(lane >= k ? lane - k : lane));
        v += lane >= k ? o : 0;
    }
    return v;
}
__device__ __forceinline__ int64_t wave_sum_i64(int64_t v, int lane)
{
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const uint32_t lo = lane_get((uint32_t)v, (uint32_t)(lane ^ k));
        const uint32_t hi = lane_get((uint32_t)((uint64_t)v >> 32), (uint32_t)(lane ^ k));
        v += (int64_t)((uint64_t)hi << 32 | lo);
    }
    return v;
}

// The chunk size of the batch: a multiple of a workgroup's step.
__device__ __forceinline__ int plan_chunk(const AttnK &a, int lane)
{
    int64_t keys = 0;
    for (int b = lane; b < a.n_seqs; b += 64)
        keys += seq_span(a, seq_len(a, b));
    keys = wave_sum_i64(keys, lane) * a.n_kv_heads * a.row_tiles;
    constexpr int STEP = ATT_TILE * ATT_WAVES;
    int64_t c = (keys / ATT_TARGET + STEP) / STEP * STEP;
    c = c < ATT_MIN_CHUNK ? ATT_MIN_CHUNK : c;
    return __builtin_amdgcn_readfirstlane((int)c);
}
__device__ __forceinline__ int plan_chunks(const AttnK &a, int span, int chunk)
{
    return !a.split || span <= chunk ? 1 : (span + chunk - 1) / chunk;
}
// A workgroup's share of the batch.
struct Unit {
    int b, kvh, tile, chunk, n_chunks, len, chunk_keys;
};
// Unit u of the plan; false past the last one.  per = units of one chunk of
// one sequence.
__device__ __forceinline__ bool plan_unit(const AttnK &a, uint32_t u, int lane, Unit *o)
{
    const uint32_t per = (uint32_t)(a.n_kv_heads * a.row_tiles);
    int chunk = 0;
    uint32_t rest;
    if (!a.split) {
        o->b = (int)(u / per);
        rest = u % per;
        o->len = seq_len(a, o->b);
        o->n_chunks = 1;
        o->chunk = 0;
    } else {
        chunk = plan_chunk(a, lane);
        int64_t left = u;
        bool found = false;
        for (int b0 = 0; b0 < a.n_seqs && !found; b0 += 64) {
            const int b = b0 + lane;
            const int len = b < a.n_seqs ? seq_len(a, b) : 0;
            const int n = b < a.n_seqs ? plan_chunks(a, seq_span(a, len), chunk) : 0;
            const int s = wave_scan(n, lane);
            // The first sequence whose units end past u.
            const uint64_t past = __builtin_amdgcn_ballot_w64((int64_t)s * per > left);
            if (past) {
                const int w = __builtin_ctzll(past);
                o->b = b0 + w;
                o->len = __builtin_amdgcn_readlane(len, w);
                o->n_chunks = __builtin_amdgcn_readlane(n, w);
                left -= (int64_t)(__builtin_amdgcn_readlane(s, w) - o->n_chunks) * per;
                found = true;
            } else {
                left -= (int64_t)__builtin_amdgcn_readlane(s, 63) * per;
            }
        }
        if (!found)
            return false;
        rest = (uint32_t)left % per;
        o->chunk = (int)((uint32_t)left / per);
    }
    // The last row tile sees the most keys: it goes first.
    o->tile = a.row_tiles - 1 - (int)(rest / (uint32_t)a.n_kv_heads);
    o->kvh = (int)(rest % (uint32_t)a.n_kv_heads);
    // Equal chunks of a sequence.
    constexpr int STEP = ATT_TILE * ATT_WAVES;
    const int span = seq_span(a, o->len);
    o->chunk_keys = o->n_chunks == 1 ? 0x40000000
                                     : ((span + o->n_chunks - 1) / o->n_chunks + STEP - 1) / STEP * STEP;
    return true;
}

__device__ __forceinline__ float max4_groups(float v)
{
    uint2_t r = __builtin_amdgcn_permlane16_swap(f2u(v), f2u(v), false, false);
    v = __builtin_fmaxf(u2f(r[0]), u2f(r[1]));
    r = __builtin_amdgcn_permlane32_swap(f2u(v), f2u(v), false, false);
    return __builtin_fmaxf(u2f(r[0]), u2f(r[1]));
}
__device__ __forceinline__ float sum4_groups(float v) { return sum32_f32(sum16_f32(v)); }

// One tile's cache data of a lane.
template <int D>
struct KvTile {
    static constexpr int KW = D / 32;                // dwords of a key's codes per lane
    static constexpr int VB = D / 32;                // bytes of a value's codes per lane
    uint32_t kc[2][KW], kb[2];
    f32x4_t ks[2], vs[2];
    uint32_t vc[8][VB > 4 ? VB / 4 : 1], vb[8];
};

// Where a tile's two 16-key halves lie: the page (as the table holds it) and the
// slot in it.  The rows are formed where they are used, so that the table's
// loads have a step's time to arrive.
struct TilePages {
    int64_t page[2];
    int slot[2];
};
__device__ __forceinline__ TilePages tile_pages(const AttnK &a, const int64_t *table, int t0)
{
    TilePages o;
    const int last = (int)(a.max_pages * a.page_size) - 16;
#pragma unroll
    for (int s = 0; s < 2; s++) {
        int t = t0 + 16 * s;
        t = t < last ? t : last;                     // halves past the table: masked by length
        const uint32_t pi = udiv((uint32_t)t, a.page_div);
        o.page[s] = table[pi];
        o.slot[s] = t - (int)pi * a.page_size;
    }
    return o;
}

template <int D>
__device__ __forceinline__ void load_tile(KvTile<D> &x, const AttnK &a, const TilePages &pages,
                                          int kvh, int l, int g)
{
    constexpr int KW = KvTile<D>::KW, VB = KvTile<D>::VB;
#pragma unroll
    for (int s = 0; s < 2; s++) {
        int64_t page = pages.page[s];
        page = page < 0 ? 0 : page >= a.n_pages ? a.n_pages - 1 : page;
        const int64_t r = (page * a.n_kv_heads + kvh) * a.page_size + pages.slot[s];
        const uint8_t *kc = a.k + r * (D / 2) + (uint32_t)(l * (D / 2) + g * (D / 8));
        const uint8_t *kb = a.kbs + r * (D / 16) + (uint32_t)(l * (D / 16) + g * (D / 64));
        if constexpr (KW == 2) {
            const uint2 c = ld8(kc);
            x.kc[s][0] = c.x;
            x.kc[s][1] = c.y;
            x.kb[s] = *kb;
        } else {
#pragma unroll
            for (int j = 0; j < KW / 4; j++) {
                const uint4 c = ld16(kc + 16 * j);
                x.kc[s][4 * j] = c.x;
                x.kc[s][4 * j + 1] = c.y;
                x.kc[s][4 * j + 2] = c.z;
                x.kc[s][4 * j + 3] = c.w;
            }
            if constexpr (KW == 4)
                x.kb[s] = *reinterpret_cast<const uint16_t *>(kb);
            else
                x.kb[s] = *reinterpret_cast<const uint32_t *>(kb);
        }
        x.ks[s] = *reinterpret_cast<const f32x4_t *>(a.ks + r + 4 * g);
        x.vs[s] = *reinterpret_cast<const f32x4_t *>(a.vs + r + 4 * g);
        const uint8_t *vc = a.v + r * (D / 2) + (uint32_t)(4 * g * (D / 2) + l * VB);
        const uint8_t *vb = a.vbs + r * (D / 16) + (uint32_t)(4 * g * (D / 16) + l * (D / 16) / 16);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint8_t *p = vc + i * (D / 2);
            if constexpr (VB == 2)
                x.vc[4 * s + i][0] = *reinterpret_cast<const uint16_t *>(p);
            else if constexpr (VB == 4)
                x.vc[4 * s + i][0] = *reinterpret_cast<const uint32_t *>(p);
            else {
                const uint2 c = ld8(p);
                x.vc[4 * s + i][0] = c.x;
                x.vc[4 * s + i][1] = c.y;
            }
            x.vb[4 * s + i] = vb[i * (D / 16)];
        }
    }
}

// E4M3 byte -> FP16 (exact).
__device__ __forceinline__ _Float16 e4m3_f16(uint32_t byte) { return (_Float16)e4m3_value(byte); }

template <int J>
__device__ __forceinline__ f16x2_t pair_f16(uint32_t codes)
{
    return __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, J));
}
__device__ __forceinline__ f16x8_t cat8(f16x2_t a, f16x2_t b, f16x2_t c, f16x2_t d)
{
    return f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// Eight elements (one dword of codes) under one block scale.
__device__ __forceinline__ f16x8_t oct_f16(uint32_t codes, f16x2_t d)
{
    return cat8(pair_f16<0>(codes) * d, pair_f16<1>(codes) * d, pair_f16<2>(codes) * d,
                pair_f16<3>(codes) * d);
}
__device__ __forceinline__ f16x2_t pair_f16_dyn(uint32_t codes, int j)
{
    return j == 0 ? pair_f16<0>(codes) : j == 1 ? pair_f16<1>(codes)
         : j == 2 ? pair_f16<2>(codes) : pair_f16<3>(codes);
}

// State of a wavefront's 16 RT rows.  Row (lane % 16) of tile rt: running
// maximum m of the scores (log2 units), this lane's part of the sum l, the
// running maximum w of p s_v relative to m, and O^T in units of 2^(e - 14).
template <int D, int RT>
struct Rows {
    f16x8_t q[RT][D / 32];
    float c[RT];                                     // score factor of the row
    float m[RT], l[RT], w[RT];
    int e[RT];
    f32x4_t o[RT][D / 16];
};

template <int D, int RT, bool MASKED>
__device__ __forceinline__ void attend(Rows<D, RT> &st, const KvTile<D> &x, int t0, int len,
                                       const int (&lo)[RT], const int (&hi)[RT], int g)
{
    constexpr int KK = D / 32;
    // Scores: two 16-key halves, KK steps of 8 elements per lane group.
    f32x4_t s[2][RT];
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
            s[h][rt] = f32x4_t{};
#pragma unroll
        for (int kk = 0; kk < KK; kk++) {
            // The D/4 elements of a lane hold D/64 blocks of 16 (two dwords each).
            const _Float16 d = e4m3_f16((x.kb[h] >> (8 * (kk / 2))) & 0xFFu);
            const f16x8_t kf = oct_f16(x.kc[h][kk], f16x2_t{d, d});
#pragma unroll
            for (int rt = 0; rt < RT; rt++)
                s[h][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, st.q[rt][kk], s[h][rt], 0, 0,
                                                                   0);
        }
    }
    f32x4_t vs[2] = {x.vs[0], x.vs[1]};
    if constexpr (MASKED) {
        // Slots past the length may hold anything: their value scales count as 0.
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (t0 + 16 * (j >> 2) + 4 * g + (j & 3) >= len)
                vs[j >> 2][j & 3] = 0.0f;
    }
    f16x8_t p8[RT], p8lo[RT];
    bool any_low = false;
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        float z[8], tm = NO_MAX;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            z[j] = s[j >> 2][rt][j & 3] * (x.ks[j >> 2][j & 3] * st.c[rt]);
            if constexpr (MASKED) {
                const int t = t0 + 16 * (j >> 2) + 4 * g + (j & 3);
                z[j] = t >= lo[rt] && t < hi[rt] ? z[j] : NO_MAX;
            }
            tm = __builtin_fmaxf(tm, z[j]);
        }
        tm = max4_groups(tm);
        const float mn = __builtin_fmaxf(st.m[rt], tm);
        const float al = __builtin_amdgcn_exp2f(st.m[rt] - mn);
        float sum = 0.0f, pw[8], wm = 0.0f, pm = 1.0e30f;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float p = __builtin_amdgcn_exp2f(z[j] - mn);
            if constexpr (MASKED)
                p = z[j] == NO_MAX ? 0.0f : p;
            sum += p;
            pw[j] = p * vs[j >> 2][j & 3];
            wm = __builtin_fmaxf(wm, pw[j]);
            pm = __builtin_fminf(pm, pw[j]);
        }
        wm = max4_groups(wm);
        const float wn = __builtin_fmaxf(st.w[rt] * al, wm);
        int e = (int)(f2u(wn) >> 23) - 127;
        // Twelve binades above the smallest normal number: 2^(14 - e) stays finite.
        e = e < -112 ? -112 : e;
        const float up = u2f((uint32_t)(14 - e + 127) << 23);       // 2^(14 - e)
        const float f = __builtin_ldexpf(al, st.e[rt] - e);
        st.m[rt] = mn;
        st.l[rt] = __builtin_fmaf(st.l[rt], al, sum);
        st.w[rt] = wn;
        st.e[rt] = e;
#pragma unroll
        for (int j = 0; j < D / 16; j++)
            st.o[rt][j] *= f;
        p8lo[rt] = f16x8_t{};
        if (__builtin_amdgcn_ballot_w64(pm * up < LOW) != 0) {      // zeros too: harmless
            any_low = true;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float x = pw[j] * up;
                p8lo[rt][j] = (_Float16)(x < LOW ? x * LOW_UP : 0.0f);
                p8[rt][j] = (_Float16)(x < LOW ? 0.0f : x);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                p8[rt][j] = (_Float16)(pw[j] * up);
        }
    }
    // Values: pairs of keys (2i, 2i + 1) of the lane group's eight.
    f16x2_t vd[4];
    uint32_t ev[4][KvTile<D>::VB > 4 ? 2 : 1], od[4][KvTile<D>::VB > 4 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t b0 = x.vb[2 * i], b1 = x.vb[2 * i + 1];
        if constexpr (MASKED) {
            const int t = t0 + 16 * (i >> 1) + 4 * g + 2 * (i & 1);
            b0 = t < len ? b0 : 0;
            b1 = t + 1 < len ? b1 : 0;
        }
        vd[i] = f16x2_t{e4m3_f16(b0), e4m3_f16(b1)};
#pragma unroll
        for (int wd = 0; wd < (KvTile<D>::VB > 4 ? 2 : 1); wd++) {
            const uint32_t c0 = x.vc[2 * i][wd], c1 = x.vc[2 * i + 1][wd];
            ev[i][wd] = (c0 & 0x0F0F0F0Fu) | ((c1 << 4) & 0xF0F0F0F0u);
            od[i][wd] = ((c0 >> 4) & 0x0F0F0F0Fu) | (c1 & 0xF0F0F0F0u);
        }
    }
    auto values = [&](int j) {
        f16x2_t v[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = pair_f16_dyn((j & 1) ? od[i][j >> 3] : ev[i][j >> 3], (j >> 1) & 3) * vd[i];
        return cat8(v[0], v[1], v[2], v[3]);
    };
#pragma unroll
    for (int j = 0; j < D / 16; j++) {
        const f16x8_t vf = values(j);
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
            st.o[rt][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p8[rt], st.o[rt][j], 0, 0, 0);
    }
    if (any_low) {
        // Decoded anew: kept from the first round they would cost every step's registers.
#pragma unroll
        for (int i = 0; i < 4; i++)
            asm("" : "+v"(ev[i][0]), "+v"(od[i][0]));
#pragma unroll
        for (int j = 0; j < D / 16; j++) {
            const f16x8_t vf = values(j);
#pragma unroll
            for (int rt = 0; rt < RT; rt++) {
                const f32x4_t o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p8lo[rt], f32x4_t{},
                                                                         0, 0, 0);
                st.o[rt][j] += o * (1.0f / LOW_UP);
            }
        }
    }
}

template <int D, int RT>
__global__ void __launch_bounds__(ATT_THREADS, RT == 1 && D <= 128 ? 2 : 1)
    nvfp4_attention_kernel(AttnK a)
{
    constexpr int ROWS = 16 * RT;
    __shared__ float lds_ml[ATT_WAVES][ROWS][2];
    // Rows padded by four floats: the 16 rows a store touches miss each other's banks.
    __shared__ __attribute__((aligned(16))) float lds_o[ATT_WAVES][ROWS][D + 4];

    const int lane = (int)lane_id(), l = lane & 15, g = lane >> 4, wave = wave_in_group();
    Unit un;
    if (!plan_unit(a, wg_id(), lane, &un))
        return;
    const int tile = un.tile, kvh = un.kvh, b = un.b, len = un.len;

    // Keys the tile's rows see: [kmin, kmax); this workgroup's part of them.
    const int r0 = tile * ROWS;
    const int r1 = r0 + ROWS < a.rows ? r0 + ROWS : a.rows;
    const int first = len - a.q_len + (int)udiv((uint32_t)r0, a.group_div);
    const int last = len - a.q_len + (int)udiv((uint32_t)(r1 - 1), a.group_div);
    const int kmax = a.causal ? (last + 1 < 0 ? 0 : last + 1) : len;
    int kmin = a.causal && a.window > 0 ? first - a.window + 1 : 0;
    kmin = kmin < 0 ? 0 : kmin & ~(ATT_TILE - 1);
    const int64_t start64 = (int64_t)kmin + (int64_t)un.chunk * un.chunk_keys;
    const int start = start64 < kmax ? (int)start64 : kmax;
    const int stop = kmax - start < un.chunk_keys ? kmax : start + un.chunk_keys;

    Rows<D, RT> st;
    int lo[RT], hi[RT];
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const int r = r0 + 16 * rt + l < a.rows ? r0 + 16 * rt + l : a.rows - 1;
        const int qi = (int)udiv((uint32_t)r, a.group_div);
        const int pos = len - a.q_len + qi;
        hi[rt] = a.causal ? pos + 1 : len;
        lo[rt] = a.causal && a.window > 0 ? pos - a.window + 1 : 0;
        const int64_t qrow = ((int64_t)b * a.q_len + qi) * a.n_heads + kvh * a.group +
                             (r - qi * a.group);
        const uint16_t *qp = a.q + qrow * D + g * (D / 4);
        uint4 raw[D / 32];
        uint32_t am = 0;
#pragma unroll
        for (int kk = 0; kk < D / 32; kk++) {
            raw[kk] = ld16(qp + 8 * kk);
            am = pk_max_u16(am, pk_max_u16(pk_max_u16(raw[kk].x & 0x7FFF7FFFu,
                                                      raw[kk].y & 0x7FFF7FFFu),
                                           pk_max_u16(raw[kk].z & 0x7FFF7FFFu,
                                                      raw[kk].w & 0x7FFF7FFFu)));
        }
        am = max32_u32(max16_u32(hmax_u16(am)));
        // Largest magnitude into [2^14, 2^15): exact for values within 2^-31 of it.
        const int e = (int)(am >> 7) - 127 - 14;
        st.c[rt] = __builtin_ldexpf(a.scale, e);
#pragma unroll
        for (int kk = 0; kk < D / 32; kk++) {
            const uint32_t w[4] = {raw[kk].x, raw[kk].y, raw[kk].z, raw[kk].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                st.q[rt][kk][2 * i] = (_Float16)__builtin_ldexpf(bf16_lo(w[i]), -e);
                st.q[rt][kk][2 * i + 1] = (_Float16)__builtin_ldexpf(bf16_hi(w[i]), -e);
            }
        }
        st.m[rt] = NO_MAX;
        st.l[rt] = 0.0f;
        st.w[rt] = 0.0f;
        st.e[rt] = -112;
#pragma unroll
        for (int j = 0; j < D / 16; j++)
            st.o[rt][j] = f32x4_t{};
    }

    const int64_t *table = a.table + (int64_t)b * a.max_pages;
    constexpr int STEP = ATT_TILE * ATT_WAVES;
    // Keys every row sees: a tile inside [full_lo, full_hi) needs no mask.
    const int full_hi = a.causal ? (first + 1 < len ? first + 1 : len) : len;
    const int full_lo = a.causal && a.window > 0 ? last - a.window + 1 : 0;
    int t0 = start + wave * ATT_TILE;
    if (t0 < stop) {
        // Two register sets take turns: while one tile is worked on, the next one's
        // loads are in flight and the page of the one after is looked up (steps past
        // the last read the last tile again).
        const int t_last = t0 + (stop - 1 - t0) / STEP * STEP;
        auto at = [&](int t) { return tile_pages(a, table, t < t_last ? t : t_last); };
        auto work = [&](const KvTile<D> &x, int t) {
            if (t >= full_lo && t + ATT_TILE <= full_hi)
                attend<D, RT, false>(st, x, t, len, lo, hi, g);
            else
                attend<D, RT, true>(st, x, t, len, lo, hi, g);
        };
        KvTile<D> x0, x1;
        load_tile<D>(x0, a, at(t0), kvh, l, g);
        TilePages next = at(t0 + STEP);
        for (;;) {
            load_tile<D>(x1, a, next, kvh, l, g);
            next = at(t0 + 2 * STEP);
            work(x0, t0);
            if (t0 == t_last)
                break;
            load_tile<D>(x0, a, next, kvh, l, g);
            next = at(t0 + 3 * STEP);
            work(x1, t0 + STEP);
            t0 += 2 * STEP;
            if (t0 > t_last)
                break;
        }
    }

    // Join the four wavefronts.
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        st.l[rt] = sum4_groups(st.l[rt]);
        if (g == 0) {
            lds_ml[wave][16 * rt + l][0] = st.m[rt];
            lds_ml[wave][16 * rt + l][1] = st.l[rt];
        }
    }
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const int r = 16 * rt + l;
        float m = NO_MAX;
#pragma unroll
        for (int w = 0; w < ATT_WAVES; w++)
            m = __builtin_fmaxf(m, lds_ml[w][r][0]);
        const float f = __builtin_ldexpf(__builtin_amdgcn_exp2f(st.m[rt] - m), st.e[rt] - 14);
        // Element 4g + i of lane column l, tile j: d = (4g + i) D/16 + j.
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < D / 16; j++)
                lds_o[wave][r][(4 * g + i) * (D / 16) + j] = st.o[rt][j][i] * f;
    }
    __syncthreads();
    constexpr int PER = D / 8;                       // 8 elements per thread
    for (int i = (int)tid(); i < (r1 - r0) * PER; i += ATT_THREADS) {
        const int r = i / PER, d = 8 * (i % PER);
        float m = NO_MAX, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < ATT_WAVES; w++)
            m = __builtin_fmaxf(m, lds_ml[w][r][0]);
#pragma unroll
        for (int w = 0; w < ATT_WAVES; w++)
            sum += lds_ml[w][r][1] * __builtin_amdgcn_exp2f(lds_ml[w][r][0] - m);
        float o[8] = {};
#pragma unroll
        for (int w = 0; w < ATT_WAVES; w++)
#pragma unroll
            for (int j = 0; j < 8; j++)
                o[j] += lds_o[w][r][d + j];
        const int qi = (int)udiv((uint32_t)(r0 + r), a.group_div);
        const int64_t qrow = ((int64_t)b * a.q_len + qi) * a.n_heads + kvh * a.group +
                             (r0 + r - qi * a.group);
        if (un.n_chunks == 1) {
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            u32x4_t v;
#pragma unroll
            for (int j = 0; j < 4; j++)
                v[j] = (uint32_t)bf16_rne(o[2 * j] * inv) |
                       (uint32_t)bf16_rne(o[2 * j + 1] * inv) << 16;
            *reinterpret_cast<u32x4_t *>(a.out + qrow * D + d) = v;
            if (a.lse && d == 0)
                a.lse[qrow] = sum > 0.0f ? (m + __builtin_amdgcn_logf(sum)) * LN2
                                         : -__builtin_inff();
        } else {
            const int64_t pr = (int64_t)wg_id() * ROWS + r;
            if (d == 0) {
                a.part_ml[2 * pr] = m;
                a.part_ml[2 * pr + 1] = sum;
            }
            if (sum > 0.0f)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    *reinterpret_cast<f32x4_t *>(a.part_o + pr * D + d + 4 * h) =
                        f32x4_t{o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]};
        }
    }
}

// Joins the chunks of one row per wavefront: sum_c 2^(m_c - m) O_c / sum.
// Rows of one chunk were written by their workgroup.
template <int D>
__global__ void __launch_bounds__(256) nvfp4_attention_join_kernel(AttnK a)
{
    const int lane = (int)lane_id();
    const int64_t row = (int64_t)wg_id() * 4 + wave_in_group();
    if (row >= (int64_t)a.n_seqs * a.q_len * a.n_heads)
        return;
    constexpr int V = D / 64;
    const int head = (int)(row % a.n_heads), qi = (int)(row / a.n_heads % a.q_len);
    const int b = (int)(row / a.n_heads / a.q_len);
    const int chunk = plan_chunk(a, lane);
    const int n = plan_chunks(a, seq_span(a, seq_len(a, b)), chunk);
    if (n == 1)
        return;
    int64_t before = 0;                             // chunks of the sequences before b
    for (int i = lane; i < b; i += 64)
        before += plan_chunks(a, seq_span(a, seq_len(a, i)), chunk);
    before = wave_sum_i64(before, lane);
    const int r = qi * a.group + head % a.group;
    const int64_t per = (int64_t)a.n_kv_heads * a.row_tiles;
    const int64_t unit = before * per +
                         (int64_t)(a.row_tiles - 1 - r / a.tile_rows) * a.n_kv_heads +
                         head / a.group;
    const int64_t p0 = unit * a.tile_rows + r % a.tile_rows, step = per * a.tile_rows;
    float m = NO_MAX;
    for (int c = lane; c < n; c += 64) {
        const float *ml = a.part_ml + 2 * (p0 + c * step);
        m = __builtin_fmaxf(m, ml[1] > 0.0f ? ml[0] : NO_MAX);
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1)
        m = __builtin_fmaxf(m, lane_get(m, (uint32_t)(lane ^ k)));
    // Lane c holds the factor of chunk c0 + c; the parts are loaded eight at a time
    // (a chunk without keys has none: its slot is read, but not used).
    float sum = 0.0f, o[V] = {};
    for (int c0 = 0; c0 < n; c0 += 64) {
        const int c = c0 + lane < n ? c0 + lane : n - 1;
        const float *ml = a.part_ml + 2 * (p0 + c * step);
        const float lc = c0 + lane < n ? ml[1] : 0.0f;
        const float f = lc > 0.0f ? __builtin_amdgcn_exp2f(ml[0] - m) : 0.0f;
        sum = __builtin_fmaf(lc, f, sum);
        const int cn = n - c0 < 64 ? n - c0 : 64;
        for (int i = 0; i < cn; i += 8) {
            float v[8][V];
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const int ck = c0 + (i + k < cn ? i + k : cn - 1);
                const float *p = a.part_o + (p0 + ck * step) * D + lane;
#pragma unroll
                for (int j = 0; j < V; j++)
                    v[k][j] = p[64 * j];
            }
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const int ik = i + k < cn ? i + k : cn - 1;
                const float fk = u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(f), ik));
                if (i + k < cn && fk > 0.0f)
#pragma unroll
                    for (int j = 0; j < V; j++)
                        o[j] = __builtin_fmaf(v[k][j], fk, o[j]);
            }
        }
    }
    sum = wave_sum_f32(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int j = 0; j < V; j++)
        a.out[row * D + 64 * j + lane] = bf16_rne(o[j] * inv);
    if (a.lse && lane == 0)
        a.lse[row] = sum > 0.0f ? (m + __builtin_amdgcn_logf(sum)) * LN2 : -__builtin_inff();
}

// Row tiles of a launch, and the most units its plan can have: a chunk more
// per (sequence, head, row tile) than its share of ATT_TARGET.
struct AttnPlan {
    int rt, row_tiles;
    bool split;
    int64_t units;
};
AttnPlan attention_plan(int64_t n_seqs, int64_t q_len, int64_t n_heads, int64_t n_kv_heads,
                        int64_t head_dim, int64_t max_keys)
{
    const int64_t rows = q_len * (n_heads / n_kv_heads);
    // More rows share a key's decoding, as far as a wavefront's registers go: 64 rows
    // of 64 elements, 32 of 128, 16 of 256.
    const int most_rt = head_dim == 64 ? 4 : head_dim == 128 ? 2 : 1;
    const int want_rt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    const int rt = want_rt < most_rt ? want_rt : most_rt;
    const int64_t row_tiles = (rows + 16 * rt - 1) / (16 * rt);
    const int64_t base = n_seqs * n_kv_heads * row_tiles;
    // With enough row tiles to fill the chip, or keys for one chunk, none is split.
    const bool split = base < ATT_TARGET && max_keys > ATT_MIN_CHUNK;
    const int64_t most = base * ((max_keys + ATT_MIN_CHUNK - 1) / ATT_MIN_CHUNK);
    const int64_t units = !split ? base : most < ATT_TARGET + base ? most : ATT_TARGET + base;
    return AttnPlan{rt, (int)row_tiles, split, units};
}

}  // namespace

int64_t nvfp4_attention_workspace(int64_t n_seqs, int64_t q_len, int64_t n_heads,
                                  int64_t n_kv_heads, int64_t head_dim, int64_t max_keys)
{
    const AttnPlan p = attention_plan(n_seqs, q_len, n_heads, n_kv_heads, head_dim, max_keys);
    return p.split ? p.units * 16 * p.rt * (head_dim + 2) * 4 : 0;
}

template <int D, int RT>
static void attention_launch(const AttnK &k, int64_t wgs, hipStream_t stream)
{
    hipLaunchKernelGGL((nvfp4_attention_kernel<D, RT>), dim3((unsigned)wgs), dim3(ATT_THREADS), 0,
                       stream, k);
}

hipError_t launch_nvfp4_attention(const AttnArgs &a, void *workspace, hipStream_t stream)
{
    const int64_t max_keys = a.max_pages * a.page_size;
    const AttnPlan p = attention_plan(a.n_seqs, a.q_len, a.n_heads, a.n_kv_heads, a.head_dim,
                                      max_keys);
    const int64_t n_rows = a.n_seqs * a.q_len * a.n_heads;
    float *ml = static_cast<float *>(workspace);
    const int group = (int)(a.n_heads / a.n_kv_heads);
    const AttnK k{a.q, a.k, a.kbs, a.ks, a.v, a.vbs, a.vs, a.block_table, a.seq_lens, a.n_pages,
                  a.max_pages, (int)a.q_len, (int)a.n_heads, (int)a.n_kv_heads, group,
                  (int)a.page_size, (int)(a.q_len * group), make_div((uint32_t)a.page_size),
                  make_div((uint32_t)group), a.scale * LOG2E, a.causal ? 1 : 0,
                  (int)(a.window < 0x7FFFFFFF ? a.window : 0x7FFFFFFF), (int)a.n_seqs,
                  p.row_tiles, 16 * p.rt, p.split, a.out, a.lse, ml,
                  p.split ? ml + p.units * 16 * p.rt * 2 : nullptr};
    const int64_t wgs = p.units;
    if (a.head_dim == 64)
        p.rt == 1 ? attention_launch<64, 1>(k, wgs, stream)
        : p.rt == 2 ? attention_launch<64, 2>(k, wgs, stream)
                    : attention_launch<64, 4>(k, wgs, stream);
    else if (a.head_dim == 128)
        p.rt == 1 ? attention_launch<128, 1>(k, wgs, stream)
                  : attention_launch<128, 2>(k, wgs, stream);
    else
        attention_launch<256, 1>(k, wgs, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.split)
        return e;
    const dim3 grid((unsigned)((n_rows + 3) / 4)), block(256);
    auto join = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, k);
    };
    if (a.head_dim == 64)
        join(nvfp4_attention_join_kernel<64>);
    else if (a.head_dim == 128)
        join(nvfp4_attention_join_kernel<128>);
    else
        join(nvfp4_attention_join_kernel<256>);
    return hipGetLastError();
}

}  // namespace mxq
