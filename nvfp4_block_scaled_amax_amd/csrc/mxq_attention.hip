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
// scores, and a value's scale s_v goes into the softmax's exponent, so that
// the numerators are 2^(z + log2 s_v - m + TOP), m the running maximum of
// z + log2 s_v (to within SLACK).  They are rounded to FP16: the largest is
// 2^11 to 2^15, and one within 2^-25 of it keeps all its 11 bits whatever
// the scales are.  A step with smaller ones (whose values may be all that an
// output element is made of, where the others' codes are 0) takes those in
// further rounds of products, under 2^29, 2^58 .. as far as FP32 reaches.  The sum takes each numerator times 1 / s_v.  q is
// exact in FP16 under a power of two per row.
//   Operand order.  A lane reads the D/4 consecutive elements of a key that
// belong to its group (16 bytes at D = 128) and the queries are loaded in the
// same order.  Of a value row lane l reads elements D/16 l onwards; two keys'
// nibbles are merged byte-wise (even and odd elements), so that one
// conversion yields the pair (key t, key t + 1) of one element, which is what
// the second product's first operand holds.
//
// Pipeline.  A wavefront copies its tiles straight into LDS
// (global_load_lds, which needs no registers), ATT_STAGES tiles deep, and
// waits for its own copies by count; nothing is shared between wavefronts,
// so there is no barrier in the loop.  (Tiles in registers, one ahead: 44
// loads a tile instead of 7, and 90 registers more.)
//
// Split.  A workgroup of four wavefronts takes a chunk of the keys of one
// (sequence, key/value head, row tile), its wavefronts every fourth tile of
// it; they join through LDS.  The lengths are device data, so the chunks are
// planned on the device: every workgroup sums the lengths and derives the
// same chunk size, about ATT_TARGET equal chunks over the whole batch, so
// that long sequences take many workgroups and short ones one (with chunks
// planned on the host from the longest length, most workgroups of a ragged
// batch were empty, and those that were not sat on few XCDs: 221 us against
// 156 us with the XCDs evened out, 71 us planned here).  A sequence that
// is one chunk is written by its workgroup; otherwise partial results go to
// the workspace and a second kernel joins them.
#include <type_traits>

#include "mxq_layer.h"
#include "mxq_layer_device.h"

namespace mxq {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int ATT_WAVES = 4, ATT_THREADS = 64 * ATT_WAVES;
constexpr int ATT_TILE = 32;                        // keys per step of a wavefront
constexpr int ATT_MIN_CHUNK = 2 * ATT_TILE * ATT_WAVES;
constexpr int ATT_TARGET = 640;                    // chunks a launch aims at
constexpr int WIDE_WAVES = 8, WIDE_THREADS = 64 * WIDE_WAVES;       // many query rows: see below
constexpr int WIDE_RT = 2, WIDE_ROWS = 16 * WIDE_RT * WIDE_WAVES;
constexpr int WIDE_TARGET = 480;                   // chunks of its launch (232: 145 us, 1000: 144)
constexpr int WIDE_TILES = 200;                    // least row tiles of 32 for it
constexpr float NO_MAX = -1.0e30f;                  // running maximum before the first key
constexpr float TOP = 11.0f, SLACK = 4.0f;          // numerators: 2^TOP at m, 2^15 at m + SLACK
constexpr float LOW_LOG2 = -14.0f, LOW = 0x1p-14f;  // smaller ones go to further rounds,
constexpr float LOW_UP = 0x1p29f;                   // each under this factor more
constexpr float MIN_VS = 0x1p-100f;                 // value scales below count as 0
constexpr float ZERO_VS = 0x1p-8f;                  // the scale of a tile without other ones
constexpr float MAX_SUM = 0x1p90f, SUM_STEP = 40.0f;  // a larger sum raises m by this much
constexpr int ATT_STAGES = 2;                      // tiles in LDS per wavefront

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
    int n_seqs, row_tiles, tile_rows, target;        // target: chunks of the launch
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
    const int w = a.window + a.tile_rows + ATT_TILE;
    return w < len ? w : len;
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
    int64_t c = (keys / a.target + STEP) / STEP * STEP;
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

// The cache rows of a tile's two 16-key halves (their first keys; a half lies
// in one page, so its 16 rows are consecutive).
struct TileRows {
    int64_t r[2];
};
// Rows of a wavefront's next 64 tiles, one tile a lane.  Looked up tile by tile
// with scalar loads, the page table cost every step a memory latency: LDS
// reads wait for the same counter.
struct RowWindow {
    uint32_t lo[2], hi[2];
};
__device__ __forceinline__ RowWindow row_window(const AttnK &a, const int64_t *table, int kvh,
                                                int t0, int step, int t_last, int lane)
{
    RowWindow w;
    const int last = (int)(a.max_pages * a.page_size) - 16;
    // Tiles past the wavefront's last stand for it.
    const int n = (t_last - t0) / step;
    const int tile = t0 + (lane < n ? lane : n) * step;
#pragma unroll
    for (int s = 0; s < 2; s++) {
        int t = tile + 16 * s;
        t = t < last ? t : last;                     // halves past the table: masked by length
        const uint32_t pi = udiv((uint32_t)t, a.page_div);
        int64_t page = table[pi];
        page = page < 0 ? 0 : page >= a.n_pages ? a.n_pages - 1 : page;
        const int64_t r = (page * a.n_kv_heads + kvh) * a.page_size + (t - (int)pi * a.page_size);
        w.lo[s] = (uint32_t)r;
        w.hi[s] = (uint32_t)((uint64_t)r >> 32);
    }
    return w;
}
__device__ __forceinline__ TileRows window_rows(const RowWindow &w, int i)
{
    TileRows o;
#pragma unroll
    for (int s = 0; s < 2; s++)
        o.r[s] = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)w.hi[s], i) << 32 |
                           (uint32_t)__builtin_amdgcn_readlane((int)w.lo[s], i));
    return o;
}

// A tile in LDS: codes of the 32 keys, codes of the values, block scales of
// both, and the FP32 scales (keys, then values).
template <int D>
struct Stage {
    static constexpr int CODES = 32 * (D / 2), BLOCKS = 32 * (D / 16);
    static constexpr int BLOCK_ROOM = BLOCKS < 256 ? 256 : BLOCKS;     // whole 64-lane copies
    static constexpr int K = 0, V = CODES, KB = 2 * CODES, VB = KB + BLOCK_ROOM,
                         S = VB + BLOCK_ROOM, BYTES = S + 256;
    static constexpr int COPIES = 2 * (CODES / 1024) + 2 * (BLOCK_ROOM / 256) + 1;
};

// Copies of 16 or 4 bytes a lane from per-lane addresses to LDS bytes lds + 16 lane
// (4 lane).  The compiler does not track them: the loop counts them, and the wait
// state that the copy needs after the write of M0 is the s_nop.
__device__ __forceinline__ void to_lds16(const uint8_t *p, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(p), "s"(lds)
                 : "memory", "m0");
}
// The same from a wave-uniform base and a lane's offset.
__device__ __forceinline__ void to_lds16(const uint8_t *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}
__device__ __forceinline__ void to_lds4(const uint8_t *p, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
                 :
                 : "v"(p), "s"(lds)
                 : "memory", "m0");
}
// Waits until at most N of the wavefront's copies are outstanding.
template <int N>
__device__ __forceinline__ void wait_copies()
{
    static_assert(N >= 0 && N < 64, "vmcnt field");
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

template <int D>
__device__ __forceinline__ void copy_tile(const AttnK &a, const TileRows &rows, uint32_t lds,
                                          int lane)
{
    using St = Stage<D>;
    // Byte i of a half's 16 rows is byte i from its first row.
    constexpr int HALF = St::CODES / 2, BHALF = St::BLOCKS / 2;
#pragma unroll
    for (int c = 0; c < St::CODES / 1024; c++) {
        if constexpr (HALF >= 1024) {
            constexpr int PER = HALF / 1024;         // copies of a half
            const int64_t r = rows.r[c / PER] * (D / 2) + 1024 * (c % PER);
            to_lds16(a.k + r, (uint32_t)(16 * lane), lds + St::K + 1024 * c);
            to_lds16(a.v + r, (uint32_t)(16 * lane), lds + St::V + 1024 * c);
        } else {
            const int64_t r = (lane & 32 ? rows.r[1] : rows.r[0]) * (D / 2) + 16 * (lane & 31);
            to_lds16(a.k + r, lds + St::K);
            to_lds16(a.v + r, lds + St::V);
        }
    }
#pragma unroll
    for (int c = 0; c < St::BLOCK_ROOM / 256; c++) {
        // D = 64: the upper lanes read what the lower ones do.
        const int at = (256 * c + 4 * lane) % St::BLOCKS;
        const int64_t r = (at >= BHALF ? rows.r[1] : rows.r[0]) * (D / 16) + at % BHALF;
        to_lds4(a.kbs + r, lds + St::KB + 256 * c);
        to_lds4(a.vbs + r, lds + St::VB + 256 * c);
    }
    const int64_t r = (lane & 16 ? rows.r[1] : rows.r[0]) + (lane & 15);
    to_lds4(reinterpret_cast<const uint8_t *>((lane & 32 ? a.vs : a.ks) + r), lds + St::S);
}

// Two E4M3 bytes -> FP16 (exact).
__device__ __forceinline__ f16x2_t e4m3_pair_f16(uint32_t bytes)
{
    return __builtin_bit_cast(f16x2_t,
                              __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 1.0f, false));
}

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
// maximum m of the numerators' exponents z + log2 s_v, this lane's part of
// the sum l, and O^T; l and O in units of 2^(m - TOP).
template <int D, int RT>
struct Rows {
    f16x8_t q[RT][D / 32];
    float c[RT];                                     // score factor of the row
    float m[RT], l[RT];
    f32x4_t o[RT][D / 16];
};

// A lane's address in LDS, opaque, so that the accesses from it take their
// constant distances as instruction offsets (else each is an addition).
typedef __attribute__((address_space(3))) const uint8_t *lds_cptr;
__device__ __forceinline__ lds_cptr lds_at(uint32_t address)
{
    asm("" : "+v"(address));
    return (lds_cptr)(uintptr_t)address;
}
template <typename T>
__device__ __forceinline__ T lds_ld(lds_cptr p)
{
    return *reinterpret_cast<__attribute__((address_space(3))) const T *>(p);
}

// Step kk of a lane's D/4 elements of a key, which hold D/64 blocks of 16 (two dwords
// each).
__device__ __forceinline__ f16x8_t key_f16(uint32_t codes, uint32_t blocks, int kk)
{
    const f16x2_t d = e4m3_pair_f16(blocks >> (16 * (kk / 4)));
    const _Float16 dk = d[(kk / 2) & 1];
    return oct_f16(codes, f16x2_t{dk, dk});
}

// Values as operands: pairs of keys (2i, 2i + 1) of the lane group's eight, their
// codes merged (even and odd elements), and their block scales.
template <int VW>
struct ValuePairs {
    f16x2_t vd[4];
    uint32_t ev[4][VW], od[4][VW];
    __device__ __forceinline__ ValuePairs(const uint32_t (&vc)[8][VW], const uint32_t (&vb)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            vd[i] = e4m3_pair_f16(vb[2 * i] | vb[2 * i + 1] << 8);
#pragma unroll
            for (int w = 0; w < VW; w++) {
                const uint32_t c0 = vc[2 * i][w], c1 = vc[2 * i + 1][w];
                ev[i][w] = (c0 & 0x0F0F0F0Fu) | ((c1 << 4) & 0xF0F0F0F0u);
                od[i][w] = ((c0 >> 4) & 0x0F0F0F0Fu) | (c1 & 0xF0F0F0F0u);
            }
        }
    }
    // Element j of the lane's D/16, eight keys.
    __device__ __forceinline__ f16x8_t operator()(int j) const
    {
        f16x2_t v[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = pair_f16_dyn((j & 1) ? od[i][j >> 3] : ev[i][j >> 3], (j >> 1) & 3) * vd[i];
        return cat8(v[0], v[1], v[2], v[3]);
    }
    // The same, decoded anew where it is called: shared with the other uses, the
    // decoded values would stay in registers.
    __device__ __forceinline__ f16x8_t again(int j) const
    {
        f16x2_t v[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint32_t c = (j & 1) ? od[i][j >> 3] : ev[i][j >> 3];
            asm volatile("" : "+v"(c));
            v[i] = pair_f16_dyn(c, (j >> 1) & 3) * vd[i];
        }
        return cat8(v[0], v[1], v[2], v[3]);
    }
};

// lv = log2 s_v, rv = 2^-lv of the lane group's eight values, whose block scales are
// vb.  A value scale of 0 (below MIN_VS) stands for a row of zeros, and slots that no
// row of the tile sees (outside keys [klo, khi): past the length, before the
// window) may hold anything: their block scales count as 0, and they take
// part in the sum under the largest scale of the tile.  In a tile of zeros that is
// ZERO_VS, about the scale of values of 1, within FP32's range of every other: m
// follows it, and a sum that began under 2^-100 would overflow at 2^17 keys or
// vanish beside scales above 2^26.
template <bool MASKED>
__device__ __forceinline__ void value_scales(const f32x4_t (&vs)[2], uint32_t (&vb)[8],
                                             float (&lv)[8], float (&rv)[8], int t0, int klo,
                                             int khi, int g)
{
    float vmin = vs[0][0];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        lv[j] = vs[j >> 2][j & 3];
        vmin = __builtin_fminf(vmin, lv[j]);
    }
    if (MASKED || __builtin_amdgcn_ballot_w64(vmin < MIN_VS) != 0) {
        float vz = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int t = t0 + 16 * (j >> 2) + 4 * g + (j & 3);
            const bool live = lv[j] >= MIN_VS && t >= klo && t < khi;
            vb[j] = live ? vb[j] : 0;
            lv[j] = live ? lv[j] : 0.0f;
            vz = __builtin_fmaxf(vz, lv[j]);
        }
        vz = max4_groups(vz);
        vz = vz > 0.0f ? vz : ZERO_VS;
#pragma unroll
        for (int j = 0; j < 8; j++)
            lv[j] = lv[j] > 0.0f ? lv[j] : vz;
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
        lv[j] = __builtin_amdgcn_logf(lv[j]);
        rv[j] = __builtin_amdgcn_exp2f(-lv[j]);
    }
}

// The softmax of a tile's scores s and its products with the values: value(j) are
// the values' operands, again(j) the same for further rounds.
template <int D, int RT, bool MASKED, typename Value, typename Again>
__device__ __forceinline__ void weigh(Rows<D, RT> &st, const f32x4_t (&s)[2][RT],
                                      const f32x4_t (&ks)[2], const float (&lv)[8],
                                      const float (&rv)[8], int t0, const int (&lo)[RT],
                                      const int (&hi)[RT], int g, Value value, Again again)
{
    f16x8_t p8[RT];
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        float z[8], zx = NO_MAX, zn = -NO_MAX;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            z[j] = __builtin_fmaf(s[j >> 2][rt][j & 3], ks[j >> 2][j & 3] * st.c[rt], lv[j]);
            if constexpr (MASKED) {
                const int t = t0 + 16 * (j >> 2) + 4 * g + (j & 3);
                const bool see = t >= lo[rt] && t < hi[rt];
                zn = __builtin_fminf(zn, see ? z[j] : -NO_MAX);
                z[j] = see ? z[j] : NO_MAX;
            } else {
                zn = __builtin_fminf(zn, z[j]);
            }
            zx = __builtin_fmaxf(zx, z[j]);
        }
        // m follows the maximum only when that is past m + SLACK: with m exact, nearly
        // every step of a short chunk had some row whose maximum rose.  It also rises
        // where the sum, whose terms are up to 2^(TOP + SLACK) / s_v, nears FP32's range.
        zx = max4_groups(zx);
        if (__builtin_amdgcn_ballot_w64(zx > st.m[rt] + SLACK || st.l[rt] > MAX_SUM) != 0) {
            float mn = zx > st.m[rt] + SLACK ? zx : st.m[rt];
            if (max4_groups(st.l[rt]) > MAX_SUM)
                mn = __builtin_fmaxf(mn, st.m[rt] + SUM_STEP);
            const float al = __builtin_amdgcn_exp2f(st.m[rt] - mn);
            st.m[rt] = mn;
            st.l[rt] *= al;
#pragma unroll
            for (int j = 0; j < D / 16; j++)
                st.o[rt][j] *= al;
        }
        const float base = st.m[rt] - TOP;
        float p[8], sum[2] = {};
#pragma unroll
        for (int j = 0; j < 8; j++) {
            p[j] = __builtin_amdgcn_exp2f(z[j] - base);
            if constexpr (MASKED)                    // a row that has seen no key: m = NO_MAX
                p[j] = z[j] == NO_MAX ? 0.0f : p[j];
            sum[j & 1] = __builtin_fmaf(p[j], rv[j], sum[j & 1]);
        }
        st.l[rt] += sum[0] + sum[1];
        if (__builtin_amdgcn_ballot_w64(zn - base < LOW_LOG2) != 0) {
            // Numerators in [bound / LOW_UP, bound), each round 29 bits further down.
            float bound = LOW, up = LOW_UP, down = 1.0f / LOW_UP, bits = LOW_LOG2;
#pragma unroll 1
            do {
                f16x8_t plo;
#pragma unroll
                for (int j = 0; j < 8; j++)
                    plo[j] = (_Float16)(p[j] < bound && p[j] >= bound * (1.0f / LOW_UP) ? p[j] * up
                                                                                      : 0.0f);
#pragma unroll
                for (int j = 0; j < D / 16; j++) {
                    const f32x4_t o = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        again(j), plo, f32x4_t{}, 0, 0, 0);
                    st.o[rt][j] += o * down;
                    __builtin_amdgcn_sched_barrier(0);               // one at a time: registers
                }
                bound *= 1.0f / LOW_UP;
                up *= LOW_UP;
                down *= 1.0f / LOW_UP;
                bits -= 29.0f;
            } while (bits > -126.0f && __builtin_amdgcn_ballot_w64(zn - base < bits) != 0);
#pragma unroll
            for (int j = 0; j < 8; j++)
                p[j] = p[j] < LOW ? 0.0f : p[j];
        }
#pragma unroll
        for (int j = 0; j < 8; j++)
            p8[rt][j] = (_Float16)p[j];
    }
#pragma unroll
    for (int j = 0; j < D / 16; j++) {
        const f16x8_t vf = value(j);
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
            st.o[rt][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p8[rt], st.o[rt][j], 0, 0, 0);
        if (j & 1)
            __builtin_amdgcn_sched_barrier(0);
    }
}

// One step: the tile at LDS address x (keys t0 ..).
template <int D, int RT, bool MASKED>
__device__ __forceinline__ void attend(Rows<D, RT> &st, uint32_t x, int t0, int klo, int khi,
                                       const int (&lo)[RT], const int (&hi)[RT], int l, int g)
{
    using St = Stage<D>;
    constexpr int KK = D / 32;
    // Scores: two 16-key halves, KK steps of 8 elements per lane group.
    f32x4_t s[2][RT];
#pragma unroll
    for (int rt = 0; rt < RT; rt++)
        s[0][rt] = s[1][rt] = f32x4_t{};
    uint32_t kc[2][KK], kb[2];
    const lds_cptr pk = lds_at(x + St::K + l * (D / 2) + g * (D / 8));
    const lds_cptr pkb = lds_at(x + St::KB + l * (D / 16) + g * (D / 64));
#pragma unroll
    for (int h = 0; h < 2; h++) {
        if constexpr (KK == 2) {
            const u32x2_t c = lds_ld<u32x2_t>(pk + 16 * h * (D / 2));
            kc[h][0] = c[0];
            kc[h][1] = c[1];
            kb[h] = lds_ld<uint8_t>(pkb + 16 * h * (D / 16));
        } else {
#pragma unroll
            for (int j = 0; j < KK / 4; j++) {
                const u32x4_t c = lds_ld<u32x4_t>(pk + 16 * h * (D / 2) + 16 * j);
#pragma unroll
                for (int w = 0; w < 4; w++)
                    kc[h][4 * j + w] = c[w];
            }
            if constexpr (KK == 4)
                kb[h] = lds_ld<uint16_t>(pkb + 16 * h * (D / 16));
            else
                kb[h] = lds_ld<uint32_t>(pkb + 16 * h * (D / 16));
        }
    }
#pragma unroll
    for (int kk = 0; kk < KK; kk++) {
        f16x8_t kf[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            kf[h] = key_f16(kc[h][kk], kb[h], kk);
        }
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                s[h][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[h], st.q[rt][kk], s[h][rt],
                                                                   0, 0, 0);
    }
    // The lane group's eight keys, and their values' codes and block scales.
    const lds_cptr ps = lds_at(x + St::S + 16 * g);
    const lds_cptr pv = lds_at(x + St::V + 4 * g * (D / 2) + l * (D / 32));
    const lds_cptr pvb = lds_at(x + St::VB + 4 * g * (D / 16) + l * (D / 16) / 16);
    constexpr int VW = D == 256 ? 2 : 1;             // dwords of a key's codes per lane
    f32x4_t ks[2], vs[2];
    uint32_t vc[8][VW], vb[8];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        ks[h] = lds_ld<f32x4_t>(ps + 64 * h);
        vs[h] = lds_ld<f32x4_t>(ps + 128 + 64 * h);
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const int key = 16 * (j >> 2) + (j & 3);
        if constexpr (D == 64)
            vc[j][0] = lds_ld<uint16_t>(pv + key * (D / 2));
        else if constexpr (D == 128)
            vc[j][0] = lds_ld<uint32_t>(pv + key * (D / 2));
        else {
            const u32x2_t w = lds_ld<u32x2_t>(pv + key * (D / 2));
            vc[j][0] = w[0];
            vc[j][1] = w[1];
        }
        vb[j] = lds_ld<uint8_t>(pvb + key * (D / 16));
    }
    float lv[8], rv[8];
    value_scales<MASKED>(vs, vb, lv, rv, t0, klo, khi, g);
    const ValuePairs<VW> v(vc, vb);
    weigh<D, RT, MASKED>(st, s, ks, lv, rv, t0, lo, hi, g, v, [&](int j) { return v.again(j); });
}

// What rows r0 .. r1 - 1 of a sequence of len keys see: keys [klo, kmax) at most, of
// which every row sees [full_lo, full_hi); kmin is the first key of klo's tile.
struct Span {
    int kmin, klo, kmax, full_lo, full_hi;
};
__device__ __forceinline__ Span row_span(const AttnK &a, int r0, int r1, int len)
{
    const int first = len - a.q_len + (int)udiv((uint32_t)r0, a.group_div);
    const int last = len - a.q_len + (int)udiv((uint32_t)(r1 - 1), a.group_div);
    Span s;
    s.kmax = a.causal ? (last + 1 < 0 ? 0 : last + 1) : len;
    const int klo = a.causal && a.window > 0 ? first - a.window + 1 : 0;
    s.klo = klo < 0 ? 0 : klo;
    s.kmin = s.klo & ~(ATT_TILE - 1);
    s.full_hi = a.causal ? (first + 1 < len ? first + 1 : len) : len;
    s.full_lo = a.causal && a.window > 0 ? last - a.window + 1 : 0;
    return s;
}

// Loads a wavefront's query rows r0 .. and starts their state; row (lane % 16) of
// tile rt sees keys [lo, hi).
template <int D, int RT>
__device__ __forceinline__ void start_rows(const AttnK &a, Rows<D, RT> &st, int (&lo)[RT],
                                           int (&hi)[RT], int r0, int b, int kvh, int len, int l,
                                           int g)
{
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
#pragma unroll
        for (int j = 0; j < D / 16; j++)
            st.o[rt][j] = f32x4_t{};
    }
}

template <int D, int RT>
__global__ void __launch_bounds__(ATT_THREADS, D * RT <= 128 ? 3 : 2)
    nvfp4_attention_kernel(AttnK a)
{
    constexpr int ROWS = 16 * RT;
    // The wavefronts' tiles; after the loop their sums: rows padded by four floats, so
    // that the 16 rows a store touches miss each other's banks.
    constexpr int TILE_BYTES = ATT_WAVES * ATT_STAGES * Stage<D>::BYTES;
    constexpr int SUM_BYTES = ATT_WAVES * ROWS * (D + 4) * 4;
    __shared__ __attribute__((aligned(16))) uint8_t
        lds[TILE_BYTES > SUM_BYTES ? TILE_BYTES : SUM_BYTES];
    __shared__ float lds_ml[ATT_WAVES][ROWS][2];
    float(*lds_o)[ROWS][D + 4] = reinterpret_cast<float(*)[ROWS][D + 4]>(lds);

    const int lane = (int)lane_id(), l = lane & 15, g = lane >> 4, wave = wave_in_group();
    Unit un;
    if (!plan_unit(a, wg_id(), lane, &un))
        return;
    const int tile = un.tile, kvh = un.kvh, b = un.b, len = un.len;

    // Keys the tile's rows see, and this workgroup's part of them.
    const int r0 = tile * ROWS;
    const int r1 = r0 + ROWS < a.rows ? r0 + ROWS : a.rows;
    const Span sp = row_span(a, r0, r1, len);
    const int64_t start64 = (int64_t)sp.kmin + (int64_t)un.chunk * un.chunk_keys;
    const int start = start64 < sp.kmax ? (int)start64 : sp.kmax;
    const int stop = sp.kmax - start < un.chunk_keys ? sp.kmax : start + un.chunk_keys;

    Rows<D, RT> st;
    int lo[RT], hi[RT];
    start_rows<D, RT>(a, st, lo, hi, r0, b, kvh, len, l, g);

    const int64_t *table = a.table + (int64_t)b * a.max_pages;
    constexpr int STEP = ATT_TILE * ATT_WAVES;
    int t0 = start + wave * ATT_TILE;
    if (t0 < stop) {
        // Tiles go round ATT_STAGES buffers.  Steps past the last copy the last tile
        // again, so that the count of copies in flight is the same in every step.
        using St = Stage<D>;
        const int t_last = t0 + (stop - 1 - t0) / STEP * STEP;
        const uint8_t *mine = lds + wave * ATT_STAGES * St::BYTES;
        const uint32_t mine32 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)mine;
        RowWindow win = row_window(a, table, kvh, t0, STEP, t_last, lane);
#pragma unroll
        for (int i = 0; i < ATT_STAGES - 1; i++)
            copy_tile<D>(a, window_rows(win, i), mine32 + i * St::BYTES, lane);
        int buf = 0, ahead = ATT_STAGES - 1;         // place in the window of the next copy
        auto step = [&](auto masked) {
            if (ahead == 64) {
                const int tn = t0 + (ATT_STAGES - 1) * STEP;
                win = row_window(a, table, kvh, tn < t_last ? tn : t_last, STEP, t_last, lane);
                ahead = 0;
            }
            const int fill = buf == 0 ? ATT_STAGES - 1 : buf - 1;
            copy_tile<D>(a, window_rows(win, ahead), mine32 + fill * St::BYTES, lane);
            ahead++;
            wait_copies<(ATT_STAGES - 1) * St::COPIES>();
            attend<D, RT, decltype(masked)::value>(st, mine32 + buf * St::BYTES, t0, sp.klo,
                                                   sp.kmax, lo, hi, l, g);
            // The tile has been read before the next step's copies overwrite it.
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
            buf = buf == ATT_STAGES - 1 ? 0 : buf + 1;
            t0 += STEP;
        };
        // Loops of their own for tiles that need no mask and for the others: both
        // forms in one loop took 90 registers more.
        auto full = [&] { return t0 >= sp.full_lo && t0 + ATT_TILE <= sp.full_hi; };
        while (t0 <= t_last) {
            while (t0 <= t_last && full())
                step(std::false_type{});
            while (t0 <= t_last && !full())
                step(std::true_type{});
        }
        wait_copies<0>();
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
    __syncthreads();                                 // no wavefront reads tiles any more
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const int r = 16 * rt + l;
        float m = NO_MAX;
#pragma unroll
        for (int w = 0; w < ATT_WAVES; w++)
            m = __builtin_fmaxf(m, lds_ml[w][r][0]);
        const float f = __builtin_amdgcn_exp2f(st.m[rt] - m);
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
                a.lse[qrow] = sum > 0.0f ? (m - TOP + __builtin_amdgcn_logf(sum)) * LN2
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

// Many query rows of 64 elements (chunks of a prompt).  A workgroup of eight
// wavefronts takes WIDE_ROWS rows, and a step's four tiles are decoded once for all
// of them: wavefronts 0 to 3 decode the keys of one tile each, 4 to 7 the values,
// and leave them in LDS as the operands of the products, a lane's 16 bytes
// after another's.  The next step's codes are loaded to registers meanwhile.
// 3 chunks of 509 queries of 16 heads over up to 8192 keys: 118 us and 22 us for the
// join, against 182 us where every 32 rows decode the keys anew; the issue of
// vector instructions is what bounds both (62 % of the cycles here).  With
// 128 registers for four wavefronts a SIMD instead of two it spills: 191 us.
// Rows of 128 elements have fewer decodings per product and gain nothing (120
// against 116 us for 4 chunks of 200 queries over 4000 keys).
template <int D>
struct Decoded {
    static constexpr int KF = D / 16, VF = D / 16;   // operands of 1 KiB
    static constexpr int K = 0, V = 1024 * KF, KS = V + 1024 * VF, LV = KS + 128, RV = LV + 128,
                         BYTES = RV + 128;
};

// A wavefront's part of a tile as loaded.  Keys: c[h KK + kk], b[h] of half h, s[0][0]
// the FP32 scale of key lane % 32.  Values: c[j], b[j] of key j of the lane
// group's eight, s their FP32 scales.
template <int D>
struct RawPart {
    static constexpr int KK = D / 32;
    uint32_t c[8], b[8];
    f32x4_t s[2];

    __device__ __forceinline__ void load_keys(const AttnK &a, const TileRows &rows, int lane)
    {
        const int l = lane & 15, g = lane >> 4;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int64_t r = rows.r[h] + l;
            const uint8_t *pc = a.k + r * (D / 2) + g * (D / 8);
            const uint8_t *pb = a.kbs + r * (D / 16) + g * (D / 64);
            const uint2 w = ld8(pc);
            c[2 * h] = w.x;
            c[2 * h + 1] = w.y;
            b[h] = *pb;
        }
        s[0][0] = a.ks[(lane & 16 ? rows.r[1] : rows.r[0]) + l];
    }
    __device__ __forceinline__ void load_values(const AttnK &a, const TileRows &rows, int lane)
    {
        const int l = lane & 15, g = lane >> 4;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t r = rows.r[j >> 2] + 4 * g + (j & 3);
            c[j] = *reinterpret_cast<const uint16_t *>(a.v + r * (D / 2) + l * (D / 32));
            b[j] = a.vbs[r * (D / 16) + l * (D / 16) / 16];
            s[j >> 2][j & 3] = a.vs[r];
        }
    }
    __device__ __forceinline__ void decode_keys(uint8_t *out, int lane) const
    {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int kk = 0; kk < KK; kk++)
                *reinterpret_cast<f16x8_t *>(out + Decoded<D>::K + 1024 * (h * KK + kk) +
                                             16 * lane) = key_f16(c[h * KK + kk], b[h], kk);
        if (lane < 32)
            *reinterpret_cast<float *>(out + Decoded<D>::KS + 4 * lane) = s[0][0];
    }
    template <bool MASKED>
    __device__ __forceinline__ void decode_values(uint8_t *out, int t0, int klo, int khi,
                                                  int lane)
    {
        const int g = lane >> 4;
        float lv[8], rv[8];
        value_scales<MASKED>(s, b, lv, rv, t0, klo, khi, g);
        uint32_t codes[8][1];
#pragma unroll
        for (int j = 0; j < 8; j++)
            codes[j][0] = c[j];
        const ValuePairs<1> v(codes, b);
#pragma unroll
        for (int j = 0; j < D / 16; j++)
            *reinterpret_cast<f16x8_t *>(out + Decoded<D>::V + 1024 * j + 16 * lane) = v(j);
        if ((lane & 15) == 0)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                *reinterpret_cast<f32x4_t *>(out + Decoded<D>::LV + 64 * h + 16 * g) =
                    f32x4_t{lv[4 * h], lv[4 * h + 1], lv[4 * h + 2], lv[4 * h + 3]};
                *reinterpret_cast<f32x4_t *>(out + Decoded<D>::RV + 64 * h + 16 * g) =
                    f32x4_t{rv[4 * h], rv[4 * h + 1], rv[4 * h + 2], rv[4 * h + 3]};
            }
    }
};

// One decoded tile (keys t0 ..) and a wavefront's rows.
template <int D, int RT, bool MASKED>
__device__ __forceinline__ void attend_decoded(Rows<D, RT> &st, const uint8_t *x, int t0,
                                               const int (&lo)[RT], const int (&hi)[RT], int lane)
{
    using De = Decoded<D>;
    constexpr int KK = D / 32;
    const int g = lane >> 4;
    const uint32_t x32 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)x;
    const lds_cptr mine = lds_at(x32 + 16 * lane), group = lds_at(x32 + De::KS + 16 * g);
    f32x4_t s[2][RT];
#pragma unroll
    for (int rt = 0; rt < RT; rt++)
        s[0][rt] = s[1][rt] = f32x4_t{};
#pragma unroll
    for (int kk = 0; kk < KK; kk++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const f16x8_t kf = lds_ld<f16x8_t>(mine + De::K + 1024 * (h * KK + kk));
#pragma unroll
            for (int rt = 0; rt < RT; rt++)
                s[h][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, st.q[rt][kk], s[h][rt], 0,
                                                                  0, 0);
        }
    f32x4_t ks[2];
    float lv[8], rv[8];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        ks[h] = lds_ld<f32x4_t>(group + 64 * h);
        const f32x4_t vl = lds_ld<f32x4_t>(group + (De::LV - De::KS) + 64 * h);
        const f32x4_t vr = lds_ld<f32x4_t>(group + (De::RV - De::KS) + 64 * h);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            lv[4 * h + i] = vl[i];
            rv[4 * h + i] = vr[i];
        }
    }
    // Further rounds read the values again: kept, they would take registers.
    weigh<D, RT, MASKED>(
        st, s, ks, lv, rv, t0, lo, hi, g,
        [&](int j) { return lds_ld<f16x8_t>(mine + De::V + 1024 * j); },
        [&](int j) { return lds_ld<f16x8_t>(lds_at(x32 + 16 * lane) + De::V + 1024 * j); });
}

template <int D>
__global__ void __launch_bounds__(WIDE_THREADS, 2) nvfp4_attention_wide_kernel(AttnK a)
{
    constexpr int RT = WIDE_RT, STEP = ATT_TILE * ATT_WAVES;
    __shared__ __attribute__((aligned(16))) uint8_t lds[ATT_WAVES * Decoded<D>::BYTES];
    const int lane = (int)lane_id(), l = lane & 15, g = lane >> 4, wave = wave_in_group();
    Unit un;
    if (!plan_unit(a, wg_id(), lane, &un))
        return;
    const int kvh = un.kvh, b = un.b, len = un.len;
    const int r0 = un.tile * WIDE_ROWS;
    const int r1 = r0 + WIDE_ROWS < a.rows ? r0 + WIDE_ROWS : a.rows;
    const Span sp = row_span(a, r0, r1, len);
    const int64_t start64 = (int64_t)sp.kmin + (int64_t)un.chunk * un.chunk_keys;
    const int start = start64 < sp.kmax ? (int)start64 : sp.kmax;
    const int stop = sp.kmax - start < un.chunk_keys ? sp.kmax : start + un.chunk_keys;

    Rows<D, RT> st;
    int lo[RT], hi[RT];
    const int w0 = r0 + 16 * RT * wave;              // the wavefront's first row
    start_rows<D, RT>(a, st, lo, hi, w0, b, kvh, len, l, g);

    if (start < stop) {                              // the same for the whole workgroup
        const int64_t *table = a.table + (int64_t)b * a.max_pages;
        const int steps = (stop - start + STEP - 1) / STEP;
        const bool values = wave >= ATT_WAVES;
        const int part = ATT_TILE * (wave & (ATT_WAVES - 1));
        const int t_last = start + part + (steps - 1) * STEP;
        uint8_t *out = lds + (wave & (ATT_WAVES - 1)) * Decoded<D>::BYTES;
        RowWindow win = row_window(a, table, kvh, start + part, STEP, t_last, lane);
        RawPart<D> raw;
        auto load = [&](int i) {
            const TileRows rows = window_rows(win, i);
            values ? raw.load_values(a, rows, lane) : raw.load_keys(a, rows, lane);
        };
        load(0);
        int t = start, ahead = 1;                    // place in the window of the next load
        auto step = [&](auto masked) {
            constexpr bool MASKED = decltype(masked)::value;
            __syncthreads();                         // the last step's tiles have been read
            if (values)
                raw.template decode_values<MASKED>(out, t + part, sp.klo, sp.kmax, lane);
            else
                raw.decode_keys(out, lane);
            if (ahead == 64) {
                const int tn = t + part + STEP;
                win = row_window(a, table, kvh, tn < t_last ? tn : t_last, STEP, t_last, lane);
                ahead = 0;
            }
            load(ahead);                             // past the last step: the last tile again
            ahead++;
            __syncthreads();
#pragma unroll 1
            for (int i = 0; i < ATT_WAVES; i++) {
                const int t0 = t + ATT_TILE * i;
                if (t0 >= stop)
                    break;
                attend_decoded<D, RT, MASKED>(st, lds + i * Decoded<D>::BYTES, t0, lo, hi, lane);
            }
            t += STEP;
        };
        auto full = [&] { return t >= sp.full_lo && t + STEP <= sp.full_hi; };
        while (t < stop) {
            while (t < stop && full())
                step(std::false_type{});
            while (t < stop && !full())
                step(std::true_type{});
        }
    }

    // A lane holds, of row l of tile rt, elements (4g + i) D/16 + j.
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const float sum = sum4_groups(st.l[rt]), m = st.m[rt];
        const int r = w0 + 16 * rt + l;
        if (r >= r1)
            continue;
        if (un.n_chunks == 1) {
            const int qi = (int)udiv((uint32_t)r, a.group_div);
            const int64_t qrow = ((int64_t)b * a.q_len + qi) * a.n_heads + kvh * a.group +
                                 (r - qi * a.group);
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint32_t v[D / 32];
#pragma unroll
                for (int j = 0; j < D / 32; j++)
                    v[j] = (uint32_t)bf16_rne(st.o[rt][2 * j][i] * inv) |
                           (uint32_t)bf16_rne(st.o[rt][2 * j + 1][i] * inv) << 16;
                *reinterpret_cast<u32x2_t *>(a.out + qrow * D + (4 * g + i) * (D / 16)) =
                    u32x2_t{v[0], v[1]};
            }
            if (a.lse && g == 0)
                a.lse[qrow] = sum > 0.0f ? (m - TOP + __builtin_amdgcn_logf(sum)) * LN2
                                         : -__builtin_inff();
        } else {
            const int64_t pr = (int64_t)wg_id() * WIDE_ROWS + (r - r0);
            if (g == 0) {
                a.part_ml[2 * pr] = m;
                a.part_ml[2 * pr + 1] = sum;
            }
            if (sum > 0.0f)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    *reinterpret_cast<f32x4_t *>(a.part_o + pr * D + (4 * g + i) * (D / 16)) =
                        f32x4_t{st.o[rt][0][i], st.o[rt][1][i], st.o[rt][2][i], st.o[rt][3][i]};
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
        a.lse[row] = sum > 0.0f ? (m - TOP + __builtin_amdgcn_logf(sum)) * LN2 : -__builtin_inff();
}

// Row tiles of a launch, and the most units its plan can have: a chunk more
// per (sequence, head, row tile) than its share of ATT_TARGET.
struct AttnPlan {
    int rt, row_tiles, tile_rows, target;            // rt = 0: the kernel for many rows
    bool split;
    int64_t units;
};
AttnPlan attention_plan(int64_t n_seqs, int64_t q_len, int64_t n_heads, int64_t n_kv_heads,
                        int64_t head_dim, int64_t max_keys)
{
    const int64_t rows = q_len * (n_heads / n_kv_heads);
    // The kernel for many rows where they fill the chip: 224 tiles of 32 rows over
    // 2000 keys take 42 us against 48, but 36 tiles over 4000 keys 40 us against 34.
    const bool wide = head_dim == 64 && rows > 32 &&
                      n_seqs * n_kv_heads * ((rows + 31) / 32) >= WIDE_TILES;
    // Otherwise, more rows share a key's decoding as far as a wavefront's registers go
    // without spilling: 32 rows of 64 or 128 elements, 16 of 256.
    const int rt = wide ? 0 : rows <= 16 || head_dim == 256 ? 1 : 2;
    const int tile_rows = wide ? WIDE_ROWS : 16 * rt, target = wide ? WIDE_TARGET : ATT_TARGET;
    const int64_t row_tiles = (rows + tile_rows - 1) / tile_rows;
    const int64_t base = n_seqs * n_kv_heads * row_tiles;
    // With enough row tiles to fill the chip, or keys for one chunk, none is split.
    const bool split = base < target && max_keys > ATT_MIN_CHUNK;
    const int64_t most = base * ((max_keys + ATT_MIN_CHUNK - 1) / ATT_MIN_CHUNK);
    const int64_t units = !split ? base : most < target + base ? most : target + base;
    return AttnPlan{rt, (int)row_tiles, tile_rows, target, split, units};
}

}  // namespace

int64_t nvfp4_attention_workspace(int64_t n_seqs, int64_t q_len, int64_t n_heads,
                                  int64_t n_kv_heads, int64_t head_dim, int64_t max_keys)
{
    const AttnPlan p = attention_plan(n_seqs, q_len, n_heads, n_kv_heads, head_dim, max_keys);
    return p.split ? p.units * p.tile_rows * (head_dim + 2) * 4 : 0;
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
    // A window of all keys and queries is none, and positions less it fit 32 bits.
    const int64_t most = max_keys + a.q_len, window = a.window < most ? a.window : most;
    const AttnK k{a.q, a.k, a.kbs, a.ks, a.v, a.vbs, a.vs, a.block_table, a.seq_lens, a.n_pages,
                  a.max_pages, (int)a.q_len, (int)a.n_heads, (int)a.n_kv_heads, group,
                  (int)a.page_size, (int)(a.q_len * group), make_div((uint32_t)a.page_size),
                  make_div((uint32_t)group), a.scale * LOG2E, a.causal ? 1 : 0,
                  (int)window, (int)a.n_seqs, p.row_tiles, p.tile_rows, p.target, p.split, a.out,
                  a.lse, ml, p.split ? ml + p.units * p.tile_rows * 2 : nullptr};
    const int64_t wgs = p.units;
    if (p.rt == 0)
        hipLaunchKernelGGL(nvfp4_attention_wide_kernel<64>, dim3((unsigned)wgs),
                           dim3(WIDE_THREADS), 0, stream, k);
    else if (a.head_dim == 64)
        p.rt == 1 ? attention_launch<64, 1>(k, wgs, stream)
                  : attention_launch<64, 2>(k, wgs, stream);
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
