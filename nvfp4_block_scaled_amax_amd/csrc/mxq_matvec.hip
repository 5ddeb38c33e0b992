// mxq_matvec.hip -- products of few rows with NVFP4 weights: a decode step's
// projections (dense) and experts (expert-sorted rows, the gate/up pair with
// SwiGLU in the epilogue).  C[m][n] = s_x[m] s_b[n] sum_k x[m][k]
// dec(code[n][k]) dec(block scale[n][k/16]), fp32 accumulation.
//
// What bounds it: the weights, 9/16 byte an element, each read once; the
// arithmetic is one conversion and one packed multiply per code pair, about
// half of what the VALU can do while HBM delivers the pair.  So every row
// count takes the same path: 16x16x32 FP16 matrix instructions with 16 weight
// rows as their first operand and up to 16 activation rows as the second
// (rows past M repeat the last one and are not stored).
//
// Weights.  dec(code) dec(block scale) is an exact FP16 value.  In a unit of
// 128 K values lane (n, g) = (lane % 16, lane / 16) holds the 32 values k =
// 32 g .. of row n: one 16-byte load of codes and two block scales.  Which
// 8 of them enter instruction q of four is the same for both operands, so
// the lane's own order serves.
//
// Activations are staged once per workgroup in LDS as FP16, 128 values of a
// row under one power of two (their largest magnitude in [2^14, 2^15)), so
// that BF16 values enter exactly unless they are 2^-30 below that; per-token
// NVFP4 ones enter as dec(code) dec(block scale).  FP32 ones are rounded to
// FP16's 11 bits, three more than a BF16 result has: two FP16 parts of each
// (22 bits) take twice the LDS, so that a row of the largest K no longer fits,
// and twice the matrix instructions (13 x 128256 x 2048 35 -> 46 us, 4 x 7168 x
// 18432 67 -> 131 us, the experts of 48 tokens 85 -> 92 us).  A unit's product starts
// from zero and joins the row's sum under the running largest exponent, so
// no sum overflows where the result does not, nor loses more than 2^-149 of the
// row's largest values' part.  The FP32 scales' exponents join that one.
//
// Split.  Of few weights (below MV_WHOLE_K_TILES tiles of 16 rows) a
// workgroup's four wavefronts share K unit by unit and join through LDS for
// every tile: that fills more of the chip.  Of many, every wavefront takes
// tiles of its own and loads them in memory's order (see MvLine).  Either
// way the next loads are issued before the current ones are multiplied.
// Measured in graphs of ten calls: 1 x 2048 x 2048 4.7 us; 13 x 128257 x 2048
// 35 us (151 MB: 4.3 TB/s); 1 x 1000000 x 2048 250 us (4.6 TB/s).
#include <type_traits>

#include "mxq_layer.h"
#include "mxq_layer_device.h"

namespace mxq {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Wavefronts of a workgroup that splits K among them; one whose wavefronts take
// whole tiles has up to MV_MAX_WAVES, which share the staged rows (13 x 128257 x
// 2048: 47 us with four, 41 us with sixteen).  Experts have fewer rows to share and
// fewer tiles, and keep four (8 tokens: 47 us, with eight 51 us).
constexpr int MV_SPLIT = 4, MV_MAX_WAVES = 16;
constexpr int MV_UNIT = 128;                      // K values per unit
constexpr int MV_XROW = MV_UNIT * 2 + 16;         // a row's unit in LDS, padded: 16 rows at one
                                                  // offset fall in distinct banks
constexpr int MV_STAGE = 4;                       // units of rows loaded at once when staging
constexpr int MV_RROW = 20;                       // floats per row of a wavefront's partial tile
constexpr int MV_MAX_ROWS = 32;                   // activation rows of a workgroup
constexpr int MV_LDS = 160 * 1024;                // a workgroup's most
constexpr int64_t MV_CU_WAVES = 20;               // wavefronts a compute unit is given
constexpr int64_t MV_WHOLE_K_TILES = 2048;        // 16-row tiles from which wavefronts take whole ones
// Units of a wavefront's loads: strided ones of nw weights when K is split,
// consecutive ones of a whole tile.
constexpr int mv_block(int nw) { return nw == 1 ? 4 : 2; }
constexpr int MV_LINE = 4;
constexpr int MV_TURN = MV_LINE * 1024 + 512;     // a wavefront's LDS to turn a block in

struct MvArgs {
    ActX x;
    WeightB w, up;                                // up.codes == nullptr: no gate
    const float *scales;
    Div per_scale;                                // rows of the weight per FP32 scale
    int64_t N, K;
    int rows;                                     // activation rows per pass (dense)
    int M, passes;                                // dense
    int waves;                                    // wavefronts of a workgroup
    int tiles, wgs_n;                             // 16-row weight tiles, workgroups sharing them
    // Experts: rows of x, sorted by segment.
    int64_t n_tokens, total_rows;
    const int64_t *row_tokens, *seg_offsets;
    int n_groups;
    int chunk_rows;                               // activation rows staged at once
    void *c;
};

__device__ __forceinline__ f16x2_t e4m3_pair(uint32_t bytes)
{
    return __builtin_bit_cast(f16x2_t,
                              __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 1.0f, false));
}
template <int J>
__device__ __forceinline__ f16x2_t code_pair(uint32_t codes)
{
    return __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, J));
}
// Eight values (one dword of codes) under block scale d.
__device__ __forceinline__ f16x8_t oct(uint32_t codes, _Float16 d)
{
    const f16x2_t d2 = {d, d};
    const f16x2_t a = code_pair<0>(codes) * d2, b = code_pair<1>(codes) * d2,
                  c = code_pair<2>(codes) * d2, e = code_pair<3>(codes) * d2;
    return f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// The mantissa of an FP32 scale, in [1/2, 1); its exponent goes to e.
__device__ __forceinline__ float mantissa(float scale, int *e)
{
    *e += __builtin_amdgcn_frexp_expf(scale);
    return __builtin_amdgcn_frexp_mantf(scale);
}
// sum * scale * 2^e, in FP32's range where the result is.
__device__ __forceinline__ float scaled(float sum, float scale, int e)
{
    const float v = sum * mantissa(scale, &e);
    return __builtin_ldexpf(v, e);
}
// What a lane loads of an activation row's unit: 8 values.
struct ActRaw {
    uint4 a, b;
};
template <int FMT>
__device__ __forceinline__ ActRaw act_load(const ActX &x, int64_t row, int64_t k, int64_t K)
{
    ActRaw r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (k >= K)                                   // K % 64 == 0: all 8 values or none
        return r;
    if constexpr (FMT == MXQ_X_BF16) {
        r.a = ld16(reinterpret_cast<const uint16_t *>(x.x) + row * K + k);
    } else if constexpr (FMT == MXQ_X_F32) {
        r.a = ld16(reinterpret_cast<const float *>(x.x) + row * K + k);
        r.b = ld16(reinterpret_cast<const float *>(x.x) + row * K + k + 4);
    } else {
        r.a.x = *reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(x.x) +
                                                    row * (K >> 1) + (k >> 1));
        r.a.y = x.bs[row * (K >> 4) + (k >> 4)];
    }
    return r;
}
// The FP16 values of a row's unit (16 lanes, 8 values each) and its exponent.
template <int FMT>
__device__ __forceinline__ f16x8_t act_f16(const ActRaw &r, int *e)
{
    if constexpr (FMT == MXQ_X_NVFP4) {
        *e = 0;
        return oct(r.a.x, e4m3_pair(r.a.y)[0]);
    } else {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            f[i] = FMT == MXQ_X_F32 ? u2f(w[i]) : (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t b = f2u(f[i]) & 0x7FFFFFFFu;
            am = am > b ? am : b;
        }
        am = max(am, dpp<DPP_XOR1>(am));
        am = max(am, dpp<DPP_XOR2>(am));
        am = max(am, dpp<DPP_HALF_MIRROR>(am));
        am = max(am, dpp<DPP_MIRROR>(am));
        *e = (int)(am >> 23) - 127 - 14;
        f16x8_t v;
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = (_Float16)__builtin_ldexpf(f[i], -*e);
        return v;
    }
}

// Stages rows [0, rows) of the activations (row r is row src(r) of x) into
// LDS; columns past K are zero.  ex[unit * rows + r] is the unit's exponent.
// Each 16 lanes take a unit of a row, MV_STAGE of them loaded at once.
template <int FMT, typename Src>
__device__ __forceinline__ void stage_rows(uint8_t *xs, int *ex, const ActX &x, int rows,
                                           int units, int64_t K, int waves, Src src)
{
    const int GROUPS = 4 * waves;
    const int l16 = (int)(tid() & 15), total = rows * units;
    for (int p0 = (int)(tid() >> 4); p0 < total; p0 += GROUPS * MV_STAGE) {
        ActRaw raw[MV_STAGE];
#pragma unroll
        for (int j = 0; j < MV_STAGE; j++) {
            const int p = p0 + GROUPS * j < total ? p0 + GROUPS * j : total - 1;
            const int u = (int)((uint32_t)p / (uint32_t)rows);
            raw[j] = act_load<FMT>(x, src(p - u * rows), (int64_t)MV_UNIT * u + 8 * l16, K);
        }
#pragma unroll
        for (int j = 0; j < MV_STAGE; j++) {
            const int p = p0 + GROUPS * j;
            int e;
            const f16x8_t v = act_f16<FMT>(raw[j], &e);
            if (p < total) {
                *reinterpret_cast<f16x8_t *>(xs + p * MV_XROW + 16 * l16) = v;
                if (l16 == 0)
                    ex[p] = e;
            }
        }
    }
}

// One wavefront's loads of up to mv_block units of a weight tile (of NW
// weights: gate and up).
template <int NW>
struct MvBlock {
    static constexpr int U = mv_block(NW);
    u32x4_t c[NW][U];
    uint32_t s[NW][U];
};
template <int NW>
__device__ __forceinline__ void load_block(MvBlock<NW> &b, const WeightB *w, int64_t row, int u0,
                                           int units, int64_t K, int g)
{
#pragma unroll
    for (int j = 0; j < mv_block(NW); j++) {
        const int u = u0 + MV_SPLIT * j;
        if (u < units) {
            // The half unit that ends a K of 64 (mod 128): the upper lane groups read the
            // lower ones' codes, against zero activations.
            const int gk = MV_UNIT * u + 32 * g < K ? g : g & 1;
#pragma unroll
            for (int i = 0; i < NW; i++) {
                b.c[i][j] = *reinterpret_cast<const u32x4_t *>(w[i].codes + row * (K >> 1) +
                                                               64 * u + 16 * gk);
                b.s[i][j] = *reinterpret_cast<const uint16_t *>(w[i].bs + row * (K >> 4) + 8 * u +
                                                                2 * gk);
            }
        }
    }
}

// A wavefront's sums of one tile: lane (m, g) holds C[m][n0 + 4g + i] of MT
// groups of 16 activation rows, in units of 2^e.
template <int NW, int MT>
struct MvSums {
    f32x4_t a[NW][MT];
    int e[MT];
};

template <int NW, int MT>
__device__ __forceinline__ void multiply_block(MvSums<NW, MT> &st, const MvBlock<NW> &b,
                                               const uint8_t *xs, const int *ex, int rows, int u0,
                                               int units, int l, int g)
{
#pragma unroll
    for (int j = 0; j < mv_block(NW); j++) {
        const int u = u0 + MV_SPLIT * j;
        if (u >= units)
            break;
        f32x4_t d[NW][MT];
        int e[MT];
        const uint8_t *xp[MT];
#pragma unroll
        for (int t = 0; t < MT; t++) {
            const int r = 16 * t + l < rows ? 16 * t + l : rows - 1;
            xp[t] = xs + (int64_t)(u * rows + r) * MV_XROW + 64 * g;
            e[t] = ex[u * rows + r];
#pragma unroll
            for (int i = 0; i < NW; i++)
                d[i][t] = f32x4_t{};
        }
#pragma unroll
        for (int q = 0; q < 4; q++) {
            f16x8_t xf[MT];
#pragma unroll
            for (int t = 0; t < MT; t++)
                xf[t] = *reinterpret_cast<const f16x8_t *>(xp[t] + 16 * q);
#pragma unroll
            for (int i = 0; i < NW; i++) {
                const f16x8_t wf = oct(b.c[i][j][q], e4m3_pair(b.s[i][j])[q >> 1]);
#pragma unroll
                for (int t = 0; t < MT; t++)
                    d[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf, xf[t], d[i][t], 0, 0, 0);
            }
        }
#pragma unroll
        for (int t = 0; t < MT; t++) {
            const int en = e[t] > st.e[t] ? e[t] : st.e[t];
            const float fo = __builtin_ldexpf(1.0f, st.e[t] - en), fd = __builtin_ldexpf(1.0f, e[t] - en);
            st.e[t] = en;
#pragma unroll
            for (int i = 0; i < NW; i++)
#pragma unroll
                for (int k = 0; k < 4; k++)
                    st.a[i][t][k] = __builtin_fmaf(st.a[i][t][k], fo, d[i][t][k] * fd);
        }
    }
}

// The loads of up to MV_LINE consecutive units of a whole tile, in memory's
// order: 256 consecutive bytes of each of four rows an instruction (64 bytes
// of sixteen rows, the order of the matrix instructions, reach 3.9 TB/s,
// these 5.7).  They are turned into that order through LDS, a wavefront by
// itself: slot s of row r holds 16-byte piece s ^ r, so that sixteen rows at
// one piece fall in distinct banks.
struct MvLine {
    u32x4_t c[4];
    uint32_t s[2];
};
__device__ __forceinline__ void load_line(MvLine &b, const WeightB &w, int64_t row0,
                                          int64_t last_row, int u0, int64_t K, int lane)
{
    const int pieces = (int)(K >> 5), sbytes = (int)(K >> 4);
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int r = 4 * j + (lane >> 4);
        int p = 4 * u0 + ((lane & 15) ^ r);
        p = p < pieces ? p : pieces - 1;             // past K: any codes, against zeros
        const int64_t row = row0 + r < last_row ? row0 + r : last_row;
        b.c[j] = *reinterpret_cast<const u32x4_t *>(w.codes + row * (K >> 1) + 16 * p);
    }
    const int64_t row = row0 + (lane >> 2) < last_row ? row0 + (lane >> 2) : last_row;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        int o = 8 * (u0 + (lane & 3)) + 4 * h;
        o = o < sbytes ? o : sbytes - 4;
        b.s[h] = *reinterpret_cast<const uint32_t *>(w.bs + row * sbytes + o);
    }
}
template <int MT>
__device__ __forceinline__ void multiply_line(MvSums<1, MT> &st, const MvLine &b, uint8_t *turn,
                                              const uint8_t *xs, const int *ex, int rows, int u0,
                                              int units, int lane)
{
    const int l = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < 4; j++)
        *reinterpret_cast<u32x4_t *>(turn + 1024 * j + 16 * lane) = b.c[j];
    *reinterpret_cast<u32x2_t *>(turn + 4096 + 8 * lane) = u32x2_t{b.s[0], b.s[1]};
    // The block's sums join under the largest of its exponents and the sum's own.
    int xr[MT];
    float f[MV_LINE][MT];
#pragma unroll
    for (int t = 0; t < MT; t++) {
        xr[t] = 16 * t + l < rows ? 16 * t + l : rows - 1;
        int e[MV_LINE], en = st.e[t];
#pragma unroll
        for (int j = 0; j < MV_LINE; j++) {
            e[j] = u0 + j < units ? ex[(u0 + j) * rows + xr[t]] : -1000;
            en = e[j] > en ? e[j] : en;
        }
        st.a[0][t] *= __builtin_ldexpf(1.0f, st.e[t] - en);
        st.e[t] = en;
#pragma unroll
        for (int j = 0; j < MV_LINE; j++)
            f[j][t] = __builtin_ldexpf(1.0f, e[j] - en);
    }
#pragma unroll
    for (int j = 0; j < MV_LINE; j++) {
        if (u0 + j >= units)
            break;
        const u32x4_t c = *reinterpret_cast<const u32x4_t *>(turn + 256 * l +
                                                             16 * ((4 * j + g) ^ l));
        const f16x2_t sc = e4m3_pair(*reinterpret_cast<const uint16_t *>(turn + 4096 + 32 * l +
                                                                         8 * j + 2 * g));
        f32x4_t d[MT];
#pragma unroll
        for (int t = 0; t < MT; t++)
            d[t] = f32x4_t{};
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const f16x8_t wf = oct(c[q], sc[q >> 1]);
#pragma unroll
            for (int t = 0; t < MT; t++) {
                const f16x8_t xf = *reinterpret_cast<const f16x8_t *>(
                    xs + ((u0 + j) * rows + xr[t]) * MV_XROW + 64 * g + 16 * q);
                d[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf, xf, d[t], 0, 0, 0);
            }
        }
#pragma unroll
        for (int t = 0; t < MT; t++)
#pragma unroll
            for (int k = 0; k < 4; k++)
                st.a[0][t][k] = __builtin_fmaf(d[t][k], f[j][t], st.a[0][t][k]);
    }
}

// The tiles t0, t0 + step, ... of one weight (rows row0 ..) times the staged
// rows; out(m, n, sums, e) ends each element with the sums of the NW weights
// in units of 2^e.
template <int NW, int MT, typename Out>
__device__ __forceinline__ void split_tiles(const WeightB *w, int64_t row0, int64_t N, int64_t K,
                                          int tiles, int t0, int step, const uint8_t *xs,
                                          const int *ex, int rows, int units, float *red,
                                          int *red_e, MvBlock<NW> &first, Out out)
{
    const int lane = (int)lane_id(), l = lane & 15, g = lane >> 4, wave = wave_in_group();
    constexpr int PART = 16 * MT * MV_RROW;                  // floats of a wavefront's tile
    constexpr int SPAN = MV_SPLIT * mv_block(NW);            // units of a block
    const int blocks = (units + SPAN - 1) / SPAN, u0 = wave;
    auto tile_row = [&](int t) {
        const int64_t n = (int64_t)16 * t + l;
        return row0 + (n < N ? n : N - 1);
    };
    MvBlock<NW> cur = first;
    int parity = 0;
    for (int t = t0; t < tiles; t += step) {
        MvSums<NW, MT> st;
#pragma unroll
        for (int i = 0; i < MT; i++) {
            st.e[i] = -300;
#pragma unroll
            for (int k = 0; k < NW; k++)
                st.a[k][i] = f32x4_t{};
        }
        for (int b = 0; b < blocks; b++) {
            MvBlock<NW> nx;
            const bool more = b + 1 < blocks;
            if (more || t + step < tiles)
                load_block<NW>(nx, w, tile_row(more ? t : t + step),
                                   u0 + (more ? SPAN * (b + 1) : 0), units, K, g);
            multiply_block<NW, MT>(st, cur, xs, ex, rows, u0 + SPAN * b, units, l, g);
            cur = nx;
        }
        {
            float *mine = red + (parity * MV_SPLIT + wave) * NW * PART;
            int *mine_e = red_e + (parity * MV_SPLIT + wave) * 16 * MT;
#pragma unroll
            for (int i = 0; i < MT; i++) {
                if (g == 0)
                    mine_e[16 * i + l] = st.e[i];
#pragma unroll
                for (int k = 0; k < NW; k++)
                    *reinterpret_cast<f32x4_t *>(mine + k * PART + (16 * i + l) * MV_RROW +
                                                 4 * g) = st.a[k][i];
            }
            __syncthreads();
            // Tile t's partials are read here and overwritten two tiles on, behind the
            // next tile's barrier.
            for (int o = (int)tid(); o < 16 * rows; o += 64 * MV_SPLIT) {
                const int m = o >> 4, n = o & 15;
                int e = -300;
#pragma unroll
                for (int v = 0; v < MV_SPLIT; v++) {
                    const int ev = red_e[(parity * MV_SPLIT + v) * 16 * MT + m];
                    e = e > ev ? e : ev;
                }
                float s[NW];
#pragma unroll
                for (int k = 0; k < NW; k++) {
                    s[k] = 0.0f;
#pragma unroll
                    for (int v = 0; v < MV_SPLIT; v++)
                        s[k] += __builtin_ldexpf(
                            red[(parity * MV_SPLIT + v) * NW * PART + k * PART + m * MV_RROW + n],
                            red_e[(parity * MV_SPLIT + v) * 16 * MT + m] - e);
                }
                if ((int64_t)16 * t + n < N)
                    out(m, (int64_t)16 * t + n, s, e);
            }
            parity ^= 1;
        }
    }
}

// The same by a wavefront alone: tiles t0, t0 + step, ..., all of K each, one
// weight after the other.
template <int NW, int MT, typename Out>
__device__ __forceinline__ void whole_tiles(const WeightB *w, int64_t row0, int64_t N, int64_t K,
                                            int tiles, int t0, int step, const uint8_t *xs,
                                            const int *ex, int rows, int units, uint8_t *turn,
                                            MvLine &first, Out out)
{
    const int lane = (int)lane_id(), l = lane & 15, g = lane >> 4;
    const int blocks = (units + MV_LINE - 1) / MV_LINE;
    MvLine cur = first;
    for (int t = t0; t < tiles; t += step) {
        MvSums<1, MT> st[NW];
#pragma unroll
        for (int i = 0; i < NW; i++) {
#pragma unroll
            for (int m = 0; m < MT; m++) {
                st[i].e[m] = -300;
                st[i].a[0][m] = f32x4_t{};
            }
            for (int b = 0; b < blocks; b++) {
                MvLine nx;
                const bool more = b + 1 < blocks, here = more || i + 1 < NW;
                if (here || t + step < tiles)
                    load_line(nx, w[more ? i : i + 1 < NW ? i + 1 : 0],
                              row0 + 16 * (int64_t)(here ? t : t + step), row0 + N - 1,
                              more ? MV_LINE * (b + 1) : 0, K, lane);
                multiply_line<MT>(st[i], cur, turn, xs, ex, rows, MV_LINE * b, units, lane);
                cur = nx;
            }
        }
        // Lane (m, g) holds four consecutive columns of row m, every weight's under the
        // same exponent (the row's largest).
#pragma unroll
        for (int m = 0; m < MT; m++)
            if (16 * m + l < rows)
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const int64_t n = (int64_t)16 * t + 4 * g + c;
                    float v[NW];
#pragma unroll
                    for (int i = 0; i < NW; i++)
                        v[i] = st[i].a[0][m][c];
                    if (n < N)
                        out(16 * m + l, n, v, st[0].e[m]);
                }
    }
}

// LDS of a launch: staged rows, their exponents, then two parities of the
// wavefronts' partial tiles (K split, waves = 0) or each wavefront's room to
// turn its loads in.
struct MvLds {
    int ex, red, red_e, bytes;
};
__host__ __device__ inline MvLds mv_lds(int rows, int units, int nw, int mt, int waves)
{
    MvLds o;
    o.ex = rows * units * MV_XROW;
    o.red = o.ex + (rows * units * 4 + 15) / 16 * 16;
    o.red_e = o.red + (waves ? waves * MV_TURN : 2 * MV_SPLIT * nw * 16 * mt * MV_RROW * 4);
    o.bytes = o.red_e + (waves ? 0 : 2 * MV_SPLIT * 16 * mt * 4);
    return o;
}

template <bool BF16_OUT, int FMT, int MT, bool WHOLE>
__global__ void __launch_bounds__(64 * (WHOLE ? MV_MAX_WAVES : MV_SPLIT))
    nvfp4_matvec_kernel(MvArgs a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int units = (int)((a.K + MV_UNIT - 1) / MV_UNIT);
    const int wg = (int)(wg_id() / (uint32_t)a.passes), pass = (int)(wg_id() % (uint32_t)a.passes);
    const int m0 = pass * a.rows, rows = a.M - m0 < a.rows ? a.M - m0 : a.rows;
    const MvLds o = mv_lds(a.rows, units, 1, MT, WHOLE ? a.waves : 0);
    int *ex = reinterpret_cast<int *>(lds + o.ex);
    const int lane = (int)lane_id(), wave = wave_in_group();
    auto src = [&](int r) { return (int64_t)m0 + r; };
    auto out = [&](int m, int64_t nn, const float *s, int e) {
        float v = s[0];
        if constexpr (FMT == MXQ_X_NVFP4)
            v *= mantissa(a.x.s[m0 + m], &e);
        st_elem<BF16_OUT>(a.c, (m0 + m) * a.N + nn,
                          scaled(v, a.scales[udiv((uint32_t)nn, a.per_scale)], e));
    };
    if constexpr (WHOLE) {
        const int t0 = wg * a.waves + wave;
        MvLine first;
        load_line(first, a.w, (int64_t)16 * t0, a.N - 1, 0, a.K, lane);
        stage_rows<FMT>(lds, ex, a.x, rows, units, a.K, a.waves, src);
        __syncthreads();
        whole_tiles<1, MT>(&a.w, 0, a.N, a.K, a.tiles, t0, a.wgs_n * a.waves, lds, ex, rows, units,
                           lds + o.red + wave * MV_TURN, first, out);
    } else {
        const int64_t n = (int64_t)16 * wg + (lane & 15);
        MvBlock<1> first;
        load_block<1>(first, &a.w, n < a.N ? n : a.N - 1, wave, units, a.K, lane >> 4);
        stage_rows<FMT>(lds, ex, a.x, rows, units, a.K, a.waves, src);
        __syncthreads();
        split_tiles<1, MT>(&a.w, 0, a.N, a.K, a.tiles, wg, a.wgs_n, lds, ex, rows, units,
                           reinterpret_cast<float *>(lds + o.red),
                           reinterpret_cast<int *>(lds + o.red_e), first, out);
    }
}

// The expert of slot s (the s-th segment that has rows) and its rows.
__device__ __forceinline__ bool find_segment(const int64_t *off, int n_groups, int64_t total,
                                             int slot, int *expert, int64_t *r0, int64_t *r1)
{
    const int lane = (int)lane_id();
    for (int e0 = 0; e0 < n_groups; e0 += 64) {
        const int e = e0 + lane;
        int64_t a = 0, b = 0;
        if (e < n_groups) {
            a = off[e];
            b = off[e + 1];
            a = a < 0 ? 0 : a;
            b = b > total ? total : b;
        }
        uint64_t some = __builtin_amdgcn_ballot_w64(b > a);
        const int n = __builtin_popcountll(some);
        if (slot < n) {
            for (; slot > 0; slot--)
                some &= some - 1;
            const int src = __builtin_ctzll(some);
            *expert = e0 + src;
            *r0 = __builtin_amdgcn_readlane((int)a, src);    // at most 2^30 rows
            *r1 = __builtin_amdgcn_readlane((int)b, src);
            return true;
        }
        slot -= n;
    }
    return false;
}

template <bool BF16_OUT, int FMT, int MT, bool WHOLE, bool GATED>
__global__ void __launch_bounds__(64 * (WHOLE ? MV_MAX_WAVES : MV_SPLIT))
    nvfp4_expert_kernel(MvArgs a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int NW = GATED ? 2 : 1;
    const int units = (int)((a.K + MV_UNIT - 1) / MV_UNIT);
    const int wg = (int)(wg_id() % (uint32_t)a.wgs_n);
    int e = 0;
    int64_t r0 = 0, r1 = 0;
    if (!find_segment(a.seg_offsets, a.n_groups, a.total_rows, (int)(wg_id() / (uint32_t)a.wgs_n),
                      &e, &r0, &r1))
        return;
    const MvLds o = mv_lds(a.chunk_rows, units, NW, MT, WHOLE ? a.waves : 0);
    int *ex = reinterpret_cast<int *>(lds + o.ex);
    const int lane = (int)lane_id(), wave = wave_in_group();
    const WeightB w[2] = {a.w, a.up};
    const int64_t row0 = (int64_t)e * a.N;
    const float scale = a.scales[e];
    for (int64_t c0 = r0; c0 < r1; c0 += a.chunk_rows) {
        const int rows = (int)(r1 - c0 < a.chunk_rows ? r1 - c0 : a.chunk_rows);
        auto src = [&](int r) {
            int64_t x = c0 + r;
            if constexpr (GATED) {
                x = a.row_tokens[x];
                x = x < 0 ? 0 : x >= a.n_tokens ? a.n_tokens - 1 : x;
            }
            return x;
        };
        auto out = [&](int m, int64_t nn, const float *s, int ee) {
            float sx = 1.0f;
            if constexpr (FMT == MXQ_X_NVFP4)
                sx = mantissa(a.x.s[src(m)], &ee);
            float v = scaled(s[0] * sx, scale, ee);
            if constexpr (GATED)
                v = silu_f32(v) * scaled(s[NW - 1] * sx, scale, ee);
            st_elem<BF16_OUT>(a.c, (c0 + m) * a.N + nn, v);
        };
        auto stage = [&] {
            if (c0 != r0)
                __syncthreads();                  // the last chunk's rows have been read
            stage_rows<FMT>(lds, ex, a.x, rows, units, a.K, a.waves, src);
            __syncthreads();
        };
        if constexpr (WHOLE) {
            const int t0 = wg * a.waves + wave;
            MvLine first;
            load_line(first, w[0], row0 + 16 * (int64_t)t0, row0 + a.N - 1, 0, a.K, lane);
            stage();
            whole_tiles<NW, MT>(w, row0, a.N, a.K, a.tiles, t0, a.wgs_n * a.waves, lds, ex, rows,
                                units, lds + o.red + wave * MV_TURN, first, out);
        } else {
            const int64_t n = (int64_t)16 * wg + (lane & 15);
            MvBlock<NW> first;
            load_block<NW>(first, w, row0 + (n < a.N ? n : a.N - 1), wave, units, a.K, lane >> 4);
            stage();
            split_tiles<NW, MT>(w, row0, a.N, a.K, a.tiles, wg, a.wgs_n, lds, ex, rows, units,
                                reinterpret_cast<float *>(lds + o.red),
                                reinterpret_cast<int *>(lds + o.red_e), first, out);
        }
    }
}

// Rows staged at once: at most `want`, as LDS holds them beside the rest
// (one row of the largest K always fits).
int staged_rows(int64_t want, int units, int nw, int waves)
{
    int r = (int)(want < MV_MAX_ROWS ? want : MV_MAX_ROWS);
    while (r > 1 && mv_lds(r, units, nw, (r + 15) / 16, waves).bytes > MV_LDS)
        r--;
    return r;
}
// Wavefronts of a workgroup that takes whole tiles: as many as fit beside the
// rows, 0 if not even four do.
int whole_waves(int64_t rows, int units, int nw, int most)
{
    const int r = (int)(rows < MV_MAX_ROWS ? rows : MV_MAX_ROWS);
    for (int w = most; w >= 4; w /= 2)
        if (mv_lds(r, units, nw, (r + 15) / 16, w).bytes <= MV_LDS)
            return w;
    return 0;
}

// Workgroups that the chip's 256 compute units hold with `lds` bytes each, at
// most MV_CU_WAVES wavefronts a unit: a launch of about as many stages its
// activations least often (32 x 8192 x 4096 BF16: 30 us with 512 workgroups,
// 37 us with 1024; 48 x 5120 x 2048: 17 and 23).
int64_t resident_target(int64_t lds, int waves)
{
    const int64_t per_cu = MV_LDS / lds, most = MV_CU_WAVES / waves;
    return 256 * (per_cu < 1 ? 1 : per_cu > most ? most : per_cu);
}

template <typename F>
void with_format(int fmt, bool bf16_out, F f)
{
    auto by_out = [&](auto format) {
        if (bf16_out)
            f(std::true_type{}, format);
        else
            f(std::false_type{}, format);
    };
    if (fmt == MXQ_X_BF16)
        by_out(std::integral_constant<int, MXQ_X_BF16>{});
    else if (fmt == MXQ_X_F32)
        by_out(std::integral_constant<int, MXQ_X_F32>{});
    else
        by_out(std::integral_constant<int, MXQ_X_NVFP4>{});
}

}  // namespace

hipError_t launch_nvfp4_matvec(const ActX &x, const WeightB &b, const float *scales,
                               int64_t rows_per_scale, int64_t M, int64_t N, int64_t K,
                               bool bf16_out, void *c, hipStream_t stream)
{
    MvArgs a{};
    a.x = x;
    a.w = b;
    a.scales = scales;
    a.per_scale = make_div((uint32_t)(rows_per_scale < N ? rows_per_scale : N));
    a.N = N;
    a.K = K;
    a.M = (int)M;
    a.tiles = (int)((N + 15) / 16);
    a.c = c;
    const int units = (int)((K + MV_UNIT - 1) / MV_UNIT);
    const int whole = a.tiles >= MV_WHOLE_K_TILES ? whole_waves(M, units, 1, MV_MAX_WAVES) : 0;
    const int most = staged_rows(M, units, 1, whole);
    a.passes = (int)((M + most - 1) / most);
    a.rows = (int)((M + a.passes - 1) / a.passes);
    a.waves = whole ? whole : MV_SPLIT;
    const int mt = (a.rows + 15) / 16;
    const size_t lds = (size_t)mv_lds(a.rows, units, 1, mt, whole).bytes;
    const int64_t work = whole ? (a.tiles + whole - 1) / whole : a.tiles;
    const int64_t share = (resident_target((int64_t)lds, a.waves) + a.passes - 1) / a.passes;
    a.wgs_n = (int)(work < share ? work : share);
    const dim3 grid((unsigned)(a.wgs_n * a.passes)), block(64 * a.waves);
    with_format(x.fmt, bf16_out, [&](auto out, auto fmt) {
        constexpr bool OUT = decltype(out)::value;
        constexpr int FMT = decltype(fmt)::value;
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, lds, stream, a); };
        if (mt == 1)
            whole ? go(nvfp4_matvec_kernel<OUT, FMT, 1, true>)
                  : go(nvfp4_matvec_kernel<OUT, FMT, 1, false>);
        else
            whole ? go(nvfp4_matvec_kernel<OUT, FMT, 2, true>)
                  : go(nvfp4_matvec_kernel<OUT, FMT, 2, false>);
    });
    return hipGetLastError();
}

bool expert_grid_ok(int64_t n_groups, int64_t, int64_t N)
{
    return n_groups * ((N + 3) / 4) < ((int64_t)1 << 24);
}

hipError_t launch_nvfp4_expert_matvec(const ActX &x, int64_t n_tokens, const int64_t *row_tokens,
                                      const int64_t *seg_offsets, int64_t n_groups,
                                      int64_t total_rows, const WeightB &w, const WeightB &up,
                                      const float *scales, int64_t N, int64_t K, bool bf16_out,
                                      void *c, hipStream_t stream)
{
    MvArgs a{};
    a.x = x;
    a.w = w;
    a.up = up;
    a.scales = scales;
    a.N = N;
    a.K = K;
    a.n_tokens = n_tokens;
    a.total_rows = total_rows;
    a.row_tokens = row_tokens;
    a.seg_offsets = seg_offsets;
    a.n_groups = (int)n_groups;
    a.tiles = (int)((N + 15) / 16);
    a.c = c;
    // One slot per expert that can have rows.  Rows staged at once: three even shares,
    // which few experts exceed (they take their weights twice, from L2).
    const int64_t slots = n_groups < total_rows ? n_groups : total_rows;
    const int64_t even = 3 * ((total_rows + slots - 1) / slots);
    const bool gated = up.codes != nullptr;
    const int nw = gated ? 2 : 1, units = (int)((K + MV_UNIT - 1) / MV_UNIT);
    const int64_t want = total_rows < even ? total_rows : even;
    const int whole = slots * a.tiles >= MV_WHOLE_K_TILES ? whole_waves(want, units, nw, MV_SPLIT) : 0;
    a.chunk_rows = staged_rows(want, units, nw, whole);
    a.waves = whole ? whole : MV_SPLIT;
    const int mt = (a.chunk_rows + 15) / 16;
    const size_t lds = (size_t)mv_lds(a.chunk_rows, units, nw, mt, whole).bytes;
    // Equal shares of an expert's tiles, for about as many workgroups as fit the chip.
    const int64_t target = resident_target((int64_t)lds, a.waves);
    const int64_t per = (target + slots - 1) / slots;
    const int64_t work = whole ? (a.tiles + whole - 1) / whole : a.tiles;
    const int64_t each = work <= per ? 1 : (work + per - 1) / per;
    a.wgs_n = (int)((work + each - 1) / each);
    const dim3 grid((unsigned)(a.wgs_n * slots)), block(64 * a.waves);
    with_format(x.fmt, bf16_out, [&](auto out, auto fmt) {
        constexpr bool OUT = decltype(out)::value;
        constexpr int FMT = decltype(fmt)::value;
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, lds, stream, a); };
        auto by_split = [&](auto mtc, auto gate) {
            constexpr int MT = decltype(mtc)::value;
            constexpr bool GATED = decltype(gate)::value;
            whole ? go(nvfp4_expert_kernel<OUT, FMT, MT, true, GATED>)
                  : go(nvfp4_expert_kernel<OUT, FMT, MT, false, GATED>);
        };
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        if (mt == 1)
            gated ? by_split(One{}, std::true_type{}) : by_split(One{}, std::false_type{});
        else
            gated ? by_split(Two{}, std::true_type{}) : by_split(Two{}, std::false_type{});
    });
    return hipGetLastError();
}

}  // namespace mxq
