// mxq_api.cpp -- the C ABI of libmxq (declared in include/mxq.h): host-side
// validation, then the launch.  Nothing here allocates device memory.
#include "mxq.h"

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "mxq_launch.h"
#include "mxq_layer.h"

namespace {

// One array argument: its extent in bytes, required alignment, and whether
// the call writes it.
struct Buf {
    const void *p;
    int64_t bytes;
    int align;
    bool output;
};

constexpr int64_t MAX_ELEMS = (int64_t)1 << 62;
// GEMM tiles address their 256 rows with 32-bit offsets.
constexpr int64_t MAX_GEMM_K = (int64_t)1 << 23;
constexpr int64_t MAX_GRID_ROWS = mxq::MAX_TOKEN_ROWS;   // per-token NVFP4: one workgroup per row
constexpr int64_t MAX_BLOCKS = 0xFFFFFFFF;        // 16-element blocks indexed in 32 bits
constexpr int64_t MAX_MXFP8_COLS = (int64_t)1 << 26;  // 32-row tile offsets fit 32 bits
constexpr int64_t MAX_COPY_FLOOR_BYTES = (int64_t)1 << 35;
// Layer operators: one workgroup of at most 256 threads per token, and the
// sizes the few-row products and the attention index with 32 bits.
constexpr int64_t MAX_LAYER_TOKENS = (int64_t)1 << 24;
constexpr int64_t MAX_MATVEC_ROWS = 64, MAX_MATVEC_N = (int64_t)1 << 24;
constexpr int64_t MAX_MATVEC_K = (int64_t)1 << 16, MAX_MATVEC_GROUPS = (int64_t)1 << 16;
constexpr int64_t MAX_ATTN_ROWS = (int64_t)1 << 25, MAX_ATTN_KEYS = (int64_t)1 << 30;
constexpr int64_t MAX_CACHE_ROWS = (int64_t)1 << 40;

bool size_ok(int64_t a, int64_t b)
{
    return a > 0 && b > 0 && a <= MAX_ELEMS / b;
}

// The MXFP8 tile launches over `row_tiles` 32-row tiles of `cols` columns
// fit one grid.
bool mxfp8_grid_ok(int64_t row_tiles, int64_t cols)
{
    return row_tiles <= MAX_ELEMS / cols && mxq::mxfp8_tiles(row_tiles, cols) <= mxq::MAX_MXFP8_TILES;
}

// One allocation of the current device: [base, base + size).
struct Range {
    uintptr_t base;
    uint64_t size;
};

bool inside(const Buf &b, const Range &r)
{
    const uintptr_t p = (uintptr_t)b.p;
    return p >= r.base && (uint64_t)(p - r.base) + (uint64_t)b.bytes <= r.size;
}

// Device memory of the current device, and [p, p + bytes) inside one
// allocation, whose range is returned in *r.
int check_device(const Buf &b, int device, Range *r)
{
    hipPointerAttribute_t attr;
    if (hipPointerGetAttributes(&attr, b.p) != hipSuccess) {
        (void)hipGetLastError();
        return MXQ_ERR_DEVICE;
    }
    if (attr.type != hipMemoryTypeDevice || attr.device != device)
        return MXQ_ERR_DEVICE;
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    if (hipMemGetAddressRange(&base, &size, const_cast<void *>(b.p)) != hipSuccess) {
        (void)hipGetLastError();
        return MXQ_ERR_DEVICE;
    }
    *r = Range{(uintptr_t)base, (uint64_t)size};
    if (!inside(b, *r))
        return MXQ_ERR_DEVICE;
    return MXQ_OK;
}

bool overlaps(const Buf &a, const Buf &b)
{
    const uintptr_t a0 = (uintptr_t)a.p, a1 = a0 + (uintptr_t)a.bytes;
    const uintptr_t b0 = (uintptr_t)b.p, b1 = b0 + (uintptr_t)b.bytes;
    return a0 < b1 && b0 < a1;
}

// Alignment, device residency and extent of every buffer, then pairwise
// overlap between any output and any other buffer.
int check_bufs(const Buf *bufs, int n)
{
    for (int i = 0; i < n; i++)
        if (((uintptr_t)bufs[i].p) % (uintptr_t)bufs[i].align != 0)
            return MXQ_ERR_ALIGN;
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess) {
        (void)hipGetLastError();
        return MXQ_ERR_DEVICE;
    }
    // A buffer inside an allocation already queried in this call (same
    // device, device memory) needs no runtime query of its own: each query
    // costs about 0.4 us of host time, which bounds back-to-back launches
    // of small kernels.
    Range seen[16];
    int n_seen = 0;
    for (int i = 0; i < n; i++) {
        bool known = false;
        for (int k = 0; k < n_seen && !known; k++)
            known = inside(bufs[i], seen[k]);
        if (known)
            continue;
        Range r{0, 0};
        const int st = check_device(bufs[i], device, &r);
        if (st != MXQ_OK)
            return st;
        if (n_seen < 16)
            seen[n_seen++] = r;
    }
    for (int i = 0; i < n; i++)
        for (int j = i + 1; j < n; j++)
            if ((bufs[i].output || bufs[j].output) && overlaps(bufs[i], bufs[j]))
                return MXQ_ERR_ALIAS;
    return MXQ_OK;
}

int launched(hipError_t e)
{
    return e == hipSuccess ? MXQ_OK : MXQ_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int mxq_version(void)
{
    return MXQ_VERSION;
}

const char *mxq_status_string(int status)
{
    switch (status) {
    case MXQ_OK: return "ok";
    case MXQ_ERR_NULL: return "a required pointer is NULL";
    case MXQ_ERR_SIZE: return "a size is not positive (or too large), or n_groups < 1";
    case MXQ_ERR_SHAPE: return "rows/cols not divisible as the format requires";
    case MXQ_ERR_ALIGN: return "a pointer is not aligned as required (16 bytes for vector-accessed arrays)";
    case MXQ_ERR_ALIAS: return "an output overlaps an input or another output";
    case MXQ_ERR_OFFSETS: return "inconsistent combination of optional outputs";
    case MXQ_ERR_DEVICE: return "an array is not device memory of the current device, or extends past the end of its allocation";
    case MXQ_ERR_LAUNCH: return "kernel launch failed";
    case MXQ_ERR_ARG: return "unknown format argument";
    default: return "unknown status";
    }
}

int mxq_mxfp8_quantize_rowcol(const uint16_t *x, int64_t rows, int64_t cols, uint8_t *row_codes,
                              uint8_t *row_scales, uint8_t *col_codes, uint8_t *col_scales,
                              void *stream)
{
    if (!x)
        return MXQ_ERR_NULL;
    if ((row_codes == nullptr) != (row_scales == nullptr) ||
        (col_codes == nullptr) != (col_scales == nullptr) || (!row_codes && !col_codes))
        return MXQ_ERR_OFFSETS;
    if (!size_ok(rows, cols) || cols > MAX_MXFP8_COLS || !mxfp8_grid_ok((rows + 31) / 32, cols))
        return MXQ_ERR_SIZE;
    if (cols % 32 != 0 || (col_codes && rows % 32 != 0))
        return MXQ_ERR_SHAPE;
    const int64_t n = rows * cols;
    Buf b[5];
    int k = 0;
    b[k++] = {x, 2 * n, 16, false};
    if (row_codes) {
        b[k++] = {row_codes, n, 16, true};
        b[k++] = {row_scales, n / 32, 1, true};
    }
    if (col_codes) {
        b[k++] = {col_codes, n, 16, true};
        b[k++] = {col_scales, n / 32, 8, true};
    }
    const int st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_mxfp8_dense(x, rows, cols, row_codes, row_scales, col_codes,
                                            col_scales, nullptr, 0, (hipStream_t)stream));
}

int mxq_mxfp8_quantize_ocp_floor(const uint16_t *x, int64_t rows, int64_t cols,
                                 uint8_t *row_codes, uint8_t *row_scales, uint8_t *col_codes,
                                 uint8_t *col_scales, void *stream)
{
    if (!x)
        return MXQ_ERR_NULL;
    if ((row_codes == nullptr) != (row_scales == nullptr) ||
        (col_codes == nullptr) != (col_scales == nullptr) || (!row_codes && !col_codes))
        return MXQ_ERR_OFFSETS;
    if (!size_ok(rows, cols) || cols > MAX_MXFP8_COLS || !mxfp8_grid_ok((rows + 31) / 32, cols))
        return MXQ_ERR_SIZE;
    if (cols % 32 != 0 || (col_codes && rows % 32 != 0))
        return MXQ_ERR_SHAPE;
    const int64_t n = rows * cols;
    Buf b[5];
    int k = 0;
    b[k++] = {x, 2 * n, 16, false};
    if (row_codes) {
        b[k++] = {row_codes, n, 16, true};
        b[k++] = {row_scales, n / 32, 1, true};
    }
    if (col_codes) {
        b[k++] = {col_codes, n, 16, true};
        b[k++] = {col_scales, n / 32, 8, true};
    }
    const int st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_mxfp8_ocp_floor(x, rows, cols, row_codes, row_scales, col_codes,
                                                col_scales, (hipStream_t)stream));
}

int mxq_mxfp8_quantize_rowcol_t(const uint16_t *x, int64_t rows, int64_t cols,
                                uint8_t *row_codes, uint8_t *row_scales, uint8_t *col_codes_t,
                                uint8_t *col_scales_t, void *stream)
{
    if (!x || !col_codes_t || !col_scales_t)
        return MXQ_ERR_NULL;
    if ((row_codes == nullptr) != (row_scales == nullptr))
        return MXQ_ERR_OFFSETS;
    if (!size_ok(rows, cols) || cols > MAX_MXFP8_COLS || !mxfp8_grid_ok((rows + 31) / 32, cols))
        return MXQ_ERR_SIZE;
    if (cols % 32 != 0 || rows % 32 != 0)
        return MXQ_ERR_SHAPE;
    const int64_t n = rows * cols;
    Buf b[5];
    int k = 0;
    b[k++] = {x, 2 * n, 16, false};
    b[k++] = {col_codes_t, n, 16, true};
    b[k++] = {col_scales_t, n / 32, 1, true};
    if (row_codes) {
        b[k++] = {row_codes, n, 16, true};
        b[k++] = {row_scales, n / 32, 1, true};
    }
    const int st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_mxfp8_colt(x, rows, cols, row_codes, row_scales, col_codes_t,
                                           col_scales_t, (hipStream_t)stream));
}

int mxq_nvfp4_quantize_per_token(const uint16_t *x, int64_t rows, int64_t cols, uint8_t *codes,
                                 uint8_t *block_scales, float *token_scales, void *stream)
{
    if (!x || !codes || !block_scales || !token_scales)
        return MXQ_ERR_NULL;
    if (!size_ok(rows, cols) || rows > MAX_GRID_ROWS)
        return MXQ_ERR_SIZE;
    if (cols % 16 != 0)
        return MXQ_ERR_SHAPE;
    const int64_t n = rows * cols;
    const Buf b[4] = {{x, 2 * n, 16, false},
                      {codes, n / 2, 16, true},
                      {block_scales, n / 16, 1, true},
                      {token_scales, 4 * rows, 4, true}};
    const int st = check_bufs(b, 4);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_nvfp4_per_token(x, rows, cols, codes, block_scales, token_scales,
                                                (hipStream_t)stream));
}

int mxq_nvfp4_quantize_per_token_approx(const uint16_t *x, int64_t rows, int64_t cols,
                                        uint8_t *codes, uint8_t *block_scales,
                                        float *token_scales, void *stream)
{
    if (!x || !codes || !block_scales || !token_scales)
        return MXQ_ERR_NULL;
    if (!size_ok(rows, cols) || rows > MAX_GRID_ROWS || cols > 4096)
        return MXQ_ERR_SIZE;
    if (cols % 16 != 0)
        return MXQ_ERR_SHAPE;
    const int64_t n = rows * cols;
    const Buf b[4] = {{x, 2 * n, 16, false},
                      {codes, n / 2, 16, true},
                      {block_scales, n / 16, 1, true},
                      {token_scales, 4 * rows, 4, true}};
    const int st = check_bufs(b, 4);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_nvfp4_approx(x, rows, cols, codes, block_scales, token_scales,
                                             (hipStream_t)stream));
}

int mxq_nvfp4_quantize_gateup_pair(const uint16_t *gate, const uint16_t *up, int64_t n_experts,
                                   int64_t rows, int64_t cols, uint8_t *gate_codes,
                                   uint8_t *gate_block_scales, uint8_t *up_codes,
                                   uint8_t *up_block_scales, float *scope_scales, void *stream)
{
    if (!gate || !gate_codes || !gate_block_scales || !scope_scales)
        return MXQ_ERR_NULL;
    const bool has_up = up != nullptr;
    if ((up_codes != nullptr) != has_up || (up_block_scales != nullptr) != has_up)
        return MXQ_ERR_OFFSETS;
    if (!size_ok(rows, cols) || n_experts <= 0 || !size_ok(n_experts, rows * cols))
        return MXQ_ERR_SIZE;
    if (cols % 16 != 0)
        return MXQ_ERR_SHAPE;
    const int64_t n = n_experts * rows * cols;
    if (n / 16 > MAX_BLOCKS || n_experts > mxq::MAX_GRID_ITEMS / 64 ||
        mxq::scoped_amax_workgroups(n_experts, rows * cols, has_up) >
            mxq::MAX_SCOPED_AMAX_WORKGROUPS)
        return MXQ_ERR_SIZE;
    Buf b[7];
    int k = 0;
    b[k++] = {gate, 2 * n, 16, false};
    b[k++] = {gate_codes, n / 2, 16, true};
    b[k++] = {gate_block_scales, n / 16, 1, true};
    b[k++] = {scope_scales, 4 * n_experts, 4, true};
    if (has_up) {
        b[k++] = {up, 2 * n, 16, false};
        b[k++] = {up_codes, n / 2, 16, true};
        b[k++] = {up_block_scales, n / 16, 1, true};
    }
    const int st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_nvfp4_scoped(gate, up, n_experts, rows, cols, gate_codes,
                                             gate_block_scales, up_codes, up_block_scales,
                                             scope_scales, (hipStream_t)stream));
}

int mxq_nvfp4_quantize_gateup_pair_amax(const uint16_t *gate, const uint16_t *up,
                                        const uint16_t *scope_amax, int64_t n_experts,
                                        int64_t rows, int64_t cols, uint8_t *gate_codes,
                                        uint8_t *gate_block_scales, uint8_t *up_codes,
                                        uint8_t *up_block_scales, float *scope_scales,
                                        void *stream)
{
    if (!gate || !scope_amax || !gate_codes || !gate_block_scales || !scope_scales)
        return MXQ_ERR_NULL;
    const bool has_up = up != nullptr;
    if ((up_codes != nullptr) != has_up || (up_block_scales != nullptr) != has_up)
        return MXQ_ERR_OFFSETS;
    if (!size_ok(rows, cols) || n_experts <= 0 || !size_ok(n_experts, rows * cols))
        return MXQ_ERR_SIZE;
    if (cols % 16 != 0)
        return MXQ_ERR_SHAPE;
    const int64_t n = n_experts * rows * cols;
    if (n / 16 > MAX_BLOCKS || n_experts > mxq::MAX_GRID_ITEMS / 64)
        return MXQ_ERR_SIZE;
    Buf b[8];
    int k = 0;
    b[k++] = {gate, 2 * n, 16, false};
    b[k++] = {scope_amax, 2 * n_experts, 2, false};
    b[k++] = {gate_codes, n / 2, 16, true};
    b[k++] = {gate_block_scales, n / 16, 1, true};
    b[k++] = {scope_scales, 4 * n_experts, 4, true};
    if (has_up) {
        b[k++] = {up, 2 * n, 16, false};
        b[k++] = {up_codes, n / 2, 16, true};
        b[k++] = {up_block_scales, n / 16, 1, true};
    }
    const int st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_nvfp4_scoped_amax(gate, up, scope_amax, n_experts, rows, cols,
                                                  gate_codes, gate_block_scales, up_codes,
                                                  up_block_scales, scope_scales,
                                                  (hipStream_t)stream));
}

int mxq_dequantize_bf16(int fmt, const uint8_t *codes, const uint8_t *scales,
                        const float *fp32_scales, int64_t rows_per_fp32_scale, int64_t rows,
                        int64_t cols, uint16_t *out, void *stream)
{
    if (fmt != MXQ_FMT_MXFP8_ROW && fmt != MXQ_FMT_MXFP8_COL && fmt != MXQ_FMT_NVFP4)
        return MXQ_ERR_ARG;
    if (!codes || !scales || !out || (fmt == MXQ_FMT_NVFP4 && !fp32_scales))
        return MXQ_ERR_NULL;
    if (!size_ok(rows, cols) || (fmt == MXQ_FMT_NVFP4 && rows_per_fp32_scale < 1))
        return MXQ_ERR_SIZE;
    const int64_t n = rows * cols;
    if (n / 16 > MAX_BLOCKS)
        return MXQ_ERR_SIZE;
    if (fmt == MXQ_FMT_NVFP4) {
        if (cols % 16 != 0)
            return MXQ_ERR_SHAPE;
        const int64_t n_scales = (rows + rows_per_fp32_scale - 1) / rows_per_fp32_scale;
        const Buf b[4] = {{codes, n / 2, 8, false},
                          {scales, n / 16, 1, false},
                          {fp32_scales, 4 * n_scales, 4, false},
                          {out, 2 * n, 16, true}};
        const int st = check_bufs(b, 4);
        if (st != MXQ_OK)
            return st;
        return launched(mxq::launch_dequant_nvfp4(codes, scales, fp32_scales, rows_per_fp32_scale,
                                                  rows, cols, out, (hipStream_t)stream));
    }
    const bool col = fmt == MXQ_FMT_MXFP8_COL;
    if (cols % 32 != 0 || (col && rows % 32 != 0))
        return MXQ_ERR_SHAPE;
    const Buf b[3] = {{codes, n, 16, false}, {scales, n / 32, col ? 16 : 1, false},
                      {out, 2 * n, 16, true}};
    const int st = check_bufs(b, 3);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_dequant_mxfp8(col, codes, scales, rows, cols, out,
                                              (hipStream_t)stream));
}

int mxq_quantize_dequant_bf16(int fmt, const uint16_t *x, int64_t rows, int64_t cols,
                              uint8_t *codes, uint8_t *scales, float *token_scales,
                              uint16_t *out, void *stream)
{
    if (fmt != MXQ_FMT_MXFP8_ROW && fmt != MXQ_FMT_NVFP4)
        return MXQ_ERR_ARG;
    if (!x || !out)
        return MXQ_ERR_NULL;
    if ((codes == nullptr) != (scales == nullptr) ||
        (fmt == MXQ_FMT_MXFP8_ROW && token_scales != nullptr))
        return MXQ_ERR_OFFSETS;
    if (!size_ok(rows, cols))
        return MXQ_ERR_SIZE;
    const int64_t n = rows * cols;
    Buf b[5];
    int k = 0;
    b[k++] = {x, 2 * n, 16, false};
    b[k++] = {out, 2 * n, 16, true};
    if (fmt == MXQ_FMT_NVFP4) {
        if (rows > MAX_GRID_ROWS)
            return MXQ_ERR_SIZE;
        if (cols % 16 != 0)
            return MXQ_ERR_SHAPE;
        if (codes) {
            b[k++] = {codes, n / 2, 16, true};
            b[k++] = {scales, n / 16, 1, true};
        }
        if (token_scales)
            b[k++] = {token_scales, 4 * rows, 4, true};
        const int st = check_bufs(b, k);
        if (st != MXQ_OK)
            return st;
        return launched(mxq::launch_nvfp4_qdq(x, rows, cols, codes, scales, token_scales, out,
                                              (hipStream_t)stream));
    }
    if (cols > MAX_MXFP8_COLS || !mxfp8_grid_ok((rows + 31) / 32, cols))
        return MXQ_ERR_SIZE;
    if (cols % 32 != 0)
        return MXQ_ERR_SHAPE;
    if (codes) {
        b[k++] = {codes, n, 16, true};
        b[k++] = {scales, n / 32, 1, true};
    }
    const int st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_mxfp8_row_qdq(x, rows, cols, codes, scales, out,
                                              (hipStream_t)stream));
}

int mxq_mxfp8_gemm(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b,
                   const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, int out_dtype,
                   void *c, void *stream)
{
    if (out_dtype != MXQ_OUT_F32 && out_dtype != MXQ_OUT_BF16)
        return MXQ_ERR_ARG;
    if (!a || !a_scales || !b || !b_scales || !c)
        return MXQ_ERR_NULL;
    if (!size_ok(M, K) || !size_ok(N, K) || !size_ok(M, 4 * N))   // C up to 4 bytes
        return MXQ_ERR_SIZE;
    if (K % 128 != 0)
        return MXQ_ERR_SHAPE;
    if (K > MAX_GEMM_K || ((M + 255) / 256) * ((N + 255) / 256) > mxq::MAX_GEMM_TILES)
        return MXQ_ERR_SIZE;
    const int esz = out_dtype == MXQ_OUT_F32 ? 4 : 2;
    const Buf bb[5] = {{a, M * K, 16, false},
                       {a_scales, M * (K / 32), 4, false},
                       {b, N * K, 16, false},
                       {b_scales, N * (K / 32), 4, false},
                       {c, esz * M * N, esz, true}};
    const int st = check_bufs(bb, 5);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_mxfp8_gemm(a, a_scales, b, b_scales, M, N, K,
                                           out_dtype == MXQ_OUT_BF16, c, (hipStream_t)stream));
}

int mxq_mxfp8_grouped_gemm(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b,
                           const uint8_t *b_scales, const int64_t *seg_offsets, int64_t n_groups,
                           int64_t total_rows, int64_t N, int64_t K, int out_dtype, void *c,
                           void *stream)
{
    if (out_dtype != MXQ_OUT_F32 && out_dtype != MXQ_OUT_BF16)
        return MXQ_ERR_ARG;
    if (!a || !a_scales || !b || !b_scales || !seg_offsets || !c)
        return MXQ_ERR_NULL;
    if (!size_ok(total_rows, K) || !size_ok(N, K) || !size_ok(total_rows, 4 * N) || n_groups < 1 ||
        !size_ok(n_groups, N * K) || n_groups > MAX_ELEMS / 8 - 1)
        return MXQ_ERR_SIZE;
    if (K % 128 != 0)
        return MXQ_ERR_SHAPE;
    if (K > MAX_GEMM_K || total_rows > MAX_ELEMS / 4 - 255 ||
        mxq::grouped_gemm_mtiles(total_rows, n_groups) > mxq::MAX_GEMM_TILES ||
        mxq::grouped_gemm_mtiles(total_rows, n_groups) * ((N + 255) / 256) > mxq::MAX_GEMM_TILES)
        return MXQ_ERR_SIZE;
    const int esz = out_dtype == MXQ_OUT_F32 ? 4 : 2;
    const Buf bb[6] = {{a, total_rows * K, 16, false},
                       {a_scales, total_rows * (K / 32), 4, false},
                       {b, n_groups * N * K, 16, false},
                       {b_scales, n_groups * N * (K / 32), 4, false},
                       {seg_offsets, 8 * (n_groups + 1), 8, false},
                       {c, esz * total_rows * N, esz, true}};
    const int st = check_bufs(bb, 6);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_mxfp8_grouped_gemm(a, a_scales, b, b_scales, seg_offsets,
                                                   n_groups, total_rows, N, K,
                                                   out_dtype == MXQ_OUT_BF16, c,
                                                   (hipStream_t)stream));
}

// Shared by the two grouped transposed entry points; rc == nullptr: the
// columnwise copy alone.
static int grouped_colt(const uint16_t *x, int64_t total_rows, int64_t cols,
                        const int64_t *seg_offsets, int64_t n_groups, uint8_t *rc, uint8_t *rs,
                        uint8_t *codes_t, uint8_t *scales_t, int64_t *block_offsets,
                        void *stream)
{
    if (!size_ok(total_rows, cols) || cols > MAX_MXFP8_COLS || n_groups < 1 ||
        n_groups > ((int64_t)1 << 40) || total_rows > MAX_ELEMS / 4)
        return MXQ_ERR_SIZE;
    const int64_t pitch = mxq::grouped_colt_pitch(total_rows, n_groups);
    if (!size_ok(pitch, cols) || !mxfp8_grid_ok(pitch / 32, cols))
        return MXQ_ERR_SIZE;
    if (cols % 32 != 0)
        return MXQ_ERR_SHAPE;
    const int64_t n = total_rows * cols;
    Buf b[7] = {{x, 2 * n, 16, false},
                {seg_offsets, 8 * (n_groups + 1), 8, false},
                {codes_t, pitch * cols, 16, true},
                {scales_t, pitch / 32 * cols, 4, true},
                {block_offsets, 8 * (n_groups + 1), 8, true},
                {rc, n, 16, true},
                {rs, n / 32, 1, true}};
    const int st = check_bufs(b, rc ? 7 : 5);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_mxfp8_grouped_colt(x, total_rows, cols, seg_offsets, n_groups,
                                                   rc, rs, codes_t, scales_t, block_offsets,
                                                   (hipStream_t)stream));
}

int mxq_mxfp8_grouped_colwise_t(const uint16_t *x, int64_t total_rows, int64_t cols,
                                const int64_t *seg_offsets, int64_t n_groups, uint8_t *codes_t,
                                uint8_t *scales_t, int64_t *block_offsets, void *stream)
{
    if (!x || !seg_offsets || !codes_t || !scales_t || !block_offsets)
        return MXQ_ERR_NULL;
    return grouped_colt(x, total_rows, cols, seg_offsets, n_groups, nullptr, nullptr, codes_t,
                        scales_t, block_offsets, stream);
}

int mxq_mxfp8_grouped_quantize_rowcol_t(const uint16_t *x, int64_t total_rows, int64_t cols,
                                        const int64_t *seg_offsets, int64_t n_groups,
                                        uint8_t *row_codes, uint8_t *row_scales,
                                        uint8_t *codes_t, uint8_t *scales_t,
                                        int64_t *block_offsets, void *stream)
{
    if (!x || !seg_offsets || !row_codes || !row_scales || !codes_t || !scales_t ||
        !block_offsets)
        return MXQ_ERR_NULL;
    return grouped_colt(x, total_rows, cols, seg_offsets, n_groups, row_codes, row_scales,
                        codes_t, scales_t, block_offsets, stream);
}

int mxq_mxfp8_grouped_wgrad(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b,
                            const uint8_t *b_scales, const int64_t *block_offsets,
                            int64_t n_groups, int64_t M, int64_t N, int64_t pitch, int out_dtype,
                            void *c, void *stream)
{
    if (out_dtype != MXQ_OUT_F32 && out_dtype != MXQ_OUT_BF16)
        return MXQ_ERR_ARG;
    if (!a || !a_scales || !b || !b_scales || !block_offsets || !c)
        return MXQ_ERR_NULL;
    if (!size_ok(M, pitch) || !size_ok(N, pitch) || !size_ok(M, 4 * N) || n_groups < 1 ||
        !size_ok(n_groups, 4 * M * N) || n_groups > MAX_ELEMS / 8 - 1)
        return MXQ_ERR_SIZE;
    if (pitch % 128 != 0)
        return MXQ_ERR_SHAPE;
    if (pitch > MAX_GEMM_K ||
        n_groups * ((M + 255) / 256) * ((N + 255) / 256) > mxq::MAX_GEMM_TILES)
        return MXQ_ERR_SIZE;
    const int esz = out_dtype == MXQ_OUT_F32 ? 4 : 2;
    const Buf bb[6] = {{a, M * pitch, 16, false},
                       {a_scales, M * (pitch / 32), 4, false},
                       {b, N * pitch, 16, false},
                       {b_scales, N * (pitch / 32), 4, false},
                       {block_offsets, 8 * (n_groups + 1), 8, false},
                       {c, esz * n_groups * M * N, esz, true}};
    const int st = check_bufs(bb, 6);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_mxfp8_grouped_wgrad(a, a_scales, b, b_scales, block_offsets,
                                                    n_groups, M, N, pitch,
                                                    out_dtype == MXQ_OUT_BF16, c,
                                                    (hipStream_t)stream));
}

int mxq_nvfp4_grouped_gemm(const uint8_t *a, const uint8_t *a_block_scales, const float *a_scales,
                           const uint8_t *b, const uint8_t *b_block_scales, const float *b_scales,
                           const int64_t *seg_offsets, int64_t n_groups, int64_t total_rows,
                           int64_t N, int64_t K, int out_dtype, void *c, void *stream)
{
    if (out_dtype != MXQ_OUT_F32 && out_dtype != MXQ_OUT_BF16)
        return MXQ_ERR_ARG;
    if (!a || !a_block_scales || !a_scales || !b || !b_block_scales || !b_scales ||
        !seg_offsets || !c)
        return MXQ_ERR_NULL;
    if (!size_ok(total_rows, K) || !size_ok(N, K) || !size_ok(total_rows, 4 * N) ||
        n_groups < 1 || !size_ok(n_groups, N * K) || n_groups > MAX_ELEMS / 8 - 1)
        return MXQ_ERR_SIZE;
    if (K % 64 != 0)
        return MXQ_ERR_SHAPE;
    if (K > MAX_GEMM_K || total_rows > MAX_ELEMS / 4 - 255 ||
        mxq::grouped_gemm_mtiles(total_rows, n_groups) > mxq::MAX_GEMM_TILES ||
        mxq::grouped_gemm_mtiles(total_rows, n_groups) * ((N + 255) / 256) > mxq::MAX_GEMM_TILES)
        return MXQ_ERR_SIZE;
    const int esz = out_dtype == MXQ_OUT_F32 ? 4 : 2;
    const Buf bb[8] = {{a, total_rows * (K / 2), 16, false},
                       {a_block_scales, total_rows * (K / 16), 4, false},
                       {a_scales, 4 * total_rows, 4, false},
                       {b, n_groups * N * (K / 2), 16, false},
                       {b_block_scales, n_groups * N * (K / 16), 4, false},
                       {b_scales, 4 * n_groups, 4, false},
                       {seg_offsets, 8 * (n_groups + 1), 8, false},
                       {c, esz * total_rows * N, esz, true}};
    const int st = check_bufs(bb, 8);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_nvfp4_grouped_gemm(a, a_block_scales, a_scales, b,
                                                   b_block_scales, b_scales, seg_offsets,
                                                   n_groups, total_rows, N, K,
                                                   out_dtype == MXQ_OUT_BF16, c,
                                                   (hipStream_t)stream));
}

int mxq_nvfp4_gemm(const uint8_t *a, const uint8_t *a_block_scales, const float *a_scales,
                   int64_t rows_per_a_scale, const uint8_t *b, const uint8_t *b_block_scales,
                   const float *b_scales, int64_t rows_per_b_scale, int64_t M, int64_t N,
                   int64_t K, int out_dtype, void *c, void *stream)
{
    if (out_dtype != MXQ_OUT_F32 && out_dtype != MXQ_OUT_BF16)
        return MXQ_ERR_ARG;
    if (!a || !a_block_scales || !a_scales || !b || !b_block_scales || !b_scales || !c)
        return MXQ_ERR_NULL;
    if (!size_ok(M, K) || !size_ok(N, K) || !size_ok(M, 4 * N) || rows_per_a_scale < 1 ||
        rows_per_b_scale < 1)
        return MXQ_ERR_SIZE;
    if (K % 64 != 0)
        return MXQ_ERR_SHAPE;
    if (K > MAX_GEMM_K || ((M + 255) / 256) * ((N + 255) / 256) > mxq::MAX_GEMM_TILES)
        return MXQ_ERR_SIZE;
    const int esz = out_dtype == MXQ_OUT_F32 ? 4 : 2;
    const Buf bb[7] = {{a, M * K / 2, 16, false},
                       {a_block_scales, M * (K / 16), 4, false},
                       {a_scales, 4 * ((M + rows_per_a_scale - 1) / rows_per_a_scale), 4, false},
                       {b, N * K / 2, 16, false},
                       {b_block_scales, N * (K / 16), 4, false},
                       {b_scales, 4 * ((N + rows_per_b_scale - 1) / rows_per_b_scale), 4, false},
                       {c, esz * M * N, esz, true}};
    const int st = check_bufs(bb, 7);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_nvfp4_gemm(a, a_block_scales, a_scales, rows_per_a_scale, b,
                                           b_block_scales, b_scales, rows_per_b_scale, M, N, K,
                                           out_dtype == MXQ_OUT_BF16, c, (hipStream_t)stream));
}

int mxq_grouped_quantize(int fmt, const uint16_t *x, int64_t total_rows, int64_t cols,
                         const int64_t *seg_offsets, int64_t n_groups, const mxq_grouped_out *out,
                         void *stream)
{
    if (fmt != MXQ_FMT_MXFP8_ROWCOL && fmt != MXQ_FMT_NVFP4)
        return MXQ_ERR_ARG;
    if (!x || !seg_offsets || !out)
        return MXQ_ERR_NULL;
    if (!size_ok(total_rows, cols) || n_groups < 1 || n_groups > MAX_ELEMS / 8)
        return MXQ_ERR_SIZE;
    const int64_t n = total_rows * cols;
    if (fmt == MXQ_FMT_NVFP4) {
        if (!out->codes || !out->block_scales || !out->token_scales)
            return MXQ_ERR_NULL;
        if (total_rows > MAX_GRID_ROWS)
            return MXQ_ERR_SIZE;
        if (cols % 16 != 0)
            return MXQ_ERR_SHAPE;
        const Buf b[5] = {{x, 2 * n, 16, false},
                          {seg_offsets, 8 * (n_groups + 1), 8, false},
                          {out->codes, n / 2, 16, true},
                          {out->block_scales, n / 16, 1, true},
                          {out->token_scales, 4 * total_rows, 4, true}};
        const int st = check_bufs(b, 5);
        if (st != MXQ_OK)
            return st;
        // Per-token outputs do not depend on the segments.
        return launched(mxq::launch_nvfp4_per_token(x, total_rows, cols, out->codes,
                                                    out->block_scales, out->token_scales,
                                                    (hipStream_t)stream));
    }
    uint8_t *rc = out->row_codes, *rs = out->row_scales, *cc = out->col_codes,
            *cs = out->col_scales;
    int64_t *P = out->col_scale_offsets;
    if ((rc == nullptr) != (rs == nullptr) || (cc == nullptr) != (cs == nullptr) ||
        (cc != nullptr) != (P != nullptr) || (!rc && !cc))
        return MXQ_ERR_OFFSETS;
    if (cols % 32 != 0)
        return MXQ_ERR_SHAPE;
    if (cols > MAX_MXFP8_COLS)
        return MXQ_ERR_SIZE;
    const int64_t scale_rows = total_rows / 32 + n_groups;
    if (scale_rows > MAX_ELEMS / cols ||
        !mxfp8_grid_ok(cc ? scale_rows : (total_rows + 31) / 32, cols))
        return MXQ_ERR_SIZE;
    Buf b[7];
    int k = 0;
    b[k++] = {x, 2 * n, 16, false};
    b[k++] = {seg_offsets, 8 * (n_groups + 1), 8, false};
    if (rc) {
        b[k++] = {rc, n, 16, true};
        b[k++] = {rs, n / 32, 1, true};
    }
    if (cc) {
        b[k++] = {cc, n, 16, true};
        b[k++] = {cs, scale_rows * cols, 8, true};
        b[k++] = {P, 8 * (n_groups + 1), 8, true};
    }
    const int st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    if (!cc) {
        // Rowwise only: identical to the dense call over all rows.
        return launched(mxq::launch_mxfp8_dense(x, total_rows, cols, rc, rs, nullptr, nullptr,
                                                nullptr, 0, (hipStream_t)stream));
    }
    return launched(mxq::launch_mxfp8_grouped(x, total_rows, cols, seg_offsets, n_groups, rc, rs,
                                              cc, cs, P, nullptr, 0, (hipStream_t)stream));
}

int mxq_grouped_quantize_dispatch(int fmt, const uint16_t *x, int64_t n_tokens, int64_t cols,
                                  int64_t top_k, const int64_t *token_rows,
                                  const int64_t *row_tokens, int64_t total_rows,
                                  const int64_t *seg_offsets, int64_t n_groups,
                                  const mxq_grouped_out *out, void *stream)
{
    if (fmt != MXQ_FMT_MXFP8_ROWCOL && fmt != MXQ_FMT_NVFP4)
        return MXQ_ERR_ARG;
    if (!x || !out)
        return MXQ_ERR_NULL;
    if (!size_ok(n_tokens, cols) || !size_ok(total_rows, cols))
        return MXQ_ERR_SIZE;
    const int64_t nx = n_tokens * cols, n = total_rows * cols;
    if (fmt == MXQ_FMT_NVFP4) {
        if (!token_rows || !out->codes || !out->block_scales || !out->token_scales)
            return MXQ_ERR_NULL;
        if (top_k < 1 || !size_ok(n_tokens, top_k) || n_tokens > MAX_GRID_ROWS)
            return MXQ_ERR_SIZE;
        if (cols % 16 != 0)
            return MXQ_ERR_SHAPE;
        const Buf b[5] = {{x, 2 * nx, 16, false},
                          {token_rows, 8 * n_tokens * top_k, 8, false},
                          {out->codes, n / 2, 16, true},
                          {out->block_scales, n / 16, 1, true},
                          {out->token_scales, 4 * total_rows, 4, true}};
        const int st = check_bufs(b, 5);
        if (st != MXQ_OK)
            return st;
        return launched(mxq::launch_nvfp4_dispatch(x, n_tokens, cols, token_rows, top_k,
                                                   total_rows, out->codes, out->block_scales,
                                                   out->token_scales, (hipStream_t)stream));
    }
    if (!row_tokens)
        return MXQ_ERR_NULL;
    uint8_t *rc = out->row_codes, *rs = out->row_scales, *cc = out->col_codes,
            *cs = out->col_scales;
    int64_t *P = out->col_scale_offsets;
    if ((rc == nullptr) != (rs == nullptr) || (cc == nullptr) != (cs == nullptr) ||
        (cc != nullptr) != (P != nullptr) || (!rc && !cc))
        return MXQ_ERR_OFFSETS;
    if (cc && !seg_offsets)
        return MXQ_ERR_NULL;
    if (cc && (n_groups < 1 || n_groups > MAX_ELEMS / 8))
        return MXQ_ERR_SIZE;
    if (cols % 32 != 0)
        return MXQ_ERR_SHAPE;
    if (cols > MAX_MXFP8_COLS)
        return MXQ_ERR_SIZE;
    const int64_t scale_rows = total_rows / 32 + (cc ? n_groups : 0);
    if (scale_rows > MAX_ELEMS / cols ||
        !mxfp8_grid_ok(cc ? scale_rows : (total_rows + 31) / 32, cols))
        return MXQ_ERR_SIZE;
    Buf b[8];
    int k = 0;
    b[k++] = {x, 2 * nx, 16, false};
    b[k++] = {row_tokens, 8 * total_rows, 8, false};
    if (rc) {
        b[k++] = {rc, n, 16, true};
        b[k++] = {rs, n / 32, 1, true};
    }
    if (cc) {
        b[k++] = {seg_offsets, 8 * (n_groups + 1), 8, false};
        b[k++] = {cc, n, 16, true};
        b[k++] = {cs, scale_rows * cols, 8, true};
        b[k++] = {P, 8 * (n_groups + 1), 8, true};
    }
    const int st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    if (!cc)
        return launched(mxq::launch_mxfp8_dense(x, total_rows, cols, rc, rs, nullptr, nullptr,
                                                row_tokens, n_tokens, (hipStream_t)stream));
    return launched(mxq::launch_mxfp8_grouped(x, total_rows, cols, seg_offsets, n_groups, rc, rs,
                                              cc, cs, P, row_tokens, n_tokens,
                                              (hipStream_t)stream));
}

int mxq_copy_floor(const void *src, int64_t src_bytes, void *dst, int64_t dst_bytes,
                   void *stream)
{
    if (!src || !dst)
        return MXQ_ERR_NULL;
    if (src_bytes <= 0 || dst_bytes <= 0 || src_bytes > MAX_COPY_FLOOR_BYTES ||
        dst_bytes > MAX_COPY_FLOOR_BYTES)
        return MXQ_ERR_SIZE;
    if (src_bytes % 16 != 0 || dst_bytes % 16 != 0)
        return MXQ_ERR_SHAPE;
    const Buf b[2] = {{src, src_bytes, 16, false}, {dst, dst_bytes, 16, true}};
    const int st = check_bufs(b, 2);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_copy_floor(src, src_bytes, dst, dst_bytes, (hipStream_t)stream));
}

// ---------------------------------------------------------------------------
// Layer operators
// ---------------------------------------------------------------------------

static bool route_sizes_ok(int64_t n_tokens, int64_t n_experts)
{
    return n_tokens > 0 && n_experts > 0 && n_tokens < MAX_LAYER_TOKENS &&
           n_experts <= mxq::MAX_EXPERTS;
}

static bool dtype_ok(int dtype)
{
    return dtype == MXQ_OUT_F32 || dtype == MXQ_OUT_BF16;
}

// By bits, hidden from the compiler as bits of a float: under -fno-honor-nans
// it may otherwise merge the test with a comparison and lose the NaN.
static bool finite_f32(float f)
{
    uint32_t u;
    memcpy(&u, &f, sizeof u);
    __asm__("" : "+r"(u));
    return (u & 0x7F800000u) != 0x7F800000u;
}

int64_t mxq_moe_route_workspace(int64_t n_tokens, int64_t n_experts)
{
    return route_sizes_ok(n_tokens, n_experts) ? mxq::moe_route_workspace(n_tokens, n_experts)
                                               : 0;
}

int mxq_moe_route(int dtype, const void *logits, const float *bias, int64_t n_tokens,
                  int64_t n_experts, const mxq_route_params *params, float *weights,
                  int64_t *experts, int64_t *token_rows, int64_t *row_tokens,
                  int64_t *seg_offsets, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(dtype))
        return MXQ_ERR_ARG;
    if (!logits || !params || !weights || !experts)
        return MXQ_ERR_NULL;
    const mxq_route_params p = *params;
    if ((p.scoring != MXQ_SCORE_SOFTMAX && p.scoring != MXQ_SCORE_SIGMOID) ||
        (p.group_topk != 1 && p.group_topk != 2) || !finite_f32(p.scale))
        return MXQ_ERR_ARG;
    const bool maps = token_rows != nullptr;
    if ((row_tokens != nullptr) != maps || (seg_offsets != nullptr) != maps)
        return MXQ_ERR_OFFSETS;
    if (!route_sizes_ok(n_tokens, n_experts) || p.top_k < 1 || p.top_k > n_experts ||
        p.top_k > mxq::MAX_TOP_K || n_tokens > mxq::MAX_COPIES / p.top_k || p.n_groups < 1 ||
        p.n_groups > 64 || p.topk_groups < 1 || p.topk_groups > p.n_groups)
        return MXQ_ERR_SIZE;
    if (n_experts % p.n_groups != 0)
        return MXQ_ERR_SHAPE;
    const int64_t need = maps ? mxq::moe_route_workspace(n_tokens, n_experts) : 0;
    if (need > 0 && !workspace)
        return MXQ_ERR_NULL;
    if (workspace_bytes < need)
        return MXQ_ERR_SIZE;
    const int esz = dtype == MXQ_OUT_F32 ? 4 : 2;
    const int64_t copies = n_tokens * p.top_k;
    Buf b[8];
    int k = 0;
    b[k++] = {logits, esz * n_tokens * n_experts, esz, false};
    b[k++] = {weights, 4 * copies, 4, true};
    b[k++] = {experts, 8 * copies, 8, true};
    if (bias)
        b[k++] = {bias, 4 * n_experts, 4, false};
    if (maps) {
        b[k++] = {token_rows, 8 * copies, 8, true};
        b[k++] = {row_tokens, 8 * copies, 8, true};
        b[k++] = {seg_offsets, 8 * (n_experts + 1), 8, true};
        b[k++] = {workspace, need, 16, true};
    }
    const int st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_moe_route(dtype == MXQ_OUT_BF16, logits, bias, n_tokens,
                                          n_experts, p, weights, experts, token_rows, row_tokens,
                                          seg_offsets, workspace, (hipStream_t)stream));
}

int mxq_moe_route_backward(int dtype, const float *d_weights, const void *logits,
                           const int64_t *experts, int64_t n_tokens, int64_t n_experts,
                           int64_t top_k, int scoring, int renormalize, float scale,
                           void *d_logits, void *stream)
{
    if (!dtype_ok(dtype) || (scoring != MXQ_SCORE_SOFTMAX && scoring != MXQ_SCORE_SIGMOID) ||
        !finite_f32(scale))
        return MXQ_ERR_ARG;
    if (!d_weights || !logits || !experts || !d_logits)
        return MXQ_ERR_NULL;
    if (!route_sizes_ok(n_tokens, n_experts) || top_k < 1 || top_k > mxq::MAX_TOP_K ||
        n_tokens > mxq::MAX_COPIES / top_k)
        return MXQ_ERR_SIZE;
    const int esz = dtype == MXQ_OUT_F32 ? 4 : 2;
    const Buf b[4] = {{d_weights, 4 * n_tokens * top_k, 4, false},
                      {logits, esz * n_tokens * n_experts, esz, false},
                      {experts, 8 * n_tokens * top_k, 8, false},
                      {d_logits, esz * n_tokens * n_experts, esz, true}};
    const int st = check_bufs(b, 4);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_moe_route_backward(
        dtype == MXQ_OUT_BF16, d_weights, logits, experts, n_tokens, n_experts, top_k,
        scoring == MXQ_SCORE_SIGMOID, renormalize != 0, scale, d_logits, (hipStream_t)stream));
}

static int combine_sizes(int64_t total_rows, int64_t n_tokens, int64_t top_k, int64_t cols)
{
    if (!size_ok(total_rows, 4 * cols) || cols > MAX_ELEMS / 4 || n_tokens < 1 ||
        n_tokens >= MAX_LAYER_TOKENS || top_k < 1 || top_k > mxq::MAX_TOP_K ||
        !size_ok(n_tokens, 4 * cols))
        return MXQ_ERR_SIZE;
    return cols % 8 != 0 ? MXQ_ERR_SHAPE : MXQ_OK;
}

int mxq_moe_combine(int dtype, const void *rows, int64_t total_rows, const int64_t *token_rows,
                    const float *weights, int64_t n_tokens, int64_t top_k, int64_t cols,
                    int out_dtype, void *out, void *stream)
{
    if (!dtype_ok(dtype) || !dtype_ok(out_dtype))
        return MXQ_ERR_ARG;
    if (!rows || !token_rows || !weights || !out)
        return MXQ_ERR_NULL;
    int st = combine_sizes(total_rows, n_tokens, top_k, cols);
    if (st != MXQ_OK)
        return st;
    const int esz = dtype == MXQ_OUT_F32 ? 4 : 2;
    const Buf b[4] = {{rows, esz * total_rows * cols, 16, false},
                      {token_rows, 8 * n_tokens * top_k, 8, false},
                      {weights, 4 * n_tokens * top_k, 4, false},
                      {out, (out_dtype == MXQ_OUT_F32 ? 4 : 2) * n_tokens * cols, 16, true}};
    st = check_bufs(b, 4);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_moe_combine(dtype == MXQ_OUT_BF16, rows, total_rows, token_rows,
                                            weights, n_tokens, top_k, cols,
                                            out_dtype == MXQ_OUT_BF16, out,
                                            (hipStream_t)stream));
}

int mxq_moe_combine_backward(int dtype, const void *d_out, const void *rows, int64_t total_rows,
                             const int64_t *token_rows, const float *weights,
                             const int64_t *seg_offsets, int64_t n_groups, int64_t n_tokens,
                             int64_t top_k, int64_t cols, void *d_rows, float *d_weights,
                             void *stream)
{
    if (!dtype_ok(dtype))
        return MXQ_ERR_ARG;
    if (!d_out || !rows || !token_rows || !weights || !d_rows || !d_weights)
        return MXQ_ERR_NULL;
    if (seg_offsets && (n_groups < 1 || n_groups > MAX_ELEMS / 8 - 1))
        return MXQ_ERR_SIZE;
    int st = combine_sizes(total_rows, n_tokens, top_k, cols);
    if (st != MXQ_OK)
        return st;
    const int esz = dtype == MXQ_OUT_F32 ? 4 : 2;
    Buf b[7];
    int k = 0;
    b[k++] = {d_out, esz * n_tokens * cols, 16, false};
    b[k++] = {rows, esz * total_rows * cols, 16, false};
    b[k++] = {token_rows, 8 * n_tokens * top_k, 8, false};
    b[k++] = {weights, 4 * n_tokens * top_k, 4, false};
    b[k++] = {d_rows, esz * total_rows * cols, 16, true};
    b[k++] = {d_weights, 4 * n_tokens * top_k, 4, true};
    if (seg_offsets)
        b[k++] = {seg_offsets, 8 * (n_groups + 1), 8, false};
    st = check_bufs(b, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_moe_combine_backward(
        dtype == MXQ_OUT_BF16, d_out, rows, total_rows, token_rows, weights, seg_offsets,
        n_groups, n_tokens, top_k, cols, d_rows, d_weights, (hipStream_t)stream));
}

// The activation operand of the few-row products: format, pointers, then
// (after the sizes) its buffers appended to b.
static int act_args(int x_fmt, const void *x, const uint8_t *xbs, const float *xs)
{
    if (x_fmt != MXQ_X_BF16 && x_fmt != MXQ_X_F32 && x_fmt != MXQ_X_NVFP4)
        return MXQ_ERR_ARG;
    if (!x || (x_fmt == MXQ_X_NVFP4 && (!xbs || !xs)))
        return MXQ_ERR_NULL;
    if (x_fmt != MXQ_X_NVFP4 && (xbs || xs))
        return MXQ_ERR_OFFSETS;
    return MXQ_OK;
}
static int act_bufs(Buf *b, const mxq::ActX &x, int64_t rows, int64_t K)
{
    if (x.fmt == MXQ_X_NVFP4) {
        b[0] = {x.x, rows * (K / 2), 16, false};
        b[1] = {x.bs, rows * (K / 16), 4, false};
        b[2] = {x.s, 4 * rows, 4, false};
        return 3;
    }
    b[0] = {x.x, rows * K * (x.fmt == MXQ_X_F32 ? 4 : 2), 16, false};
    return 1;
}

int mxq_nvfp4_matvec(int x_fmt, const void *x, const uint8_t *x_block_scales,
                     const float *x_scales, const uint8_t *b, const uint8_t *b_block_scales,
                     const float *b_scales, int64_t rows_per_b_scale, int64_t M, int64_t N,
                     int64_t K, int out_dtype, void *c, void *stream)
{
    if (!dtype_ok(out_dtype))
        return MXQ_ERR_ARG;
    int st = act_args(x_fmt, x, x_block_scales, x_scales);
    if (st != MXQ_OK)
        return st;
    if (!b || !b_block_scales || !b_scales || !c)
        return MXQ_ERR_NULL;
    if (M < 1 || M > MAX_MATVEC_ROWS || N < 1 || N > MAX_MATVEC_N || K < 1 || K > MAX_MATVEC_K ||
        rows_per_b_scale < 1)
        return MXQ_ERR_SIZE;
    if (K % 64 != 0)
        return MXQ_ERR_SHAPE;
    const mxq::ActX ax{x_fmt, x, x_block_scales, x_scales};
    const int esz = out_dtype == MXQ_OUT_F32 ? 4 : 2;
    Buf bb[7];
    int k = act_bufs(bb, ax, M, K);
    bb[k++] = {b, N * (K / 2), 16, false};
    bb[k++] = {b_block_scales, N * (K / 16), 4, false};
    bb[k++] = {b_scales, 4 * ((N - 1) / rows_per_b_scale + 1), 4, false};
    bb[k++] = {c, esz * M * N, esz, true};
    st = check_bufs(bb, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_nvfp4_matvec(ax, mxq::WeightB{b, b_block_scales}, b_scales,
                                             rows_per_b_scale, M, N, K,
                                             out_dtype == MXQ_OUT_BF16, c, (hipStream_t)stream));
}

static bool expert_sizes_ok(int64_t n_groups, int64_t total_rows, int64_t N, int64_t K)
{
    return n_groups >= 1 && n_groups <= MAX_MATVEC_GROUPS && total_rows >= 1 &&
           total_rows <= mxq::MAX_COPIES && N >= 1 && N <= MAX_MATVEC_N && K >= 1 &&
           K <= MAX_MATVEC_K && mxq::expert_grid_ok(n_groups, total_rows, N);
}

int mxq_nvfp4_expert_matvec(int x_fmt, const void *x, const uint8_t *x_block_scales,
                            const float *x_scales, const uint8_t *b,
                            const uint8_t *b_block_scales, const float *b_scales,
                            const int64_t *seg_offsets, int64_t n_groups, int64_t total_rows,
                            int64_t N, int64_t K, int out_dtype, void *c, void *stream)
{
    if (!dtype_ok(out_dtype))
        return MXQ_ERR_ARG;
    int st = act_args(x_fmt, x, x_block_scales, x_scales);
    if (st != MXQ_OK)
        return st;
    if (!b || !b_block_scales || !b_scales || !seg_offsets || !c)
        return MXQ_ERR_NULL;
    if (!expert_sizes_ok(n_groups, total_rows, N, K))
        return MXQ_ERR_SIZE;
    if (K % 64 != 0)
        return MXQ_ERR_SHAPE;
    const mxq::ActX ax{x_fmt, x, x_block_scales, x_scales};
    const int esz = out_dtype == MXQ_OUT_F32 ? 4 : 2;
    Buf bb[8];
    int k = act_bufs(bb, ax, total_rows, K);
    bb[k++] = {b, n_groups * N * (K / 2), 16, false};
    bb[k++] = {b_block_scales, n_groups * N * (K / 16), 4, false};
    bb[k++] = {b_scales, 4 * n_groups, 4, false};
    bb[k++] = {seg_offsets, 8 * (n_groups + 1), 8, false};
    bb[k++] = {c, esz * total_rows * N, esz, true};
    st = check_bufs(bb, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_nvfp4_expert_matvec(
        ax, total_rows, nullptr, seg_offsets, n_groups, total_rows,
        mxq::WeightB{b, b_block_scales}, mxq::WeightB{nullptr, nullptr}, b_scales, N, K,
        out_dtype == MXQ_OUT_BF16, c, (hipStream_t)stream));
}

int mxq_nvfp4_expert_gateup(int x_fmt, const void *x, const uint8_t *x_block_scales,
                            const float *x_scales, int64_t n_tokens, const int64_t *row_tokens,
                            const int64_t *seg_offsets, int64_t n_groups, int64_t total_rows,
                            const uint8_t *gate, const uint8_t *gate_block_scales,
                            const uint8_t *up, const uint8_t *up_block_scales,
                            const float *scope_scales, int64_t N, int64_t K, int out_dtype,
                            void *h, void *stream)
{
    if (!dtype_ok(out_dtype))
        return MXQ_ERR_ARG;
    int st = act_args(x_fmt, x, x_block_scales, x_scales);
    if (st != MXQ_OK)
        return st;
    if (!row_tokens || !seg_offsets || !gate || !gate_block_scales || !up || !up_block_scales ||
        !scope_scales || !h)
        return MXQ_ERR_NULL;
    if (n_tokens < 1 || n_tokens > mxq::MAX_COPIES ||
        !expert_sizes_ok(n_groups, total_rows, N, K))
        return MXQ_ERR_SIZE;
    if (K % 64 != 0)
        return MXQ_ERR_SHAPE;
    const mxq::ActX ax{x_fmt, x, x_block_scales, x_scales};
    const int esz = out_dtype == MXQ_OUT_F32 ? 4 : 2;
    Buf bb[11];
    int k = act_bufs(bb, ax, n_tokens, K);
    bb[k++] = {row_tokens, 8 * total_rows, 8, false};
    bb[k++] = {seg_offsets, 8 * (n_groups + 1), 8, false};
    bb[k++] = {gate, n_groups * N * (K / 2), 16, false};
    bb[k++] = {gate_block_scales, n_groups * N * (K / 16), 4, false};
    bb[k++] = {up, n_groups * N * (K / 2), 16, false};
    bb[k++] = {up_block_scales, n_groups * N * (K / 16), 4, false};
    bb[k++] = {scope_scales, 4 * n_groups, 4, false};
    bb[k++] = {h, esz * total_rows * N, esz, true};
    st = check_bufs(bb, k);
    if (st != MXQ_OK)
        return st;
    return launched(mxq::launch_nvfp4_expert_matvec(
        ax, n_tokens, row_tokens, seg_offsets, n_groups, total_rows,
        mxq::WeightB{gate, gate_block_scales}, mxq::WeightB{up, up_block_scales}, scope_scales,
        N, K, out_dtype == MXQ_OUT_BF16, h, (hipStream_t)stream));
}

// Status of the attention's sizes (without the pages, which only the call has).
static int attention_sizes(int64_t n_seqs, int64_t q_len, int64_t n_heads, int64_t n_kv_heads,
                           int64_t head_dim, int64_t max_keys)
{
    if (n_seqs < 1 || q_len < 1 || n_heads < 1 || n_kv_heads < 1 || max_keys < 1 ||
        n_seqs > MAX_ATTN_ROWS || q_len > MAX_ATTN_ROWS || n_heads > MAX_ATTN_ROWS ||
        n_seqs * q_len > MAX_ATTN_ROWS || n_seqs * q_len * n_heads > MAX_ATTN_ROWS ||
        max_keys > MAX_ATTN_KEYS)
        return MXQ_ERR_SIZE;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || n_heads % n_kv_heads != 0)
        return MXQ_ERR_SHAPE;
    return MXQ_OK;
}

int64_t mxq_nvfp4_attention_workspace(int64_t n_seqs, int64_t q_len, int64_t n_heads,
                                      int64_t n_kv_heads, int64_t head_dim, int64_t max_keys)
{
    if (attention_sizes(n_seqs, q_len, n_heads, n_kv_heads, head_dim, max_keys) != MXQ_OK)
        return 0;
    return mxq::nvfp4_attention_workspace(n_seqs, q_len, n_heads, n_kv_heads, head_dim, max_keys);
}

int mxq_nvfp4_attention(const uint16_t *q, const mxq_nvfp4_cache *k, const mxq_nvfp4_cache *v,
                        const int64_t *block_table, const int64_t *seq_lens, int64_t n_seqs,
                        int64_t q_len, int64_t n_heads, int64_t n_kv_heads, int64_t head_dim,
                        int64_t n_pages, int64_t page_size, int64_t max_pages,
                        float softmax_scale, int causal, int64_t window, uint16_t *out,
                        float *lse, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!q || !k || !v || !block_table || !seq_lens || !out || !k->codes || !k->block_scales ||
        !k->scales || !v->codes || !v->block_scales || !v->scales)
        return MXQ_ERR_NULL;
    if (!finite_f32(softmax_scale))
        return MXQ_ERR_ARG;
    if (softmax_scale <= 0.0f || window < 0 || (!causal && window != 0))
        return MXQ_ERR_ARG;
    if (n_pages < 1 || page_size < 1 || max_pages < 1 || n_kv_heads < 1 ||
        page_size > MAX_ATTN_KEYS || max_pages > MAX_ATTN_KEYS / page_size ||
        n_kv_heads > MAX_ATTN_ROWS || n_pages > MAX_CACHE_ROWS / page_size / n_kv_heads)
        return MXQ_ERR_SIZE;
    const int sz = attention_sizes(n_seqs, q_len, n_heads, n_kv_heads, head_dim,
                                   max_pages * page_size);
    if (sz != MXQ_OK)
        return sz;
    if (page_size % 16 != 0)
        return MXQ_ERR_SHAPE;
    const int64_t need = mxq::nvfp4_attention_workspace(n_seqs, q_len, n_heads, n_kv_heads,
                                                        head_dim, max_pages * page_size);
    if (need > 0 && !workspace)
        return MXQ_ERR_NULL;
    if (workspace_bytes < need)
        return MXQ_ERR_SIZE;
    const int64_t rows = n_pages * n_kv_heads * page_size, nq = n_seqs * q_len * n_heads;
    Buf b[13];
    int i = 0;
    b[i++] = {q, 2 * nq * head_dim, 16, false};
    for (const mxq_nvfp4_cache *c : {k, v}) {
        b[i++] = {c->codes, rows * (head_dim / 2), 16, false};
        b[i++] = {c->block_scales, rows * (head_dim / 16), 8, false};
        b[i++] = {c->scales, 4 * rows, 16, false};
    }
    b[i++] = {block_table, 8 * n_seqs * max_pages, 8, false};
    b[i++] = {seq_lens, 8 * n_seqs, 8, false};
    b[i++] = {out, 2 * nq * head_dim, 16, true};
    if (lse)
        b[i++] = {lse, 4 * nq, 4, true};
    if (need > 0)
        b[i++] = {workspace, need, 16, true};
    const int st = check_bufs(b, i);
    if (st != MXQ_OK)
        return st;
    const mxq::AttnArgs a{q, k->codes, k->block_scales, k->scales, v->codes, v->block_scales,
                          v->scales, block_table, seq_lens, n_seqs, q_len, n_heads, n_kv_heads,
                          head_dim, n_pages, page_size, max_pages, softmax_scale, causal != 0,
                          window, out, lse};
    return launched(mxq::launch_nvfp4_attention(a, workspace, (hipStream_t)stream));
}

}  // extern "C"
