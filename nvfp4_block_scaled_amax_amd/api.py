"""Tensor-level helpers over the C ABI: allocate outputs with torch.empty on
the input's device and call the library.  BF16 inputs may be torch.bfloat16 or
int16/uint16 tensors of bit patterns; they must be contiguous HIP tensors.

`stream` (by default the current one) is where a call's kernels run.  Its
outputs are memory of the current stream, as any tensor made there, so a caller
that names another stream orders the two and keeps inputs and outputs until
the kernels have run; what a call holds besides belongs to `stream` itself."""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional

import torch

from . import _binding as B


def _bf16_bits(x: torch.Tensor) -> torch.Tensor:
    if x.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        if not x.is_contiguous():
            raise ValueError("input must be contiguous")
        return x
    raise TypeError(f"expected a BF16 tensor (or its int16 bits), got {x.dtype}")


def _empty(shape, dtype, like):
    return like.new_empty(shape, dtype=dtype)


class MXFP8RowCol(NamedTuple):
    row_codes: Optional[torch.Tensor]
    row_scales: Optional[torch.Tensor]
    col_codes: Optional[torch.Tensor]
    col_scales: Optional[torch.Tensor]


def mxfp8_quantize_rowcol(x, rowwise: bool = True, colwise: bool = True,
                          stream=None) -> MXFP8RowCol:
    x = _bf16_bits(x)
    rows, cols = x.shape
    u8 = torch.uint8
    rc = _empty((rows, cols), u8, x) if rowwise else None
    rs = _empty((rows, cols // 32), u8, x) if rowwise else None
    cc = _empty((rows, cols), u8, x) if colwise else None
    cs = _empty((rows // 32, cols), u8, x) if colwise else None
    B.mxq_mxfp8_quantize_rowcol(x, rows, cols, rc, rs, cc, cs, stream)
    return MXFP8RowCol(rc, rs, cc, cs)


def mxfp8_quantize_rowcol_t(x, rowwise: bool = True, stream=None) -> MXFP8RowCol:
    """Both MXFP8 copies, the columnwise one transposed: col_codes [cols][rows],
    col_scales [cols][rows/32] (K-contiguous for a GEMM contracting over rows)."""
    x = _bf16_bits(x)
    rows, cols = x.shape
    u8 = torch.uint8
    rc = _empty((rows, cols), u8, x) if rowwise else None
    rs = _empty((rows, cols // 32), u8, x) if rowwise else None
    cc = _empty((cols, rows), u8, x)
    cs = _empty((cols, rows // 32), u8, x)
    B.mxq_mxfp8_quantize_rowcol_t(x, rows, cols, rc, rs, cc, cs, stream)
    return MXFP8RowCol(rc, rs, cc, cs)


def mxfp8_quantize_ocp_floor(x, rowwise: bool = True, colwise: bool = True,
                             stream=None) -> MXFP8RowCol:
    """Comparison variant: both MXFP8 copies under the OCP MX scale rule
    (floor(log2 amax) - 8, saturating at 448), which clips."""
    x = _bf16_bits(x)
    rows, cols = x.shape
    u8 = torch.uint8
    rc = _empty((rows, cols), u8, x) if rowwise else None
    rs = _empty((rows, cols // 32), u8, x) if rowwise else None
    cc = _empty((rows, cols), u8, x) if colwise else None
    cs = _empty((rows // 32, cols), u8, x) if colwise else None
    B.mxq_mxfp8_quantize_ocp_floor(x, rows, cols, rc, rs, cc, cs, stream)
    return MXFP8RowCol(rc, rs, cc, cs)


class NVFP4(NamedTuple):
    codes: torch.Tensor
    block_scales: torch.Tensor
    fp32_scales: torch.Tensor


def nvfp4_quantize_per_token(x, stream=None) -> NVFP4:
    x = _bf16_bits(x)
    rows, cols = x.shape
    codes = _empty((rows, cols // 2), torch.uint8, x)
    bs = _empty((rows, cols // 16), torch.uint8, x)
    ts = _empty((rows,), torch.float32, x)
    B.mxq_nvfp4_quantize_per_token(x, rows, cols, codes, bs, ts, stream)
    return NVFP4(codes, bs, ts)


def nvfp4_quantize_per_token_approx(x, stream=None) -> NVFP4:
    """Opt-in approximate per-token NVFP4 (not the contract): one
    reciprocal-multiply and one conversion per block scale and per code."""
    x = _bf16_bits(x)
    rows, cols = x.shape
    codes = _empty((rows, cols // 2), torch.uint8, x)
    bs = _empty((rows, cols // 16), torch.uint8, x)
    ts = _empty((rows,), torch.float32, x)
    B.mxq_nvfp4_quantize_per_token_approx(x, rows, cols, codes, bs, ts, stream)
    return NVFP4(codes, bs, ts)


def nvfp4_quantize_per_tensor(x, stream=None) -> NVFP4:
    """Comparison variant: NVFP4 of an activation tensor with ONE FP32 scale
    for the whole tensor (the batch-dependent scope the per-token recipe
    replaces); the weight-export call with a single one-tensor scope."""
    x = _bf16_bits(x)
    rows, cols = x.shape
    codes = _empty((1, rows, cols // 2), torch.uint8, x)
    bs = _empty((1, rows, cols // 16), torch.uint8, x)
    s = _empty((1,), torch.float32, x)
    B.mxq_nvfp4_quantize_gateup_pair(x, None, 1, rows, cols, codes, bs, None, None, s, stream)
    return NVFP4(codes[0], bs[0], s)


class GateUpNVFP4(NamedTuple):
    gate_codes: torch.Tensor
    gate_block_scales: torch.Tensor
    up_codes: Optional[torch.Tensor]
    up_block_scales: Optional[torch.Tensor]
    scope_scales: torch.Tensor


def nvfp4_quantize_gateup_pair(gate, up=None, stream=None) -> GateUpNVFP4:
    gate = _bf16_bits(gate)
    E, rows, cols = gate.shape
    gc = _empty((E, rows, cols // 2), torch.uint8, gate)
    gb = _empty((E, rows, cols // 16), torch.uint8, gate)
    uc = ub = None
    if up is not None:
        up = _bf16_bits(up)
        if up.shape != gate.shape:
            raise ValueError("gate and up must have the same shape")
        uc = torch.empty_like(gc)
        ub = torch.empty_like(gb)
    sc = _empty((E,), torch.float32, gate)
    B.mxq_nvfp4_quantize_gateup_pair(gate, up, E, rows, cols, gc, gb, uc, ub, sc, stream)
    return GateUpNVFP4(gc, gb, uc, ub, sc)


def nvfp4_quantize_gateup_pair_amax(gate, up, scope_amax, stream=None) -> GateUpNVFP4:
    """The export with each scope's amax supplied: scope_amax is a device
    tensor of n_experts BF16 values (torch.bfloat16 or int16 bits)."""
    gate = _bf16_bits(gate)
    E, rows, cols = gate.shape
    amax = _bf16_bits(scope_amax)
    if amax.numel() != E:
        raise ValueError("scope_amax must hold one value per expert")
    gc = _empty((E, rows, cols // 2), torch.uint8, gate)
    gb = _empty((E, rows, cols // 16), torch.uint8, gate)
    uc = ub = None
    if up is not None:
        up = _bf16_bits(up)
        if up.shape != gate.shape:
            raise ValueError("gate and up must have the same shape")
        uc = torch.empty_like(gc)
        ub = torch.empty_like(gb)
    sc = _empty((E,), torch.float32, gate)
    B.mxq_nvfp4_quantize_gateup_pair_amax(gate, up, amax, E, rows, cols, gc, gb, uc, ub, sc,
                                          stream)
    return GateUpNVFP4(gc, gb, uc, ub, sc)


def dequantize_bf16(fmt: int, codes, scales, fp32_scales=None, rows_per_fp32_scale: int = 1,
                    stream=None) -> torch.Tensor:
    """Returns a torch.bfloat16 tensor [rows][cols]."""
    rows = codes.shape[0] if codes.dim() == 2 else codes.shape[0] * codes.shape[1]
    last = codes.shape[-1]
    cols = 2 * last if fmt == B.MXQ_FMT_NVFP4 else last
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device=codes.device)
    B.mxq_dequantize_bf16(fmt, codes, scales, fp32_scales, rows_per_fp32_scale, rows, cols, out,
                          stream)
    return out


class QuantDequant(NamedTuple):
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    fp32_scales: Optional[torch.Tensor]     # NVFP4 only
    dequant: torch.Tensor                    # torch.bfloat16 [rows][cols]


def quantize_dequant_bf16(fmt: int, x, keep_codes: bool = True, stream=None) -> QuantDequant:
    """Rowwise MXFP8 (fmt MXQ_FMT_MXFP8_ROW) or per-token NVFP4 and the BF16
    dequantization of the result, in one pass; keep_codes=False stores only
    the dequantized copy."""
    x = _bf16_bits(x)
    rows, cols = x.shape
    u8 = torch.uint8
    codes = scales = ts = None
    if fmt == B.MXQ_FMT_NVFP4:
        if keep_codes:
            codes, scales = _empty((rows, cols // 2), u8, x), _empty((rows, cols // 16), u8, x)
            ts = _empty((rows,), torch.float32, x)
    elif keep_codes:
        codes, scales = _empty((rows, cols), u8, x), _empty((rows, cols // 32), u8, x)
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device=x.device)
    B.mxq_quantize_dequant_bf16(fmt, x, rows, cols, codes, scales, ts, out, stream)
    return QuantDequant(codes, scales, ts, out)


def mxfp8_gemm(a_codes, a_scales, b_codes, b_scales, out_dtype=torch.bfloat16,
               stream=None) -> torch.Tensor:
    """C = A x B^T on MXFP8 operands (rowwise copies: a [M][K], b [N][K] with
    [.][K/32] E8M0 scales); returns C [M][N] as fp32 or BF16."""
    M, K = a_codes.shape
    N = b_codes.shape[0]
    c = torch.empty((M, N), dtype=out_dtype, device=a_codes.device)
    code = B.MXQ_OUT_BF16 if out_dtype == torch.bfloat16 else B.MXQ_OUT_F32
    B.mxq_mxfp8_gemm(a_codes, a_scales, b_codes, b_scales, M, N, K, code, c, stream)
    return c


def mxfp8_grouped_gemm(a_codes, a_scales, b_codes, b_scales, seg_offsets,
                       out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """Per-expert C[r] = A[r] x B_e^T for the rows r of each segment e of
    seg_offsets (device int64 [G+1]): a [R][K] and a_scales [R][K/32] are the
    expert-sorted rowwise MXFP8 copy, b [G][N][K] and b_scales [G][N][K/32]
    the experts' weights; returns C [R][N] as fp32 or BF16 (rows outside
    every segment left unwritten)."""
    R, K = a_codes.shape
    G, N = b_codes.shape[0], b_codes.shape[1]
    c = torch.empty((R, N), dtype=out_dtype, device=a_codes.device)
    code = B.MXQ_OUT_BF16 if out_dtype == torch.bfloat16 else B.MXQ_OUT_F32
    B.mxq_mxfp8_grouped_gemm(a_codes, a_scales, b_codes, b_scales, seg_offsets, G, R, N, K, code,
                             c, stream)
    return c


class GroupedColT(NamedTuple):
    codes_t: torch.Tensor         # [cols][pitch]
    scales_t: torch.Tensor        # [cols][pitch / 32]
    block_offsets: torch.Tensor   # [G + 1] int64: segment e's first 32-row block


def grouped_colt_pitch(total_rows: int, n_groups: int) -> int:
    """Row pitch of the grouped transposed columnwise copy."""
    return -(-total_rows // 128) * 128 + 128 * n_groups


def mxfp8_grouped_colwise_t(x, seg_offsets, stream=None) -> GroupedColT:
    """The grouped columnwise MXFP8 copy of the expert-sorted rows x [R][cols],
    transposed with every segment padded to 128 rows (the weight-gradient
    operand layout)."""
    x = _bf16_bits(x)
    R, cols = x.shape
    G = seg_offsets.numel() - 1
    pitch = grouped_colt_pitch(R, G)
    out = GroupedColT(_empty((cols, pitch), torch.uint8, x),
                      _empty((cols, pitch // 32), torch.uint8, x),
                      _empty((G + 1,), torch.int64, x))
    B.mxq_mxfp8_grouped_colwise_t(x, R, cols, seg_offsets, G, out.codes_t, out.scales_t,
                                  out.block_offsets, stream)
    return out


def mxfp8_grouped_quantize_rowcol_t(x, seg_offsets, stream=None):
    """From one read of the expert-sorted rows x [R][cols]: the rowwise MXFP8
    copy (codes [R][cols], scales [R][cols/32], as the grouped quantize writes
    it) and the grouped transposed padded columnwise copy.  Returns
    (row_codes, row_scales, GroupedColT)."""
    x = _bf16_bits(x)
    R, cols = x.shape
    G = seg_offsets.numel() - 1
    pitch = grouped_colt_pitch(R, G)
    rc = _empty((R, cols), torch.uint8, x)
    rs = _empty((R, cols // 32), torch.uint8, x)
    out = GroupedColT(_empty((cols, pitch), torch.uint8, x),
                      _empty((cols, pitch // 32), torch.uint8, x),
                      _empty((G + 1,), torch.int64, x))
    B.mxq_mxfp8_grouped_quantize_rowcol_t(x, R, cols, seg_offsets, G, rc, rs, out.codes_t,
                                          out.scales_t, out.block_offsets, stream)
    return rc, rs, out


def mxfp8_grouped_wgrad(a: GroupedColT, b: GroupedColT, out_dtype=torch.float32,
                        stream=None) -> torch.Tensor:
    """Per-expert C_e = A_e x B_e^T contracting over each segment's rows, from
    two grouped transposed copies over the same segments (a from dY, b from
    X: C_e = dW_e); returns C [G][M][N]."""
    M, pitch = a.codes_t.shape
    N = b.codes_t.shape[0]
    G = a.block_offsets.numel() - 1
    c = torch.empty((G, M, N), dtype=out_dtype, device=a.codes_t.device)
    code = B.MXQ_OUT_BF16 if out_dtype == torch.bfloat16 else B.MXQ_OUT_F32
    B.mxq_mxfp8_grouped_wgrad(a.codes_t, a.scales_t, b.codes_t, b.scales_t, a.block_offsets, G,
                              M, N, pitch, code, c, stream)
    return c


def nvfp4_grouped_gemm(a_codes, a_block_scales, a_scales, b_codes, b_block_scales, b_scales,
                       seg_offsets, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """Per-expert C[r] = a_scales[r] b_scales[e] A[r] x B_e^T for the rows r of
    each segment e of seg_offsets (device int64 [G+1]): a [R][K/2] codes,
    [R][K/16] block scales and [R] FP32 scales (the grouped per-token NVFP4
    copy); b [G][N][K/2], [G][N][K/16] and [G] FP32 scope scales (the
    experts' exported weights); returns C [R][N] as fp32 or BF16."""
    R, K = a_codes.shape[0], 2 * a_codes.shape[1]
    G, N = b_codes.shape[0], b_codes.shape[1]
    c = torch.empty((R, N), dtype=out_dtype, device=a_codes.device)
    code = B.MXQ_OUT_BF16 if out_dtype == torch.bfloat16 else B.MXQ_OUT_F32
    B.mxq_nvfp4_grouped_gemm(a_codes, a_block_scales, a_scales, b_codes, b_block_scales, b_scales,
                             seg_offsets, G, R, N, K, code, c, stream)
    return c


def nvfp4_gemm(a_codes, a_block_scales, a_scales, b_codes, b_block_scales, b_scales,
               rows_per_a_scale: int = 1, rows_per_b_scale: Optional[int] = None,
               out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """C = A x B^T on NVFP4 operands (a [M][K/2], b [N][K/2], E4M3 block
    scales per 16, FP32 scales per rows_per_*_scale rows; by default one per
    token of A and one for all of B)."""
    M, half = a_codes.shape
    N, K = b_codes.shape[0], 2 * half
    rpb = N if rows_per_b_scale is None else rows_per_b_scale
    c = torch.empty((M, N), dtype=out_dtype, device=a_codes.device)
    code = B.MXQ_OUT_BF16 if out_dtype == torch.bfloat16 else B.MXQ_OUT_F32
    B.mxq_nvfp4_gemm(a_codes, a_block_scales, a_scales, rows_per_a_scale, b_codes,
                     b_block_scales, b_scales, rpb, M, N, K, code, c, stream)
    return c


class GroupedMXFP8(NamedTuple):
    row_codes: torch.Tensor
    row_scales: torch.Tensor
    col_codes: torch.Tensor
    col_scales: torch.Tensor          # capacity rows; the first P[G] are written
    col_scale_offsets: torch.Tensor


def grouped_quantize_mxfp8(x, seg_offsets, stream=None) -> GroupedMXFP8:
    x = _bf16_bits(x)
    R, cols = x.shape
    G = seg_offsets.numel() - 1
    u8 = torch.uint8
    out = GroupedMXFP8(_empty((R, cols), u8, x), _empty((R, cols // 32), u8, x),
                       _empty((R, cols), u8, x), _empty((R // 32 + G, cols), u8, x),
                       _empty((G + 1,), torch.int64, x))
    B.mxq_grouped_quantize(B.MXQ_FMT_MXFP8_ROWCOL, x, R, cols, seg_offsets, G,
                           out._asdict(), stream)
    return out


def grouped_quantize_nvfp4(x, seg_offsets, stream=None) -> NVFP4:
    x = _bf16_bits(x)
    R, cols = x.shape
    G = seg_offsets.numel() - 1
    res = NVFP4(_empty((R, cols // 2), torch.uint8, x), _empty((R, cols // 16), torch.uint8, x),
                _empty((R,), torch.float32, x))
    B.mxq_grouped_quantize(B.MXQ_FMT_NVFP4, x, R, cols, seg_offsets, G,
                           {"codes": res.codes, "block_scales": res.block_scales,
                            "token_scales": res.fp32_scales}, stream)
    return res


def dispatch_quantize_mxfp8(tokens, row_tokens, seg_offsets, stream=None) -> GroupedMXFP8:
    """Grouped MXFP8 row+col of the expert-sorted rows tokens[row_tokens[r]],
    read straight from the unpermuted tokens."""
    tokens = _bf16_bits(tokens)
    T, cols = tokens.shape
    R = row_tokens.numel()
    G = seg_offsets.numel() - 1
    u8 = torch.uint8
    out = GroupedMXFP8(_empty((R, cols), u8, tokens), _empty((R, cols // 32), u8, tokens),
                       _empty((R, cols), u8, tokens), _empty((R // 32 + G, cols), u8, tokens),
                       _empty((G + 1,), torch.int64, tokens))
    B.mxq_grouped_quantize_dispatch(B.MXQ_FMT_MXFP8_ROWCOL, tokens, T, cols, 0, None,
                                    row_tokens, R, seg_offsets, G, out._asdict(), stream)
    return out


def dispatch_quantize_nvfp4(tokens, token_rows, total_rows, stream=None) -> NVFP4:
    """Per-token NVFP4 of every token, written to its rows token_rows[t][c]
    of a [total_rows] expert-sorted layout."""
    tokens = _bf16_bits(tokens)
    T, cols = tokens.shape
    top_k = token_rows.shape[1]
    res = NVFP4(_empty((total_rows, cols // 2), torch.uint8, tokens),
                _empty((total_rows, cols // 16), torch.uint8, tokens),
                _empty((total_rows,), torch.float32, tokens))
    B.mxq_grouped_quantize_dispatch(B.MXQ_FMT_NVFP4, tokens, T, cols, top_k, token_rows, None,
                                    total_rows, None, 0,
                                    {"codes": res.codes, "block_scales": res.block_scales,
                                     "token_scales": res.fp32_scales}, stream)
    return res


# ---------------------------------------------------------------------------
# Layer operators
# ---------------------------------------------------------------------------

def _dtype_code(t: torch.Tensor, what: str) -> int:
    if t.dtype == torch.bfloat16:
        return B.MXQ_OUT_BF16
    if t.dtype == torch.float32:
        return B.MXQ_OUT_F32
    raise TypeError(f"{what} must be BF16 or FP32, got {t.dtype}")


def _out_code(dtype) -> int:
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    return B.MXQ_OUT_BF16 if dtype == torch.bfloat16 else B.MXQ_OUT_F32


def _arg(t, what: str, dtype, shape):
    """A tensor argument of the given dtype and shape (None: any size), contiguous.
    A small call checks up to twenty of these while its kernel takes a few
    microseconds, so an argument that fits takes three comparisons."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    s = t.shape
    if s != shape:
        fits = len(s) == len(shape)
        if fits:
            for n, w in zip(s, shape):
                if n != w and w is not None:
                    fits = False
        if not fits:
            raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(s)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _on(stream):
    """What a call allocates for itself and lets go on return belongs to the
    stream that its kernels run on: memory of another stream could go to that
    stream's next allocation while they still use it."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


def _workspace(nbytes: int, like, stream):
    if not nbytes:
        return None
    if stream is None:
        return _empty((nbytes,), torch.uint8, like)
    with _on(stream):
        return _empty((nbytes,), torch.uint8, like)


class Routing(NamedTuple):
    weights: torch.Tensor                    # [T][top_k] FP32
    experts: torch.Tensor                    # [T][top_k] int64, -1: none left
    token_rows: Optional[torch.Tensor]       # [T][top_k] int64, -1: no row
    row_tokens: Optional[torch.Tensor]       # [T * top_k] int64
    seg_offsets: Optional[torch.Tensor]      # [n_experts + 1] int64


def moe_route(logits, top_k: int, bias=None, scoring: int = B.MXQ_SCORE_SOFTMAX,
              n_expert_groups: int = 1, topk_groups: int = 1, group_topk: int = 1,
              renormalize: bool = True, scale: float = 1.0, maps: bool = True,
              stream=None) -> Routing:
    """Experts, weights and the dispatch's index maps of each token from its
    router logits [T][n_experts] (BF16 or FP32); bias [n_experts] FP32 moves
    the selection only.  maps=False leaves the maps out (None)."""
    code = _dtype_code(logits, "logits")
    T, E = _arg(logits, "logits", logits.dtype, (None, None)).shape
    if bias is not None:
        _arg(bias, "bias", torch.float32, (E,))
    w = _empty((T, top_k), torch.float32, logits)
    e = _empty((T, top_k), torch.int64, logits)
    tr = rt = seg = ws = None
    nbytes = 0
    if maps:
        tr = _empty((T, top_k), torch.int64, logits)
        rt = _empty((T * top_k,), torch.int64, logits)
        seg = _empty((E + 1,), torch.int64, logits)
        nbytes = B.mxq_moe_route_workspace(T, E)
        ws = _workspace(nbytes, logits, stream)
    params = B.mxq_route_params(top_k, n_expert_groups, topk_groups, group_topk, scoring,
                                int(renormalize), scale)
    B.mxq_moe_route(code, logits, bias, T, E, params, w, e, tr, rt, seg, ws, nbytes, stream)
    return Routing(w, e, tr, rt, seg)


def moe_route_backward(d_weights, logits, experts, scoring: int = B.MXQ_SCORE_SOFTMAX,
                       renormalize: bool = True, scale: float = 1.0, stream=None) -> torch.Tensor:
    """d_logits of the router's weights, the selection held fixed."""
    code = _dtype_code(logits, "logits")
    T, E = _arg(logits, "logits", logits.dtype, (None, None)).shape
    k = _arg(experts, "experts", torch.int64, (T, None)).shape[1]
    _arg(d_weights, "d_weights", torch.float32, (T, k))
    d = torch.empty_like(logits)
    B.mxq_moe_route_backward(code, d_weights, logits, experts, T, E, k, scoring, renormalize,
                             scale, d, stream)
    return d


def moe_combine(rows, token_rows, weights, out_dtype=None, stream=None) -> torch.Tensor:
    """out[t] = sum_c weights[t][c] rows[token_rows[t][c]], [T][cols], in
    out_dtype (by default the dtype of rows, BF16 or FP32)."""
    code = _dtype_code(rows, "rows")
    R, cols = _arg(rows, "rows", rows.dtype, (None, None)).shape
    T, k = _arg(token_rows, "token_rows", torch.int64, (None, None)).shape
    _arg(weights, "weights", torch.float32, (T, k))
    out_dtype = rows.dtype if out_dtype is None else out_dtype
    out_code = _out_code(out_dtype)
    out = _empty((T, cols), out_dtype, rows)
    B.mxq_moe_combine(code, rows, R, token_rows, weights, T, k, cols, out_code, out, stream)
    return out


def moe_combine_backward(d_out, rows, token_rows, weights, seg_offsets=None, stream=None):
    """(d_rows, d_weights) of moe_combine.  With the router's seg_offsets the
    rows past the last segment get zeros; other rows that no entry of
    token_rows names are left unwritten."""
    code = _dtype_code(rows, "rows")
    R, cols = _arg(rows, "rows", rows.dtype, (None, None)).shape
    T, k = _arg(token_rows, "token_rows", torch.int64, (None, None)).shape
    _arg(weights, "weights", torch.float32, (T, k))
    _arg(d_out, "d_out", rows.dtype, (T, cols))
    G = 0
    if seg_offsets is not None:
        G = _arg(seg_offsets, "seg_offsets", torch.int64, (None,)).numel() - 1
    d_rows = torch.empty_like(rows)
    d_w = _empty((T, k), torch.float32, rows)
    B.mxq_moe_combine_backward(code, d_out, rows, R, token_rows, weights, seg_offsets, G, T, k,
                               cols, d_rows, d_w, stream)
    return d_rows, d_w


def _activations(x):
    """(format, codes or values, block scales, FP32 scales, rows, K) of an
    activation operand: a BF16 or FP32 tensor [rows][K] or an NVFP4 tuple."""
    if isinstance(x, tuple):
        x = NVFP4(*x)
        rows, half = _arg(x.codes, "x codes", torch.uint8, (None, None)).shape
        _arg(x.block_scales, "x block scales", torch.uint8, (rows, half // 8))
        _arg(x.fp32_scales, "x FP32 scales", torch.float32, (rows,))
        return B.MXQ_X_NVFP4, x.codes, x.block_scales, x.fp32_scales, rows, 2 * half
    code = _dtype_code(x, "x")
    rows, K = _arg(x, "x", x.dtype, (None, None)).shape
    return (B.MXQ_X_BF16 if code == B.MXQ_OUT_BF16 else B.MXQ_X_F32), x, None, None, rows, K


def _nvfp4_weight(codes, block_scales, lead, K, what):
    """N of a weight [*lead][N][K] in NVFP4."""
    shape = (*lead, None, K // 2)
    N = _arg(codes, f"{what} codes", torch.uint8, shape).shape[-2]
    _arg(block_scales, f"{what} block scales", torch.uint8, (*lead, N, K // 16))
    return N


def nvfp4_matvec(x, b_codes, b_block_scales, b_scales, rows_per_b_scale: Optional[int] = None,
                 out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """C = x W^T for few rows x (at most 64): BF16 or FP32 [M][K], or an NVFP4
    tuple of per-token rows; W [N][K] in NVFP4 with one FP32 scale per
    rows_per_b_scale rows (by default one for all).  BF16 and NVFP4 activations
    enter the products exactly, FP32 ones rounded to 11 bits.  Returns C [M][N]."""
    fmt, xv, xbs, xs, M, K = _activations(x)
    N = _nvfp4_weight(b_codes, b_block_scales, (), K, "b")
    rpb = N if rows_per_b_scale is None else rows_per_b_scale
    if rpb > 0:
        _arg(b_scales, "b scales", torch.float32, (-(-N // rpb),))
    code = _out_code(out_dtype)
    c = _empty((M, N), out_dtype, xv)
    B.mxq_nvfp4_matvec(fmt, xv, xbs, xs, b_codes, b_block_scales, b_scales, rpb, M, N, K, code,
                       c, stream)
    return c


def nvfp4_expert_matvec(x, b_codes, b_block_scales, b_scales, seg_offsets,
                        out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """C[r] = x[r] W_e^T for the rows r of each segment e of seg_offsets: x
    [R][K] expert-sorted (as nvfp4_matvec), W [G][N][K] in NVFP4 with one FP32
    scale per expert.  Rows outside every segment are left unwritten."""
    fmt, xv, xbs, xs, R, K = _activations(x)
    G = _arg(seg_offsets, "seg_offsets", torch.int64, (None,)).numel() - 1
    N = _nvfp4_weight(b_codes, b_block_scales, (G,), K, "b")
    _arg(b_scales, "b scales", torch.float32, (G,))
    code = _out_code(out_dtype)
    c = _empty((R, N), out_dtype, xv)
    B.mxq_nvfp4_expert_matvec(fmt, xv, xbs, xs, b_codes, b_block_scales, b_scales, seg_offsets, G,
                              R, N, K, code, c, stream)
    return c


def nvfp4_expert_gateup(x, gateup: GateUpNVFP4, row_tokens, seg_offsets,
                        out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """h[r] = silu(x[t] gate_e^T) * (x[t] up_e^T), t = row_tokens[r], for the
    rows r of each segment e: x [T][K] unpermuted tokens (as nvfp4_matvec),
    gateup the experts' exported pair.  Returns h [R][N]."""
    fmt, xv, xbs, xs, T, K = _activations(x)
    G = _arg(seg_offsets, "seg_offsets", torch.int64, (None,)).numel() - 1
    R = _arg(row_tokens, "row_tokens", torch.int64, (None,)).numel()
    if gateup.up_codes is None:
        raise ValueError("gateup must hold the up projection")
    N = _nvfp4_weight(gateup.gate_codes, gateup.gate_block_scales, (G,), K, "gate")
    if _nvfp4_weight(gateup.up_codes, gateup.up_block_scales, (G,), K, "up") != N:
        raise ValueError("gate and up must have the same shape")
    _arg(gateup.scope_scales, "scope scales", torch.float32, (G,))
    code = _out_code(out_dtype)
    h = _empty((R, N), out_dtype, xv)
    B.mxq_nvfp4_expert_gateup(fmt, xv, xbs, xs, T, row_tokens, seg_offsets, G, R,
                              gateup.gate_codes, gateup.gate_block_scales, gateup.up_codes,
                              gateup.up_block_scales, gateup.scope_scales, N, K, code, h, stream)
    return h


def nvfp4_expert_layer(x, routing: Routing, gateup: GateUpNVFP4, down: GateUpNVFP4,
                       stream=None) -> torch.Tensor:
    """The expert layer of a decode step: the routed experts' gate/up with
    SwiGLU, down, and the weighted return to the tokens.  x [T][K] BF16, FP32
    or NVFP4; gateup and down as nvfp4_quantize_gateup_pair exports them (down
    with up=None).  Intermediates are FP32 tensors, of which the down product
    holds its activations in FP16 under powers of two (as nvfp4_matvec); returns
    BF16 [T][N]."""
    with _on(stream):
        h = nvfp4_expert_gateup(x, gateup, routing.row_tokens, routing.seg_offsets, stream=stream)
        y = nvfp4_expert_matvec(h, down.gate_codes, down.gate_block_scales, down.scope_scales,
                                routing.seg_offsets, stream=stream)
    return moe_combine(y, routing.token_rows, routing.weights, torch.bfloat16, stream)


class Attention(NamedTuple):
    out: torch.Tensor          # [n_seqs][q_len][n_heads][head_dim] BF16
    lse: torch.Tensor          # [n_seqs][q_len][n_heads] FP32


def nvfp4_cache_rows(pages, slots, n_kv_heads: int, page_size: int) -> torch.Tensor:
    """Rows of an NVFP4 cache, [T][n_kv_heads] int64, of tokens at slot slots[t] of
    page pages[t]: the token_rows under which dispatch_quantize_nvfp4's
    library call writes their keys (or values) into the cache."""
    heads = torch.arange(n_kv_heads, device=pages.device)
    return (pages[:, None] * n_kv_heads + heads) * page_size + slots[:, None]


def nvfp4_cache_append(x, rows, cache: NVFP4, stream=None) -> None:
    """Quantize keys or values x [T][n_kv_heads][head_dim] (BF16) into the rows
    [T][n_kv_heads] of the cache; a row of -1 is dropped."""
    x = _bf16_bits(x)
    T, H, D = x.shape
    _arg(rows, "rows", torch.int64, (T, H))
    n = _arg(cache.codes, "cache codes", torch.uint8, (None, D // 2)).shape[0]
    _arg(cache.block_scales, "cache block scales", torch.uint8, (n, D // 16))
    _arg(cache.fp32_scales, "cache FP32 scales", torch.float32, (n,))
    B.mxq_grouped_quantize_dispatch(B.MXQ_FMT_NVFP4, x, T * H, D, 1, rows, None, n, None, 0,
                                    {"codes": cache.codes, "block_scales": cache.block_scales,
                                     "token_scales": cache.fp32_scales}, stream)


def nvfp4_attention(q, k: NVFP4, v: NVFP4, block_table, seq_lens, n_kv_heads: int,
                    page_size: int, softmax_scale: Optional[float] = None, causal: bool = True,
                    window: int = 0, stream=None) -> Attention:
    """Attention of q [n_seqs][q_len][n_heads][head_dim] (BF16) over a paged
    cache of NVFP4 keys and values (rows [n_pages * n_kv_heads * page_size], see
    nvfp4_cache_rows); block_table [n_seqs][max_pages] and seq_lens [n_seqs]
    int64.  The queries are the last q_len positions of their sequence;
    softmax_scale is 1/sqrt(head_dim) by default."""
    _arg(q, "q", torch.bfloat16, (None, None, None, None))
    n_seqs, q_len, n_heads, D = q.shape
    n_rows = _arg(k.codes, "k codes", torch.uint8, (None, D // 2)).shape[0]
    _arg(v.codes, "v codes", torch.uint8, (n_rows, D // 2))
    _arg(k.block_scales, "k block scales", torch.uint8, (n_rows, D // 16))
    _arg(v.block_scales, "v block scales", torch.uint8, (n_rows, D // 16))
    _arg(k.fp32_scales, "k FP32 scales", torch.float32, (n_rows,))
    _arg(v.fp32_scales, "v FP32 scales", torch.float32, (n_rows,))
    max_pages = _arg(block_table, "block_table", torch.int64, (n_seqs, None)).shape[1]
    _arg(seq_lens, "seq_lens", torch.int64, (n_seqs,))
    per_page = n_kv_heads * page_size
    if per_page < 1 or n_rows % per_page != 0:
        raise ValueError("the cache must hold n_pages * n_kv_heads * page_size rows")
    scale = D ** -0.5 if softmax_scale is None else softmax_scale
    out = torch.empty_like(q)
    lse = _empty((n_seqs, q_len, n_heads), torch.float32, q)
    nbytes = B.mxq_nvfp4_attention_workspace(n_seqs, q_len, n_heads, n_kv_heads, D,
                                             max_pages * page_size)
    B.mxq_nvfp4_attention(q, k, v, block_table, seq_lens, n_seqs, q_len, n_heads, n_kv_heads, D,
                          n_rows // per_page, page_size, max_pages, scale, causal, window, out,
                          lse, _workspace(nbytes, q, stream), nbytes, stream)
    return Attention(out, lse)
