"""The layer operators on the GPU against plain 64-bit forms (layer_ref).
Tolerances count roundings: half a step of an output's type relative to its
value, and for fp32 sums one half step per addition of the sum of the terms'
magnitudes.  Selections and index maps are compared for equality."""
import numpy as np
import pytest
import torch

import layer_ref as R
import nvfp4_block_scaled_amax_amd as mxq
from nvfp4_block_scaled_amax_amd import api
from nvfp4_block_scaled_amax_amd import workloads as W
from gpu_util import announce, dev, host, require_gpu

pytestmark = pytest.mark.gpu

SOFTMAX, SIGMOID = mxq.MXQ_SCORE_SOFTMAX, mxq.MXQ_SCORE_SIGMOID


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def bf16(a):
    """float64 values rounded to BF16 values."""
    return W.bf16_to_f64(W.bf16_bits(a))


def put(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def close(got, want, tol, what):
    got = got.detach().cpu().double().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got[np.isfinite(want)]).all(), what
    fin = np.isfinite(want)
    assert (got[~fin] == want[~fin]).all(), what
    err = np.where(fin, np.abs(np.where(fin, got, 0) - np.where(fin, want, 0)), 0)
    bad = np.argwhere(err > tol)
    assert bad.size == 0, (what, len(bad), tuple(bad[0]), got[tuple(bad[0])],
                           want[tuple(bad[0])], np.broadcast_to(tol, want.shape)[tuple(bad[0])])


# ---------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------

def params(top_k, scoring=SOFTMAX, groups=1, topk_groups=1, group_topk=1, renorm=True, scale=1.0):
    return dict(top_k=top_k, scoring=scoring, n_groups=groups, topk_groups=topk_groups,
                group_topk=group_topk, renormalize=renorm, scale=scale)


def run_route(x, bias, p, dtype, maps=True):
    return api.moe_route(put(x, dtype), p["top_k"], bias=None if bias is None else
                         put(bias, torch.float32), scoring=p["scoring"],
                         n_expert_groups=p["n_groups"], topk_groups=p["topk_groups"],
                         group_topk=p["group_topk"], renormalize=p["renormalize"],
                         scale=p["scale"], maps=maps)


def check_route(x, bias, p, dtype, name):
    """x holds values of the dtype exactly."""
    announce(f"route {name} {x.shape} {p}")
    r = run_route(x, bias, p, dtype)
    torch.cuda.synchronize()
    w, e, tr, rt, seg = R.route(x, bias, p)
    for got, want, what in ((r.experts, e, "experts"), (r.token_rows, tr, "token_rows"),
                            (r.row_tokens, rt, "row_tokens"), (r.seg_offsets, seg, "seg")):
        got = got.cpu().numpy()
        assert np.array_equal(got, want), (name, what, np.argwhere(got != want)[:3])
    close(r.weights, w, np.abs(w) * 2.0 ** -20 + 1e-37, f"{name} weights")
    return r


def logits(rng, T, E, dtype):
    x = rng.normal(0, 1.5, (T, E))
    return bf16(x) if dtype == torch.bfloat16 else x.astype(np.float32).astype(np.float64)


ROUTES = [
    (1, 8, params(2)), (1, 256, params(8, SIGMOID, 8, 4, 2, True, 2.5)),
    (3, 7, params(7, SOFTMAX, renorm=False)), (63, 60, params(4)), (64, 128, params(8)),
    (65, 128, params(8, SIGMOID)), (257, 160, params(6, SOFTMAX, 8, 3, 1, False, 16.0)),
    (300, 1, params(1)), (40, 1024, params(64, SIGMOID, 16, 9, 2)), (129, 72, params(5, SIGMOID,
     4, 2, 2, False)), (1000, 64, params(1, SOFTMAX)), (33, 192, params(3, SOFTMAX, 64, 5, 2)),
    (17, 100, params(10, SIGMOID, 50, 7, 2)), (2048, 33, params(2, SOFTMAX, 3, 2, 2)),
]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,p", ROUTES)
def test_route(T, E, p, dtype, bias):
    rng = np.random.default_rng(T * 1000 + E)
    x = logits(rng, T, E, dtype)
    b = rng.normal(0, 0.1, E).astype(np.float32).astype(np.float64) if bias else None
    check_route(x, b, p, dtype, f"random {T}x{E}")


@pytest.mark.parametrize("scoring", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("bias", [None, 0.0])
def test_route_ties_go_to_the_lowest_expert(scoring, bias):
    rng = np.random.default_rng(3)
    T, E = 200, 96
    x = rng.integers(-2, 3, (T, E)).astype(np.float64)       # many equal logits
    x[:7] = 0.0
    b = None if bias is None else np.zeros(E)
    check_route(x, b, params(9, scoring), torch.bfloat16, "ties")
    check_route(x, b, params(6, scoring, 8, 3, 1), torch.float32, "ties in groups")
    check_route(x, b, params(6, scoring, 8, 3, 2), torch.float32, "ties in group sums")


@pytest.mark.parametrize("scoring", [SOFTMAX, SIGMOID])
def test_route_near_ties_are_decided_exactly(scoring):
    """Keys that agree to 2^-30: fp32 scores cannot order them."""
    rng = np.random.default_rng(8)
    T, E = 300, 64
    x = np.float32(1.0) + rng.integers(-3, 4, (T, E)) * np.float32(2.0 ** -23)
    x = x.astype(np.float32).astype(np.float64)
    b = (rng.integers(-3, 4, E) * 2.0 ** -26).astype(np.float32).astype(np.float64)
    check_route(x, b, params(8, scoring), torch.float32, "near ties")
    check_route(x, b, params(8, scoring, 8, 4, 1), torch.float32, "near ties in groups")


@pytest.mark.parametrize("scoring", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masked_experts_and_rows(scoring, groups):
    rng = np.random.default_rng(5)
    T, E = 150, 32
    x = rng.normal(0, 2, (T, E)).astype(np.float32).astype(np.float64)
    x[rng.random((T, E)) < 0.6] = -np.inf
    x[::9] = -np.inf                                         # whole rows
    x[1::9, 1:] = -np.inf                                    # one expert left
    x[2, 4] = np.inf
    x[3, 5] = np.nan
    x[4] = -3.0e38                                           # the type's lowest values
    x[5, 3:] = 3.0e38
    for b in (None, rng.normal(0, 0.1, E).astype(np.float32).astype(np.float64)):
        check_route(x, b, params(6, scoring, groups, 2 if groups > 1 else 1, 2), torch.float32,
                    "masked")
    b[::3] = -np.inf                                         # disabled experts
    check_route(x, b, params(6, scoring, groups, 2 if groups > 1 else 1, 1), torch.float32,
                "disabled experts")
    check_route(np.full((70, E), -np.inf), None, params(2, scoring, groups), torch.bfloat16,
                "nothing to select")


def test_route_without_maps_and_large_logits():
    rng = np.random.default_rng(6)
    x = (rng.normal(0, 60, (50, 40))).astype(np.float32).astype(np.float64)
    p = params(4, SIGMOID, renorm=False)
    r = run_route(x, None, p, torch.float32, maps=False)
    torch.cuda.synchronize()
    assert r.token_rows is None and r.row_tokens is None and r.seg_offsets is None
    w, e = R.route(x, None, p)[:2]
    assert np.array_equal(r.experts.cpu().numpy(), e)
    close(r.weights, w, np.abs(w) * 2.0 ** -20 + 1e-37, "weights")


def test_route_feeds_the_dispatch(orc):
    """The maps drive the fused dispatch: its rows are the tokens' rows."""
    rng = np.random.default_rng(9)
    T, E = 77, 16
    x = rng.normal(0, 1, (T, E)).astype(np.float32)
    x[5] = -np.inf
    r = run_route(x.astype(np.float64), None, params(3), torch.float32)
    tok = W.student_t_activations(T, 64, 11)
    q = api.dispatch_quantize_nvfp4(dev(tok), r.token_rows, T * 3)
    m = api.dispatch_quantize_mxfp8(dev(tok), r.row_tokens, r.seg_offsets)
    torch.cuda.synchronize()
    rows = int(r.seg_offsets[-1])
    rt = r.row_tokens.cpu().numpy()[:rows]
    assert rows == 3 * (T - 1)
    c, b, s = orc.nvfp4_per_token(tok[rt])
    assert np.array_equal(host(q.codes)[:rows], c) and np.array_equal(host(q.fp32_scales)[:rows], s)
    rc, rs = orc.mxfp8_rowwise(tok[rt])
    assert np.array_equal(host(m.row_codes)[:rows], rc)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("scoring", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (65, 60, 4), (33, 160, 6), (9, 1024, 64),
                                   (130, 128, 8), (20, 3, 3)])
def test_route_backward(T, E, k, scoring, renorm, dtype):
    announce(f"route backward {T}x{E} k={k} {scoring} {renorm} {dtype}")
    rng = np.random.default_rng(T + E)
    x = logits(rng, T, E, dtype)
    x[rng.random((T, E)) < 0.1] = -np.inf
    x[:1] = -np.inf
    experts = R.route(x, None, params(k, scoring))[1]
    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    d = api.moe_route_backward(put(dw, torch.float32), put(x, dtype), put(experts, torch.int64),
                               scoring, renorm, 1.5)
    torch.cuda.synchronize()
    want, mag = R.route_backward(dw.astype(np.float64), x, experts, scoring, renorm, 1.5)
    # Scores within 2^-20, at most 64 + 1024 / 64 + 6 fp32 additions per sum.
    tol = mag * (2.0 ** -19 + 90 * 2.0 ** -24) + 1e-37
    if dtype == torch.bfloat16:
        tol = tol + np.abs(want) * R.HALF_BF16
    close(d, want, tol, "d_logits")


@pytest.mark.parametrize("scoring", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(scoring, renorm):
    """Central differences of the weights in 64 bits, step 2^-17: truncation
    2^-34 times third derivatives (at most a few), far below 2^-19."""
    rng = np.random.default_rng(12)
    T, E, k, h = 6, 12, 4, 2.0 ** -17
    x = rng.normal(0, 1, (T, E)).astype(np.float32).astype(np.float64)
    experts = R.route(x, None, params(k, scoring))[1]
    dw = rng.normal(0, 1, (T, k)).astype(np.float32).astype(np.float64)

    def loss(z):
        return (dw * R.route_weights(z, experts, scoring, renorm, 2.0)).sum(1)
    want = np.zeros((T, E))
    for e in range(E):
        up, dn = x.copy(), x.copy()
        up[:, e] += h
        dn[:, e] -= h
        want[:, e] = (loss(up) - loss(dn)) / (2 * h)
    d = api.moe_route_backward(put(dw, torch.float32), put(x, torch.float32),
                               put(experts, torch.int64), scoring, renorm, 2.0)
    mag = R.route_backward(dw, x, experts, scoring, renorm, 2.0)[1]
    close(d, want, mag * (2.0 ** -19 + 90 * 2.0 ** -24) + 2.0 ** -28, "differences")


def test_route_backward_ignores_experts_out_of_range():
    rng = np.random.default_rng(13)
    x = rng.normal(0, 1, (4, 10))
    x = x.astype(np.float32).astype(np.float64)
    bad = np.array([[0, -1, 10, 3], [-5, 1 << 40, 2, 9], [10, 11, 12, 13], [1, 2, 3, 4]])
    clean = np.where((bad < 0) | (bad >= 10), -1, bad)
    dw = rng.normal(0, 1, (4, 4)).astype(np.float32)
    a = api.moe_route_backward(put(dw, torch.float32), put(x, torch.float32),
                               put(bad, torch.int64))
    want, mag = R.route_backward(dw.astype(np.float64), x, clean, SOFTMAX, True, 1.0)
    close(a, want, mag * (2.0 ** -19 + 90 * 2.0 ** -24) + 1e-37, "out of range")


# ---------------------------------------------------------------------------
# Combine
# ---------------------------------------------------------------------------

def combine_case(rng, T, k, cols, dtype, drop=0.1):
    rows = rng.normal(0, 1, (T * k, cols))
    rows = bf16(rows) if dtype == torch.bfloat16 else rows.astype(np.float32).astype(np.float64)
    perm = rng.permutation(T * k).reshape(T, k).astype(np.int64)
    perm[rng.random((T, k)) < drop] = -1
    w = rng.random((T, k)).astype(np.float32)
    return rows, perm, w


COMBINES = [(1, 1, 8), (1, 8, 2048), (5, 3, 96), (33, 8, 200), (7, 2, 4104), (64, 64, 16),
            (3, 6, 8192)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,cols", COMBINES)
def test_combine(T, k, cols, dtype):
    announce(f"combine {T}x{k}x{cols} {dtype}")
    rng = np.random.default_rng(T + cols)
    rows, tr, w = combine_case(rng, T, k, cols, dtype)
    tr[0, 0] = -1
    tr[T - 1] = -1                                   # a token with no copy
    if T > 1:
        tr[0, k - 1] = T * k                         # out of range
    want, mag = R.combine(rows, tr, w.astype(np.float64))
    for out in (torch.float32, torch.bfloat16):
        got = api.moe_combine(put(rows, dtype), put(tr, torch.int64), put(w, torch.float32), out)
        assert got.dtype == out
        tol = mag * k * 2.0 ** -24 + (np.abs(want) * R.HALF_BF16 if out == torch.bfloat16 else 0)
        close(got, want, tol * 1.0001, "combine")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,cols", COMBINES)
def test_combine_backward(T, k, cols, dtype):
    announce(f"combine backward {T}x{k}x{cols} {dtype}")
    rng = np.random.default_rng(T + cols)
    rows, _, w = combine_case(rng, T, k, cols, dtype)
    experts = rng.integers(-1, 5, (T, k))
    tr, _, seg = R.maps(experts, 5)
    d = rng.normal(0, 1, (T, cols))
    d = bf16(d) if dtype == torch.bfloat16 else d.astype(np.float32).astype(np.float64)
    d_rows, d_w = api.moe_combine_backward(put(d, dtype), put(rows, dtype), put(tr, torch.int64),
                                           put(w, torch.float32), put(seg, torch.int64))
    torch.cuda.synchronize()
    want = np.zeros_like(rows)
    t, c = np.nonzero(tr >= 0)
    want[tr[t, c]] = w[t, c, None].astype(np.float64) * d[t]
    half = R.HALF_BF16 if dtype == torch.bfloat16 else 2.0 ** -24
    close(d_rows, want, np.abs(want) * (half * 1.0001 + 2.0 ** -24), "d_rows")
    terms = d[:, None, :] * rows[np.maximum(tr, 0)]
    want = np.where(tr >= 0, terms.sum(2), 0.0)
    close(d_w, want, np.abs(terms).sum(2) * (cols / 16 + 32) * 2.0 ** -24, "d_weights")


def test_combine_backward_leaves_unnamed_rows():
    """Without segments only the rows that are named change."""
    rng = np.random.default_rng(2)
    T, k, cols = 6, 2, 64
    rows, _, w = combine_case(rng, T, k, cols, torch.bfloat16)
    tr = np.full((T, k), -1, np.int64)
    tr[:, 0] = 2 * np.arange(T)
    d = put(bf16(rng.normal(0, 1, (T, cols))), torch.bfloat16)
    rw = put(rows, torch.bfloat16)
    d_rows = torch.full_like(rw, 7.0)
    d_w = torch.empty(T, k, device="cuda")
    mxq.mxq_moe_combine_backward(mxq.MXQ_OUT_BF16, d, rw, T * k, put(tr, torch.int64),
                                 put(w, torch.float32), None, 0, T, k, cols, d_rows, d_w)
    torch.cuda.synchronize()
    assert (d_rows[1::2] == 7.0).all() and not (d_rows[0::2] == 7.0).all(1).any()
    assert (d_w[:, 1] == 0).all()


# ---------------------------------------------------------------------------
# Few-row products
# ---------------------------------------------------------------------------

X_KINDS = ["bf16", "f32", "nvfp4"]


def activation(rng, rows, K, kind):
    """(operand for the API, its values in 64 bits [rows][K], the row factor
    sx, largest relative error of a value held in FP16)."""
    if kind == "nvfp4":
        c, b, s = R.random_nvfp4(rng, rows, K)
        return api.NVFP4(dev(c), dev(b), dev(s)), R.decode(c, b), s.astype(np.float64), 0.0
    x = rng.standard_t(3, (rows, K)) * np.exp2(rng.uniform(-20, 20, (rows, 1)))
    if kind == "bf16":
        return put(bf16(x), torch.bfloat16), bf16(x), np.ones(rows), 0.0
    x = x.astype(np.float32).astype(np.float64)
    return put(x, torch.float32), x, np.ones(rows), R.HALF_FP16


def product(xv, sx, w, sb, held):
    """C and its tolerance (without the output's rounding): the FP16 holding
    (relative held, and 2^-39 of the row's largest), fp32 sums of at most
    K / 16 + 32 additions, two scale products."""
    K = xv.shape[1]
    want = (xv @ w.T) * sx[:, None] * sb[None, :]
    mag = (np.abs(xv) @ np.abs(w).T) * np.abs(sx)[:, None] * np.abs(sb)[None, :]
    floor = 2.0 ** -39 * np.abs(xv).max(1)[:, None] * np.abs(w).sum(1)[None, :] \
        * np.abs(sx)[:, None] * np.abs(sb)[None, :]
    return want, mag * (held + (K / 16 + 34) * 2.0 ** -23) + floor


MATVECS = [(1, 1, 64), (1, 130, 2048), (2, 17, 192), (3, 65, 576), (5, 300, 1024), (8, 31, 64),
           (16, 257, 2048), (17, 40, 320), (33, 100, 704), (64, 129, 1344), (13, 16, 8192),
           (4, 48, 65536)]


@pytest.mark.parametrize("kind", X_KINDS)
@pytest.mark.parametrize("M,N,K", MATVECS)
def test_matvec(M, N, K, kind):
    announce(f"matvec {M}x{N}x{K} {kind}")
    rng = np.random.default_rng(M * 7 + N + K)
    x, xv, sx, held = activation(rng, M, K, kind)
    c, b, _ = R.random_nvfp4(rng, N, K)
    w = R.decode(c, b)
    for rpb in (N, 1, 16):
        s = np.exp2(rng.uniform(-9, -3, -(-N // rpb))).astype(np.float32)
        want, tol = product(xv, sx, w, np.repeat(s, rpb)[:N].astype(np.float64), held)
        for out in (torch.float32, torch.bfloat16):
            got = api.nvfp4_matvec(x, dev(c), dev(b), dev(s), rpb, out)
            torch.cuda.synchronize()
            assert got.dtype == out
            close(got, want, tol + (np.abs(want) * R.HALF_BF16 * 1.001
                                    if out == torch.bfloat16 else 0), f"matvec {rpb} {out}")


def test_matvec_zero_and_tiny_rows():
    rng = np.random.default_rng(4)
    M, N, K = 6, 40, 512
    x = bf16(rng.normal(0, 1, (M, K)))
    x[0] = 0.0
    x[1, 1:] = 0.0
    x[2] = bf16(x[2] * 2.0 ** -126)                  # BF16 subnormals among them
    x[3] = bf16(x[3] * 2.0 ** 125)
    x[4, :256] = 0.0
    c, b, _ = R.random_nvfp4(rng, N, K, lo=0)        # zero and subnormal block scales
    c[:, ::3] = 0
    s = np.full(1, 2.0 ** -20, np.float32)
    want, tol = product(x, np.ones(M), R.decode(c, b), np.repeat(s, N).astype(np.float64), 0.0)
    got = api.nvfp4_matvec(put(x, torch.bfloat16), dev(c), dev(b), dev(s), None, torch.float32)
    close(got, want, tol + 1e-44, "tiny")
    assert (got[0] == 0).all()


def segments(rng, G, R_rows, empty=0.5):
    """Ragged segments with empty ones, the last rows in no segment."""
    sizes = rng.multinomial(R_rows - R_rows // 8, np.where(
        (u := rng.random(G)) < empty, 1e-12, u) / np.where(u < empty, 1e-12, u).sum())
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)


EXPERTS = [(4, 1, 40, 64), (4, 9, 65, 320), (16, 40, 130, 768), (128, 8, 48, 256),
           (3, 200, 33, 128), (70, 64, 17, 64), (1, 37, 100, 2048)]


@pytest.mark.parametrize("kind", X_KINDS)
@pytest.mark.parametrize("G,rows,N,K", EXPERTS)
def test_expert_matvec(G, rows, N, K, kind):
    announce(f"expert matvec {G} {rows}x{N}x{K} {kind}")
    rng = np.random.default_rng(G + rows + N)
    x, xv, sx, held = activation(rng, rows, K, kind)
    c, b, s = R.random_nvfp4(rng, G * N, K)
    s = s[:G]
    seg = segments(rng, G, rows)
    got = torch.full((rows, N), 5.0, device="cuda")
    args = (x.codes, x.block_scales, x.fp32_scales) if kind == "nvfp4" else (x, None, None)
    mxq.mxq_nvfp4_expert_matvec(X_KINDS.index(kind), *args, dev(c), dev(b), dev(s), dev(seg), G,
                                rows, N, K, mxq.MXQ_OUT_F32, got)
    torch.cuda.synchronize()
    want, tol = np.full((rows, N), 5.0), np.zeros((rows, N))
    w = R.decode(c, b).reshape(G, N, K)
    for e in range(G):
        a, z = seg[e], seg[e + 1]
        if z > a:
            want[a:z], tol[a:z] = product(xv[a:z], sx[a:z], w[e], np.full(N, float(s[e])), held)
    close(got, want, tol, "expert matvec")


@pytest.mark.parametrize("kind", X_KINDS)
@pytest.mark.parametrize("G,rows,N,K", EXPERTS)
def test_expert_gateup(G, rows, N, K, kind):
    announce(f"expert gateup {G} {rows}x{N}x{K} {kind}")
    rng = np.random.default_rng(G + rows + N + 1)
    T = max(1, rows // 2)
    x, xv, sx, held = activation(rng, T, K, kind)
    gc, gb, s = R.random_nvfp4(rng, G * N, K)
    uc, ub, _ = R.random_nvfp4(rng, G * N, K)
    s = (s[:G] * 2.0 ** -6).astype(np.float32)
    seg = segments(rng, G, rows)
    rt = rng.integers(0, T, rows)
    rt[-1] = -1
    pair = api.GateUpNVFP4(*(dev(a.reshape(G, N, -1)) for a in (gc, gb, uc, ub)), dev(s))
    for out in (torch.float32, torch.bfloat16):
        got = api.nvfp4_expert_gateup(x, pair, dev(rt), dev(seg), out)
        torch.cuda.synchronize()
        n = seg[-1]
        rr = np.maximum(rt, 0)[:n]
        e_of = np.searchsorted(seg, np.arange(n), side="right") - 1
        g, tg, u, tu = (np.zeros((n, N)) for _ in range(4))
        for e in np.unique(e_of):
            i = np.nonzero(e_of == e)[0]
            sc = np.full(N, float(s[e]))
            g[i], tg[i] = product(xv[rr[i]], sx[rr[i]], R.decode(gc, gb).reshape(G, N, K)[e], sc, held)
            u[i], tu[i] = product(xv[rr[i]], sx[rr[i]], R.decode(uc, ub).reshape(G, N, K)[e], sc, held)
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        want = silu * u
        # |silu'| <= 1.1; silu itself within 2^-20.
        tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(silu) * tu + np.abs(want) * 2.0 ** -20 + 1e-36
        if out == torch.bfloat16:
            tol = tol + np.abs(want) * R.HALF_BF16
        close(got[:n], want, tol, "gateup")


def test_expert_layer_matches_its_parts():
    rng = np.random.default_rng(21)
    T, E, H, I, k = 9, 12, 256, 192, 3
    x = put(bf16(rng.normal(0, 1, (T, H))), torch.bfloat16)
    gate, up = (dev(W.bf16_bits(rng.normal(0, 0.05, (E, I, H)))) for _ in range(2))
    down = dev(W.bf16_bits(rng.normal(0, 0.05, (E, H, I))))
    pair = api.nvfp4_quantize_gateup_pair(gate, up)
    dn = api.nvfp4_quantize_gateup_pair(down)
    r = api.moe_route(put(rng.normal(0, 1, (T, E)), torch.float32), k)
    got = api.nvfp4_expert_layer(x, r, pair, dn)
    torch.cuda.synchronize()
    xs, e = x.cpu().double().numpy(), r.experts.cpu().numpy()
    w = r.weights.cpu().double().numpy()

    def dec(c, b, s):
        return R.decode(host(c), host(b)) * host(s).astype(np.float64)[:, None, None]
    g, u, d = (dec(*a) for a in ((pair.gate_codes, pair.gate_block_scales, pair.scope_scales),
                                 (pair.up_codes, pair.up_block_scales, pair.scope_scales),
                                 (dn.gate_codes, dn.gate_block_scales, dn.scope_scales)))
    want, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for c in range(k):
            a, b = g[e[t, c]] @ xs[t], u[e[t, c]] @ xs[t]
            h = a / (1 + np.exp(-a)) * b
            mag = np.abs(d[e[t, c]]) @ np.abs(h)
            want[t] += w[t, c] * (d[e[t, c]] @ h)
            # h held in FP16 for the second product; fp32 sums on both sides.
            tol[t] += w[t, c] * mag * (R.HALF_FP16 + (H + I) * 2.0 ** -20)
    close(got, want, tol + np.abs(want) * R.HALF_BF16, "expert layer")


def test_malformed_segments_stay_in_bounds():
    rng = np.random.default_rng(23)
    G, rows, N, K = 5, 12, 40, 128
    x, *_ = activation(rng, rows, K, "bf16")
    c, b, s = R.random_nvfp4(rng, G * N, K)
    out = torch.full((rows + 8, N), 5.0, device="cuda")
    for seg in ([-5, 100, 3, 3, 2, 1 << 40], [4, 2, 9, 1 << 62, -(1 << 62), 12]):
        announce(f"malformed segments {seg}")
        mxq.mxq_nvfp4_expert_matvec(mxq.MXQ_X_BF16, x, None, None, dev(c), dev(b), dev(s[:G].copy()),
                                    dev(np.array(seg, np.int64)), G, rows, N, K, mxq.MXQ_OUT_F32,
                                    out[4:4 + rows])
        torch.cuda.synchronize()
        assert (out[:4] == 5.0).all() and (out[4 + rows:] == 5.0).all()


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def attention_case(rng, lens, Q, H, Hkv, D, page, max_pages=None, spread=8.0):
    B = len(lens)
    per = max(1, max(-(-n // page) for n in lens))
    max_pages = per if max_pages is None else max_pages
    n_pages = B * max_pages + 2
    table = rng.permutation(n_pages)[:B * max_pages].reshape(B, max_pages).astype(np.int64)
    rows = n_pages * Hkv * page
    k = R.random_nvfp4(rng, rows, D, zero_rows=0.05)
    v = R.random_nvfp4(rng, rows, D, zero_rows=0.05)
    q = bf16(rng.normal(0, 1, (B, Q, H, D)) * np.exp2(rng.uniform(-spread, 0, (B, Q, H, 1))))
    return q, k, v, table, np.array(lens, np.int64)


def run_attention(q, k, v, table, lens, Hkv, page, scale, causal, window):
    return api.nvfp4_attention(put(q, torch.bfloat16), api.NVFP4(*(dev(a) for a in k)),
                               api.NVFP4(*(dev(a) for a in v)), dev(table), dev(lens), Hkv, page,
                               scale, causal, window)


def check_attention(case, Hkv, page, name, scale=None, causal=True, window=0):
    q, k, v, table, lens = case
    D = q.shape[3]
    announce(f"attention {name} q={q.shape} lens={lens[:4]} kv={Hkv} page={page} w={window}")
    r = run_attention(q, k, v, table, lens, Hkv, page, scale, causal, window)
    torch.cuda.synchronize()
    kk, vv = (R.decode(c, b) * s[:, None].astype(np.float64) for c, b, s in (k, v))
    sc = float(np.float32(D ** -0.5 if scale is None else scale))
    want, lse, mag, terms = R.attention(q, kk, vv, table, lens, Hkv, page, sc, causal, window)
    # Scores: fp32 sums of D products and four factors.  The numerators: FP16.
    # Sums over keys: one rounding per 16 keys and level of the joins.
    n = max(1, int(lens.max()))
    delta = terms * (D + 24) * 2.0 ** -23 + 2.0 ** -20
    tol = mag * (R.HALF_FP16 + 2 * delta[..., None] + (n / 16 + 64) * 2.0 ** -23)
    close(r.out, want, tol + np.abs(want) * R.HALF_BF16 * 1.001 + 1e-36, f"{name} out")
    close(r.lse, lse, delta + (n / 16 + 64) * 2.0 ** -23 + np.abs(np.where(
        np.isfinite(lse), lse, 0)) * 2.0 ** -22, f"{name} lse")
    return r


ATTENTIONS = [
    # lens, q_len, heads, kv heads, head dim, page
    ([1], 1, 1, 1, 128, 16), ([17, 1, 0, 33], 1, 8, 1, 128, 16), ([31, 32, 65], 1, 8, 2, 64, 32),
    ([300, 7], 1, 20, 4, 256, 48), ([130, 64, 15], 2, 6, 2, 128, 64), ([3, 40], 5, 3, 3, 64, 16),
    ([500], 1, 32, 2, 128, 128), ([45, 200], 33, 4, 1, 64, 16), ([100, 64], 64, 5, 5, 128, 32),
    ([1200], 3, 16, 1, 128, 16), ([90], 20, 17, 1, 256, 16), ([2000, 3000], 1, 4, 4, 64, 80),
]


@pytest.mark.parametrize("lens,Q,H,Hkv,D,page", ATTENTIONS)
def test_attention(lens, Q, H, Hkv, D, page):
    rng = np.random.default_rng(sum(lens) + H)
    check_attention(attention_case(rng, lens, Q, H, Hkv, D, page), Hkv, page, "causal")


@pytest.mark.parametrize("lens,Q,H,Hkv,page,causal,window", [
    ([300, 201], 200, 16, 16, 16, True, 0), ([700, 64, 0], 70, 64, 32, 48, True, 0),
    ([520, 33], 100, 32, 32, 32, True, 40), ([260, 130], 100, 40, 20, 16, False, 0),
])
def test_attention_many_rows(lens, Q, H, Hkv, page, causal, window):
    """Enough query rows of 64 elements to fill the chip, in one part and in several,
    some of them before the first key; slots past the length hold anything."""
    rng = np.random.default_rng(53)
    q, k, v, table, lens = case = attention_case(rng, lens, Q, H, Hkv, 64, page)
    r = check_attention(case, Hkv, page, "many rows", causal=causal, window=window)
    live = np.zeros(k[0].shape[0], bool)
    for b, n in enumerate(lens):
        t = np.arange(n)
        for h in range(Hkv):
            live[(table[b][t // page] * Hkv + h) * page + t % page] = True
    for c, bs, s in (k, v):
        c[~live], bs[~live], s[~live] = 0xFF, 0x7F, np.nan
    again = run_attention(q, k, v, table, lens, Hkv, page, None, causal, window)
    torch.cuda.synchronize()
    assert torch.equal(again.out, r.out) and torch.equal(again.lse, r.lse)


@pytest.mark.parametrize("window", [1, 5, 16, 100])
def test_attention_window(window):
    rng = np.random.default_rng(window)
    check_attention(attention_case(rng, [200, 3, 64, 0, 37], 4, 6, 2, 128, 32), 2, 32, "window",
                    window=window)
    check_attention(attention_case(rng, [257], 40, 2, 1, 64, 16), 1, 16, "window chunk",
                    window=window)


def test_attention_not_causal_and_scale():
    rng = np.random.default_rng(31)
    check_attention(attention_case(rng, [50, 1, 0, 99], 7, 4, 2, 64, 16), 2, 16, "all keys",
                    causal=False)
    check_attention(attention_case(rng, [70], 1, 4, 2, 128, 16), 2, 16, "scale", scale=0.5)


def test_attention_queries_before_the_first_key():
    """q_len longer than the sequence: the first queries see nothing."""
    rng = np.random.default_rng(32)
    r = check_attention(attention_case(rng, [3, 0, 1], 6, 4, 2, 128, 16), 2, 16, "short")
    assert torch.isneginf(r.lse[1]).all() and (r.out[1] == 0).all()
    assert torch.isneginf(r.lse[0, :3]).all()


def test_attention_long_sequence_in_parts():
    """Enough keys to be split over many workgroups, few rows."""
    rng = np.random.default_rng(33)
    check_attention(attention_case(rng, [9001, 4097], 1, 4, 1, 128, 64), 1, 64, "long")


def test_attention_slots_past_the_length_hold_anything():
    """NaN scales and codes past the length and in pages not named."""
    rng = np.random.default_rng(34)
    q, k, v, table, lens = attention_case(rng, [37, 5, 50], 2, 4, 2, 128, 16)
    want = run_attention(q, k, v, table, lens, 2, 16, None, True, 0)
    live = np.zeros(k[0].shape[0], bool)
    for b, n in enumerate(lens):
        t = np.arange(n)
        for h in range(2):
            live[(table[b][t // 16] * 2 + h) * 16 + t % 16] = True
    for a in (k, v):
        a[1][~live] = 0x7F                              # E4M3 NaN
        a[2][~live] = np.nan
    got = run_attention(q, k, v, table, lens, 2, 16, None, True, 0)
    torch.cuda.synchronize()
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)


def test_attention_bad_pages_and_lengths_stay_in_bounds():
    """Pages and lengths out of range are clamped; the well-formed sequence
    beside them keeps its result."""
    rng = np.random.default_rng(35)
    q, k, v, table, lens = attention_case(rng, [40, 40, 40], 1, 4, 2, 64, 16)
    want = run_attention(q, k, v, table, lens, 2, 16, None, True, 0)
    table[1] = [-1, 1 << 40, 10 ** 6][:table.shape[1]]
    lens[2] = 1 << 50
    lens[1] = 33
    got = run_attention(q, k, v, table, lens, 2, 16, None, True, 0)
    torch.cuda.synchronize()
    assert torch.equal(got.out[0], want.out[0])
    lens[2] = -7
    got = run_attention(q, k, v, table, lens, 2, 16, None, True, 0)
    torch.cuda.synchronize()
    assert (got.out[2] == 0).all() and torch.isneginf(got.lse[2]).all()


def test_attention_value_scales_far_apart():
    """Values whose scales differ by 2^24 under scores that favour the small
    ones: the small ones' part keeps its precision."""
    rng = np.random.default_rng(36)
    case = attention_case(rng, [80], 1, 4, 1, 128, 16, spread=0.0)
    s = case[2][2]
    s[:] = np.where(rng.random(s.size) < 0.5, 2.0 ** -24, 1.0).astype(np.float32)
    check_attention(case, 1, 16, "scales apart")
    s[:] = 0.0
    check_attention(case, 1, 16, "zero values")


def test_attention_append_then_read(orc):
    """Keys and values quantized into the cache by the append are what the
    attention reads: the oracle's quantization at the same rows."""
    rng = np.random.default_rng(37)
    B, Hkv, D, page, n = 3, 2, 128, 16, 21
    k = W.bf16_bits(rng.normal(0, 1, (B * n, Hkv, D)))
    v = W.bf16_bits(rng.normal(0, 1, (B * n, Hkv, D)))
    table = rng.permutation(7)[:6].reshape(B, 2).astype(np.int64)
    t = np.tile(np.arange(n), B)
    pages, slots = table[np.repeat(np.arange(B), n), t // page], t % page
    cache = [api.NVFP4(torch.zeros(7 * Hkv * page, D // 2, dtype=torch.uint8, device="cuda"),
                       torch.zeros(7 * Hkv * page, D // 16, dtype=torch.uint8, device="cuda"),
                       torch.zeros(7 * Hkv * page, device="cuda")) for _ in range(2)]
    rows = api.nvfp4_cache_rows(dev(pages), dev(slots), Hkv, page)
    api.nvfp4_cache_append(dev(k), rows, cache[0])
    api.nvfp4_cache_append(dev(v), rows, cache[1])
    q = bf16(rng.normal(0, 1, (B, 1, 6, D)))
    lens = np.full(B, n, np.int64)
    got = api.nvfp4_attention(put(q, torch.bfloat16), *cache, dev(table), dev(lens), Hkv, page)
    torch.cuda.synchronize()
    host_rows = rows.cpu().numpy().reshape(-1)
    for bits, c in ((k, cache[0]), (v, cache[1])):
        want = orc.nvfp4_per_token(bits.reshape(-1, D))
        for w, g in zip(want, c):
            assert np.array_equal(host(g)[host_rows], w)
    args = [tuple(host(a) for a in c) for c in cache]
    again = run_attention(q, *args, table, lens, Hkv, page, None, True, 0)
    assert torch.equal(again.out, got.out)


# ---------------------------------------------------------------------------
# Streams, graphs, repeatability
# ---------------------------------------------------------------------------

def layer_calls(seed=41):
    """One call of every operator, as functions of no arguments."""
    rng = np.random.default_rng(seed)
    T, E, k, H, I = 24, 16, 4, 256, 128
    x = put(bf16(rng.normal(0, 1, (T, H))), torch.bfloat16)
    lg = put(rng.normal(0, 1, (T, E)), torch.float32)
    bias = put(rng.normal(0, 0.1, E), torch.float32)
    pair = api.nvfp4_quantize_gateup_pair(*(dev(W.bf16_bits(rng.normal(0, 0.05, (E, I, H))))
                                            for _ in range(2)))
    dn = api.nvfp4_quantize_gateup_pair(dev(W.bf16_bits(rng.normal(0, 0.05, (E, H, I)))))
    r = api.moe_route(lg, k, bias=bias, scoring=SIGMOID)
    q, kc, vc, table, lens = attention_case(rng, [700, 300], 1, 8, 2, 64, 16)
    q, table, lens = put(q, torch.bfloat16), dev(table), dev(lens)
    kc, vc = api.NVFP4(*(dev(a) for a in kc)), api.NVFP4(*(dev(a) for a in vc))
    dout = put(bf16(rng.normal(0, 1, (T, H))), torch.bfloat16)
    y = put(bf16(rng.normal(0, 1, (T * k, H))), torch.bfloat16)
    torch.cuda.synchronize()
    return [
        lambda: tuple(api.moe_route(lg, k, bias=bias, scoring=SIGMOID)),
        lambda: (api.moe_route_backward(r.weights, lg, r.experts, SIGMOID),),
        lambda: (api.moe_combine(y, r.token_rows, r.weights),),
        lambda: api.moe_combine_backward(dout, y, r.token_rows, r.weights, r.seg_offsets),
        lambda: (api.nvfp4_matvec(x, pair.gate_codes[0], pair.gate_block_scales[0],
                                  pair.scope_scales[:1]),),
        lambda: (api.nvfp4_expert_layer(x, r, pair, dn),),
        lambda: tuple(api.nvfp4_attention(q, kc, vc, table, lens, 2, 16)),
    ]


def test_same_bytes_again_and_on_another_stream():
    for i, f in enumerate(layer_calls()):
        announce(f"repeat call {i}")
        first = f()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            second = f()
        side.synchronize()
        for a, b in zip(first, second):
            assert torch.equal(a, b), i


def test_captured_in_one_graph():
    calls = layer_calls(43)
    want = [f() for f in calls]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [f() for f in calls]
    for rep in range(3):
        announce(f"graph replay {rep}")
        for outs in got:
            for t in outs:
                t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(want, got)):
            for s, t in zip(a, b):
                assert torch.equal(s, t), (rep, i)


def test_api_refuses_wrong_arguments():
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    idx = torch.zeros(4, 2, device="cuda", dtype=torch.int64)
    w = torch.zeros(4, 2, device="cuda")
    with pytest.raises(TypeError):
        api.moe_route(x.to(torch.float16), 2)
    with pytest.raises(ValueError):
        api.moe_route(x.t(), 2)
    with pytest.raises(TypeError):
        api.moe_route(x, 2, bias=torch.zeros(64, device="cuda", dtype=torch.float64))
    with pytest.raises(mxq.MXQError):
        api.moe_route(x, 65)
    with pytest.raises(ValueError):
        api.moe_combine(x, idx, w[:3])
    with pytest.raises(TypeError):
        api.moe_combine(x, idx.int(), w)
    codes = torch.zeros(8, 32, device="cuda", dtype=torch.uint8)
    bs = torch.zeros(8, 4, device="cuda", dtype=torch.uint8)
    one = torch.zeros(1, device="cuda")
    with pytest.raises(ValueError):
        api.nvfp4_matvec(x[:, :32].contiguous(), codes, bs, one)
    with pytest.raises(TypeError):
        api.nvfp4_matvec(x, codes, bs, one, out_dtype=torch.float16)
    with pytest.raises(mxq.MXQError):
        api.nvfp4_matvec(torch.zeros(65, 64, device="cuda"), codes, bs, one)
    q = torch.zeros(1, 1, 2, 64, device="cuda", dtype=torch.bfloat16)
    cache = api.NVFP4(torch.zeros(32, 32, device="cuda", dtype=torch.uint8),
                      torch.zeros(32, 4, device="cuda", dtype=torch.uint8),
                      torch.zeros(32, device="cuda"))
    table, lens = torch.zeros(1, 1, device="cuda", dtype=torch.int64), torch.zeros(
        1, device="cuda", dtype=torch.int64)
    with pytest.raises(ValueError):
        api.nvfp4_attention(q, cache, cache, table, lens, 3, 16)
    with pytest.raises(mxq.MXQError):
        api.nvfp4_attention(q, cache, cache, table, lens, 2, 16, causal=False, window=4)
    with pytest.raises(TypeError):
        api.nvfp4_attention(q.float(), cache, cache, table, lens, 2, 16)


# ---------------------------------------------------------------------------
# The operators together
# ---------------------------------------------------------------------------

def nvfp4_f64(w):
    return R.decode(host(w.codes), host(w.block_scales)) * host(w.fp32_scales)[:, None].astype(
        np.float64)


def test_decode_block_in_a_graph():
    """Steps of the example's block replayed from a graph give the bytes of the
    eager steps of a second block, and each operator's output follows from
    what the step handed to it."""
    from examples.moe_block import DecodeBlock, Shape
    s = Shape(hidden=256, inter=128, experts=12, top_k=3, heads=8, kv_heads=2, head_dim=64, page=16)
    n, context = 3, 30
    announce("decode block")
    eager, block = (DecodeBlock(s, n, context, 48, seed=3) for _ in range(2))
    rng = np.random.default_rng(43)
    xs = [put(bf16(rng.normal(0, 1, (n, s.hidden))), torch.bfloat16) for _ in range(5)]
    x = xs[0].clone()
    block.step(x)
    eager.step(xs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, parts = block.step(x)
    for xi in xs[1:]:
        x.copy_(xi)
        graph.replay()
        want, other = eager.step(xi)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(parts["att"], other["att"])
        assert torch.equal(parts["rows"], other["rows"])
    assert block.lens.tolist() == [context + 5] * n

    kk, vv = (nvfp4_f64(c) for c in block.cache)
    q = parts["q"].cpu().double().numpy()[:, None]
    sc = float(np.float32(s.head_dim ** -0.5))
    want, _, mag, terms = R.attention(q, kk, vv, host(block.table), host(block.lens), s.kv_heads,
                                      s.page, sc, True, 0)
    delta = terms * (s.head_dim + 24) * 2.0 ** -23 + 2.0 ** -20
    tol = mag * (R.HALF_FP16 + 2 * delta[..., None] + (35 / 16 + 64) * 2.0 ** -23)
    close(parts["att"], want, tol + np.abs(want) * R.HALF_BF16 * 1.001, "attention of the step")
    h2 = parts["h2"].cpu().double().numpy()
    w = block.w_router
    want, tol = product(h2, np.ones(n), R.decode(host(w.codes), host(w.block_scales)),
                        np.repeat(host(w.fp32_scales), s.experts).astype(np.float64), 0.0)
    close(parts["logits"], want, tol, "router logits of the step")
    r = parts["routing"]
    _, experts, *_ = R.route(parts["logits"].cpu().double().numpy(), None, params(s.top_k))
    assert np.array_equal(host(r.experts), experts)
    y = api.nvfp4_expert_layer(parts["h2"], r, block.gateup, block.down)
    torch.cuda.synchronize()
    assert torch.equal(y, parts["y"])


def test_train_step():
    """Values that MXFP8 holds exactly: every product of the step is exact, so
    what is left is the BF16 rounding of each result."""
    from examples.moe_block import train_step
    rng = np.random.default_rng(47)
    T, E, K, N, k = 50, 6, 256, 128, 2
    announce("train step")
    x, w, g = (rng.integers(-2, 3, shape).astype(np.float64)
               for shape in ((T, K), (E, N, K), (T, N)))
    z = rng.uniform(-3, 0, (T, E)).astype(np.float32).astype(np.float64)
    pick = np.sort(np.argsort(rng.random((T, E)), 1)[:, :k], 1)
    np.put_along_axis(z, pick, 1.0, 1)                       # two equal experts: weights of 1/2
    s = train_step(put(x, torch.bfloat16), put(z, torch.float32), put(w, torch.bfloat16),
                   put(g, torch.bfloat16), k)
    torch.cuda.synchronize()
    y = bf16(np.einsum("tk,tcnk->tcn", x, w[pick]))
    want = 0.5 * y.sum(1)
    tiny = 2.0 ** -20 * np.abs(y).sum(1)
    close(s.out, want, tiny + np.abs(want) * R.HALF_BF16, "out")
    dx = bf16(np.einsum("tn,tcnk->tck", 0.5 * g, w[pick]))
    close(s.d_tokens, dx.sum(1), np.abs(dx.sum(1)) * R.HALF_BF16 + 2.0 ** -20 * np.abs(dx).sum(1),
          "d_tokens")
    de = np.zeros((E, N, K))
    for t in range(T):
        for e in pick[t]:
            de[e] += np.outer(0.5 * g[t], x[t])
    close(s.d_experts, de, np.zeros(de.shape), "d_experts")
    dw = np.einsum("tn,tcn->tc", g, y)
    # The two weights' fp32 sums, then the router's gradient: test_route_backward's bound.
    dmag = np.einsum("tn,tcn->tc", np.abs(g), np.abs(y))
    want, _ = R.route_backward(dw, z, pick, SOFTMAX, True, 1.0)
    _, mag = R.route_backward(dmag, z, pick, SOFTMAX, True, 1.0)
    close(s.d_logits, want, mag * (2.0 ** -19 + (90 + N) * 2.0 ** -24) + 1e-37, "d_logits")
