"""The layer operators on the GPU at the edges of their ranges, against the
64-bit forms of layer_ref with the tolerances of test_layer_gpu."""
import numpy as np
import pytest
import torch

import layer_ref as R
import nvfp4_block_scaled_amax_amd as mxq
from nvfp4_block_scaled_amax_amd import api
from nvfp4_block_scaled_amax_amd import workloads as W
from gpu_util import announce, dev, require_gpu
from test_layer_gpu import (X_KINDS, activation, attention_case, bf16, check_attention, check_route, close,
                            params, product, put, run_attention, segments)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# ---------------------------------------------------------------------------
# A stream named in the call
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("raw", [False, True])
def test_named_stream_keeps_what_the_call_lets_go(raw):
    """The side stream is busy when the calls return; what the current stream
    allocates and fills meanwhile must not be what they still use."""
    rng = np.random.default_rng(61)
    T, E, k, H, I = 200, 16, 4, 256, 128
    x = put(bf16(rng.normal(0, 1, (T, H))), torch.bfloat16)
    lg = put(rng.normal(0, 1, (T, E)), torch.float32)
    pair = api.nvfp4_quantize_gateup_pair(*(dev(W.bf16_bits(rng.normal(0, 0.05, (E, I, H))))
                                            for _ in range(2)))
    dn = api.nvfp4_quantize_gateup_pair(dev(W.bf16_bits(rng.normal(0, 0.05, (E, H, I)))))
    r = api.moe_route(lg, k)
    q, kc, vc, table, lens = attention_case(rng, [700, 300], 1, 8, 2, 64, 16)
    q, table, lens = put(q, torch.bfloat16), dev(table), dev(lens)
    kc, vc = api.NVFP4(*(dev(a) for a in kc)), api.NVFP4(*(dev(a) for a in vc))
    calls = [lambda s: tuple(api.moe_route(lg, k, stream=s)),
             lambda s: (api.nvfp4_expert_layer(x, r, pair, dn, stream=s),),
             lambda s: tuple(api.nvfp4_attention(q, kc, vc, table, lens, 2, 16, stream=s))]
    side = torch.cuda.Stream()
    for i, f in enumerate(calls):
        announce(f"named stream, call {i}")
        want = f(None)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = f(side.cuda_stream if raw else side)
        # Sizes of the temporaries: the workspaces, and h and y of the expert layer.
        taken = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
                 for n in (mxq.mxq_moe_route_workspace(T, E), T * k * I * 4, T * k * H * 4,
                           mxq.mxq_nvfp4_attention_workspace(2, 1, 8, 2, 64, 704))]
        torch.cuda.synchronize()
        assert all(bool((t == 0x5A).all()) for t in taken), i
        for a, b in zip(want, got):
            assert torch.equal(a, b), i


# ---------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(7, 24, 4), (70, 24, 4), (40, 300, 20)])
def test_a_disabled_expert_stays_in_the_softmax(T, E, k, dtype):
    """The bias moves the selection only: with experts at a bias of -inf (or NaN),
    the likeliest among them, the others keep the scores of the softmax over all
    experts, in the keys and in the weights."""
    announce(f"disabled experts {T}x{E} {dtype}")
    rng = np.random.default_rng(T + E)
    x = rng.normal(0, 1.5, (T, E))
    x[:, 0] += 4.0
    x = bf16(x) if dtype == torch.bfloat16 else x.astype(np.float32).astype(np.float64)
    b = rng.normal(0, 0.05, E).astype(np.float32).astype(np.float64)
    b[::5] = -np.inf
    b[5] = np.nan
    r = api.moe_route(put(x, dtype), k, bias=put(b, torch.float32), renormalize=False)
    torch.cuda.synchronize()
    s = R.scores(x, mxq.MXQ_SCORE_SOFTMAX)
    key = np.where(b > -np.inf, s + np.where(b > -np.inf, b, 0.0), -np.inf)
    want = np.argsort(-key, 1, kind="stable")[:, :k]
    assert np.array_equal(r.experts.cpu().numpy(), want)
    w = np.take_along_axis(s, want, 1)
    got = r.weights.cpu().double().numpy()
    assert (np.abs(got - w) <= w * 2.0 ** -20).all()
    # The function whose gradient moe_route_backward gives.
    assert np.array_equal(w, R.route_weights(x, want, mxq.MXQ_SCORE_SOFTMAX, False, 1.0))


@pytest.mark.parametrize("scoring", [mxq.MXQ_SCORE_SOFTMAX, mxq.MXQ_SCORE_SIGMOID])
@pytest.mark.parametrize("T,E,groups,at", [(32, 128, 64, 1e6), (2000, 128, 64, 4096.0),
                                           (3000, 96, 32, 300.0), (500, 512, 16, 32768.0)])
def test_group_sums_of_keys_that_cancel(T, E, groups, at, scoring):
    """A group's two best keys, large of either sign: their sum is small, but FP32 holds
    each only to 2^-24 of its size."""
    announce(f"group sums {T}x{E} {scoring}")
    rng = np.random.default_rng(T + E)
    x = rng.normal(0, 1.0, (T, E)).astype(np.float32).astype(np.float64)
    per = E // groups
    b = np.where(np.arange(E) % per == 0, at, -at)
    b[np.arange(E) % per > 1] = -np.inf
    # Both experts of the best group: only the sums decide.
    check_route(x, b, params(2, scoring, groups, 1, 2), torch.float32, "group sums")
    check_route(x, b, params(6, scoring, groups, groups // 4, 2), torch.float32, "group sums")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("scoring", [mxq.MXQ_SCORE_SOFTMAX, mxq.MXQ_SCORE_SIGMOID])
@pytest.mark.parametrize("T,E,k", [(200, 60, 30), (40, 640, 50), (3000, 16, 9)])
def test_weights_of_logits_far_apart(T, E, k, scoring, renorm, dtype):
    """Weights keep their 2^-20 where the logits differ by tens, a difference that FP32
    rounds to 2^-19."""
    rng = np.random.default_rng(T + E)
    x = rng.normal(0, 14.0, (T, E))
    x = bf16(x) if dtype == torch.bfloat16 else x.astype(np.float32).astype(np.float64)
    check_route(x, None, params(k, scoring, renorm=renorm, scale=1.5), dtype, "far apart")


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,Q,H,Hkv,D,page", [
    ([3, 0, 1, 40], 6, 4, 2, 128, 16), ([5, 2], 40, 2, 1, 256, 16),
    ([150, 3, 260], 200, 16, 16, 64, 16),                # the kernel for many rows
    ([1500], 1, 8, 2, 64, 32), ([700, 9], 30, 4, 1, 128, 48),
])
def test_attention_window_past_every_key(lens, Q, H, Hkv, D, page):
    """However wide, a window that holds all keys is none, also for queries that
    stand before the first key."""
    rng = np.random.default_rng(sum(lens) + Q)
    case = attention_case(rng, lens, Q, H, Hkv, D, page)
    want = check_attention(case, Hkv, page, "no window")
    for window in (max(lens) + Q, (1 << 30) + 5, (1 << 31) - 2, (1 << 31) - 1, 1 << 31, 1 << 62,
                   (1 << 63) - 1):
        got = run_attention(*case, Hkv, page, None, True, window)
        torch.cuda.synchronize()
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse), window


@pytest.mark.parametrize("n,Q,H,Hkv,D,page", [
    (140000, 1, 4, 1, 128, 64), (140001, 1, 2, 1, 64, 128), (150000, 2, 1, 1, 256, 16),
    (140000, 100, 64, 1, 64, 64),                        # the kernel for many rows
    (33000, 5, 40, 8, 128, 64),
])
@pytest.mark.parametrize("values", ["none", "last", "tiny", "huge"])
def test_attention_sum_over_many_keys_of_small_or_no_values(n, Q, H, Hkv, D, page, values):
    """Equal scores: lse is the log of the number of keys seen and out the values' mean,
    also where values are zeros (all of them, or all but the last thousand) or have scales
    at either end of their range."""
    announce(f"attention sums n={n} Q={Q} H={H} D={D} {values}")
    rng = np.random.default_rng(n + D)
    pages = -(-n // page)
    rows = pages * Hkv * page
    k = (np.zeros((rows, D // 2), np.uint8), np.zeros((rows, D // 16), np.uint8),
         np.zeros(rows, np.float32))
    codes, blocks, _ = R.random_nvfp4(rng, 1024, D)
    at = np.arange(rows) % 1021
    v = [codes[at], blocks[at], np.zeros(rows, np.float32)]
    t = (np.arange(rows) // (page * Hkv)) * page + np.arange(rows) % page
    scale = {"none": 0.0, "last": 2.0 ** -10, "tiny": 2.0 ** -100, "huge": 2.0 ** 100}[values]
    v[2][(t >= n - 1000) | (values == "tiny")] = scale
    q = bf16(rng.normal(0, 1, (1, Q, H, D)))
    r = run_attention(q, k, v, np.arange(pages)[None], np.array([n]), Hkv, page, None, True, 0)
    torch.cuda.synchronize()
    seen = n - Q + 1 + np.arange(Q)
    terms = (seen.max() / 16 + 64) * 2.0 ** -23          # one rounding per 16 keys and join
    lse = r.lse.cpu().double().numpy()[0]
    assert np.isfinite(lse).all()
    assert (np.abs(lse - np.log(seen)[:, None]) <= terms + 2.0 ** -17).all()
    got = r.out.cpu().double().numpy()[0].reshape(Q, Hkv, H // Hkv, D)
    table = R.decode(codes, blocks)
    for h in range(Hkv):
        sel = (np.arange(n) // page * Hkv + h) * page + np.arange(n) % page
        vals = table[at[sel]] * v[2][sel, None].astype(np.float64)
        total, mag = np.cumsum(vals, 0)[seen - 1], np.cumsum(np.abs(vals), 0)[seen - 1]
        want, mag = total / seen[:, None], mag / seen[:, None]
        tol = mag * (R.HALF_FP16 + 2 * terms) + np.abs(want) * R.HALF_BF16 * 1.001
        assert (np.abs(got[:, h] - want[:, None]) <= tol[:, None]).all(), h


# ---------------------------------------------------------------------------
# The router's gradient where scores are near 0 or 1
# ---------------------------------------------------------------------------

def log_sigmoid(x):
    return -np.logaddexp(0.0, -x)


def renormalized_gradient(dw, x, experts, scoring):
    """d_logits of weights s_i / sum of the selected s, from the logarithms of the
    scores, and the sum of its terms' magnitudes."""
    live = experts >= 0
    xc = np.where(live, np.take_along_axis(x, np.maximum(experts, 0), 1), -np.inf)
    ls = np.where(live, log_sigmoid(np.where(live, xc, 0.0)) if scoring else xc, -np.inf)
    top = ls.max(1, keepdims=True)
    w = np.exp(ls - np.where(top > -np.inf, top, 0.0))
    w /= np.maximum(w.sum(1, keepdims=True), 1e-300)
    g = np.where(live, dw, 0.0)
    diff = g[:, :, None] - g[:, None, :]
    down = np.exp(log_sigmoid(-np.where(live, xc, 0.0))) if scoring else 1.0
    out, mag = np.zeros_like(x), np.zeros_like(x)
    for a, d in ((out, diff), (mag, np.abs(diff))):
        v = w * (d * w[:, None, :]).sum(2) * down
        t, c = np.nonzero(live)
        a[t, experts[t, c]] = v[t, c]
    return out, mag


def check_gradient(x, experts, dw, scoring, renorm, want, mag, name):
    """Scores within 2^-19, one rounding of each term and sum, at most 20 terms."""
    announce(f"gradient {name} {x.shape}")
    d = api.moe_route_backward(put(dw, torch.float32), put(x, torch.float32),
                               put(experts, torch.int64), scoring, renorm)
    torch.cuda.synchronize()
    got = d.cpu().double().numpy()
    bad = np.argwhere(~(np.abs(got - want) <= mag * (2.0 ** -17 + 25 * 2.0 ** -24) + 1e-37))
    assert bad.size == 0, (name, len(bad), tuple(bad[0]), got[tuple(bad[0])], want[tuple(bad[0])])


SMALL = {
    "sigmoids of -95": (mxq.MXQ_SCORE_SIGMOID, -95.0, 4.0),
    "sigmoids of -1000": (mxq.MXQ_SCORE_SIGMOID, -1000.0, 4.0),
    "sigmoids about 0": (mxq.MXQ_SCORE_SIGMOID, 0.0, 3.0),
    "sigmoids of 25": (mxq.MXQ_SCORE_SIGMOID, 25.0, 6.0),
    "softmax 100 below the largest": (mxq.MXQ_SCORE_SOFTMAX, -100.0, 3.0),
    "softmax 1e4 below the largest": (mxq.MXQ_SCORE_SOFTMAX, -1e4, 3.0),
}


@pytest.mark.parametrize("name", SMALL)
@pytest.mark.parametrize("T,E,k", [(33, 20, 6), (9, 300, 20)])
def test_gradient_of_renormalized_small_scores(T, E, k, name):
    """The weights depend on the scores' ratios alone, and so does their gradient,
    however small the selected scores: with an expert disabled that has nearly all
    of the softmax, or sigmoids below FP32's range."""
    scoring, at, spread = SMALL[name]
    rng = np.random.default_rng(E)
    x = rng.normal(at, spread, (T, E)).astype(np.float32).astype(np.float64)
    x[:, 3] = 2.0                                        # disabled by the bias
    x[0, 5:] = -np.inf
    b = np.zeros(E, np.float32)
    b[3] = -np.inf
    xt = put(x, torch.float32)
    r = api.moe_route(xt, k, bias=put(b, torch.float32), scoring=scoring, scale=1.0)
    experts = r.experts.cpu().numpy()
    assert not (experts == 3).any()
    dw = rng.normal(0, 1, (T, k)).astype(np.float32).astype(np.float64)
    want, mag = renormalized_gradient(dw, x, experts, scoring)
    check_gradient(x, experts, dw, scoring, True, want, mag, name)


@pytest.mark.parametrize("T,E,k", [(40, 16, 5), (9, 300, 20), (3, 1024, 64)])
def test_gradient_of_scores_near_one(T, E, k):
    """Sigmoids to either side of 1 - 2^-24, and a softmax that one selected expert
    has nearly all of: 1 - s is what the gradient is made of."""
    rng = np.random.default_rng(T + E)
    experts = np.argsort(rng.random((T, E)), 1)[:, :k]
    experts[:, -1] = -1
    dw = rng.normal(0, 1, (T, k)).astype(np.float32).astype(np.float64)
    g = np.zeros((T, E))
    np.put_along_axis(g, experts[:, :-1], dw[:, :-1], 1)

    x = rng.uniform(-30, 60, (T, E)).astype(np.float32).astype(np.float64)
    want = g * np.exp(log_sigmoid(x) + log_sigmoid(-x))
    check_gradient(x, experts, dw, mxq.MXQ_SCORE_SIGMOID, False, want, np.abs(want), "sigmoids")

    # The first choice has all but about e^-a of the softmax.
    x = rng.normal(0, 1, (T, E))
    np.put_along_axis(x, experts[:, :1], rng.uniform(10, 40, (T, 1)), 1)
    x = x.astype(np.float32).astype(np.float64)
    s = np.exp(x - x.max(1, keepdims=True))
    s /= s.sum(1, keepdims=True)
    selected = np.zeros((T, E), bool)
    np.put_along_axis(selected, experts[:, :-1], True, 1)
    # sum_j ds_j s_j over all experts: dx_e = s_e sum_j (ds_e - ds_j) s_j, term by term.
    diff = g[:, :, None] - g[:, None, :]
    want, mag = (s * (d * s[:, None, :]).sum(2) for d in (diff, np.abs(diff)))
    check_gradient(x, experts, dw, mxq.MXQ_SCORE_SOFTMAX, False, want, mag, "softmax")


# ---------------------------------------------------------------------------
# Few-row products of many weights: wavefronts that take whole tiles of 16
# weight rows, from 2048 tiles on
# ---------------------------------------------------------------------------

def tiles(n):
    return -(-n // 16)


@pytest.mark.parametrize("kind", X_KINDS)
@pytest.mark.parametrize("M,N,K", [
    (1, 32777, 64), (13, 32790, 192), (16, 32768, 128), (17, 33001, 320), (64, 32801, 704),
    (33, 40007, 576), (1, 65551, 448), (24, 32769, 2112), (17, 32785, 2048), (5, 32783, 6208),
])
def test_matvec_of_many_weights(M, N, K, kind):
    """Ends of K inside a unit of 128 and a block of 512, of N inside a tile and a round
    of the wavefronts; one and two groups of 16 rows, one and several passes."""
    assert tiles(N) >= 2048
    announce(f"matvec {M}x{N}x{K} {kind}")
    rng = np.random.default_rng(M + N + K)
    x, xv, sx, held = activation(rng, M, K, kind)
    c, b, _ = R.random_nvfp4(rng, N, K)
    c[-1], b[-1] = c[0], b[0]
    w = R.decode(c, b)
    for rpb, out in ((N, torch.bfloat16), (16, torch.float32)):
        s = np.exp2(rng.uniform(-9, -3, -(-N // rpb))).astype(np.float32)
        want, tol = product(xv, sx, w, np.repeat(s, rpb)[:N].astype(np.float64), held)
        got = api.nvfp4_matvec(x, dev(c), dev(b), dev(s), rpb, out)
        torch.cuda.synchronize()
        close(got, want, tol + (np.abs(want) * R.HALF_BF16 * 1.001
                                if out == torch.bfloat16 else 0), f"matvec {rpb} {out}")


@pytest.mark.parametrize("kind", X_KINDS)
@pytest.mark.parametrize("G,rows,N,K", [
    (128, 200, 257, 192), (70, 90, 480, 320), (64, 300, 1000, 704), (40, 41, 830, 64),
    (16, 600, 2050, 128), (130, 1000, 250, 64), (24, 50, 1370, 1088),
])
def test_experts_of_many_weights(G, rows, N, K, kind):
    """The same per expert, alone and as the gated pair, with segments larger than the
    rows staged at once."""
    assert min(G, rows) * tiles(N) >= 2048
    announce(f"experts {G} {rows}x{N}x{K} {kind}")
    rng = np.random.default_rng(G + rows + N)
    seg = segments(rng, G, rows)
    T = max(1, rows // 3)
    rt = rng.integers(0, T, rows)
    rt[0] = -1
    x, xv, sx, held = activation(rng, rows, K, kind)
    xt, xtv, sxt, _ = activation(rng, T, K, kind)
    (gc, gb, s), (uc, ub, _) = (R.random_nvfp4(rng, G * N, K) for _ in range(2))
    s = (s[:G] * 2.0 ** -6).astype(np.float32)
    gd, gbd, ud, ubd = (dev(a.reshape(G, N, -1)) for a in (gc, gb, uc, ub))
    got = torch.full((rows, N), 5.0, device="cuda")
    args = (x.codes, x.block_scales, x.fp32_scales) if kind == "nvfp4" else (x, None, None)
    mxq.mxq_nvfp4_expert_matvec(X_KINDS.index(kind), *args, gd, gbd, dev(s), dev(seg), G, rows, N,
                                K, mxq.MXQ_OUT_F32, got)
    h = api.nvfp4_expert_gateup(xt, api.GateUpNVFP4(gd, gbd, ud, ubd, dev(s)), dev(rt), dev(seg),
                                torch.float32)
    torch.cuda.synchronize()
    assert (got[seg[-1]:] == 5.0).all()
    for e in range(G):
        a, z = seg[e], seg[e + 1]
        if z == a:
            continue
        at = slice(e * N, (e + 1) * N)
        wg, wu, sc = R.decode(gc[at], gb[at]), R.decode(uc[at], ub[at]), np.full(N, float(s[e]))
        want, tol = product(xv[a:z], sx[a:z], wg, sc, held)
        close(got[a:z], want, tol, f"expert {e}")
        t = np.maximum(rt[a:z], 0)
        (g, tg), (u, tu) = (product(xtv[t], sxt[t], w, sc, held) for w in (wg, wu))
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        # |silu'| <= 1.1; silu itself within 2^-20.
        tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(silu) * tu + np.abs(silu * u) * 2.0 ** -20
        close(h[a:z], silu * u, tol + 1e-36, f"gated pair of expert {e}")


@pytest.mark.parametrize("kind", X_KINDS)
@pytest.mark.parametrize("at", [-112, 112])
@pytest.mark.parametrize("G,rows,N,K", [(3, 9, 40, 192), (128, 200, 257, 192)])
def test_products_of_scales_far_apart(G, rows, N, K, at, kind):
    """Activations about 2^at under weights about 2^-at: results about 1, whatever a part
    of the product alone would be."""
    announce(f"scales far apart {G} {rows}x{N}x{K} {kind} 2^{at}")
    rng = np.random.default_rng(G + rows)
    if kind == "nvfp4":
        c, b, _ = R.random_nvfp4(rng, rows, K)
        sx = np.exp2(at + rng.uniform(-12, -4, rows)).astype(np.float32)
        x, xv, sx, held = api.NVFP4(dev(c), dev(b), dev(sx)), R.decode(c, b), sx.astype(np.float64), 0.0
    else:
        xv = bf16(rng.normal(0, 1, (rows, K)) * 2.0 ** at)
        x = put(xv, torch.bfloat16 if kind == "bf16" else torch.float32)
        sx, held = np.ones(rows), R.HALF_FP16 if kind == "f32" else 0.0
    gc, gb, _ = R.random_nvfp4(rng, G * N, K)
    s = np.exp2(-at + rng.uniform(-14, -9, G)).astype(np.float32)
    seg = segments(rng, G, rows)
    gd, gbd = (dev(a.reshape(G, N, -1)) for a in (gc, gb))
    rt = np.arange(rows)
    y = api.nvfp4_expert_matvec(x, gd, gbd, dev(s), dev(seg), torch.float32)
    h = api.nvfp4_expert_gateup(x, api.GateUpNVFP4(gd, gbd, gd, gbd, dev(s)), dev(rt), dev(seg),
                                torch.float32)
    m = min(rows, 64)
    few = (api.NVFP4(*(t[:m] for t in x)) if kind == "nvfp4" else x[:m])
    e0 = int(np.argmax(np.diff(seg)))
    dense = api.nvfp4_matvec(few, gd[e0], gbd[e0], dev(s[e0:e0 + 1].copy()), None, torch.float32)
    torch.cuda.synchronize()
    for e in range(G):
        a, z = seg[e], seg[e + 1]
        if z == a:
            continue
        w, sc = R.decode(gc[e * N:(e + 1) * N], gb[e * N:(e + 1) * N]), np.full(N, float(s[e]))
        want, tol = product(xv[a:z], sx[a:z], w, sc, held)
        close(y[a:z], want, tol, f"expert {e}")
        with np.errstate(over="ignore"):
            silu = want / (1 + np.exp(-want))
        close(h[a:z], silu * want, 1.1 * tol * (np.abs(want) + tol) + np.abs(silu) * tol
              + np.abs(silu * want) * 2.0 ** -20 + 1e-36, f"gated pair of expert {e}")
        if e == e0:
            close(dense, *product(xv[:m], sx[:m], w, sc, held), "dense")


# ---------------------------------------------------------------------------
# Attention over long walks and large batches
# ---------------------------------------------------------------------------

def shared_pages_case(rng, lens, Q, H, Hkv, D, page, n_pages):
    """As attention_case, the sequences' tables drawn from the same few pages."""
    per = max(1, max(-(-n // page) for n in lens))
    table = rng.integers(0, n_pages, (len(lens), per))
    rows = n_pages * Hkv * page
    k, v = (R.random_nvfp4(rng, rows, D, zero_rows=0.05) for _ in "kv")
    q = bf16(rng.normal(0, 1, (len(lens), Q, H, D)) * 0.25)
    return q, k, v, table, np.array(lens, np.int64)


@pytest.mark.parametrize("lens,Q,H,Hkv,D,page,causal,window", [
    ([17000] + [40, 0, 300] * 53, 1, 8, 4, 64, 16, True, 0),
    ([9000, 8200] + [7] * 159, 1, 4, 4, 128, 48, True, 8500),
    ([8500] + [33] * 29, 33, 16, 16, 64, 16, True, 0),   # the kernel for many rows
    ([100] * 15 + [17000] + [64] * 14, 33, 16, 16, 64, 64, False, 0),
])
def test_attention_walks_past_a_window_of_pages(lens, Q, H, Hkv, D, page, causal, window):
    """One workgroup per sequence and head, whose wavefronts look pages up 64 tiles at a
    time: sequences of 8192 keys and more need a second look-up, and a third."""
    rng = np.random.default_rng(max(lens) + D)
    check_attention(shared_pages_case(rng, lens, Q, H, Hkv, D, page, 200), Hkv, page, "long walk",
                    causal=causal, window=window)


@pytest.mark.parametrize("B,Q,H,Hkv,D", [(65, 1, 4, 2, 128), (130, 1, 6, 1, 64), (200, 3, 2, 1, 256),
                                         (70, 40, 3, 3, 64)])
def test_attention_parts_of_more_than_64_sequences(B, Q, H, Hkv, D):
    """The plan's prefix sums over the sequences in more than one round, with empty
    sequences and long ones in every round."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in np.exp2(rng.uniform(0, 11, B))]
    lens[3] = lens[B - 1] = 0
    lens[64] = 4000
    check_attention(shared_pages_case(rng, lens, Q, H, Hkv, D, 32, 300), Hkv, 32, "large batch")


@pytest.mark.parametrize("lens,Q,H,Hkv,D,page,window", [
    ([200, 77, 34], 1, 8, 2, 128, 16, 20), ([333, 40], 3, 4, 2, 64, 16, 7),
    ([150], 30, 4, 1, 256, 48, 50), ([500, 260], 100, 32, 32, 64, 32, 33),
])
def test_attention_slots_before_the_window_hold_anything(lens, Q, H, Hkv, D, page, window):
    """Keys that no query sees, in the tile where the window begins, do not reach
    the result, NaN and infinite scales included."""
    rng = np.random.default_rng(window)
    q, k, v, table, lens = case = attention_case(rng, lens, Q, H, Hkv, D, page)
    want = check_attention(case, Hkv, page, "window", window=window)
    seen = np.zeros(k[0].shape[0], bool)
    for b, n in enumerate(lens):
        t = np.arange(max(0, n - Q - window + 1), n)
        for h in range(Hkv):
            seen[(table[b][t // page] * Hkv + h) * page + t % page] = True
    for bad in (np.nan, np.inf):
        for c, bs, s in (k, v):
            c[~seen], bs[~seen], s[~seen] = 0xFF, 0x7F, bad
        got = run_attention(*case, Hkv, page, None, True, window)
        torch.cuda.synchronize()
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse), bad


# ---------------------------------------------------------------------------
# Offsets past 32 bits: what a call uses stands at the end of large buffers,
# whose other bytes hold anything
# ---------------------------------------------------------------------------

def at_the_end(t, rows):
    """A tensor of `rows` rows that ends in t's."""
    big = torch.empty((rows, *t.shape[1:]), dtype=t.dtype, device="cuda")
    big[rows - t.shape[0]:] = t
    return big


def test_far_rows_of_the_router():
    announce("far rows: router")
    rng = np.random.default_rng(71)
    x = put(bf16(rng.normal(0, 1.5, (70, 1024))), torch.bfloat16)
    T = (1 << 22) + 70                                   # more than 2^32 logits
    big = at_the_end(x, T)
    want, got = (api.moe_route(t, 4, maps=False) for t in (x, big))
    dw = put(rng.normal(0, 1, (70, 4)), torch.float32)
    dx = api.moe_route_backward(dw, x, want.experts, renormalize=False)
    dbig = api.moe_route_backward(at_the_end(dw, T), big, got.experts, renormalize=False)
    torch.cuda.synchronize()
    assert torch.equal(got.experts[-70:], want.experts)
    assert torch.equal(got.weights[-70:], want.weights) and torch.equal(dbig[-70:], dx)


def test_far_rows_of_the_combine():
    announce("far rows: combine")
    rng = np.random.default_rng(72)
    T, k, cols, R_rows = 9, 3, 2056, (1 << 21) + 77      # more than 2^32 elements
    rows = put(bf16(rng.normal(0, 1, (T * k, cols))), torch.bfloat16)
    tr = torch.from_numpy(rng.permutation(T * k).reshape(T, k)).cuda()
    w, d = put(rng.random((T, k)), torch.float32), put(bf16(rng.normal(0, 1, (T, cols))), torch.bfloat16)
    big, far = at_the_end(rows, R_rows), tr + (R_rows - T * k)
    out = [api.moe_combine(*a) for a in ((rows, tr, w), (big, far, w))]
    back = [api.moe_combine_backward(d, *a) for a in ((rows, tr, w), (big, far, w))]
    torch.cuda.synchronize()
    assert torch.equal(*out) and torch.equal(back[0][1], back[1][1])
    assert torch.equal(back[1][0][-T * k:], back[0][0])


@pytest.mark.parametrize("N,K", [((1 << 24) - 5, 576)])
def test_far_rows_of_a_dense_weight(N, K):
    announce("far rows: dense weight")
    rng = np.random.default_rng(73)
    x, xv, sx, held = activation(rng, 5, K, "bf16")
    c, b, _ = R.random_nvfp4(rng, 100, K)
    s = torch.full((1,), 2.0 ** -8, device="cuda")
    got = api.nvfp4_matvec(x, at_the_end(dev(c), N), at_the_end(dev(b), N), s, None, torch.float32)
    torch.cuda.synchronize()
    want, tol = product(xv, sx, R.decode(c, b), np.full(100, 2.0 ** -8), held)
    close(got[:, -100:], want, tol, "dense")


def test_far_rows_of_the_experts():
    announce("far rows: experts")
    rng = np.random.default_rng(74)
    G, N, K, rows = 64, 32768, 4160, 7                   # 4.4 GB of codes
    x, xv, sx, held = activation(rng, rows, K, "bf16")
    c, b, _ = R.random_nvfp4(rng, 50, K)
    s = torch.full((G,), 2.0 ** -8, device="cuda")
    seg = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
    seg[-1] = rows
    codes, blocks = (at_the_end(dev(a), G * N).view(G, N, -1) for a in (c, b))
    y = api.nvfp4_expert_matvec(x, codes, blocks, s, seg)
    h = api.nvfp4_expert_gateup(x, api.GateUpNVFP4(codes, blocks, codes, blocks, s),
                                torch.arange(rows, device="cuda"), seg)
    torch.cuda.synchronize()
    want, tol = product(xv, sx, R.decode(c, b), np.full(50, 2.0 ** -8), held)
    close(y[:, -50:], want, tol, "experts")
    with np.errstate(over="ignore"):
        silu = want / (1 + np.exp(-want))
    close(h[:, -50:], silu * want, 1.1 * tol * (np.abs(want) + tol) + np.abs(silu) * tol
          + np.abs(silu * want) * 2.0 ** -20 + 1e-36, "gated pair")


@pytest.mark.parametrize("lens,Q,H,Hkv,D", [([700, 45], 1, 8, 2, 128), ([300, 201], 200, 16, 16, 64),
                                            ([90], 3, 4, 2, 256)])
def test_far_pages_of_a_cache(lens, Q, H, Hkv, D):
    announce(f"far pages: attention D={D}")
    rng = np.random.default_rng(75)
    page = 32
    q, k, v, table, lens = case = attention_case(rng, lens, Q, H, Hkv, D, page)
    want = run_attention(*case, Hkv, page, None, True, 0)
    near = k[0].shape[0]
    rows = near + (1 << 33) // D // (Hkv * page) * (Hkv * page)      # 4.3 GB of codes before them
    far = [api.NVFP4(*(at_the_end(dev(a), rows) for a in c)) for c in (k, v)]
    got = api.nvfp4_attention(put(q, torch.bfloat16), *far, dev(table + (rows - near) // (Hkv * page)),
                              dev(lens), Hkv, page)
    torch.cuda.synchronize()
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
