"""The expert layer's and the rollout decode step's operators as workloads: routing tokens to
experts, returning expert rows to tokens, products of few tokens with NVFP4 weights (dense and
per expert) and attention over a cache of NVFP4 keys and values.

Each operator has its plain form (elementary torch operations in 32 bits, 64 where a choice hangs on
it), the library's form (``own``), and its definition in 64 bits (``exact``).
"""
import math

import torch

own = False

DEV = "cuda"
NEG_INF = float("-inf")
SOFTMAX, SIGMOID = 0, 1


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # One decode step's tokens through a router of many experts with a balance bias, in groups.
        dict(name="route_decode", op="route", tokens=7, experts=256, top_k=8, scoring=SIGMOID,
             bias=True, groups=8, topk_groups=4, group_topk=2, renorm=True, scale=2.5,
             logits="float32", pad=0),
        # A training batch routed top-8 of 128 (the dispatch workload's sizes), BF16 logits.
        dict(name="route_train", op="route", tokens=32768, experts=128, top_k=8, scoring=SOFTMAX,
             bias=False, groups=1, topk_groups=1, group_topk=1, renorm=True, scale=1.0,
             logits="bfloat16", pad=0),
        # The router's gradient of a ragged batch with padding tokens, sigmoid scores.
        dict(name="route_backward", op="route_backward", tokens=20011, experts=160, top_k=6,
             scoring=SIGMOID, bias=True, groups=1, topk_groups=1, group_topk=1, renorm=True,
             scale=1.0, logits="float32", pad=37),
        # The expert rows of a training batch back to its tokens.
        dict(name="combine_train", op="combine", tokens=32768, cols=2048, top_k=8, drop=0.0,
             dtype="bfloat16"),
        # Its gradient, with some copies dropped by a capacity limit.
        dict(name="combine_backward", op="combine_backward", tokens=9001, cols=2048, top_k=8,
             drop=0.05, dtype="bfloat16"),
        # One token through a projection of the layer: the smallest call, latency.
        dict(name="matvec_one", op="matvec", m=1, n=2048, k=2048, x="bfloat16"),
        # A decode batch, quantized per token, through a vocabulary-sized weight (odd sizes).
        dict(name="matvec_batch", op="matvec", m=13, n=128257, k=2048, x="nvfp4"),
        # One token through its 8 of 128 experts (gate, up, down, weighted return).
        dict(name="experts_one", op="experts", tokens=1, experts=128, top_k=8, hidden=2048,
             inter=768),
        # A decode batch through the same experts: nearly every expert is read.
        dict(name="experts_batch", op="experts", tokens=48, experts=128, top_k=8, hidden=2048,
             inter=768),
        # The first steps of a short sequence.
        dict(name="attention_short", op="attention", seqs=1, q_len=1, heads=32, kv_heads=4,
             head_dim=128, min_len=131, max_len=131, page=16, window=0),
        # A decode batch over ragged caches, the long ones tens of thousands of tokens.
        dict(name="attention_decode", op="attention", seqs=32, q_len=1, heads=32, kv_heads=4,
             head_dim=128, min_len=1000, max_len=32768, page=64, window=0),
        # A chunk of a prompt over the cache it extends (causal).
        dict(name="attention_chunk", op="attention", seqs=3, q_len=509, heads=16, kv_heads=2,
             head_dim=64, min_len=2000, max_len=8192, page=32, window=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine", "combine_backward", "matvec",
                     "experts", "attention"])
    if op in ("route", "route_backward"):
        per_group = rng.choice([4, 5, 8, 12, 16, 32])
        groups = rng.choice([1, 1, 2, 4, 8])
        if groups == 1:
            per_group = rng.choice([8, 20, 60, 64, 72, 128, 160, 200, 256])
        experts = groups * per_group
        topk_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(10, topk_groups * per_group))
        tokens = _log_int(rng, 1, 32768)
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k,
                    scoring=rng.choice([SOFTMAX, SIGMOID]), bias=rng.random() < 0.5,
                    groups=groups, topk_groups=topk_groups, group_topk=rng.randint(1, 2),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    logits=rng.choice(["float32", "bfloat16"]),
                    pad=rng.randint(0, tokens // 4) if rng.random() < 0.5 else 0)
    if op in ("combine", "combine_backward"):
        cols = rng.choice([96, 200, 768, 1024, 2048, 2880, 4096])
        tokens = _log_int(rng, 1, 32768 if op == "combine" else 9000)
        return dict(op=op, tokens=min(tokens, 32768 * 2048 // cols), cols=cols,
                    top_k=rng.randint(1, 8), drop=rng.choice([0.0, 0.1]),
                    dtype=rng.choice(["bfloat16", "float32"]) if cols <= 1024 else "bfloat16")
    if op == "matvec":
        return dict(op=op, m=_log_int(rng, 1, 64), n=_log_int(rng, 40, 50000),
                    k=64 * _log_int(rng, 2, 128), x=rng.choice(["bfloat16", "nvfp4"]))
    if op == "experts":
        return dict(op=op, tokens=_log_int(rng, 1, 48), experts=rng.choice([8, 32, 60, 128]),
                    top_k=rng.randint(1, 8), hidden=rng.choice([512, 1024, 2048]),
                    inter=64 * rng.randint(3, 16))
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 5, 8])
    head_dim = rng.choice([64, 128, 256])
    q_len = rng.choice([1, 1, 1, 2, 5, 33, 200])
    seqs = _log_int(rng, 1, 40) if q_len <= 5 else rng.randint(1, 4)
    max_len = _log_int(rng, q_len + 1, 20000 if q_len <= 5 else 4000)
    max_len = max(q_len, min(max_len, 600000 * 4 * 128 // (seqs * kv_heads * head_dim)))
    return dict(op=op, seqs=seqs, q_len=q_len, heads=kv_heads * group, kv_heads=kv_heads,
                head_dim=head_dim, min_len=rng.randint(q_len, max_len), max_len=max_len,
                page=rng.choice([16, 32, 48, 64, 128]),
                window=rng.choice([0, 0, rng.randint(1, 1500)]))


# ---------------------------------------------------------------------------------------------
# NVFP4 operands (what a user's quantizer has stored)
# ---------------------------------------------------------------------------------------------

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_MIDPOINTS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _quantize(x, scale):
    """x [rows][cols] and one FP32 scale per row -> codes [rows][cols/2], block scales
    [rows][cols/16] (E4M3 bytes)."""
    rows, cols = x.shape
    b = x.float().view(rows, cols // 16, 16)
    s = scale.view(rows, 1)
    safe = torch.where(s > 0, s, torch.ones_like(s))
    bs = (b.abs().amax(2) / (6.0 * safe)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = bs.float() * s
    q = b / torch.where(d > 0, d, torch.ones_like(d)).unsqueeze(2)
    code = torch.bucketize(q.abs(), torch.tensor(_MIDPOINTS, device=x.device)).to(torch.uint8)
    code |= (q < 0).to(torch.uint8) << 3
    code *= (d > 0).to(torch.uint8).unsqueeze(2)
    code = code.view(rows, cols)
    return code[:, 0::2] | (code[:, 1::2] << 4), bs.view(torch.uint8)


def _quantize_rows(x):
    """Per-token NVFP4: one FP32 scale per row."""
    s = x.float().abs().amax(1) / 2688.0
    codes, bs = _quantize(x, s)
    return codes, bs, s


def _quantize_weight(x, x2=None):
    """One FP32 scale over a whole tensor (or a pair of them)."""
    a = x.float().abs().amax()
    if x2 is not None:
        a = torch.maximum(a, x2.float().abs().amax())
    s = a / 2688.0
    out = _quantize(x, s.expand(x.shape[0]))
    if x2 is None:
        return out, s
    return out, _quantize(x2, s.expand(x2.shape[0])), s


def _decode(codes, bs):
    """Values of codes under their block scales (without the FP32 scale), 32 bits."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), dim=-1)
    v = table[pair.long()].flatten(-2)
    d = bs.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, 16)) * d.unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def _logits(case, g):
    """Router logits: experts of unequal popularity; padding tokens are masked whole."""
    T, E = case["tokens"], case["experts"]
    x = 1.3 * _randn(g, T, E) + 0.5 * _randn(g, E)
    x = x.to(getattr(torch, case["logits"]))
    if case["pad"]:
        x[T - case["pad"]:] = NEG_INF
    bias = 0.05 * _randn(g, E) if case["bias"] else None
    return x, bias


def _random_maps(g, tokens, experts, top_k, drop):
    """Random distinct experts per token, as the rows of the expert-sorted layout."""
    choice = _rand(g, tokens, experts).argsort(1)[:, :top_k]
    if drop:
        choice = torch.where(_rand(g, tokens, top_k) < drop, -1, choice)
    w = _rand(g, tokens, top_k) + 0.05
    w = torch.where(choice < 0, 0.0, w / w.sum(1, keepdim=True))
    return (w, choice) + _maps(choice, experts)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = dict(case=case, op=op)
    if op in ("route", "route_backward"):
        st["logits"], st["bias"] = _logits(case, g)
        if op == "route_backward":
            T, k = case["tokens"], case["top_k"]
            st["d_weights"] = _randn(g, T, k)
            st["experts"] = _select(st["logits"], st["bias"], case)
    elif op in ("combine", "combine_backward"):
        T, C, k = case["tokens"], case["cols"], case["top_k"]
        dt = getattr(torch, case["dtype"])
        st["weights"], _, st["token_rows"], _, st["seg_offsets"] = _random_maps(
            g, T, 128, k, case["drop"])
        rows = torch.empty(T * k, C, dtype=dt, device=DEV)
        for r in rows.split(65536):
            r.copy_(_randn(g, *r.shape))
        st["rows"] = rows
        if op == "combine_backward":
            st["d_out"] = _randn(g, T, C).to(dt)
    elif op == "matvec":
        M, N, K = case["m"], case["n"], case["k"]
        w = 0.02 * _randn(g, N, K)
        (st["codes"], st["block_scales"]), s = _quantize_weight(w.to(torch.bfloat16))
        st["scale"] = s.view(1)
        x = _randn(g, M, K).to(torch.bfloat16)
        st["x"] = x if case["x"] == "bfloat16" else _quantize_rows(x)
    elif op == "experts":
        T, E, H, I = case["tokens"], case["experts"], case["hidden"], case["inter"]
        st["x"] = _randn(g, T, H).to(torch.bfloat16)
        (st["weights"], st["experts"], st["token_rows"], st["row_tokens"],
         st["seg_offsets"]) = _random_maps(g, T, E, min(case["top_k"], E), 0.0)
        gate, up, down, scales = [], [], [], []
        for _ in range(E):
            a, b, s = _quantize_weight((0.02 * _randn(g, I, H)).to(torch.bfloat16),
                                       (0.02 * _randn(g, I, H)).to(torch.bfloat16))
            c, t = _quantize_weight((0.02 * _randn(g, H, I)).to(torch.bfloat16))
            gate.append(a), up.append(b), down.append(c), scales.append((s, t))
        for name, part in (("gate", gate), ("up", up), ("down", down)):
            st[name] = tuple(torch.stack([p[i] for p in part]) for i in range(2))
        st["gateup_scales"] = torch.stack([s for s, _ in scales])
        st["down_scales"] = torch.stack([t for _, t in scales])
    else:
        B, Q, D, P = case["seqs"], case["q_len"], case["head_dim"], case["page"]
        Hkv = case["kv_heads"]
        lo, hi = case["min_len"], case["max_len"]
        lens = lo + ((hi - lo + 1) * _rand(g, B) ** 2).long().clamp(max=hi - lo)
        lens[-1] = hi
        per_seq = -(-hi // P)
        n_pages = B * per_seq
        st["q"] = _randn(g, B, Q, case["heads"], D).to(torch.bfloat16)
        st["seq_lens"] = lens
        st["block_table"] = torch.randperm(n_pages, generator=g, device=DEV).view(B, per_seq)
        for name in ("k", "v"):
            rows = n_pages * Hkv * P
            parts = [_quantize_rows(_randn(g, min(262144, rows - r), D).to(torch.bfloat16))
                     for r in range(0, rows, 262144)]
            st[name] = tuple(torch.cat([p[i] for p in parts]) for i in range(3))
    return st


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------

def _scores(logits, scoring):
    """Softmax or sigmoid scores in 64 bits; a masked logit scores 0."""
    x = logits.double()
    if scoring == SIGMOID:
        return 1.0 / (1.0 + torch.exp(-x))
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(m > NEG_INF, m, torch.zeros_like(m)))
    s = e.sum(1, keepdim=True)
    return e / torch.where(s > 0, s, torch.ones_like(s))


def _select(logits, bias, case):
    """Experts of each token in descending order of their key; -1 where none is left."""
    T, E = logits.shape
    G, gk = case["groups"], case["group_topk"]
    if bias is None and (G == 1 or gk == 1):
        key = logits.double()            # scores rise with the logits: the same order
    else:
        key = _scores(logits, case["scoring"])
        if bias is not None:
            key = key + bias.double()
        key = torch.where(logits > NEG_INF, key, NEG_INF)
    if G > 1:
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :gk]
        some = best[:, :, 0] > NEG_INF
        gs = torch.where(best > NEG_INF, best, 0.0).sum(2)
        gs = torch.where(some, gs, NEG_INF)
        keep = gs.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, keep, True)
        key = torch.where(mask.repeat_interleave(E // G, dim=1), key, NEG_INF)
    v, idx = key.sort(dim=1, descending=True, stable=True)
    k = case["top_k"]
    return torch.where(v[:, :k] > NEG_INF, idx[:, :k], -1)


def _maps(experts, n_experts):
    """token_rows, row_tokens, seg_offsets of the copies sorted by (expert, token)."""
    T, k = experts.shape
    flat = torch.where(experts < 0, n_experts, experts).reshape(-1)
    key, order = flat.sort(stable=True)
    row = torch.arange(T * k, device=flat.device)
    kept = key < n_experts
    row_tokens = torch.where(kept, order // k, -1)
    token_rows = torch.empty_like(row).scatter_(0, order, torch.where(kept, row, -1))
    bound = torch.arange(n_experts + 1, device=flat.device)
    seg = torch.searchsorted(key, bound)
    return token_rows.view(T, k), row_tokens, seg


def _plain_route(st):
    case = st["case"]
    experts = _select(st["logits"], st["bias"], case)
    s = _scores(st["logits"], case["scoring"]).gather(1, experts.clamp(min=0))
    s = torch.where(experts < 0, 0.0, s)
    if case["renorm"]:
        t = s.sum(1, keepdim=True)
        s = s / torch.where(t > 0, t, torch.ones_like(t))
    w = (case["scale"] * s).float()
    return (w, experts) + _maps(experts, case["experts"])


def _plain_route_backward(st):
    case, x = st["case"], st["logits"].float()
    e, dw = st["experts"], st["d_weights"]
    live = e >= 0
    idx = e.clamp(min=0)
    dw = torch.where(live, dw, 0.0) * case["scale"]
    if case["scoring"] == SIGMOID:
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        m = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(m > NEG_INF, m, torch.zeros_like(m)))
        t = p.sum(1, keepdim=True)
        p = p / torch.where(t > 0, t, torch.ones_like(t))
    s = torch.where(live, p.gather(1, idx), 0.0)
    if case["renorm"]:
        t = s.sum(1, keepdim=True)
        t = torch.where(t > 0, t, torch.ones_like(t))
        ds = (dw - (dw * s).sum(1, keepdim=True) / t) / t
    else:
        ds = dw
    ds = torch.where(live, ds, 0.0)
    full = torch.zeros_like(x).scatter_add_(1, idx, ds)
    if case["scoring"] == SIGMOID:
        dx = full * p * (1.0 - p)
    else:
        dx = p * (full - (full * p).sum(1, keepdim=True))
    return dx.to(st["logits"].dtype)


def _plain_combine(st):
    rows, tr, w = st["rows"], st["token_rows"], st["weights"]
    acc = torch.zeros(tr.shape[0], rows.shape[1], device=rows.device)
    for c in range(tr.shape[1]):
        wc = torch.where(tr[:, c] >= 0, w[:, c], 0.0)
        acc += wc[:, None] * rows[tr[:, c].clamp(min=0)].float()
    return acc.to(rows.dtype)


def _plain_combine_backward(st):
    rows, tr, w = st["rows"], st["token_rows"], st["weights"]
    d = st["d_out"].float()
    d_rows = torch.zeros(rows.shape[0] + 1, rows.shape[1], dtype=rows.dtype, device=rows.device)
    d_w = torch.zeros_like(w)
    for c in range(tr.shape[1]):
        live = tr[:, c] >= 0
        y = rows[tr[:, c].clamp(min=0)].float()
        d_w[:, c] = torch.where(live, (d * y).sum(1), 0.0)
        to = torch.where(live, tr[:, c], rows.shape[0])
        d_rows[to] = (w[:, c, None] * d).to(rows.dtype)
    return d_rows[:-1], d_w


def _plain_matvec(st):
    x = st["x"]
    if isinstance(x, tuple):
        x = _decode(x[0], x[1]) * x[2][:, None]
    else:
        x = x.float()
    parts = [x @ _decode(c, b).t() for c, b in zip(st["codes"].split(16384),
                                                     st["block_scales"].split(16384))]
    return (torch.cat(parts, 1) * st["scale"]).to(torch.bfloat16)


def _plain_experts(st):
    x = st["x"].float()
    T, k = st["experts"].shape
    E = st["gateup_scales"].shape[0]
    ids = st["experts"].reshape(-1)
    xr = x.repeat_interleave(k, dim=0)
    if T * k <= E // 4:
        def product(rows, w, scales):
            m = _decode(w[0][ids], w[1][ids])
            return (m * rows[:, None, :]).sum(2) * scales[ids][:, None]
        gate, up = (product(xr, st[n], st["gateup_scales"]) for n in ("gate", "up"))
        y = product(gate / (1.0 + torch.exp(-gate)) * up, st["down"], st["down_scales"])
    else:
        y = torch.zeros_like(xr)
        for e in range(E):
            sg, sd = st["gateup_scales"][e], st["down_scales"][e]
            gate = xr @ (_decode(st["gate"][0][e], st["gate"][1][e]) * sg).t()
            up = xr @ (_decode(st["up"][0][e], st["up"][1][e]) * sg).t()
            h = gate / (1.0 + torch.exp(-gate)) * up
            ye = h @ (_decode(st["down"][0][e], st["down"][1][e]) * sd).t()
            y = torch.where((ids == e)[:, None], ye, y)
    out = (y.view(T, k, -1) * st["weights"][:, :, None]).sum(1)
    return out.to(torch.bfloat16)


def _mask(case, seq_len, n_keys, device):
    """[q_len][n_keys]: True where a query sees a key (causal from the end, optional window)."""
    Q = case["q_len"]
    pos = seq_len - Q + torch.arange(Q, device=device)[:, None]
    t = torch.arange(n_keys, device=device)[None, :]
    see = t <= pos
    if case["window"]:
        see &= t > pos - case["window"]
    return see


def _plain_attention(st):
    case, q = st["case"], st["q"].float()
    B, Q, Hq, D = q.shape
    Hkv, P = case["kv_heads"], case["page"]
    G = Hq // Hkv
    outs, lses = [], []
    for b in range(B):
        pages = st["block_table"][b]
        kv = []
        for name in ("k", "v"):
            c, bs, s = (a.view(-1, Hkv, P, *a.shape[1:])[pages] for a in st[name])
            x = _decode(c, bs) * s[..., None]                    # [pages][Hkv][P][D]
            kv.append(x.transpose(0, 1).reshape(Hkv, -1, D))
        qb = q[b].view(Q, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * Q, D)
        z = torch.matmul(qb, kv[0].transpose(1, 2).contiguous()) / math.sqrt(D)
        see = _mask(case, st["seq_lens"][b], z.shape[2], z.device).repeat(G, 1)
        z = torch.where(see, z, NEG_INF)
        m = z.amax(2, keepdim=True)
        m0 = torch.where(m > NEG_INF, m, torch.zeros_like(m))
        p = torch.exp(z - m0)
        t = p.sum(2, keepdim=True)
        o = torch.matmul(p, kv[1]) / torch.where(t > 0, t, torch.ones_like(t))
        outs.append(o.view(Hkv, G, Q, D).permute(2, 0, 1, 3).reshape(Q, Hq, D))
        lses.append((m0 + torch.log(t)).view(Hkv, G, Q).permute(2, 0, 1).reshape(Q, Hq))
    return torch.stack(outs).to(torch.bfloat16), torch.stack(lses)


# ---------------------------------------------------------------------------------------------
# The library's forms
# ---------------------------------------------------------------------------------------------

def _own_run(st):
    from nvfp4_block_scaled_amax_amd import api
    case, op = st["case"], st["op"]
    if op == "route":
        r = api.moe_route(st["logits"], case["top_k"], bias=st["bias"], scoring=case["scoring"],
                          n_expert_groups=case["groups"], topk_groups=case["topk_groups"],
                          group_topk=case["group_topk"], renormalize=case["renorm"],
                          scale=case["scale"])
        return r.weights, r.experts, r.token_rows, r.row_tokens, r.seg_offsets
    if op == "route_backward":
        return api.moe_route_backward(st["d_weights"], st["logits"], st["experts"],
                                      scoring=case["scoring"], renormalize=case["renorm"],
                                      scale=case["scale"])
    if op == "combine":
        return api.moe_combine(st["rows"], st["token_rows"], st["weights"])
    if op == "combine_backward":
        # With the segments, the rows past the last one (dropped copies) get zero gradients.
        return api.moe_combine_backward(st["d_out"], st["rows"], st["token_rows"],
                                        st["weights"], seg_offsets=st["seg_offsets"])
    if op == "matvec":
        x = st["x"]
        if isinstance(x, tuple):
            x = api.NVFP4(*x)
        return api.nvfp4_matvec(x, st["codes"], st["block_scales"], st["scale"])
    if op == "experts":
        routing = api.Routing(st["weights"], st["experts"], st["token_rows"], st["row_tokens"],
                              st["seg_offsets"])
        gateup = api.GateUpNVFP4(*st["gate"], *st["up"], st["gateup_scales"])
        down = api.GateUpNVFP4(*st["down"], None, None, st["down_scales"])
        return api.nvfp4_expert_layer(st["x"], routing, gateup, down)
    out = api.nvfp4_attention(st["q"], api.NVFP4(*st["k"]), api.NVFP4(*st["v"]),
                              st["block_table"], st["seq_lens"], case["kv_heads"],
                              case["page"], window=case["window"])
    return out.out, out.lse


_PLAIN = dict(route=_plain_route, route_backward=_plain_route_backward, combine=_plain_combine,
              combine_backward=_plain_combine_backward, matvec=_plain_matvec,
              experts=_plain_experts, attention=_plain_attention)


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------------------------

def _mean_len(case):
    """Expected sequence length: lo + (hi - lo) u^2 for uniform u, one sequence at hi."""
    lo, hi, B = case["min_len"], case["max_len"], case["seqs"]
    return ((B - 1) * (lo + (hi - lo) / 3.0) + hi) / B


def work(case):
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        size = T * E * (2 if case["logits"] == "bfloat16" else 4)
        if op == "route":
            nbytes = size + T * k * (4 + 8 + 8 + 8) + 8 * (E + 1) + (4 * E if case["bias"] else 0)
        else:
            nbytes = 2 * size + T * k * (4 + 8)
        return {"bytes": nbytes, "flops": 6 * T * E}
    if op in ("combine", "combine_backward"):
        T, C, k = case["tokens"], case["cols"], case["top_k"]
        esz = 2 if case["dtype"] == "bfloat16" else 4
        rows = T * k * (1.0 - case["drop"]) * C * esz
        if op == "combine":
            return {"bytes": int(rows + T * C * esz + T * k * 12), "flops": 2 * T * k * C}
        return {"bytes": int(2 * rows + T * C * esz + T * k * 16), "flops": 3 * T * k * C}
    if op == "matvec":
        M, N, K = case["m"], case["n"], case["k"]
        x = 2 * M * K if case["x"] == "bfloat16" else M * K * 9 // 16 + 4 * M
        return {"bytes": N * K * 9 // 16 + x + 2 * M * N, "flops": 2 * M * N * K}
    if op == "experts":
        T, E, H, I = case["tokens"], case["experts"], case["hidden"], case["inter"]
        k = min(case["top_k"], E)
        read = E * (1.0 - (1.0 - k / E) ** T)
        return {"bytes": int(read * 3 * H * I * 9 / 16 + 4 * T * H + 12 * T * k),
                "flops": 6 * T * k * H * I}
    B, Q, Hq, Hkv, D = (case[n] for n in ("seqs", "q_len", "heads", "kv_heads", "head_dim"))
    n = _mean_len(case)
    pairs = B * Q * max(n - (Q - 1) / 2.0, 1.0)
    if case["window"]:
        pairs = min(pairs, B * Q * case["window"])
        n = min(n, case["window"] + Q - 1)
    row = 2 * (D // 2 + D // 16 + 4)
    return {"bytes": int(B * n * Hkv * row + 4 * B * Q * Hq * D + 4 * B * Q * Hq),
            "flops": int(4 * pairs * Hq * D)}


# ---------------------------------------------------------------------------------------------
# Definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _values64(codes, bs):
    """Decoded values from the formats' fields, in 64 bits."""
    c = torch.stack((codes.int() % 16, codes.int() // 16), -1).flatten(-2)
    mag = c % 8
    ex, man = mag // 2, (mag % 2).double()
    v = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2(ex.double() - 1.0))
    v = torch.where(c >= 8, -v, v)
    b = bs.int()
    ex, man = b // 8 % 16, (b % 8).double()
    d = torch.where(ex == 0, man * 2.0 ** -9, (8.0 + man) * torch.exp2(ex.double() - 10.0))
    return v * d.repeat_interleave(16, dim=-1)


def _exact_route(st):
    case = st["case"]
    x = st["logits"].double().cpu()
    bias = torch.zeros(case["experts"]).double() if st["bias"] is None else \
        st["bias"].double().cpu()
    T, E = x.shape
    G, k = case["groups"], case["top_k"]
    if case["scoring"] == SIGMOID:
        s = torch.sigmoid(x)
    else:
        s = torch.nan_to_num(torch.softmax(x, 1))
    by_logit = st["bias"] is None and (G == 1 or case["group_topk"] == 1)
    key = x.clone() if by_logit else s + bias
    key[x == NEG_INF] = NEG_INF
    # Experts in descending order, the lowest index first among equals.
    if G > 1:
        parts = key.view(T, G, -1).sort(dim=2, descending=True).values
        score = parts[:, :, 0].clone()
        if case["group_topk"] == 2:
            second = parts[:, :, 1] if parts.shape[2] > 1 else torch.full_like(score, NEG_INF)
            score += torch.where(second > NEG_INF, second, torch.zeros_like(second))
        rank = score.sort(dim=1, descending=True, stable=True).indices.argsort(1)
        out = (rank >= case["topk_groups"]).repeat_interleave(E // G, 1)
        key = key.masked_fill(out, NEG_INF)
    order = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    gone = key.gather(1, order) == NEG_INF
    w = s.gather(1, order).masked_fill(gone, 0.0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    w = w * case["scale"]
    experts = order.masked_fill(gone, -1)
    t_of, c_of = torch.nonzero(~gone, as_tuple=True)
    e_of = experts[t_of, c_of]
    by = torch.argsort(e_of * T + t_of)
    token_rows = torch.full((T, k), -1, dtype=torch.int64)
    token_rows[t_of[by], c_of[by]] = torch.arange(by.numel())
    row_tokens = torch.full((T * k,), -1, dtype=torch.int64)
    row_tokens[:by.numel()] = t_of[by]
    seg = torch.zeros(E + 1, dtype=torch.int64)
    seg[1:] = torch.bincount(e_of, minlength=E).cumsum(0)
    return tuple(a.to(DEV) for a in (w, experts, token_rows, row_tokens, seg))


def _exact_route_backward(st):
    """The gradient by differentiating sum(d_weights * weights) in 64 bits."""
    case = st["case"]
    x = st["logits"].double()
    dead = (x == NEG_INF).all(1)
    z = torch.where(x == NEG_INF, -1e30, x).masked_fill(dead[:, None], 0.0).requires_grad_(True)
    s = torch.sigmoid(z) if case["scoring"] == SIGMOID else torch.softmax(z, 1)
    live = st["experts"] >= 0
    w = s.gather(1, st["experts"].clamp(min=0)) * live
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + (~live.any(1, keepdim=True)).double())
    loss = (w * case["scale"] * st["d_weights"].double() * live).sum()
    dx, = torch.autograd.grad(loss, z)
    return dx.masked_fill(x == NEG_INF, 0.0)


def _exact_combine(st):
    rows, tr, w = st["rows"], st["token_rows"], st["weights"].double()
    outs = []
    for a in range(0, tr.shape[0], 2048):
        t = tr[a:a + 2048]
        y = rows[t.clamp(min=0)].double()
        outs.append((y * (w[a:a + 2048] * (t >= 0))[:, :, None]).sum(1))
    return torch.cat(outs)


def _exact_combine_backward(st):
    rows, tr, w, d = st["rows"], st["token_rows"], st["weights"].double(), st["d_out"].double()
    d_rows = torch.zeros(rows.shape, dtype=torch.float64, device=rows.device)
    d_w = torch.zeros_like(w)
    t_of, c_of = torch.nonzero(tr >= 0, as_tuple=True)
    for a in range(0, t_of.numel(), 16384):
        t, c = t_of[a:a + 16384], c_of[a:a + 16384]
        r = tr[t, c]
        d_rows[r] = w[t, c, None] * d[t]
        d_w[t, c] = (d[t] * rows[r].double()).sum(1)
    return d_rows, d_w


def _exact_matvec(st):
    x = st["x"]
    x = _values64(x[0], x[1]) * x[2].double()[:, None] if isinstance(x, tuple) else x.double()
    outs = []
    for a in range(0, st["codes"].shape[0], 8192):
        w = _values64(st["codes"][a:a + 8192], st["block_scales"][a:a + 8192])
        outs.append(torch.mm(w * st["scale"].double(), x.t().contiguous()))
    return torch.cat(outs).t().contiguous()


def _exact_experts(st):
    T, k = st["experts"].shape
    x = st["x"].double()
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    ids = st["experts"].cpu()
    for e in sorted(set(ids.reshape(-1).tolist())):
        t, c = (i.to(x.device) for i in torch.nonzero(ids == e, as_tuple=True))
        wg, wu, wd = (_values64(st[n][0][e], st[n][1][e]) for n in ("gate", "up", "down"))
        s, sd = st["gateup_scales"][e].double(), st["down_scales"][e].double()
        gate, up = x[t] @ wg.t().contiguous() * s, x[t] @ wu.t().contiguous() * s
        y = (gate * torch.sigmoid(gate) * up) @ wd.t().contiguous() * sd
        out.index_add_(0, t, y * st["weights"][t, c, None].double())
    return out


def _exact_attention(st):
    case, q = st["case"], st["q"].double()
    B, Q, Hq, D = q.shape
    Hkv, P = case["kv_heads"], case["page"]
    out = torch.zeros_like(q)
    lse = torch.zeros(B, Q, Hq, dtype=torch.float64, device=q.device)
    lens = st["seq_lens"].cpu().tolist()
    for b in range(B):
        n = lens[b]
        t = torch.arange(n, device=q.device)
        page, slot = st["block_table"][b][t // P], t % P
        see = _mask(case, n, n, q.device)
        for h in range(Hkv):
            row = (page * Hkv + h) * P + slot
            k, v = (_values64(st[m][0][row], st[m][1][row]) * st[m][2][row].double()[:, None]
                    for m in ("k", "v"))
            for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                z = torch.where(see, q[b, :, j] @ k.t().contiguous() * D ** -0.5, NEG_INF)
                lse[b, :, j] = torch.logsumexp(z, 1)
                out[b, :, j] = torch.exp(z - lse[b, :, j, None]) @ v
    return out, lse


_EXACT = dict(route=_exact_route, route_backward=_exact_route_backward, combine=_exact_combine,
              combine_backward=_exact_combine_backward, matvec=_exact_matvec,
              experts=_exact_experts, attention=_exact_attention)


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
