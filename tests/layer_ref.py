"""Plain 64-bit forms of the layer operators (CPU, numpy), written from their
definitions in include/mxq.h, and NVFP4 operands for their tests."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], np.float64)
E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
                 for e in range(16) for m in range(8)], np.float64)
HALF_BF16 = 2.0 ** -8         # half a step, relative
HALF_FP16 = 2.0 ** -11


def decode(codes, block_scales):
    """dec(code) dec(block scale), without the FP32 scale."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    return E2M1[c] * np.repeat(E4M3[block_scales], 16, axis=-1)


def random_nvfp4(rng, rows, cols, lo=0x28, hi=0x78, zero_rows=0.0):
    """Random codes under random block scales (E4M3 bytes lo..hi, all values a
    quantizer can store are below 0x7F) and FP32 row scales over 2^8."""
    codes = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    bs = rng.integers(lo, hi + 1, (rows, cols // 16)).astype(np.uint8)
    s = np.exp2(rng.uniform(-12, -4, rows)).astype(np.float32)
    s[rng.random(rows) < zero_rows] = 0.0
    return codes, bs, s


def route(x, bias, p):
    """x [T][E] float64 -> (weights float64, experts, token_rows, row_tokens, seg)."""
    T, E = x.shape
    dead = ~(x > -np.inf)                       # -inf and NaN
    x = np.where(dead, -np.inf, np.minimum(x, np.finfo(np.float32).max))
    with np.errstate(over="ignore", invalid="ignore"):
        if p["scoring"] == 1:
            s = np.where(dead, 0.0, 1.0 / (1.0 + np.exp(-np.where(dead, 0.0, x))))
        else:
            m = np.max(x, 1, keepdims=True)
            s = np.where(dead, 0.0, np.exp(np.where(dead, 0.0, x - np.where(m > -np.inf, m, 0))))
            t = s.sum(1, keepdims=True)
            s = s / np.where(t > 0, t, 1.0)
    if bias is not None:                        # disabled: no key, but a term of the softmax's sum
        dead = dead | ~(bias > -np.inf)[None, :]
    by_logit = bias is None and (p["n_groups"] == 1 or p["group_topk"] == 1)
    key = x if by_logit else np.where(dead, -np.inf, s + (0.0 if bias is None else bias[None, :]))
    G, k = p["n_groups"], p["top_k"]
    experts = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    with np.errstate(invalid="ignore"):
        # Logarithms of the scores, for ratios of scores below the range of 64 bits.
        ls = x if p["scoring"] == 0 else np.where(dead, -np.inf, -np.logaddexp(0.0, -x))
    for t in range(T):
        kt = key[t].copy()
        if G > 1:
            gs = []
            for g in kt.reshape(G, -1):
                best = sorted(v for v in g if v > -np.inf)[::-1][:p["group_topk"]]
                gs.append(sum(best) if best else -np.inf)
            keep = np.lexsort((np.arange(G), -np.array(gs)))[:p["topk_groups"]]
            out = np.ones(G, bool)
            out[keep] = False
            kt[np.repeat(out, E // G)] = -np.inf
        order = np.lexsort((np.arange(E), -kt))[:k]
        order = order[kt[order] > -np.inf]
        experts[t, :order.size] = order
        w[t, :order.size] = s[t, order]
        if p["renormalize"] and order.size:
            r = np.exp(ls[t, order] - ls[t, order].max())
            w[t, :order.size] = r / r.sum()
    return (w * p["scale"], experts) + maps(experts, E)


def maps(experts, E):
    T, k = experts.shape
    flat = experts.reshape(-1)
    idx = np.nonzero(flat >= 0)[0]
    order = idx[np.lexsort((idx, flat[idx]))]
    token_rows = np.full(T * k, -1, np.int64)
    token_rows[order] = np.arange(order.size)
    row_tokens = np.full(T * k, -1, np.int64)
    row_tokens[:order.size] = order // k
    seg = np.concatenate([[0], np.cumsum(np.bincount(flat[idx], minlength=E))]).astype(np.int64)
    return token_rows.reshape(T, k), row_tokens, seg


def scores(x, scoring):
    dead = ~(x > -np.inf)
    z = np.where(dead, 0.0, x)
    if scoring == 1:
        return np.where(dead, 0.0, 1.0 / (1.0 + np.exp(-z)))
    m = np.max(np.where(dead, -1e300, x), 1, keepdims=True)
    s = np.where(dead, 0.0, np.exp(np.where(dead, 0.0, x - m)))
    t = s.sum(1, keepdims=True)
    return s / np.where(t > 0, t, 1.0)


def route_weights(x, experts, scoring, renorm, scale):
    """The weights of a fixed selection as a function of the logits."""
    s = scores(x, scoring)
    w = np.where(experts >= 0, np.take_along_axis(s, np.maximum(experts, 0), 1), 0.0)
    if renorm:
        t = w.sum(1, keepdims=True)
        w = w / np.where(t > 0, t, 1.0)
    return scale * w


def route_backward(dw, x, experts, scoring, renorm, scale):
    """(d_logits, bound's magnitude: the sum of the terms' absolute values)."""
    s = scores(x, scoring)
    live = experts >= 0
    idx = np.maximum(experts, 0)
    g = np.where(live, dw * scale, 0.0)
    ss = np.where(live, np.take_along_axis(s, idx, 1), 0.0)
    if renorm:
        S = ss.sum(1, keepdims=True)
        S = np.where(S > 0, S, 1.0)
        ds = np.where(live, (g - (g * ss).sum(1, keepdims=True) / S) / S, 0.0)
        mag = np.where(live, (np.abs(g) + (np.abs(g) * ss).sum(1, keepdims=True) / S) / S, 0.0)
    else:
        ds, mag = g, np.abs(g)
    full, fmag = np.zeros_like(x), np.zeros_like(x)
    for c in range(experts.shape[1]):
        r = np.nonzero(live[:, c])[0]
        np.add.at(full, (r, idx[r, c]), ds[r, c])
        np.add.at(fmag, (r, idx[r, c]), mag[r, c])
    if scoring == 1:
        return full * s * (1 - s), fmag * s
    return (s * (full - (full * s).sum(1, keepdims=True)),
            s * (fmag + (fmag * s).sum(1, keepdims=True)))


def combine(rows, token_rows, w):
    """(out, sum of the terms' absolute values)."""
    live = (token_rows >= 0) & (token_rows < rows.shape[0])
    y = rows[np.where(live, token_rows, 0)] * np.where(live, w, 0.0)[:, :, None]
    return y.sum(1), np.abs(y).sum(1)


def attention(q, k, v, table, lens, H_kv, page, scale, causal, window):
    """q [B][Q][H][D]; k, v decoded rows.  (out, lse, sum_t p |v|, largest
    scale * sum_d |q k| over the keys seen)."""
    B, Q, H, D = q.shape
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, terms = np.full((B, Q, H), -np.inf), np.zeros((B, Q, H))
    for b in range(B):
        n = int(lens[b])
        t = np.arange(n)
        for h in range(H):
            row = (table[b][t // page] * H_kv + h // (H // H_kv)) * page + t % page
            kk, vv = k[row], v[row]
            for i in range(Q):
                pos = n - Q + i
                see = (t <= pos) if causal else np.ones(n, bool)
                if window:
                    see &= t > pos - window
                if not see.any():
                    continue
                z = scale * (kk[see] @ q[b, i, h])
                m = z.max()
                p = np.exp(z - m)
                lse[b, i, h] = m + np.log(p.sum())
                p /= p.sum()
                out[b, i, h] = p @ vv[see]
                mag[b, i, h] = p @ np.abs(vv[see])
                terms[b, i, h] = scale * (np.abs(kk[see]) @ np.abs(q[b, i, h])).max()
    return out, lse, mag, terms
