"""Plain 64-bit forms of the operators around the layer (routing from logits, block
norms, gradient norm and clipping), written from include/moe.h's formulas in torch on
whatever device the inputs are.  Where a test bounds an FP32 result, the form also
returns the sum of the magnitudes of the terms that the result is made of: a rounding
is off by at most 2^-24 of such a term."""
import math

import torch

U = 2.0 ** -24                     # half a step of FP32, relative
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def affinities(logits, score):
    """p, and the affinities that sum to 1, in 64 bits; logits of -inf give 0."""
    x = logits.double()
    out = x == -math.inf
    if score == "softmax":
        m = x.masked_fill(out, -math.inf).amax(1, keepdim=True)
        p = torch.where(out, 0.0, torch.exp(x - m))
        z = p.sum(1, keepdim=True)
        p = torch.where(z == 0, 0.0, p / z)
        return p, p
    p = torch.where(out, 0.0, 1 / (1 + torch.exp(-x)))
    z = p.sum(1, keepdim=True)
    return p, torch.where(z == 0, 0.0, p / z)


def order(key, n):
    """The n largest of each row, descending; equal ones by index (sort is stable)."""
    return key.sort(dim=1, descending=True, stable=True).indices[:, :n]


def route(logits, bias, cfg):
    """cfg: dict(score, n_group, topk_group, group_top, renorm, scale, k).  Returns idx, w,
    probs, p."""
    T, E = logits.shape
    p, probs = affinities(logits, cfg["score"])
    s = p + (bias.double() if bias is not None else 0.0)
    s = torch.where((logits == -math.inf) | s.isnan(), -math.inf, s)
    key = s
    if bias is None:   # the logits rank the experts
        x = logits.double()
        key = torch.where(x.isnan() | (s == -math.inf), -math.inf, x)
    G, K = cfg.get("n_group", 1), cfg.get("topk_group", 1)
    if G > 1 and K < G:
        best = s.view(T, G, E // G).sort(dim=2, descending=True).values
        score = best[:, :, :cfg.get("group_top", 2)].sum(2)
        keep = torch.zeros(T, G, dtype=torch.bool, device=s.device)
        keep.scatter_(1, order(score, K), True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, -math.inf)
    idx = order(key, cfg["k"])
    c = p.gather(1, idx)
    c = torch.where((key.gather(1, idx) == -math.inf) & ~c.isnan(), 0.0, c)
    w = cfg.get("scale", 1.0) * c
    if cfg.get("renorm", True):
        z = c.sum(1, keepdim=True)
        w = torch.where(z == 0, 0.0, w / z)
    return idx.int(), w, probs, p


def route_bwd(logits, idx, w, dw, cfg, seq_grad=None, seq_len=0):
    """dlogits and the magnitude of its terms.  Picks of weight 0 or outside [0, E) take no
    part."""
    T, E = logits.shape
    p, q = affinities(logits, cfg["score"])
    ok = (w != 0) & (idx >= 0) & (idx < E)
    at = idx.long().clamp(0, E - 1)
    dw, w = dw.double() * ok, w.double() * ok
    scale = cfg.get("scale", 1.0)
    if cfg.get("renorm", True):
        z = (p.gather(1, at) * ok).sum(1, keepdim=True)
        z = torch.where(ok.any(1, keepdim=True), z, 1.0)
        d = (scale * dw - (dw * w).sum(1, keepdim=True)) / z * ok
        mag = (abs(scale * dw) + abs(dw * w).sum(1, keepdim=True)) / z * ok
    else:
        d, mag = scale * dw * ok, abs(scale * dw) * ok
    zero = torch.zeros_like(p)
    dp, dm = zero.scatter_add(1, at, d), zero.scatter_add(1, at, mag)
    if seq_grad is not None:
        g = seq_grad.double()[torch.arange(T, device=p.device) // seq_len]
        if cfg["score"] == "softmax":
            dp, dm = dp + g, dm + g.abs()
        else:
            S = p.sum(1, keepdim=True)
            S = torch.where(S == 0, 1.0, S)
            dp = dp + (g - (q * g).sum(1, keepdim=True)) / S
            dm = dm + (g.abs() + (q * g.abs()).sum(1, keepdim=True)) / S
    if cfg["score"] == "softmax":
        return p * (dp - (p * dp).sum(1, keepdim=True)), p * (dm + (p * dm).sum(1, keepdim=True))
    x = logits.double()
    s1 = torch.where(x == -math.inf, 0.0, p / (1 + torch.exp(x)))
    return dp * s1, dm * s1


def _rows(gate, T, seq_len):
    if gate is None:
        return None
    return gate.double()[torch.arange(T, device=gate.device) // (seq_len or max(T, 1))]


def rms(v, eps):
    return (v.square().mean(1, keepdim=True) + eps).sqrt()


def block_norm(y, res, w_post, gate, w_pre, eps, alpha, beta, seq_len):
    """u, n and the magnitude of u's terms."""
    u = res.double()
    mag = u.abs()
    if y is not None:
        z = y.double()
        if w_post is not None:
            z = z / rms(z, eps) * w_post.double()
        if gate is not None:
            z = z * _rows(gate, len(y), seq_len)
        u, mag = alpha * u + beta * z, (alpha * u).abs() + (beta * z).abs()
    n = None if w_pre is None else u / rms(u, eps) * w_pre.double()
    return u, n, mag


def block_norm_bwd(dn, du, y, u, w_post, gate, w_pre, eps, alpha, beta, seq_len):
    """dict of gradients, each with the magnitude of its terms: name -> (value, magnitude)."""
    some = dn if dn is not None else du
    T, d = some.shape
    g = du.double() if du is not None else torch.zeros(T, d, dtype=torch.float64,
                                                       device=some.device)
    gm = g.abs()
    out = {}
    if dn is not None:
        uu, a = u.double(), dn.double() * w_pre.double()
        r = rms(uu, eps)
        g = g + a / r - uu * (a * uu).mean(1, keepdim=True) / r ** 3
        gm = gm + a.abs() / r + uu.abs() * (a * uu).abs().mean(1, keepdim=True) / r ** 3
        t = dn.double() * uu / r
        out["dw_pre"] = (t.sum(0), t.abs().sum(0))
    out["dres"] = (g * (alpha if y is not None else 1.0), gm * (abs(alpha) if y is not None else 1))
    if y is None:
        return out
    yy = y.double()
    q = torch.full_like(yy, beta)
    if gate is not None:
        q = q * _rows(gate, T, seq_len)
    if w_post is not None:
        r = rms(yy, eps)
        t = q * g * yy / r
        out["dw_post"] = (t.sum(0), (q.abs() * gm * yy.abs() / r).sum(0))
        q = q * w_post.double()
        b, bm = q * g, q.abs() * gm
        dy = b / r - yy * (b * yy).mean(1, keepdim=True) / r ** 3
        dm = bm / r + yy.abs() * (bm * yy.abs()).mean(1, keepdim=True) / r ** 3
        z = yy / r * w_post.double()
    else:
        dy, dm, z = q * g, q.abs() * gm, yy
    out["dy"] = (dy, dm)
    if gate is not None:
        L = seq_len or max(T, 1)
        t, tm = beta * g * z, abs(beta) * gm * z.abs()
        out["dgate"] = (torch.stack([v.sum(0) for v in t.split(L)]),
                        torch.stack([v.sum(0) for v in tm.split(L)]))
    return out


def grad_clip(grads, max_norm):
    """norm, coef, clipped gradients."""
    norm = math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))
    q = max_norm / (norm + 1e-6)
    coef = 1.0 if q >= 1.0 else q
    return norm, coef, [g.double() * coef for g in grads]


def within(got, ref, tol, what):
    """|got - ref| <= tol everywhere, NaN and infinities in the same places."""
    got, ref = got.double().cpu(), ref.double().cpu()
    tol = tol.double().cpu() if torch.is_tensor(tol) else torch.as_tensor(tol).double()
    assert torch.equal(got.isnan(), ref.isnan()), f"{what}: NaN in other places"
    fin = ref.isfinite()
    assert torch.equal(got[~fin & ~ref.isnan()], ref[~fin & ~ref.isnan()]), what
    off = (got - ref).abs().where(fin, torch.zeros(()).double())
    bad = off > tol.expand_as(off)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, the worst by "
                           f"{float((off / tol.expand_as(off).clamp_min(1e-300)).max()):.3g} times "
                           "its bound")
