"""The operators around the MoE layer, as plain formulas and as calls of the library.

Three families:
  route   the router's choice from given logits (``moe_route_topk``) and its backward
          (``moe_route_bwd``): softmax or sigmoid affinities, a selection bias, expert
          groups, top-k, renormalised and scaled weights;
  norm    the RMS norms before and after a block with the block's gate and the residual's
          scale (``moe_block_norm``), and the backward (``moe_block_norm_bwd``);
  grads   the global norm of many gradient tensors and their clipping
          (``moe_grad_clip_norm``).

``own = False``: elementary torch operations.  ``own = True``: the library's calls on
buffers that a program allocates once.
"""
import math
import random

import torch

own = False

# --------------------------------------------------------------------------- cases --


def listed():
    return [
        # one token of a decoding user: latency only (the layer's 128 experts, top 6)
        dict(name="route_token", op="route", T=1, E=128, k=6, score="softmax", n_group=1,
             topk_group=1, bias=True, scale=1.0, logits="f32", bwd=False, seq_len=0),
        # a small decode batch: sigmoid scores, 8 groups of which 4 are kept, bf16 logits
        dict(name="route_batch_groups", op="route", T=77, E=256, k=8, score="sigmoid", n_group=8,
             topk_group=4, bias=True, scale=2.5, logits="bf16", bwd=False, seq_len=0),
        # the layer workload's forward (T = 8192)
        dict(name="route_prefill", op="route", T=8192, E=128, k=6, score="softmax", n_group=1,
             topk_group=1, bias=True, scale=1.0, logits="f32", bwd=False, seq_len=0),
        # the train workload (T = 16384) with the sequence-wise balance loss's gradient
        dict(name="route_train", op="route", T=16384, E=128, k=6, score="softmax", n_group=1,
             topk_group=1, bias=True, scale=1.0, logits="f32", bwd=True, seq_len=8192),
        # the same tokens with grouped sigmoid routing over the most experts the layer takes
        dict(name="route_train_groups", op="route", T=16384, E=256, k=8, score="sigmoid",
             n_group=8, topk_group=4, bias=True, scale=2.5, logits="f32", bwd=True, seq_len=0),
        # one token between two blocks: post-norm, gated residual, next block's pre-norm
        dict(name="norm_token", op="norm", T=1, d=4096, res="bf16", gate=True, seq_len=0,
             bwd=False),
        # the layer workload's hidden states between two blocks, bf16 residual stream
        dict(name="norm_prefill", op="norm", T=8192, d=4096, res="bf16", gate=False, seq_len=0,
             bwd=False),
        # ragged training batch: an odd row count, a width that is no power of two, gates per
        # sequence, float32 residual stream
        dict(name="norm_bwd_ragged", op="norm", T=777, d=1984, res="f32", gate=True, seq_len=130,
             bwd=True),
        # the train workload's backward, gates per sequence of 8192 tokens
        dict(name="norm_bwd_train", op="norm", T=16384, d=4096, res="bf16", gate=True,
             seq_len=8192, bwd=True),
        # the gradients of a small model: 40 tensors of odd sizes, below the clipping norm
        dict(name="grads_small", op="grads", tensors=40, total=300_000, type="f32", clips=False),
        # a dense model's bf16 gradients in one packed buffer, 300 tensors of odd sizes
        dict(name="grads_mixed", op="grads", tensors=300, total=60_000_000, type="bf16",
             clips=True),
        # the layer's own FP32 gradients on one of eight expert-parallel ranks: 16 routed and
        # 2 shared experts' dW1 and dW2, and dWg
        dict(name="grads_expert_rank", op="grads", tensors=0, total=0, type="f32", clips=True,
             E=128, experts=18, d=4096, I=1408),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "grads"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        E = n_group * rng.choice([g for g in (4, 8, 12, 16, 20, 32, 48, 64, 96, 128, 160, 256)
                                  if g * n_group <= 256])
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(10, E // n_group * topk_group))
        bwd = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), n_group=n_group,
                    topk_group=topk_group, bias=rng.random() < 0.7,
                    scale=rng.choice([1.0, 1.5, 2.5]), logits=rng.choice(["f32", "bf16"]),
                    bwd=bwd, seq_len=rng.randint(128, 8192) if bwd and rng.random() < 0.5 else 0)
    if op == "norm":
        d = 64 * _log(rng, 2, 112)
        return dict(op=op, T=_log(rng, 1, 16384), d=d, res=rng.choice(["bf16", "f32"]),
                    gate=rng.random() < 0.6,
                    seq_len=_log(rng, 64, 8192) if rng.random() < 0.5 else 0,
                    bwd=rng.random() < 0.5)
    return dict(op=op, tensors=_log(rng, 1, 400), total=_log(rng, 1_000, 80_000_000),
                type=rng.choice(["f32", "bf16", "f16"]), clips=rng.random() < 0.7)


# -------------------------------------------------------------------------- inputs --

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _grad_shapes(case):
    """The tensors' sizes: the layer's own, or odd sizes spread over three decades."""
    if case["tensors"] == 0:
        n, d, i = case["experts"], case["d"], case["I"]
        return [(n, 2 * i, d), (n, d, i), (case["E"], d)]
    r = random.Random(case["total"] * 1000 + case["tensors"])
    parts = [math.exp(r.uniform(0.0, 7.0)) for _ in range(case["tensors"])]
    return [(max(1, int(case["total"] * p / sum(parts))),) for p in parts]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")    # noqa: E731
    s = {"case": case}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # x ~ N(0, 1) against gate weights of std 0.02 over d = 4096 give logits of std 1.28
        s["logits"] = (1.28 * randn(T, E)).to(TYPES[case["logits"]])
        s["bias"] = (rand(E) - 0.5) * (0.02 if case["score"] == "softmax" else 0.1) \
            if case["bias"] else None
        if case["bwd"]:
            s["dw"] = randn(T, k)
            s["seq_grad"] = 1e-3 * rand(-(-T // case["seq_len"]), E) if case["seq_len"] else None
        if own:
            import grouped_gemm_fp32_b200 as moe
            dev = dict(device="cuda")
            s["dims"] = moe.MoeDims.of(T, 4096, E, k, 0, 64, 64)
            s["cfg"] = moe.MoeRouteCfg.of(case["score"], case["n_group"], case["topk_group"],
                                          scale=case["scale"])
            s["idx"] = torch.empty(T, k, dtype=torch.int32, **dev)
            s["w"] = torch.empty(T, k, **dev)
            s["probs"] = torch.empty(T, E, **dev)
            if case["bwd"]:
                s["dlogits"] = torch.empty_like(s["logits"])
    elif case["op"] == "norm":
        T, d, rt = case["T"], case["d"], TYPES[case["res"]]
        rows = -(-T // case["seq_len"]) if case["seq_len"] else 1
        bf = torch.bfloat16
        s["y"] = (0.5 * randn(T, d) * torch.exp(randn(T, 1) * 0.3)).to(bf)
        s["w_post"] = 1.0 + 0.1 * randn(d)
        s["w_pre"] = 1.0 + 0.1 * randn(d)
        s["gate"] = 0.5 + 0.2 * randn(rows, d) if case["gate"] else None
        s["res"] = (3.0 * randn(T, d)).to(rt)      # forward: the residual; backward: u itself
        if case["bwd"]:
            s["dn"] = randn(T, d).to(bf)
            s["du"] = (0.3 * randn(T, d)).to(rt)
        if own:
            import grouped_gemm_fp32_b200 as moe
            dims = s["dims"] = moe.MoeDims.of(T, d, 8, 1, 0, 64, 64)
            cfg = s["cfg"] = moe.MoeNormCfg.of(EPS, ALPHA, BETA, seq_len=case["seq_len"])
            like = torch.empty_like
            if case["bwd"]:
                s["dy"], s["dres"] = like(s["y"]), like(s["res"])
                s["dw_post"], s["dw_pre"] = like(s["w_post"]), like(s["w_pre"])
                s["dgate"] = like(s["gate"]) if case["gate"] else None
                s["ws"] = torch.empty(moe.moe_norm_workspace_size(dims, cfg), dtype=torch.uint8,
                                      device="cuda")
            else:
                s["u"], s["n"] = like(s["res"]), like(s["y"])
    else:
        shapes, t = _grad_shapes(case), TYPES[case["type"]]
        sizes = [math.prod(x) for x in shapes]
        scale = torch.exp(2.0 * randn(len(shapes))).tolist()
        # a total norm of 12: above the clipping norm of 1, below that of 100
        unit = 1.0 / math.sqrt(sum(n * c * c for n, c in zip(sizes, scale)))
        loss_scale = 256.0 if case["type"] == "f16" else 1.0   # f16 gradients are kept in range
        s["max_norm"] = loss_scale * (1.0 if case["clips"] else 100.0)
        unit *= 12.0 * loss_scale
        s["grads"] = [(unit * c * randn(*x)).to(t) for x, c in zip(shapes, scale)]
        s["flat"] = torch.empty(sum(sizes), dtype=t, device="cuda")   # the packed bucket
        s["outs"] = [v.view(x) for v, x in zip(s["flat"].split(sizes), shapes)]
        if own:
            import grouped_gemm_fp32_b200 as moe
            s["list"] = moe.GradList(s["grads"], s["outs"])
            s["norm"], s["coef"] = torch.empty(2, 1, device="cuda").unbind(0)
            s["sumsq"] = torch.empty(1, dtype=torch.float64, device="cuda")
            s["ws"] = torch.empty(moe.moe_grad_workspace_size(len(shapes)), dtype=torch.uint8,
                                  device="cuda")
    return s


EPS, ALPHA, BETA = 1e-6, 1.0, 0.7   # norm: epsilon, weight of the residual, of the block

# --------------------------------------------------------------------- plain forms --


def _route_plain(s):
    c, logits, bias = s["case"], s["logits"], s["bias"]
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    # in 64 bits: neighbouring scores decide the choice
    x = logits.double()
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        probs = p
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
        probs = p / p.sum(1, keepdim=True)
    sel = p if bias is None else p + bias
    if G > 1:
        top2 = sel.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        order = top2.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        keep.scatter_(1, order, True)
        sel = sel.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    idx = sel.sort(dim=1, descending=True, stable=True).indices[:, :k]
    chosen = p.gather(1, idx)
    z = chosen.sum(1, keepdim=True)
    w = c["scale"] * chosen / z
    out = {"idx": idx.to(torch.int32), "w": w.float(), "probs": probs.float()}
    if c["bwd"]:
        p, w, z, probs = p.float(), w.float(), z.float(), probs.float()
        dp = (c["scale"] * s["dw"] - (s["dw"] * w).sum(1, keepdim=True)) / z
        dp = torch.zeros_like(p).scatter_(1, idx, dp)
        if s["seq_grad"] is not None:
            t = torch.arange(T, device=x.device) // c["seq_len"]
            q = s["seq_grad"][t]
            if c["score"] == "softmax":
                dp = dp + q
            else:
                total = p.sum(1, keepdim=True)
                dp = dp + (q - (probs * q).sum(1, keepdim=True)) / total
        if c["score"] == "softmax":
            dl = p * (dp - (p * dp).sum(1, keepdim=True))
        else:
            e = torch.exp(-logits.float().abs())
            dl = dp * e / ((1.0 + e) * (1.0 + e))
        out["dlogits"] = dl.to(logits.dtype)
    return out


def _gate_rows(s):
    """The gate of every token: row t // seq_len (one row for all where seq_len is 0)."""
    c, gate = s["case"], s["gate"]
    if gate is None or not c["seq_len"]:
        return gate
    return gate[torch.arange(c["T"], device=gate.device) // c["seq_len"]]


def _norm_plain(s):
    c, y = s["case"], s["y"].float()
    r1 = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    yh = y * r1
    gate = _gate_rows(s)
    if not c["bwd"]:
        z = yh * s["w_post"]
        u = ALPHA * s["res"].float() + BETA * (z if gate is None else gate * z)
        r2 = torch.rsqrt((u * u).mean(1, keepdim=True) + EPS)
        return {"u": u.to(s["res"].dtype), "n": (u * r2 * s["w_pre"]).to(torch.bfloat16)}
    u, dn = s["res"].float(), s["dn"].float()
    r2 = torch.rsqrt((u * u).mean(1, keepdim=True) + EPS)
    uh = u * r2
    dnh = dn * s["w_pre"]
    du = s["du"].float() + r2 * (dnh - uh * (dnh * uh).mean(1, keepdim=True))
    dz = BETA * (du if gate is None else gate * du)
    dyh = dz * s["w_post"]
    dy = r1 * (dyh - yh * (dyh * yh).mean(1, keepdim=True))
    out = {"dy": dy.to(torch.bfloat16), "dres": (ALPHA * du).to(s["res"].dtype),
           "dw_post": (dz * yh).sum(0), "dw_pre": (dn * uh).sum(0)}
    if gate is not None:
        t = BETA * du * yh * s["w_post"]
        n, L = s["gate"].shape[0], c["seq_len"] or c["T"]
        pad = torch.zeros(n * L - c["T"], c["d"], device=t.device)
        out["dgate"] = torch.cat([t, pad]).view(n, L, c["d"]).sum(1)
    return out


def _grads_plain(s):
    # in 64 bits: a sum over up to hundreds of millions of squares
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt().float()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["outs"])]
    return {"norm": norm.view(1), "coef": coef.view(1), "grads": s["flat"]}


# ------------------------------------------------------------------- the library's --


def _route_own(s):
    import grouped_gemm_fp32_b200 as moe
    c = s["case"]
    moe.moe_route_topk(s["dims"], s["cfg"], s["logits"], s["bias"], s["idx"], s["w"], s["probs"])
    out = {"idx": s["idx"], "w": s["w"], "probs": s["probs"]}
    if c["bwd"]:
        moe.moe_route_bwd(s["dims"], s["cfg"], s["logits"], s["idx"], s["w"], s["dw"],
                          s["seq_grad"], c["seq_len"], s["dlogits"])
        out["dlogits"] = s["dlogits"]
    return out


def _norm_own(s):
    import grouped_gemm_fp32_b200 as moe
    if not s["case"]["bwd"]:
        moe.moe_block_norm(s["dims"], s["cfg"], s["y"], s["res"], s["w_post"], s["gate"],
                           s["w_pre"], s["u"], s["n"])
        return {"u": s["u"], "n": s["n"]}
    moe.moe_block_norm_bwd(s["dims"], s["cfg"], s["dn"], s["du"], s["y"], s["res"], s["w_post"],
                           s["gate"], s["w_pre"], s["dy"], s["dres"], s["dw_post"], s["dgate"],
                           s["dw_pre"], 0, s["ws"])
    out = {"dy": s["dy"], "dres": s["dres"], "dw_post": s["dw_post"], "dw_pre": s["dw_pre"]}
    if s["gate"] is not None:
        out["dgate"] = s["dgate"]
    return out


def _grads_own(s):
    import grouped_gemm_fp32_b200 as moe
    moe.moe_grad_clip_norm(s["list"], s["max_norm"], s["sumsq"], s["norm"], s["coef"], s["ws"])
    return {"norm": s["norm"], "coef": s["coef"], "grads": s["flat"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _route_own, "norm": _norm_own, "grads": _grads_own}[op](state)
    return {"route": _route_plain, "norm": _norm_plain, "grads": _grads_plain}[op](state)


# ------------------------------------------------------------------- work and truth --


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["logits"] == "f32" else 2
        # forward: logits in; probs, picks and weights out
        byte = T * E * size + E * 4 * case["bias"] + T * E * 4 + T * k * 8
        flop = T * E * 12 + T * k * 4
        if case["bwd"]:  # logits are the same input; dw in, dlogits out
            byte += T * k * 4 + T * E * size
            byte += -(-T // case["seq_len"]) * E * 4 if case["seq_len"] else 0
            flop += T * E * 12
        return {"bytes": byte, "flops": flop}
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        r = 4 if case["res"] == "f32" else 2
        rows = (-(-T // case["seq_len"]) if case["seq_len"] else 1) * case["gate"]
        if not case["bwd"]:  # y, res in; u, n out; weights and gates
            return {"bytes": T * d * (4 + 2 * r) + d * 4 * (2 + rows), "flops": T * d * 11}
        # dn, du, y, u in; dy, dres out; weights, gates and their gradients
        return {"bytes": T * d * (6 + 3 * r) + 2 * d * 4 * (2 + rows), "flops": T * d * 30}
    n = sum(math.prod(x) for x in _grad_shapes(case))
    return {"bytes": 2 * n * (4 if case["type"] == "f32" else 2), "flops": 3 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _route_exact(case, s)
    return _norm_exact(case, s) if case["op"] == "norm" else _grads_exact(s)


def _best(v, n):
    """Which entries of each row are among its n largest, and their places: by counting the
    entries before each one (greater, or equal with a lower index)."""
    low = torch.ones(v.shape[1], v.shape[1], dtype=torch.bool, device=v.device).tril(-1)
    place = torch.cat([((q[:, None, :] > q[:, :, None]) |
                        ((q[:, None, :] == q[:, :, None]) & low)).sum(2) for q in v.split(1024)])
    return place < n, place


def _route_exact(c, s):
    x = s["logits"].double()
    T, E, k = c["T"], c["E"], c["k"]
    soft = c["score"] == "softmax"
    p = torch.softmax(x, 1) if soft else torch.sigmoid(x)
    q = p / p.sum(1, keepdim=True)
    v = p + (s["bias"].double() if s["bias"] is not None else 0.0)
    if c["n_group"] > 1:
        per = v.view(T, c["n_group"], -1)
        best = per.amax(2)
        is_best = per == best[:, :, None]
        second = per.masked_fill(is_best & (is_best.cumsum(2) == 1), -math.inf).amax(2)
        kept, _ = _best(best + second, c["topk_group"])
        v = torch.where(kept[:, :, None], per, -math.inf).reshape(T, E)
    mask, place = _best(v, k)
    idx = torch.zeros(T, E, dtype=torch.int64, device=x.device)
    idx.scatter_(1, place, torch.arange(E, device=x.device).expand(T, E))
    idx = idx[:, :k]
    z = (p * mask).sum(1, keepdim=True)
    wfull = c["scale"] * p * mask / z
    out = {"idx": idx.to(torch.int32), "w": wfull.gather(1, idx), "probs": q}
    if c["bwd"]:
        up = torch.zeros_like(p).scatter_(1, idx, s["dw"].double())
        dp = mask * (c["scale"] * up - (up * wfull).sum(1, keepdim=True)) / z
        if s["seq_grad"] is not None:
            g = s["seq_grad"].double().repeat_interleave(c["seq_len"], 0)[:T]
            dp = dp + (g - (g * q).sum(1, keepdim=True)) / p.sum(1, keepdim=True)
        out["dlogits"] = (p * dp - p * (p * dp).sum(1, keepdim=True)) if soft \
            else dp * p * torch.sigmoid(-x)
    return out


def _norm_exact(c, s):
    T, d = c["T"], c["d"]
    y, res = s["y"].double(), s["res"].double()
    w1, w2 = s["w_post"].double(), s["w_pre"].double()
    per = c["seq_len"] or T
    g = s["gate"].double().repeat_interleave(per, 0)[:T] if s["gate"] is not None \
        else torch.ones(1, 1, dtype=torch.float64, device=y.device)
    ry = (y.square().sum(1, keepdim=True) / d + EPS).sqrt()
    if not c["bwd"]:
        u = ALPHA * res + BETA * g * w1 * y / ry
        return {"u": u, "n": w2 * u / (u.square().sum(1, keepdim=True) / d + EPS).sqrt()}
    dn, ru = s["dn"].double(), (res.square().sum(1, keepdim=True) / d + EPS).sqrt()
    a = dn * w2
    du = s["du"].double() + a / ru - res * (a * res).sum(1, keepdim=True) / (d * ru ** 3)
    b = BETA * g * w1 * du
    out = {"dy": b / ry - y * (b * y).sum(1, keepdim=True) / (d * ry ** 3), "dres": ALPHA * du,
           "dw_post": (BETA * g * du * y / ry).sum(0), "dw_pre": (dn * res / ru).sum(0)}
    if s["gate"] is not None:
        t = BETA * w1 * du * y / ry
        out["dgate"] = torch.stack([q.sum(0) for q in t.split(per)])
    return out


def _grads_exact(s):
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2
                               for g in s["grads"]))
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    one = lambda v: torch.tensor([v], dtype=torch.float64, device="cuda")  # noqa: E731
    return {"norm": one(norm), "coef": one(coef),
            "grads": torch.cat([g.flatten().double() * coef for g in s["grads"]])}
