"""moe_block_norm and moe_block_norm_bwd against their 64-bit forms.

Bounds count FP32 roundings (ref64.U each, relative to the terms a result is made of):
a row's statistic is a sum of up to 16384 terms of which no path through the kernel has
more than 128 roundings, and its use takes some 32 more: E = 160 U.  A sum over tokens
adds the roundings of its longest chain, at most T / 64 + 64 additions."""
import itertools

import pytest
import torch

import grouped_gemm_fp32_b200 as moe
import ref64
from ref64 import HALF, U, within

pytestmark = pytest.mark.gpu
E = 160 * U
EPS = 1e-6
F32, BF = torch.float32, torch.bfloat16


def inputs(T, d, rt, rows=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + d)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(y=(r(T, d) * torch.exp(r(T, 1))).to(BF), res=(3 * r(T, d)).to(rt),
                w_post=1 + 0.3 * r(d), w_pre=1 + 0.3 * r(d), gate=r(rows, d) if rows else None,
                dn=r(T, d).to(BF), du=(0.5 * r(T, d)).to(rt))


def fwd(i, cfg, y=True, post=True, gate=True, pre=True, into=None, stream=None):
    T, d = i["res"].shape
    dm = moe.MoeDims.of(T, d, 8, 1, 0, 64, 64)
    pick = lambda n, on: i[n] if on else None  # noqa: E731
    u = (torch.full_like(i["res"], 7.0) if into is None else into) if y else None
    n = torch.full((T, d), 7.0, dtype=BF, device="cuda") if pre else None
    moe.moe_block_norm(dm, cfg, pick("y", y), i["res"], pick("w_post", post and y),
                       pick("gate", gate and y), pick("w_pre", pre), u, n, stream)
    return dm, u, n


def check_fwd(i, c, **on):
    cfg = moe.MoeNormCfg.of(EPS, *c)
    y, post, gate, pre = (on.get(k, True) for k in ("y", "post", "gate", "pre"))
    res = i["res"].clone()
    _, u, n = fwd(i, cfg, y, post, gate, pre)
    assert torch.equal(i["res"], res)
    ru, rn, mag = ref64.block_norm(i["y"] if y else None, i["res"],
                                   i["w_post"] if post and y else None,
                                   i["gate"] if gate and y else None, i["w_pre"] if pre else None,
                                   EPS, *c)
    if y:
        within(u, ru, E * mag + HALF[u.dtype] * ru.abs(), "u")
    if pre:
        r = ref64.rms(ru, EPS)
        within(n, rn, E * (mag / r * i["w_pre"].abs() + rn.abs()) + HALF[BF] * rn.abs() * (1 + E)
               + ref64.TINY[BF], "n")


@pytest.mark.parametrize("rt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,d,L", [(1, 4096, 0), (1, 64, 0), (3, 128, 2), (777, 1984, 130),
                                   (301, 192, 1), (64, 4160, 64), (40, 8256, 16), (9, 16384, 5),
                                   (1025, 2048, 1024), (5000, 320, 999)])
def test_forward_matches_64_bits(T, d, L, rt):
    i = inputs(T, d, rt, -(-T // L) if L else 1)
    check_fwd(i, (1.0, 0.7, L))
    check_fwd(i, (-0.5, 1.3, L), post=False)
    check_fwd(i, (1.0, 1.0, L), gate=False)
    check_fwd(i, (1.0, 2.0, L), gate=False, post=False)
    check_fwd(i, (0.8, 0.7, L), pre=False)
    check_fwd(i, (0.8, 0.7, L), y=False)


def test_forward_in_place_and_extremes():
    i = inputs(300, 512, BF, 1)
    cfg = moe.MoeNormCfg.of(EPS, 1.0, 0.5)
    _, u, n = fwd(i, cfg)
    i2 = dict(i, res=i["res"].clone())
    _, u2, n2 = fwd(i2, cfg, into=i2["res"])
    assert u2.data_ptr() == i2["res"].data_ptr() and torch.equal(u, u2) and torch.equal(n, n2)
    # rows of zeros, a row with a NaN, a row with an infinity: the others are unharmed
    i["y"][3], i["res"][3] = 0, 0
    i["y"][5, 7] = float("nan")
    i["res"][9, 100] = float("inf")
    _, u3, n3 = fwd(i, cfg)
    assert (u3[3] == 0).all() and (n3[3] == 0).all()
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[[3, 5, 9]] = False
    assert torch.equal(u3[keep], u[keep]) and torch.equal(n3[keep], n[keep])
    assert u3[5].isnan().all() and n3[5].isnan().all() and u3[9, 100].isinf()


NAMES = ("dy", "dres", "dw_post", "dgate", "dw_pre")


def bwd(i, cfg, y=True, post=True, gate=True, dn=True, du=True, acc=None, dres=None, ws=None,
        stream=None, want=NAMES):
    T, d = i["res"].shape
    dm = moe.MoeDims.of(T, d, 8, 1, 0, 64, 64)
    post, gate = post and y, gate and y
    pick = lambda n, on: i[n] if on else None  # noqa: E731
    full = lambda t: torch.full_like(t, 7.0)   # noqa: E731
    o = dict(dy=full(i["y"]) if y else None, dres=full(i["res"]) if dres is None else dres,
             dw_post=full(i["w_post"]) if post else None,
             dgate=full(i["gate"]) if gate and i["gate"] is not None else None,
             dw_pre=full(i["w_pre"]) if dn else None)
    o = {k: v if k in want else None for k, v in o.items()}
    if ws is None:
        ws = torch.full((moe.moe_norm_workspace_size(dm, cfg),), 0xFF, dtype=torch.uint8,
                        device="cuda")   # NaNs: every value read has been written before
    if acc:
        for k in ("dw_post", "dgate", "dw_pre"):
            if o[k] is not None:
                o[k].copy_(acc[k])
    moe.moe_block_norm_bwd(dm, cfg, pick("dn", dn), pick("du", du), pick("y", y),
                           pick("res", dn), pick("w_post", post), pick("gate", gate),
                           pick("w_pre", dn), o["dy"], o["dres"], o["dw_post"], o["dgate"],
                           o["dw_pre"], 1 if acc else 0, ws, stream)
    return o


def check_bwd(i, c, **on):
    cfg = moe.MoeNormCfg.of(EPS, *c)
    y, post, gate, dn, du = (on.get(k, True) for k in ("y", "post", "gate", "dn", "du"))
    gate = gate and i["gate"] is not None
    o = bwd(i, cfg, y, post, gate, dn, du)
    T = len(i["res"])
    ref = ref64.block_norm_bwd(i["dn"] if dn else None, i["du"] if du else None,
                               i["y"] if y else None, i["res"], i["w_post"] if post and y else None,
                               i["gate"] if gate and y else None, i["w_pre"], EPS, *c)
    for k in NAMES:
        assert (o[k] is not None) == (k in ref), k
        if o[k] is not None:
            v, mag = ref[k]
            tol = E * mag if k in ("dy", "dres") else (E + (T / 64 + 64) * U) * mag
            within(o[k], v, tol + HALF[o[k].dtype] * (v.abs() + tol) + ref64.TINY[o[k].dtype], k)
    again = bwd(i, cfg, y, post, gate, dn, du)
    for k in NAMES:
        assert o[k] is None or torch.equal(o[k], again[k]), k
    return o


@pytest.mark.parametrize("rt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,d,L", [(1, 4096, 0), (1, 64, 0), (3, 128, 2), (777, 1984, 130),
                                   (301, 192, 1), (64, 4160, 64), (40, 8256, 16), (9, 16384, 5),
                                   (1025, 2048, 1024), (5000, 320, 999), (2000, 4096, 700)])
def test_backward_matches_64_bits(T, d, L, rt):
    i = inputs(T, d, rt, -(-T // L) if L else 1)
    check_bwd(i, (1.0, 0.7, L))
    check_bwd(i, (-0.5, 1.3, L), post=False)
    check_bwd(i, (1.0, 1.0, L), gate=False)
    check_bwd(i, (1.0, 1.0, L), gate=False, post=False)
    check_bwd(i, (0.8, 0.7, L), dn=False)
    check_bwd(i, (0.8, 0.7, L), du=False)
    check_bwd(i, (0.8, 0.7, L), y=False)


def test_backward_accumulates_in_place_and_unwanted():
    i = inputs(500, 256, F32, 4)
    cfg = moe.MoeNormCfg.of(EPS, 0.9, 0.7, 130)
    o = bwd(i, cfg)
    base = {k: torch.randn_like(o[k]) for k in ("dw_post", "dgate", "dw_pre")}
    a = bwd(i, cfg, acc=base)
    for k, b in base.items():
        within(a[k], b.double() + o[k].double(), 3 * U * (b.abs() + o[k].abs()), k)
    # dres over dres_out
    i2 = dict(i, du=i["du"].clone())
    p = bwd(i2, cfg, dres=i2["du"])
    for k in NAMES:
        assert torch.equal(p[k], o[k]), k
    for want in (("dy", "dres"), ("dy", "dres", "dgate"), ("dy", "dres", "dw_pre")):
        p = bwd(i, cfg, want=want)
        for k in want:
            assert torch.equal(p[k], o[k]), (want, k)


def test_backward_is_the_gradient():
    # against central differences of the 64-bit forward
    T, d, L = 5, 64, 3
    i = inputs(T, d, F32, 2, seed=3)
    c = (0.9, 0.7, L)
    u, n, _ = ref64.block_norm(i["y"], i["res"], i["w_post"], i["gate"], i["w_pre"], EPS, *c)
    o = bwd(dict(i, res=u.float()), moe.MoeNormCfg.of(EPS, *c))
    p = {k: i[k].double() for k in ("y", "res", "w_post", "gate", "w_pre")}

    def loss(p):
        u, n, _ = ref64.block_norm(p["y"], p["res"], p["w_post"], p["gate"], p["w_pre"], EPS, *c)
        return float((u * i["du"].double()).sum() + (n * i["dn"].double()).sum())

    h = 1e-5
    for name, grad in (("y", "dy"), ("res", "dres"), ("w_post", "dw_post"), ("gate", "dgate"),
                       ("w_pre", "dw_pre")):
        for j in (0, 17, p[name].numel() - 1):
            v = []
            for s in (h, -h):
                q = {k: t.clone() for k, t in p.items()}
                q[name].view(-1)[j] += s
                v.append(loss(q))
            fd, got = (v[0] - v[1]) / (2 * h), float(o[grad].view(-1)[j])
            # bf16 results carry half a step of their own; differences lose ~1e-9 / 2h
            assert abs(fd - got) <= 1e-4 + (2 ** -8) * abs(fd), (name, j, fd, got)


def test_no_tokens():
    i = inputs(0, 128, BF, 1)
    cfg = moe.MoeNormCfg.of()
    fwd(i, cfg)
    o = bwd(i, cfg)
    for k in ("dw_post", "dgate", "dw_pre"):
        assert (o[k] == 0).all()
    base = {k: torch.randn_like(o[k]) for k in ("dw_post", "dgate", "dw_pre")}
    a = bwd(i, cfg, acc=base)
    for k, b in base.items():
        assert torch.equal(a[k], b)


def test_streams_and_graphs():
    i = inputs(1200, 1024, BF, 3)
    cfg = moe.MoeNormCfg.of(EPS, 1.0, 0.7, 500)
    dm, u, n = fwd(i, cfg)
    o = bwd(i, cfg)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _, u2, n2 = fwd(i, cfg, stream=s)
        o2 = bwd(i, cfg, stream=s)
    s.synchronize()
    assert torch.equal(u, u2) and torch.equal(n, n2)
    assert all(torch.equal(o[k], o2[k]) for k in NAMES)
    # two captured calls that share a workspace, replayed one after the other
    ws = torch.full((moe.moe_norm_workspace_size(dm, cfg),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    j = inputs(1200, 1024, BF, 3, seed=9)
    oj = bwd(j, cfg)
    got, graphs = [], []
    for v in (i, j):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(bwd(v, cfg, ws=ws))
        graphs.append(g)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for ref, r in ((o, got[0]), (oj, got[1])):
        assert all(torch.equal(ref[k], r[k]) for k in NAMES)


@pytest.mark.parametrize("rt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 4096, 4160, 16384])
def test_rows_of_the_largest_values(d, rt):
    # every value just below 1e18: the squares' sum over a row leaves FP32, their mean does not
    T = 5
    i = inputs(T, d, rt, 1, seed=23)
    big = 0.99e18
    for n in ("y", "res"):
        i[n] = (big * i[n].float().sign()).to(i[n].dtype)
    i["gate"] = i["gate"].clamp(-1, 1)
    i["w_post"] = i["w_post"].clamp(0.3, 0.9)
    check_fwd(i, (0.0, 1.0, 0))
    check_fwd(i, (0.5, 0.5, 0), post=False)
    check_fwd(i, (1.0, 0.7, 0), y=False)
    # of the backward the sums alone: gradients along a row's own direction, where the
    # projection takes nearly all, have their own test
    o = bwd(i, moe.MoeNormCfg.of(EPS, 1.0, 0.7))
    ref = ref64.block_norm_bwd(i["dn"], i["du"], i["y"], i["res"], i["w_post"], i["gate"],
                               i["w_pre"], EPS, 1.0, 0.7, 0)
    for k in ("dres", "dw_post", "dgate", "dw_pre"):
        v, mag = ref[k]
        tol = E * mag if k == "dres" else (E + (T / 64 + 64) * U) * mag
        within(o[k], v, tol + HALF[o[k].dtype] * (v.abs() + tol) + ref64.TINY[o[k].dtype], k)


@pytest.mark.parametrize("rt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [512, 4160, 8256])
@pytest.mark.parametrize("su,sy,sdn,eps", [(1e13, 1.0, 1.0, 1e-6), (1.0, 1e13, 1.0, 1e-6),
                                           (1e15, 1e15, 1.0, 1e-6), (1e16, 1e17, 1e-6, 1e-6),
                                           (1e17, 1e16, 1e-6, 1e-6), (1e17, 1e17, 1e-3, 1e-6),
                                           (1e-15, 1e-15, 1.0, 1e-30), (0.0, 1.0, 1.0, 1e-30),
                                           (1.0, 0.0, 1.0, 1e-30), (0.0, 0.0, 1.0, 1e-30)])
def test_backward_of_large_and_small_rows(su, sy, sdn, eps, d, rt):
    # the projections on u and y are as large as the terms they are taken from, whatever the
    # rows' size: no power of 1 / rms may leave FP32 on the way
    T = 70
    i = inputs(T, d, rt, 1, seed=21)
    i["res"] = (i["res"].float() * su).to(rt)
    i["y"] = (i["y"].float().clamp(-8, 8) * sy).to(BF)
    for n in ("dn", "du"):
        i[n] = (i[n].float() * sdn).to(i[n].dtype)
    # along u and y, so that the projections take most of it away
    i["dn"] = (i["dn"].float() + sdn * i["res"].float() / max(su, 1e-30) / 3).to(BF)
    cfg = moe.MoeNormCfg.of(eps, 0.9, 0.7)
    o = bwd(i, cfg)
    ref = ref64.block_norm_bwd(i["dn"], i["du"], i["y"], i["res"], i["w_post"], i["gate"],
                               i["w_pre"], eps, 0.9, 0.7, 0)
    for k in NAMES:
        v, mag = ref[k]
        tol = E * mag if k in ("dy", "dres") else (E + (T / 64 + 64) * U) * mag
        within(o[k], v, tol + HALF[o[k].dtype] * (v.abs() + tol) + ref64.TINY[o[k].dtype], k)


@pytest.mark.parametrize("rt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,d", [(700, 192), (333, 4160), (20, 16384)])
def test_outputs_in_the_place_of_inputs(T, d, rt):
    i = inputs(T, d, rt, 1)
    cfg = moe.MoeNormCfg.of(EPS, 0.9, 0.7)
    dm, u, n = fwd(i, cfg)
    y, res = i["y"].clone(), i["res"].clone()
    moe.moe_block_norm(dm, cfg, y, res, i["w_post"], i["gate"], i["w_pre"], res, y)
    assert torch.equal(y, n) and torch.equal(res, u)
    o = bwd(i, cfg)
    ws = torch.empty(moe.moe_norm_workspace_size(dm, cfg), dtype=torch.uint8, device="cuda")
    for dy_over, dres_over in itertools.product(("y", "dn"), ("du", "res")):
        c = {k: i[k].clone() for k in ("y", "dn", "du", "res")}
        w = {k: torch.empty_like(o[k]) for k in ("dw_post", "dgate", "dw_pre")}
        moe.moe_block_norm_bwd(dm, cfg, c["dn"], c["du"], c["y"], c["res"], i["w_post"], i["gate"],
                               i["w_pre"], c[dy_over], c[dres_over], w["dw_post"], w["dgate"],
                               w["dw_pre"], 0, ws)
        assert torch.equal(c[dy_over], o["dy"]) and torch.equal(c[dres_over], o["dres"])
        assert all(torch.equal(w[k], o[k]) for k in w)


@pytest.mark.parametrize("rt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,d", [(300, 1088), (1023, 1088), (1024, 1088), (1023, 1536), (1024, 1536),
                                 (1023, 2048), (1024, 2048), (1, 2048), (200, 1984)])
def test_backward_on_both_sides_of_one_vector_a_thread(T, d, rt):
    check_bwd(inputs(T, d, rt, -(-T // 100)), (1.0, 0.7, 100))
