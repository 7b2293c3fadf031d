"""moe_route_topk and moe_route_bwd against their 64-bit forms, and the layer's gate
GEMMs on their own (moe_gate_logits, moe_gate_bwd).

The choice has to be the 64-bit one exactly.  Bounds of FP32 results count roundings:
an affinity takes the rounding of x - max (|x - max| 2^-24), expf (2 steps of 2^-23), a
sum of up to 256 terms (at most 14 roundings on any path, twice for the chosen ones'
sum), a reciprocal and three products: (24 + |x - max|) 2^-23 of its value covers them
for p and for w."""
import itertools
import math

import pytest
import torch

import grouped_gemm_fp32_b200 as moe
import ref64
from common import dev
import synth

pytestmark = pytest.mark.gpu
SM, SG = "softmax", "sigmoid"
INF = math.inf


def make(T, E, k, seed=0, bias=True, dtype=torch.float32, std=1.28, **cfg):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cfg = dict(score=SM, n_group=1, topk_group=1, group_top=2, renorm=True, scale=1.0, k=k) | cfg
    x = (std * torch.randn(T, E, generator=g, device="cuda")).to(dtype)
    b = 0.05 * (torch.rand(E, generator=g, device="cuda") - 0.5) if bias else None
    return x, b, cfg


def call(x, b, cfg, probs=True, stream=None):
    T, E = x.shape
    k = cfg["k"]
    dm = moe.MoeDims.of(T, 64, E, k, 0, 64, 64)
    rc = moe.MoeRouteCfg.of(*[cfg[n] for n in ("score", "n_group", "topk_group", "group_top",
                                               "renorm", "scale")])
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    p = torch.full((T, E), 7.0, device="cuda") if probs else None
    moe.moe_route_topk(dm, rc, x, b, idx, w, p, stream)
    return dm, rc, idx, w, p


def spread(x):
    x = x.double().masked_fill(~x.isfinite(), 0.0)
    return (x - x.amax(1, keepdim=True)).abs()


def check(x, b, cfg):
    dm, rc, idx, w, p = call(x, b, cfg)
    ridx, rw, rp, raw = ref64.route(x, b, cfg)
    assert torch.equal(idx, ridx), (idx != ridx).nonzero()[:5]
    # sigmoid: no maximum is subtracted, and p / sum p is what stands in w and probs
    far = spread(x) if cfg["score"] == SM else torch.zeros_like(x, dtype=torch.float64)
    rel = (24 + far) * 2 ** -23
    ref64.within(p, rp, rel * rp.nan_to_num() + 2.0 ** -126, "probs")
    wrel = rel.gather(1, ridx.long()).amax(1, keepdim=True) * 2
    ref64.within(w, rw, wrel * rw.nan_to_num() + 2.0 ** -126, "weights")
    return dm, rc, idx, w, p


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("T,E,k", [(1, 128, 6), (3, 8, 2), (5, 1, 1), (130, 7, 7), (257, 33, 5),
                                   (64, 64, 8), (1000, 96, 6), (77, 256, 8), (31, 250, 40),
                                   (2, 256, 256), (4099, 128, 6)])
def test_topk_matches_64_bits(T, E, k, score):
    for dtype, bias in itertools.product((torch.float32, torch.bfloat16), (True, False)):
        check(*make(T, E, k, T + E, bias, dtype, score=score, scale=2.5))


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("E,G,K,top,k", [(256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (128, 4, 1, 2, 6),
                                         (160, 8, 3, 2, 6), (96, 3, 2, 2, 5), (60, 5, 2, 1, 4),
                                         (256, 64, 7, 2, 9), (256, 256, 9, 1, 9),
                                         (48, 16, 16, 2, 3), (250, 2, 1, 2, 100)])
def test_groups_match_64_bits(E, G, K, top, k, score):
    for dtype, bias in itertools.product((torch.float32, torch.bfloat16), (True, False)):
        check(*make(515, E, k, E + G, bias, dtype, score=score, n_group=G, topk_group=K,
                    group_top=top, scale=1.5))


def test_without_renormalisation():
    check(*make(200, 128, 6, 1, renorm=False, scale=0.5))
    check(*make(200, 128, 6, 1, renorm=False, score=SG))


@pytest.mark.parametrize("score", [SM, SG])
def test_near_and_equal_scores(score):
    # scores a few steps of FP32 apart or equal, so that FP32 alone could not order them
    T, E = 512, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    base = torch.randint(0, 4, (T, E), generator=g, device="cuda").float()
    x = base + 2.0 ** -22 * torch.randint(0, 4, (T, E), generator=g, device="cuda")
    b = 2.0 ** -26 * torch.randint(0, 8, (E,), generator=g, device="cuda").float()
    for groups in (dict(), dict(n_group=8, topk_group=3)):
        cfg = dict(score=score, n_group=1, topk_group=1, group_top=2, renorm=True, scale=1.0,
                   k=6) | groups
        check(x, b, cfg)
        check(x, None, cfg)
        check(base, torch.zeros_like(b), cfg)
        check(torch.zeros_like(x), None, cfg)       # every score equal: the first k
        check(torch.full_like(x, -3.0), b * 0, cfg)


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("groups", [dict(), dict(n_group=4, topk_group=2)])
def test_masked_experts(score, groups):
    x, b, cfg = make(64, 32, 6, 3, score=score, **groups)
    x[0] = -INF                  # a token without any expert
    x[1, 3:] = -INF              # three left for six picks
    x[2, :31] = -INF
    x[3, ::2] = -INF
    x[4, 8:16] = -INF
    check(x, b, cfg)
    check(x, None, cfg)
    b2 = b.clone()
    b2[5:30] = -INF              # experts that the bias keeps out
    _, _, idx, w, _ = check(x, b2, cfg)
    assert (w[0] == 0).all()
    assert all(len(set(r)) == 6 for r in idx.tolist())


@pytest.mark.parametrize("score", [SM, SG])
def test_lowest_values_and_wide_ranges(score):
    # the lowest value of the type in masked places is an ordinary, very small logit
    low = torch.finfo(torch.float32).min
    x, b, cfg = make(16, 64, 4, 4, score=score)
    x[:, ::3] = low
    x[1] = low
    check(x, b, cfg)
    x, b, cfg = make(64, 64, 4, 4, score=score, std=30.0)
    check(x, b, cfg)
    x = x - 200.0                # every sigmoid below FP32's normal range
    if score == SG:
        _, _, idx, w, _ = call(x, None, cfg)
        ridx, rw, _, _ = ref64.route(x, None, cfg)
        assert torch.equal(idx, ridx)
        ref64.within(w, rw, 1e-5 * rw + 2.0 ** -126, "weights of tiny affinities")


@pytest.mark.parametrize("score", [SM, SG])
def test_non_finite_logits_keep_the_choice_valid(score):
    x, b, cfg = make(40, 64, 6, 6, score=score)
    x[0, 5] = math.nan
    x[1] = math.nan
    x[2, 9] = INF
    x[3, 4] = math.nan
    x[3, 10:] = -INF
    for bias in (b, None):
        _, _, idx, w, p = call(x, bias, cfg)
        assert all(len(set(r)) == 6 and 0 <= min(r) and max(r) < 64 for r in idx.tolist())
        assert w[4:].isfinite().all() and p[4:].isfinite().all()   # other tokens unharmed
        ridx, rw, rp, _ = ref64.route(x, bias, cfg)
        assert torch.equal(idx, ridx)
        assert torch.equal(w.isnan(), rw.isnan()) and torch.equal(p.isnan(), rp.isnan())


def bwd_check(x, idx, w, dw, cfg, rc, dm, seq_grad=None, seq_len=0):
    dl = torch.full_like(x, 9.0)
    moe.moe_route_bwd(dm, rc, x, idx, w, dw, seq_grad, seq_len, dl)
    ref, mag = ref64.route_bwd(x, idx, w, dw, cfg, seq_grad, seq_len)
    # twice an affinity's bound (p and the chosen sum), and the sums over k picks and E experts
    far = spread(x).where(x != -INF, 0.0) if cfg["score"] == SM \
        else torch.zeros_like(x, dtype=torch.float64)
    rel = (64 + cfg["k"] + 2 * far.amax(1, keepdim=True)) * 2 ** -23
    ref64.within(dl, ref, rel * mag + ref64.HALF[x.dtype] * ref.abs() + 2.0 ** -126, "dlogits")
    again = torch.full_like(x, 9.0)
    moe.moe_route_bwd(dm, rc, x, idx, w, dw, seq_grad, seq_len, again)
    assert torch.equal(dl, again)
    return dl


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("T,E,k,groups,seq_len", [(1, 128, 6, {}, 0), (5, 1, 1, {}, 0),
                                                  (300, 8, 2, {}, 128), (257, 33, 5, {}, 7),
                                                  (515, 256, 8, dict(n_group=8, topk_group=4), 0),
                                                  (2000, 128, 6, {}, 1500), (9, 256, 256, {}, 4),
                                                  (130, 250, 40, {}, 0)])
def test_bwd_matches_64_bits(T, E, k, groups, seq_len, score):
    for dtype, renorm in itertools.product((torch.float32, torch.bfloat16), (True, False)):
        x, b, cfg = make(T, E, k, T * E, True, dtype, score=score, scale=2.5, renorm=renorm,
                         **groups)
        dm, rc, idx, w, _ = call(x, b, cfg)
        g = torch.Generator(device="cuda").manual_seed(T)
        dw = torch.randn(T, k, generator=g, device="cuda")
        sg = torch.randn(-(-T // seq_len), E, generator=g, device="cuda") if seq_len else None
        bwd_check(x, idx, w, dw, cfg, rc, dm, sg, seq_len)


@pytest.mark.parametrize("score", [SM, SG])
def test_bwd_is_the_gradient(score):
    # against central differences of the 64-bit forward with the choice held
    x, b, cfg = make(6, 24, 4, 8, score=score, scale=1.5)
    dm, rc, idx, w, _ = call(x, b, cfg)
    dw = torch.randn(6, 4, device="cuda")
    sg = torch.randn(2, 24, device="cuda")
    dl = bwd_check(x, idx, w, dw, cfg, rc, dm, sg, 4)

    def loss(z):
        p, q = ref64.affinities(z, score)
        c = p.gather(1, idx.long())
        w = 1.5 * c / c.sum(1, keepdim=True)
        return ((w * dw).sum() + (q * sg.double()[torch.arange(6, device="cuda") // 4]).sum())

    h, z = 1e-5, x.double()
    for t, e in ((0, int(idx[0, 0])), (1, 5), (3, 23), (5, int(idx[5, 3])), (4, 0)):
        up, dn = z.clone(), z.clone()
        up[t, e] += h
        dn[t, e] -= h
        assert abs(float((loss(up) - loss(dn)) / (2 * h)) - float(dl[t, e])) < 1e-5


@pytest.mark.parametrize("score", [SM, SG])
def test_bwd_of_masked_tokens_and_foreign_indices(score):
    x, b, cfg = make(40, 32, 6, 3, score=score)
    x[0] = -INF
    x[1, 3:] = -INF
    dm, rc, idx, w, _ = call(x, b, cfg)
    dw = torch.randn(40, 6, device="cuda")
    dl = bwd_check(x, idx, w, dw, cfg, rc, dm, torch.randn(1, 32, device="cuda"), 64)
    assert (dl[x == -INF] == 0).all()
    idx = idx.clone()
    idx[3, 1], idx[4, 0], idx[5, 2] = -1, 32, 1 << 30      # no expert: skipped
    idx[6, 1] = idx[6, 0]                                  # the same expert twice
    bwd_check(x, idx, w, dw, cfg, rc, dm)


def test_no_tokens_and_other_streams_and_graphs():
    x, b, cfg = make(0, 64, 4)
    call(x, b, cfg)
    x, b, cfg = make(700, 256, 8, score=SG, n_group=8, topk_group=4)
    _, _, idx, w, p = call(x, b, cfg)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dm, rc, idx2, w2, p2 = call(x, b, cfg, stream=s)
        dw = torch.randn(700, 8, device="cuda")
        dl = torch.empty_like(x)
        moe.moe_route_bwd(dm, rc, x, idx2, w2, dw, None, 0, dl)
    s.synchronize()
    assert torch.equal(idx, idx2) and torch.equal(w, w2) and torch.equal(p, p2)
    ref = dl.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_route_topk(dm, rc, x, b, idx2, w2, p2)
        moe.moe_route_bwd(dm, rc, x, idx2, w2, dw, None, 0, dl)
    for t in (idx2, w2, p2, dl):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx, idx2) and torch.equal(w, w2) and torch.equal(dl, ref)


@pytest.mark.parametrize("T,d,E,k", [(300, 128, 8, 2), (1000, 192, 96, 6), (129, 256, 256, 8)])
def test_gate_logits_and_bwd(T, d, E, k):
    x = dev(synth.normal_bf16(T, 1, (T, d), 1.0), True)
    wg = dev(synth.normal_f32(T, 2, (E, d), 0.05))
    dm = moe.MoeDims.of(T, d, E, k, 0, 64, 64)
    ws = torch.zeros(moe.moe_workspace_size(dm), dtype=torch.uint8, device="cuda")
    logits = torch.full((T, E), 7.0, device="cuda")
    moe.moe_gate_logits(dm, x, wg, logits, ws)
    ref = x.double() @ wg.double().T
    mag = x.double().abs() @ wg.double().abs().T
    # products exact; d / 64 blocks of 64 products in the tensor cores' FP32 (truncating:
    # a whole step of 2^-23 each) and the blocks' sums
    ref64.within(logits, ref, (64 + d // 64 + 2) * 2.0 ** -23 * mag, "logits")
    # the library's own softmax router on these logits: moe_gate_topk's choice and weights
    bias = 0.02 * (torch.rand(E, device="cuda") - 0.5)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_gate_topk(dm, x, wg, bias, idx, w, None, ws)
    cfg = dict(score=SM, n_group=1, topk_group=1, group_top=2, renorm=True, scale=1.0, k=k)
    _, _, idx2, w2, _ = call(logits, bias, cfg)
    same = (idx == idx2).all(1)
    assert same.float().mean() > 0.99
    ref64.within(w[same], w2[same], 1e-5, "weights")
    # backward
    dl = torch.randn(T, E, device="cuda")
    dx = torch.randn(T, d, device="cuda").bfloat16()
    dx0, dwg = dx.clone(), torch.full((E, d), 3.0, device="cuda")
    for acc in (0, 1):
        before = dwg.clone()
        moe.moe_gate_bwd(dm, x, wg, dl, dx if acc == 0 else dx.clone(), dwg, acc, ws)
        rw = dl.double().T @ x.double() + (before.double() if acc else 0)
        scale = (dl.double().abs().T @ x.double().abs()).amax()
        ref64.within(dwg, rw, 1e-4 * scale, "dwg")
    rx = dx0.double() + dl.double() @ wg.double()
    ref64.within(dx, rx, 1e-2 * rx.abs().amax(), "dx")
    assert moe.moe_get_device_status(ws) == 0


# ---- from 2560 tokens on, a token of up to 128 experts takes a few lanes of a warp

MANY = 2563      # an odd number: the last warp's lanes are not all taken


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("E,k", [(8, 1), (8, 8), (16, 3), (64, 8), (64, 9), (72, 16), (120, 5),
                                 (128, 16), (128, 17), (100, 6)])
def test_many_tokens_match_64_bits(E, k, score):
    for dtype, bias in itertools.product((torch.float32, torch.bfloat16), (True, False)):
        check(*make(MANY, E, k, E + k, bias, dtype, score=score, scale=2.5))
    x, b, cfg = make(MANY, E, k, E, True, torch.bfloat16, score=score)
    check(x, torch.zeros_like(b), cfg)            # many equal scores
    check(x, b.round(decimals=2), cfg)
    check(*make(MANY, E, k, E + 1, score=score, renorm=False))


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("E,G,K,top,k", [(128, 8, 4, 2, 8), (128, 4, 1, 2, 6), (128, 16, 3, 1, 9),
                                         (64, 2, 1, 2, 8), (64, 8, 3, 1, 3), (96, 3, 2, 2, 5)])
def test_groups_of_many_tokens_match_64_bits(E, G, K, top, k, score):
    for dtype, bias in itertools.product((torch.float32, torch.bfloat16), (True, False)):
        x, b, cfg = make(MANY, E, k, E + G, bias, dtype, score=score, n_group=G, topk_group=K,
                         group_top=top, scale=1.5)
        check(x, b, cfg)
        x[::3] = x[::3].round()                   # groups of equal scores too
        check(x, b, cfg)


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("E", [64, 128])
def test_many_tokens_near_equal_masked_and_extreme(E, score):
    T = MANY
    g = torch.Generator(device="cuda").manual_seed(E)
    base = torch.randint(0, 4, (T, E), generator=g, device="cuda").float()
    x = base + 2.0 ** -22 * torch.randint(0, 4, (T, E), generator=g, device="cuda")
    b = 2.0 ** -26 * torch.randint(0, 8, (E,), generator=g, device="cuda").float()
    for groups in (dict(), dict(n_group=4, topk_group=2)):
        cfg = dict(score=score, n_group=1, topk_group=1, group_top=2, renorm=True, scale=1.0,
                   k=6) | groups
        check(x, b, cfg)
        check(x, None, cfg)
        check(base, b * 0, cfg)
        y, c, _ = make(T, E, 6, 3)
        y[::5] = -INF                             # tokens without any expert beside others
        y[1::5, 3:] = -INF
        y[2::5, ::2] = -INF
        y[3::5, ::3] = torch.finfo(torch.float32).min
        check(y, c, cfg)
        c[5:E // 2] = -INF
        check(y, c, cfg)
        check(*make(T, E, 6, 4, std=30.0, **{n: cfg[n] for n in cfg if n != "k"}))
    # a token with NaN or infinite logits leaves its neighbours in the warp alone
    x, b, cfg = make(T, E, 6, 6, score=score)
    x[0, 5], x[9], x[18, 7], x[27, 1] = math.nan, math.nan, INF, -INF
    _, _, idx, w, p = call(x, b, cfg)
    ridx, rw, rp, _ = ref64.route(x, b, cfg)
    assert torch.equal(idx, ridx)
    assert torch.equal(w.isnan(), rw.isnan()) and torch.equal(p.isnan(), rp.isnan())
    fin = ~rw.isnan()
    ref64.within(w[fin], rw[fin], 2 * (24 + 16) * 2.0 ** -23 * rw[fin], "weights")


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("E,k,L", [(8, 8, 0), (64, 8, 2000), (64, 5, 0), (128, 16, 700),
                                   (128, 6, 0), (96, 7, 1), (100, 6, 130), (64, 12, 50)])
def test_bwd_of_many_tokens(E, k, L, score):
    for dtype, renorm in itertools.product((torch.float32, torch.bfloat16), (True, False)):
        x, b, cfg = make(MANY, E, k, E * k, True, dtype, score=score, scale=2.5, renorm=renorm)
        x[7] = -INF
        x[8, 3:] = -INF
        dm, rc, idx, w, _ = call(x, b, cfg)
        g = torch.Generator(device="cuda").manual_seed(E)
        dw = torch.randn(MANY, k, generator=g, device="cuda")
        sg = torch.randn(-(-MANY // L), E, generator=g, device="cuda") if L else None
        bwd_check(x, idx, w, dw, cfg, rc, dm, sg, L)
        idx = idx.clone()
        idx[3, 0], idx[4, k - 1], idx[5, 0] = -1, E, 1 << 30       # no expert: skipped
        if k > 1:
            idx[6, 1] = idx[6, 0]                 # the same expert twice
            idx[MANY - 1, k - 1] = idx[MANY - 1, 0]
        if k > 2:
            idx[100, 2] = idx[100, 1] = idx[100, 0]
        bwd_check(x, idx, w, dw, cfg, rc, dm, sg, L)


def test_many_tokens_on_unaligned_views():
    # bases off the 16-byte pieces: element-wise accesses, the same results
    x, b, cfg = make(MANY, 64, 6, 9, dtype=torch.bfloat16)
    flat = torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")
    y = flat[1:].view_as(x)
    y.copy_(x)
    _, _, i1, w1, p1 = call(x, b, cfg)
    _, _, i2, w2, p2 = call(y, b, cfg)
    assert torch.equal(i1, i2)
    ref64.within(w2, w1, 2.0 ** -20 * w1, "weights")
    ref64.within(p2, p1, 2.0 ** -20 * p1, "probs")


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("T", [50, MANY])
@pytest.mark.parametrize("groups", [dict(), dict(n_group=4, topk_group=2)])
def test_infinite_and_nan_biases(groups, T, score):
    x, b, cfg = make(T, 64, 6, 12, score=score, **groups)
    for at, v in (([3, 40, 41], INF), ([3], INF), (list(range(20, 30)), INF), ([7, 50], -INF),
                  ([9], math.nan), ([5, 6, 30], torch.finfo(torch.float32).max)):
        c = b.clone()
        c[at] = v
        _, _, idx, w, _ = call(x, c, cfg)
        ridx, rw, _, _ = ref64.route(x, c, cfg)
        assert torch.equal(idx, ridx), (at, v)
        ref64.within(w, rw, 2 * (24 + 16) * 2.0 ** -23 * rw, "weights")


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("T", [50, MANY])
@pytest.mark.parametrize("groups", [dict(), dict(n_group=4, topk_group=2)])
@pytest.mark.parametrize("E", [64, 128])
def test_picks_of_infinite_score(E, groups, T, score):
    # fewer, exactly and more experts with a bias of +inf than the token picks, in one lane's
    # experts, spread over all, and more than a warp of them
    x, b, cfg = make(T, E, 6, 12, score=score, **groups)
    step = E // 16
    for at in ([3, 40], [0, 1, 2, 3, 4], [0, 1, 2, 3, 4, 5], list(range(E - 7, E)),
               list(range(0, E, step)), list(range(5, 45)), list(range(E))):
        c = b.clone()
        c[at] = INF
        _, _, idx, w, _ = call(x, c, cfg)
        ridx, rw, _, _ = ref64.route(x, c, cfg)
        assert torch.equal(idx, ridx), at
        ref64.within(w, rw, 2 * (24 + 16) * 2.0 ** -23 * rw, "weights")


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("T", [50, MANY])
def test_biases_of_the_lowest_value_beside_groups_that_are_not_kept(T, score):
    # the picks after the first have the lowest finite score, as the experts of the groups that
    # are not kept would have, of which some stand before them
    low = torch.finfo(torch.float32).min
    x, b, cfg = make(T, 32, 6, 13, score=score, n_group=4, topk_group=1)
    for one in (12, 20, 31):
        c = torch.full_like(b, low)
        c[one] = 0.25
        _, _, idx, w, _ = call(x, c, cfg)
        ridx, rw, _, _ = ref64.route(x, c, cfg)
        assert torch.equal(idx, ridx), one
        ref64.within(w, rw, 2 * (24 + 16) * 2.0 ** -23 * rw, "weights")


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("T", [50, MANY])
@pytest.mark.parametrize("E,G", [(32, 4), (64, 4), (60, 5), (128, 16), (250, 10), (256, 64)])
def test_group_scores_beyond_fp32(E, G, T, score):
    # two of a group's scores are finite and their sum is below FP32's lowest value, or above
    # its highest: the groups are ordered by the sum all the same
    x, b, cfg = make(T, E, 3, 14, score=score, n_group=G, topk_group=2)
    low = torch.finfo(torch.float32).min
    per = E // G
    for sign in (1.0, -1.0):
        c = torch.full_like(b, sign * low)
        for g, f in ((0, 0.9), (1, 0.8), (2, 0.6), (G - 1, 0.7)):
            c[g * per:(g + 1) * per] = sign * f * low
        for y in (x, x.index_fill(1, torch.arange(per, device="cuda"), -INF)):
            _, _, idx, w, _ = call(y, c, cfg)
            ridx, rw, _, _ = ref64.route(y, c, cfg)
            assert torch.equal(idx, ridx)
            ref64.within(w, rw, 2 * (24 + 16) * 2.0 ** -23 * rw, "weights")


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("T", [50, MANY])
@pytest.mark.parametrize("E,G", [(32, 4), (128, 8), (60, 5), (256, 16)])
def test_a_group_of_one_infinite_and_masked_experts_ranks_last(E, G, T, score):
    # inf - inf as a group's score: it ranks as -inf, and topk_group groups stay all the same
    x, b, cfg = make(T, E, 3, 15, score=score, n_group=G, topk_group=2)
    per = E // G
    for one in (0, per - 1, E - 1):
        c, y = b.clone(), x.clone()
        g = one // per
        c[one] = INF
        for e in range(g * per, (g + 1) * per):
            if e != one:
                if e % 2:
                    c[e] = -INF
                else:
                    y[:, e] = -INF
        _, _, idx, w, _ = call(y, c, cfg)
        d = b.clone()
        d[g * per:(g + 1) * per] = -INF             # the same choice as without the group
        ridx, rw, _, _ = ref64.route(y, d, cfg)
        assert torch.equal(idx, ridx), one
        ref64.within(w, rw, 2 * (24 + 16) * 2.0 ** -23 * rw, "weights")
        check(y, c, cfg | dict(group_top=1))


@pytest.mark.parametrize("T,d,E", [(1, 64, 8), (300, 128, 8), (1000, 192, 96), (129, 256, 256),
                                   (2100, 320, 128)])
def test_gate_bwd_element_by_element(T, d, E):
    """Each element against the magnitude of its own terms.  The operands are split exactly
    into three bf16 planes, whose magnitudes add up to less than 1.02 of the value; a matrix
    instruction adds 16 products to the accumulator, cutting at most three steps of 2^-23 of
    the terms so far; dX drops three pairs of planes below 2^-24 each and is rounded once to
    bf16; dWg adds up to 64 partial sums."""
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, wg, dl = r(T, d).bfloat16(), 0.05 * r(E, d), r(T, E) * torch.exp(2 * r(T, 1))
    dl[::7] = 0.0
    dm = moe.MoeDims.of(T, d, E, 1, 0, 64, 64)
    ws = torch.zeros(moe.moe_workspace_size(dm), dtype=torch.uint8, device="cuda")
    dx0 = (0.01 * r(T, d)).bfloat16()
    blocks = lambda n: -(-n // 64) * 4  # noqa: E731  instructions of one plane pair
    for acc in (0, 1):
        dx, dwg = dx0.clone(), r(E, d)
        w0 = dwg.double() if acc else torch.zeros(E, d, dtype=torch.float64, device="cuda")
        moe.moe_gate_bwd(dm, x, wg, dl, dx, dwg, acc, ws)
        rx = dx0.double() + dl.double() @ wg.double()
        mag = dx0.double().abs() + dl.double().abs() @ wg.double().abs()
        tol = (18 * blocks(E) + 4) * 1.02 * 2.0 ** -23 * mag
        ref64.within(dx, rx, tol + 2.0 ** -8 * (rx.abs() + tol), "dx")
        rw = w0 + dl.double().T @ x.double()
        mag = w0.abs() + dl.double().abs().T @ x.double().abs()
        ref64.within(dwg, rw, (9 * blocks(T) + 66) * 1.02 * 2.0 ** -23 * mag, "dwg")
    assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("T", [60, MANY])
@pytest.mark.parametrize("E", [64, 128, 256])
def test_bwd_of_picks_far_below_the_others(E, T, score):
    # the bias chooses experts whose affinities are subnormal numbers of FP32 beside small ones:
    # their gradients are ordinary numbers
    x, b, cfg = make(T, E, 4, 31, score=score, scale=1.5)
    if score == SG:
        x = x - 60.0
    b = torch.zeros_like(b)
    for j, e in enumerate((3, E // 2, E - 1, 17)):
        b[e] = 2.0 - 0.1 * j
        x[:, e] = x[:, e] * 0.5 - (30.0, 90.0, 95.0, 45.0)[j] + (0.0 if score == SM else 60.0)
    dm, rc, idx, w, _ = check(x, b, cfg)
    dw = torch.randn(T, 4, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    bwd_check(x, idx, w, dw, cfg, rc, dm)
    sg = torch.randn(-(-T // 50), E, device="cuda")
    if score == SM:
        bwd_check(x, idx, w, dw, cfg, rc, dm, sg, 50)


@pytest.mark.parametrize("T", [60, MANY])
@pytest.mark.parametrize("E", [64, 128, 256])
def test_bwd_of_picks_of_tiny_sigmoids(E, T):
    x, b, cfg = make(T, E, 4, 32, score=SG, scale=1.5)
    b = torch.zeros_like(b)
    for j, e in enumerate((3, E // 2, E - 1, 17)):
        b[e] = 2.0 - 0.1 * j
        x[:, e] = x[:, e] * 0.5 - (30.0, 90.0, 97.0, 75.0)[j]
    dm, rc, idx, w, _ = check(x, b, cfg)
    dw = torch.randn(T, 4, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    bwd_check(x, idx, w, dw, cfg, rc, dm)
    bwd_check(x, idx, w, dw, cfg, rc, dm, torch.randn(-(-T // 50), E, device="cuda"), 50)


@pytest.mark.parametrize("score", [SM, SG])
@pytest.mark.parametrize("T", [60, MANY])
@pytest.mark.parametrize("E", [64, 128, 256])
def test_factors_of_any_size(E, T, score):
    # scale / (sum of the picks) leaves FP32 where the weights do not, at either end
    for scale in (1e32, -1e32, 1e-32):
        x, b, cfg = make(T, E, 4, 33, score=score, scale=scale)
        b = torch.zeros_like(b)
        for j, e in enumerate((3, E // 2, E - 1, 17)):
            b[e] = 2.0 - 0.1 * j
            x[:, e] = x[:, e] * 0.5 - 36.0
        dm, rc, idx, w, _ = call(x, b, cfg)
        ridx, rw, _, _ = ref64.route(x, b, cfg)
        assert torch.equal(idx, ridx)
        ref64.within(w, rw, 2 * (24 + 45) * 2.0 ** -23 * rw.abs(), "weights")
        assert w.isfinite().all() and (w != 0).all()
        dw = torch.randn(T, 4, generator=torch.Generator(device="cuda").manual_seed(T),
                         device="cuda")
        bwd_check(x, idx, w, dw, cfg, rc, dm)
