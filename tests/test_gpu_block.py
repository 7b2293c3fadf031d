"""The routers of other kinds, the block norms and the clipping as the layer's driver runs
them together: layer.forward / backward with a route config, layer.block_forward /
block_backward, layer.GradClip, expert parallelism with a route config, and all of it
captured in one CUDA graph.

The operators themselves are tested elsewhere; here each part of a run is checked against
the 64-bit form on the part's own inputs, or against the same calls made one by one."""
import itertools

import pytest
import torch
import torch.distributed as dist

import grouped_gemm_fp32_b200 as moe
import ref64
import synth
from common import dev, dims_of
from grouped_gemm_fp32_b200 import ep, layer

pytestmark = pytest.mark.gpu

ROW_TOL = 1e-2   # bf16 outputs, relative to max|ref| (the layer's own bar)
DW_TOL = 1e-4    # f32 sums of the same products in another order
SIGMOID = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, renorm=True, scale=2.5)
SOFTMAX = dict(score="softmax", n_group=1, topk_group=1, group_top=2, renorm=False, scale=1.0)


def case(T=300, d=128, E=16, k=4, S=1, seed=31):
    wl = synth.Workload("block", synth.Dims(T=T, d=d, E=E, k=k, S=S, I=64, P=64), seed=seed,
                        w1_std=0.05, w2_std=0.05, wg_std=0.05, backward=True)
    inp = synth.make_inputs(wl)
    t = {n: dev(inp[n], True) for n in ("x", "w1", "w2", "dout")}
    t |= {n: dev(inp[n]) for n in ("wg", "bias")}
    return dims_of(wl), t


def rcfg(c):
    return moe.MoeRouteCfg.of(**c)


def rel(got, ref):
    return float((got.double() - ref.double()).abs().max() / ref.double().abs().max())


@pytest.mark.parametrize("c", [SIGMOID, SOFTMAX], ids=["sigmoid_groups", "softmax"])
@pytest.mark.parametrize("balance", [None, (1e-2, 128)])
def test_layer_with_another_router(c, balance):
    dm, t = case()
    b = layer.MoEBuffers(dm, train=True, route=rcfg(c))
    layer.forward(b, t["x"], t["wg"], t["bias"], t["w1"], t["w2"], seq_balance=balance)
    cfg = c | dict(k=dm.k)
    idx, w, probs, _ = ref64.route(b.logits, t["bias"], cfg)
    assert torch.equal(b.topk_idx, idx)
    # the tests of moe_route_topk derive (24 + spread) 2^-23; the spread is below 20 here
    ref64.within(b.topk_w, w, 2 * 44 * 2.0 ** -23 * w, "weights")
    ref64.within(b.probs, probs, 44 * 2.0 ** -23 * probs, "probs")
    # the same experts on the same routing: the same bits
    o = layer.MoEBuffers(dm, train=True)
    layer.forward(o, t["x"], t["wg"], t["bias"], t["w1"], t["w2"],
                  routing=(b.topk_idx, b.topk_w, b.probs), seq_balance=balance)
    assert torch.equal(o.out, b.out)
    layer.backward(b, t["x"], t["dout"], t["w1"], t["w2"], wg=t["wg"])
    layer.backward(o, t["x"], t["dout"], t["w1"], t["w2"])
    assert torch.equal(o.dw1, b.dw1) and torch.equal(o.dw_comb, b.dw_comb)
    sg, L = (b.bal_grad[:-(-dm.T // 128)], 128) if balance else (None, 0)
    dl, mag = ref64.route_bwd(b.logits, b.topk_idx, b.topk_w, b.dw_comb, cfg, sg, L)
    ref64.within(b.dlogits, dl, (64 + dm.k + 40) * 2.0 ** -23 * mag + 2.0 ** -126, "dlogits")
    assert rel(b.dx, o.dx.double() + b.dlogits.double() @ t["wg"].double()) <= ROW_TOL
    assert rel(b.dwg, b.dlogits.double().T @ t["x"].double()) <= DW_TOL
    assert moe.moe_get_device_status(b.ws) == 0


def test_router_backward_needs_the_routers_logits():
    dm, t = case(T=64)
    b = layer.MoEBuffers(dm, train=True, route=rcfg(SIGMOID))
    layer.forward(b, t["x"], t["wg"], t["bias"], t["w1"], t["w2"])
    layer.forward(b, t["x"], t["wg"], t["bias"], t["w1"], t["w2"],
                  routing=(b.topk_idx.clone(), b.topk_w.clone()))
    with pytest.raises(ValueError, match="ran the router"):
        layer.backward(b, t["x"], t["dout"], t["w1"], t["w2"], wg=t["wg"])


def block_inputs(dm, rt, L, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, d = dm.T, dm.d
    rows = -(-T // L) if L else 1
    return dict(res=(2 * r(T, d)).to(rt), w_pre=1 + 0.1 * r(d), w_post=1 + 0.1 * r(d),
                w_next=1 + 0.1 * r(d), gate=0.5 + 0.1 * r(rows, d), dres_out=r(T, d).to(rt),
                dn_next=r(T, d).bfloat16())


def bounds(ref, mag, t, d):
    """Sums of d terms (d / 512 + 16 roundings on a path) and a dozen products, of the
    terms' magnitudes, and the rounding to t."""
    return (d / 512 + 40) * ref64.U * mag + ref64.HALF[t] * ref.abs() + ref64.TINY[t]


@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post,nxt,L", list(itertools.product((True, False), (True, False), (0, 130))))
def test_block(post, nxt, L, rt):
    dm, t = case()
    cfg = moe.MoeNormCfg.of(1e-5, 1.0, 0.7, L)
    a = (1e-5, 1.0, 0.7, L)
    bb = layer.BlockBuffers(dm, cfg, rt, train=True, route=rcfg(SIGMOID))
    i = block_inputs(dm, rt, L)
    kw = dict(w_post=i["w_post"] if post else None, gate=i["gate"],
              w_next=i["w_next"] if nxt else None)
    res0 = i["res"].clone()
    res_out, n_next = layer.block_forward(bb, i["res"], i["w_pre"], t["wg"], t["bias"], t["w1"],
                                          t["w2"], **kw)
    _, n, _ = ref64.block_norm(None, i["res"], None, None, i["w_pre"], *a)
    ref64.within(bb.n, n, bounds(n, n.abs(), torch.bfloat16, dm.d), "n")
    u, nn, mag = ref64.block_norm(bb.moe.out, i["res"], kw["w_post"], i["gate"], kw["w_next"], *a)
    ref64.within(res_out, u, bounds(u, mag, rt, dm.d), "res_out")
    assert torch.equal(i["res"], res0) and (n_next is not None) == nxt
    # the layer ran on n
    o = layer.MoEBuffers(dm, train=True, route=rcfg(SIGMOID))
    assert torch.equal(layer.forward(o, bb.n, t["wg"], t["bias"], t["w1"], t["w2"]), bb.moe.out)
    dres = layer.block_backward(bb, i["dres_out"], i["res"], i["w_pre"], t["wg"], t["w1"],
                                t["w2"], dn_next=i["dn_next"] if nxt else None, gamma=1e-3,
                                bias=t["bias"], **kw)
    r = ref64.block_norm_bwd(i["dn_next"] if nxt else None, i["dres_out"], bb.moe.out, res_out,
                             kw["w_post"], i["gate"], kw["w_next"], *a)
    ref64.within(bb.dy, r["dy"][0], bounds(*r["dy"], torch.bfloat16, dm.d), "dy")
    names = [("dgate", True), ("dw_post", post)]
    if nxt:
        ref64.within(bb.dw_next, r["dw_pre"][0], bounds(*r["dw_pre"], torch.float32, 512 * 40),
                     "dw_next")
    for name, on in names:
        if on:
            ref64.within(getattr(bb, name), r[name][0], bounds(*r[name], torch.float32, 512 * 40),
                         name)
    # the layer's backward from dy, then the pre-norm's
    dn, dw1, _, _ = layer.backward(o, bb.n, bb.dy, t["w1"], t["w2"], wg=t["wg"])
    assert torch.equal(dw1, bb.moe.dw1) and torch.equal(dn, bb.moe.dx)
    # what the first norm's backward stored is within its bound of r["dres"] (unrounded: a
    # second rounding of it here would be another half step), and enters with factor 1
    r2 = ref64.block_norm_bwd(dn, r["dres"][0], None, i["res"], None, None, i["w_pre"], *a)
    tol = bounds(*r2["dres"], rt, dm.d) + bounds(*r["dres"], rt, dm.d)
    ref64.within(dres, r2["dres"][0], tol, "dres")
    ref64.within(bb.dw_pre, r2["dw_pre"][0], bounds(*r2["dw_pre"], torch.float32, 512 * 40),
                 "dw_pre")


def test_two_blocks_share_a_norm():
    # block 1 hands its n_next to block 2, and block 2's gradient parts go back into block 1
    dm, t = case(T=130)
    cfg = moe.MoeNormCfg.of()
    i = block_inputs(dm, torch.float32, 0)
    one, two, sep = (layer.BlockBuffers(dm, cfg, torch.float32, train=True) for _ in range(3))
    w = (t["wg"], t["bias"], t["w1"], t["w2"])
    r1, n1 = layer.block_forward(one, i["res"], i["w_pre"], *w, w_post=i["w_post"],
                                 w_next=i["w_next"])
    r2, none = layer.block_forward(two, r1, None, *w, w_post=i["w_post"], n=n1)
    assert none is None
    s2, _ = layer.block_forward(sep, r1, i["w_next"], *w, w_post=i["w_post"])
    # n of an FP32 residual is the same number from either pass, up to its last rounding
    assert rel(n1, sep.n) <= 2.0 ** -8 and rel(r2, s2) <= ROW_TOL
    back = (t["wg"], t["w1"], t["w2"])
    dres, dn = layer.block_backward(two, i["dres_out"], r1, None, *back, w_post=i["w_post"], n=n1)
    got = layer.block_backward(one, dres, i["res"], i["w_pre"], *back, w_post=i["w_post"],
                               w_next=i["w_next"], dn_next=dn)
    a = (1e-6, 1.0, 1.0, 0)
    r = ref64.block_norm_bwd(dn, dres, one.moe.out, r1, i["w_post"], None, i["w_next"], *a)
    ref64.within(one.dy, r["dy"][0], bounds(*r["dy"], torch.bfloat16, dm.d), "dy")
    assert got.isfinite().all()
    with pytest.raises(ValueError, match="come together"):
        layer.block_backward(one, dres, i["res"], i["w_pre"], *back, w_next=i["w_next"])


def test_train_step_in_a_graph():
    """Block forward and backward and the clipping of every weight's gradient, captured once:
    replays on new inputs give the eager step's bits, and two graphs share nothing."""
    dm, t = case(seed=37)
    cfg = moe.MoeNormCfg.of(1e-6, 1.0, 1.0, 130)
    bufs = [layer.BlockBuffers(dm, cfg, train=True, route=rcfg(SIGMOID)) for _ in range(2)]
    ins = [block_inputs(dm, torch.bfloat16, 130, seed=s) for s in (3, 4)]
    clips = [layer.GradClip([b.moe.dw1, b.moe.dw2, b.moe.dwg, b.dw_pre, b.dw_post, b.dgate])
             for b in bufs]

    def step(b, i, clip):
        layer.block_forward(b, i["res"], i["w_pre"], t["wg"], t["bias"], t["w1"], t["w2"],
                            w_post=i["w_post"], gate=i["gate"], seq_balance=(1e-2, 130))
        layer.block_backward(b, i["dres_out"], i["res"], i["w_pre"], t["wg"], t["w1"], t["w2"],
                             w_post=i["w_post"], gate=i["gate"], gamma=1e-3, bias=t["bias"])
        clip.clip(1.0)

    def results(b, clip):
        m = b.moe
        return [v.clone() for v in (b.res_out, b.dres, m.dw1, m.dw2, m.dwg, b.dw_pre, b.dw_post,
                                    b.dgate, m.bias_next, m.bal_loss, clip.norm, clip.coef)]

    want = []
    for b, i, c in zip(bufs, ins, clips):
        step(b, i, c)
        want.append(results(b, c))
        grads = [v.double() for v in c.whole.grads]
        assert abs(float(torch.sqrt(sum(v.square().sum() for v in grads)))
                   - min(1.0, float(c.norm))) < 1e-5 and float(c.norm) > 1.0
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs = []
    for b, i, c in zip(bufs, ins, clips):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(b, i, c)
        graphs.append(g)
    for order in ((0, 1), (1, 0)):
        for j in order:
            for v in (bufs[j].res_out, bufs[j].dres, bufs[j].moe.dw1, clips[j].norm):
                v.zero_()
            graphs[j].replay()
        torch.cuda.synchronize()
        for j in order:
            assert all(map(torch.equal, results(bufs[j], clips[j]), want[j]))
    # new inputs in place
    for n, v in ins[1].items():
        ins[0][n].copy_(v)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(map(torch.equal, results(bufs[0], clips[0]), want[1]))


def test_host_pipeline_with_another_router():
    dm, t = case(T=128)
    pin = lambda v: v.cpu().pin_memory()  # noqa: E731
    hx, hd = [pin(t["x"])], [pin(t["dout"])]
    ho, hdx = [torch.empty_like(hx[0]).pin_memory()], [torch.empty_like(hx[0]).pin_memory()]
    pipe = layer.HostPipeline(dm, t["w1"], t["w2"], t["wg"], t["bias"], True, gamma=1e-3,
                              route=rcfg(SIGMOID))
    pipe.run(hx, hd, ho, hdx, 1)
    pipe.synchronize()
    b = layer.MoEBuffers(dm, train=True, route=rcfg(SIGMOID))
    layer.forward(b, t["x"], t["wg"], t["bias"], t["w1"], t["w2"])
    layer.backward(b, t["x"], t["dout"], t["w1"], t["w2"], wg=t["wg"], gamma=1e-3, bias=t["bias"])
    torch.cuda.synchronize()
    assert torch.equal(ho[0], b.out.cpu()) and torch.equal(hdx[0], b.dx.cpu())


@pytest.fixture
def nccl_one_rank():
    dist.init_process_group("nccl", store=dist.HashStore(), rank=0, world_size=1,
                            device_id=torch.device("cuda", 0))
    try:
        yield
    finally:
        dist.destroy_process_group()


def test_expert_parallel_with_another_router_and_clipping(nccl_one_rank):
    dm, t = case(T=257, seed=41)
    s = torch.cuda.Stream()
    ref = layer.MoEBuffers(dm, train=True, route=rcfg(SIGMOID))
    eb = ep.EPBuffers(dm, 0, 1, train=True, alloc=ep.symmetric_alloc(1, "cuda"),
                      route=rcfg(SIGMOID))
    ep.connect(eb)
    E = dm.E
    clip = layer.GradClip([eb.full.dwg, eb.loc.dw1[E:], eb.loc.dw2[E:]],
                          sharded=[eb.loc.dw1[:E], eb.loc.dw2[:E]])
    whole = layer.GradClip([ref.dwg, ref.dw1, ref.dw2])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.forward(ref, t["x"], t["wg"], t["bias"], t["w1"], t["w2"], stream=s)
        layer.backward(ref, t["x"], t["dout"], t["w1"], t["w2"], stream=s, wg=t["wg"])
        whole.clip(0.5, stream=s)
        ep.forward(eb, t["x"], t["wg"], t["bias"], t["w1"], t["w2"], stream=s)
        ep.backward(eb, t["x"], t["dout"], t["w1"], t["w2"], stream=s, wg=t["wg"])
        clip.clip(0.5, stream=s)
    s.synchronize()
    assert ep.status(eb) == 0
    assert torch.equal(eb.full.topk_idx, ref.topk_idx)
    assert rel(eb.full.out, ref.out) <= ROW_TOL and rel(eb.full.dx, ref.dx) <= ROW_TOL
    assert rel(clip.norm, whole.norm) <= DW_TOL and float(whole.norm) > 0.5
    for got, want in ((eb.full.dwg, ref.dwg), (eb.loc.dw1, ref.dw1), (eb.loc.dw2, ref.dw2)):
        assert rel(got, want) <= 2 * DW_TOL


def test_operators_after_a_fork_and_join_in_a_capture():
    """Inside a capture the operators stand behind a join of two streams, a memset and a copy,
    and between other kernels: every replay sees what those wrote."""
    T, E, k, d = 300, 64, 6, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    src, logits, bias = r(T, E), torch.zeros(T, E, device="cuda"), 0.01 * r(E)
    dm, rc = moe.MoeDims.of(T, d, E, k, 0, 64, 64), rcfg(SIGMOID | dict(n_group=8, topk_group=4))
    idx, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    dl, dw = torch.zeros(T, E, device="cuda"), r(T, k)
    y, res, wn = r(T, d).bfloat16(), torch.zeros(T, d, device="cuda"), 1 + 0.1 * r(d)
    base, u = r(T, d), torch.zeros(T, d, device="cuda")
    n = torch.zeros(T, d, device="cuda").bfloat16()
    grads = [torch.zeros(5000, device="cuda"), torch.zeros(77, device="cuda")]
    clip = layer.GradClip(grads)
    side = torch.cuda.Stream()

    def step(main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            res.copy_(base)
            res.mul_(2.0)
        logits.copy_(src)
        logits.add_(0.5)
        main.wait_stream(side)
        idx.zero_()
        moe.moe_route_topk(dm, rc, logits, bias, idx, w, None)
        moe.moe_route_bwd(dm, rc, logits, idx, w, dw, None, 0, dl)
        dl.mul_(3.0)
        u.zero_()
        moe.moe_block_norm(dm, moe.MoeNormCfg.of(), y, res, wn, None, wn, u, n)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            grads[1].fill_(2.0)
        grads[0].copy_(u.view(-1)[:5000])
        main.wait_stream(side)
        clip.clip(1.0)

    outs = [idx, w, dl, u, n, clip.norm, *grads]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(s)
    s.synchronize()
    want = [o.clone() for o in outs]
    assert float(clip.norm) > 1.0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for _ in range(3):
        for o in outs + [logits, res]:
            o.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(map(torch.equal, outs, want))
    src.mul_(-1.0)
    base.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    with torch.cuda.stream(s):
        step(s)
    s.synchronize()
    assert all(map(torch.equal, outs, got))


def test_block_refuses_a_residual_that_its_backward_would_miss():
    dm, t = case(T=64)
    bb = layer.BlockBuffers(dm, moe.MoeNormCfg.of(), train=True)
    w = torch.ones(dm.d, device="cuda")
    with pytest.raises(ValueError, match="cannot be this block's res_out"):
        layer.block_forward(bb, bb.res_out, w, t["wg"], t["bias"], t["w1"], t["w2"])


def test_exchanges_run_on_a_stream_given_by_its_handle(nccl_one_rank):
    # every call takes a stream's handle as an integer; so do the ones with an all-reduce in them
    s = torch.cuda.Stream()
    for handle in (s.cuda_stream, 0):
        with layer.on_stream(handle):
            assert torch.cuda.current_stream().cuda_stream == handle
    assert torch.cuda.current_stream().cuda_stream == 0
    x, y = torch.full((1 << 24,), 0.5, device="cuda"), torch.full((77,), 2.0, device="cuda")
    clip = layer.GradClip([y], sharded=[x])
    torch.cuda.synchronize()
    clip.clip(1.0, stream=s.cuda_stream)
    s.synchronize()
    want = (0.25 * (1 << 24) + 4.0 * 77) ** 0.5
    assert abs(float(clip.norm) - want) <= 2.0 ** -22 * want


def test_block_refuses_an_input_that_its_backward_would_miss():
    # n_next is written by the forward; the backward reads n again
    dm, t = case(T=64)
    w = torch.ones(dm.d, device="cuda")
    res = torch.randn(dm.T, dm.d, device="cuda").bfloat16()
    args = (res, None, t["wg"], t["bias"], t["w1"], t["w2"])
    bb = layer.BlockBuffers(dm, moe.MoeNormCfg.of(), train=True)
    bb.n_next.normal_()
    with pytest.raises(ValueError, match="cannot be this block's n_next"):
        layer.block_forward(bb, *args, w_next=w, n=bb.n_next)
    layer.block_forward(bb, *args, n=bb.n_next)          # not written: as any other tensor
    # without a backward one set of buffers serves a run of blocks
    run = layer.BlockBuffers(dm, moe.MoeNormCfg.of())
    run.n_next.copy_(bb.n_next)
    other = layer.BlockBuffers(dm, moe.MoeNormCfg.of())
    want = layer.block_forward(other, *args, w_next=w, n=run.n_next.clone())
    got = layer.block_forward(run, *args, w_next=w, n=run.n_next)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("W,E,k", [(2, 16, 4), (4, 32, 6)])
def test_emulated_expert_parallel_ranks_with_another_router(W, E, k):
    # every phase for every rank in turn (no kernel waits for another beside it), against the
    # layer on the concatenated batch
    T, S = 150, 1
    dm, t = case(T=T, E=E, k=k, S=S, seed=43)
    g = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, dout = [r(T, dm.d) for _ in range(W)], [r(T, dm.d) for _ in range(W)]
    wg, bias, w1, w2 = t["wg"], t["bias"], t["w1"], t["w2"]
    ref = layer.MoEBuffers(moe.MoeDims.of(W * T, dm.d, E, k, S, dm.I, dm.P), train=True,
                           route=rcfg(SIGMOID))
    layer.forward(ref, torch.cat(x), wg, bias, w1, w2)
    layer.backward(ref, torch.cat(x), torch.cat(dout), w1, w2, wg=wg)
    ebs = [ep.EPBuffers(dm, i, W, train=True, route=rcfg(SIGMOID)) for i in range(W)]
    ep.connect_emulated(ebs)
    El = E // W
    wl = [[torch.cat([w[i * El:(i + 1) * El], w[E:]]).contiguous() for w in (w1, w2)]
          for i in range(W)]
    for i, eb in enumerate(ebs):
        ep.route(eb, x[i], wg, bias)
    table = torch.stack([eb.full.counts for eb in ebs])
    for eb in ebs:
        eb.counts_all.copy_(table)
        ep.plan(eb)
    for i, eb in enumerate(ebs):
        ep.dispatch(eb, x[i])
    for i, eb in enumerate(ebs):
        ep.experts_forward(eb, x[i], *wl[i])
    out = [ep.combine(eb).clone() for eb in ebs]
    for i, eb in enumerate(ebs):
        ep.backward_dispatch(eb, dout[i])
    for i, eb in enumerate(ebs):
        ep.experts_backward(eb, x[i], dout[i], *wl[i])
    dx = [ep.unpermute_and_router(eb, x[i], wg).clone() for i, eb in enumerate(ebs)]
    torch.cuda.synchronize()
    assert all(ep.status(eb) == 0 for eb in ebs)
    full = lambda n: torch.cat([getattr(eb.full, n) for eb in ebs])  # noqa: E731
    # a token's logits and choice are the same whichever rank it is on
    assert torch.equal(full("logits"), ref.logits) and torch.equal(full("topk_idx"), ref.topk_idx)
    assert torch.equal(full("topk_w"), ref.topk_w)
    assert rel(torch.cat(out), ref.out) <= ROW_TOL and rel(torch.cat(dx), ref.dx) <= ROW_TOL
    assert rel(full("dlogits"), ref.dlogits) <= DW_TOL
    assert rel(sum(eb.full.dwg.double() for eb in ebs), ref.dwg) <= DW_TOL
    for n in ("dw1", "dw2"):
        got = torch.cat([getattr(eb.loc, n)[:El] for eb in ebs])
        assert rel(got, getattr(ref, n)[:E]) <= DW_TOL
