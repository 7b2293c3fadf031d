"""Argument and shape checks of the routers of other kinds, the block norms and the
gradient norm and clipping: refused before anything is launched (CPU only), by the C
calls with a status and by the binding with a ValueError that names the tensor."""
import ctypes
import math

import pytest
import torch

import grouped_gemm_fp32_b200 as moe
from grouped_gemm_fp32_b200 import _lib

P = ctypes.c_void_p(4096)       # an address that is never followed: checks come first
ODD = ctypes.c_void_p(4097)
OFF8 = ctypes.c_void_p(4104)    # not 16-byte aligned
NUL = None
BIG = 1 << 40
INVALID, SHAPE = -1, -2


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_gemm_fp32_b200 import build
    build.build()


def dims(T=64, d=128, E=8, k=2):
    return ctypes.byref(moe.MoeDims.of(T, d, E, k, 0, 64, 64))


def route(dm=None, cfg=None, kind=moe.MOE_F32, x=P, idx=P, w=P):
    cfg = moe.MoeRouteCfg.of() if cfg is None else cfg
    return moe.load().moe_route_topk(dims() if dm is None else dm, ctypes.byref(cfg), kind, x,
                                     NUL, idx, w, NUL, NUL)


def route_bwd(dm=None, cfg=None, kind=moe.MOE_F32, x=P, idx=P, w=P, dw=P, sg=NUL, L=0, out=P):
    cfg = moe.MoeRouteCfg.of() if cfg is None else cfg
    return moe.load().moe_route_bwd(dims() if dm is None else dm, ctypes.byref(cfg), kind, x, idx,
                                    w, dw, sg, L, out, NUL)


def test_route_refusals():
    R = moe.MoeRouteCfg.of
    for f in (route, route_bwd):
        for cfg, status in ((R(score=2), INVALID), (R(n_group=0), INVALID),
                            (R(n_group=4, topk_group=5), INVALID),
                            (R(n_group=4, topk_group=0), INVALID), (R(group_top=3), INVALID),
                            (R(scale=math.nan), INVALID), (R(scale=math.inf), INVALID),
                            (R(n_group=3, topk_group=1), SHAPE),    # 8 experts in 3 groups
                            (R(n_group=8, topk_group=3, group_top=2), SHAPE),  # groups of one
                            (R(n_group=8, topk_group=1, group_top=1), SHAPE)):  # k = 2 of 1
            assert f(cfg=cfg) == status, (f, cfg.score, cfg.n_group)
        bad = R()
        bad.renorm = 2
        assert f(cfg=bad) == INVALID
        for dm, status in ((dims(T=-1), INVALID), (dims(E=0), INVALID), (dims(k=0), INVALID),
                           (dims(E=257), SHAPE), (dims(k=9), SHAPE),
                           (dims(T=1 << 31, k=1), SHAPE), (NUL, INVALID)):
            lib = moe.load()
            cfg = ctypes.byref(R())
            got = lib.moe_route_topk(dm, cfg, 0, P, NUL, P, P, NUL, NUL) if f is route else \
                lib.moe_route_bwd(dm, cfg, 0, P, P, P, P, NUL, 0, P, NUL)
            assert got == status
        for kind in (moe.MOE_F16, -1, 7):
            assert f(kind=kind) == INVALID
        for name in ("x", "idx", "w"):
            assert f(**{name: NUL}) == INVALID
    assert route_bwd(dw=NUL) == INVALID and route_bwd(out=NUL) == INVALID
    assert route_bwd(sg=P, L=0) == INVALID
    assert moe.load().moe_route_topk(dims(), None, 0, P, NUL, P, P, NUL, NUL) == INVALID
    # no tokens: nothing is needed, nothing is launched
    assert route(dm=dims(T=0), x=NUL, idx=NUL, w=NUL) == 0
    assert route_bwd(dm=dims(T=0), x=NUL, idx=NUL, w=NUL, dw=NUL, out=NUL) == 0


def test_gate_refusals():
    L = moe.load()
    for dm, status in ((dims(d=100), SHAPE), (dims(E=12), SHAPE), (dims(T=-1), INVALID)):
        assert L.moe_gate_logits(dm, P, P, P, P, BIG, NUL) == status
        assert L.moe_gate_bwd(dm, P, P, P, P, P, 0, P, BIG, NUL) == status
    for i in range(4):
        a = [P] * 4
        a[i] = NUL
        assert L.moe_gate_logits(dims(), *a, BIG, NUL) == INVALID
    assert L.moe_gate_logits(dims(), P, P, P, P, 8, NUL) == INVALID
    for i in range(5):
        a = [P] * 5
        a[i] = NUL
        assert L.moe_gate_bwd(dims(), *a, 0, P, BIG, NUL) == INVALID
    assert L.moe_gate_bwd(dims(), P, P, P, P, P, 0, P, 8, NUL) == INVALID


def norm(dm=None, cfg=None, kind=moe.MOE_BF16, y=P, res=P, wp=P, g=P, w=P, out=P, n=P):
    cfg = moe.MoeNormCfg.of() if cfg is None else cfg
    return moe.load().moe_block_norm(dims() if dm is None else dm, ctypes.byref(cfg), kind, y, res,
                                     wp, g, w, out, n, NUL)


def norm_bwd(dm=None, cfg=None, kind=moe.MOE_BF16, dn=P, du=P, y=P, u=P, wp=P, g=P, w=P, dy=P,
             dres=P, dwp=P, dg=P, dw=P, acc=0, ws=P, nbytes=BIG):
    cfg = moe.MoeNormCfg.of() if cfg is None else cfg
    return moe.load().moe_block_norm_bwd(dims() if dm is None else dm, ctypes.byref(cfg), kind, dn,
                                         du, y, u, wp, g, w, dy, dres, dwp, dg, dw, acc, ws,
                                         nbytes, NUL)


def test_norm_refusals():
    C = moe.MoeNormCfg.of
    for f in (norm, norm_bwd):
        for cfg in (C(eps=0.0), C(eps=-1.0), C(eps=math.nan), C(eps=math.inf),
                    C(res_scale=math.nan), C(block_scale=math.inf), C(seq_len=-1)):
            assert f(cfg=cfg) == INVALID
        for dm, status in ((dims(d=96), SHAPE), (dims(d=16448), SHAPE), (dims(T=-1), INVALID),
                           (dims(T=1 << 31), SHAPE), (dims(d=0), INVALID)):
            assert f(dm=dm) == status
        for kind in (moe.MOE_F16, -1, 9):
            assert f(kind=kind) == INVALID
    for name in ("y", "res", "wp", "g", "w", "out", "n"):
        assert norm(**{name: OFF8}) == INVALID, name
    for name in ("dn", "du", "y", "u", "wp", "g", "w", "dy", "dres", "dwp", "dg", "dw", "ws"):
        assert norm_bwd(**{name: OFF8}) == INVALID, name
    # what belongs together
    assert norm(res=NUL) == INVALID and norm(out=NUL) == INVALID
    assert norm(w=NUL) == INVALID and norm(n=NUL) == INVALID
    assert norm(y=NUL) == INVALID                          # a post-norm without a block
    assert norm(y=NUL, wp=NUL, g=NUL) == INVALID           # res_out without a block
    assert norm(y=NUL, wp=NUL, g=NUL, out=NUL, w=NUL, n=NUL) == INVALID  # nothing to do
    assert norm_bwd(dn=NUL) == INVALID                     # w_pre without dn
    assert norm_bwd(dn=NUL, w=NUL, dw=NUL, du=NUL) == INVALID
    assert norm_bwd(u=NUL) == INVALID and norm_bwd(w=NUL) == INVALID
    assert norm_bwd(y=NUL) == INVALID and norm_bwd(dy=NUL) == INVALID
    assert norm_bwd(wp=NUL) == INVALID and norm_bwd(g=NUL) == INVALID   # their gradients asked
    assert norm_bwd(dres=NUL) == INVALID and norm_bwd(ws=NUL) == INVALID
    assert norm_bwd(acc=2) == INVALID
    need = moe.moe_norm_workspace_size(moe.MoeDims.of(64, 128, 8, 2, 0, 64, 64), C())
    assert need > 0 and norm_bwd(nbytes=need - 1) == INVALID
    assert moe.moe_norm_workspace_size(moe.MoeDims.of(64, 96, 8, 2, 0, 64, 64), C()) == 0
    # one gate row per sequence: the workspace grows with them
    few, many = (moe.moe_norm_workspace_size(moe.MoeDims.of(4096, 128, 8, 2, 0, 64, 64),
                                             C(seq_len=s)) for s in (0, 1))
    assert many > few
    assert norm(dm=dims(T=0)) == 0


def test_grad_refusals():
    L = moe.load()
    one = lambda **kw: (moe.MoeGrad * 1)(moe.MoeGrad(**(dict(data=4096, out=None, n=4, type=0) | kw)))  # noqa: E731,E501
    clip = lambda a, n=1, s=P, m=1.0: L.moe_grad_clip(a, n, s, ctypes.c_float(m), NUL, NUL, NUL)  # noqa: E731,E501
    for bad in (one(type=3), one(type=-1), one(n=-1), one(data=None), one(data=4097),
                one(data=4098), one(out=4098), one(out=4097, type=moe.MOE_BF16)):
        assert clip(bad) == INVALID
        assert L.moe_grad_norm(bad, 1, 0, P, NUL, P, BIG, NUL) == INVALID
        assert L.moe_grad_clip_norm(bad, 1, ctypes.c_float(1.0), P, NUL, NUL, P, BIG, NUL) == INVALID
    ok = one()
    assert clip(ok, -1) == INVALID and clip(None) == INVALID and clip(ok, s=NUL) == INVALID
    for m in (-1.0, math.nan):
        assert clip(ok, m=m) == INVALID
        assert L.moe_grad_clip_norm(ok, 1, ctypes.c_float(m), P, NUL, NUL, P, BIG, NUL) == INVALID
    need = moe.moe_grad_workspace_size(1)
    for args in ((NUL, NUL, P, BIG), (P, NUL, NUL, BIG), (P, NUL, P, need - 1)):
        assert L.moe_grad_norm(ok, 1, 0, *args, NUL) == INVALID
        assert L.moe_grad_clip_norm(ok, 1, ctypes.c_float(1.0), args[0], NUL, NUL, args[2],
                                    args[3], NUL) == INVALID
    assert L.moe_grad_norm(ok, 1, 2, P, NUL, P, BIG, NUL) == INVALID
    assert moe.moe_grad_workspace_size(-1) == 0
    assert moe.moe_grad_workspace_size(100_000) > moe.moe_grad_workspace_size(1) > 0


def test_binding_refuses_what_it_cannot_pass(monkeypatch):
    _lib._types()
    monkeypatch.setitem(_lib._TYPES, "device", lambda: 0)   # no GPU here: pretend one is current
    dm, cfg = moe.MoeDims.of(4, 128, 8, 2, 0, 64, 64), moe.MoeRouteCfg.of()
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="logits.*element type"):
        moe.moe_route_topk(dm, cfg, x.half(), None, 16, 16, None, 0)
    with pytest.raises(ValueError, match="logits: on cpu"):
        moe.moe_route_topk(dm, cfg, x, None, 16, 16, None, 0)
    with pytest.raises(ValueError, match="logits: shape"):
        moe.moe_route_topk(dm, cfg, x[:3], None, 16, 16, None, 0)
    with pytest.raises(ValueError, match="logits: not contiguous"):
        moe.moe_route_topk(dm, cfg, torch.zeros(8, 4).T, None, 16, 16, None, 0)
    n = moe.MoeNormCfg.of()
    with pytest.raises(ValueError, match="y: torch.float32"):
        moe.moe_block_norm(dm, n, torch.zeros(4, 128), torch.zeros(4, 128), None, None, None, 16,
                           None, 0)
    with pytest.raises(ValueError, match="res: unsupported"):
        moe.moe_block_norm(dm, n, None, torch.zeros(4, 128, dtype=torch.int32), None, None, 16,
                           None, 16, 0)
    with pytest.raises(ValueError, match="gradient: on cpu"):
        moe.GradList([torch.zeros(4)])
    with pytest.raises(ValueError, match="gradient: not contiguous"):
        moe.GradList([torch.zeros(4, 4).T])
    with pytest.raises(ValueError, match="unsupported element type"):
        moe.GradList([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError, match="2 gradients, 1 outs"):
        moe.GradList([1, 2], [3])


def test_routing_refuses_outputs_over_its_logits():
    R, L = moe.MoeRouteCfg.of, _lib.load()
    dm, cfg = moe.MoeDims.of(64, 128, 8, 2, 0, 64, 64), R()
    near = ctypes.c_void_p(4096 + 64 * 8 * 4 - 4)      # the last of the logits
    for out in (P, near):
        assert L.moe_route_topk(ctypes.byref(dm), ctypes.byref(cfg), moe.MOE_F32, P, NUL, P, P,
                                out, NUL) == INVALID
        assert L.moe_route_bwd(ctypes.byref(dm), ctypes.byref(cfg), moe.MOE_F32, P, P, P, P, NUL,
                               0, out, NUL) == INVALID
    for i in range(5):         # an address between two elements
        p = [P, NUL, P, P, ctypes.c_void_p(1 << 20)]
        p[i] = ODD
        assert L.moe_route_topk(ctypes.byref(dm), ctypes.byref(cfg), moe.MOE_F32, *p,
                                NUL) == INVALID
        p = [P, P, P, P, NUL, 0, ctypes.c_void_p(1 << 20)]
        p[(0, 1, 2, 3, 6)[i]] = ODD
        assert L.moe_route_bwd(ctypes.byref(dm), ctypes.byref(cfg), moe.MOE_BF16, *p,
                               NUL) == INVALID


def test_gradient_calls_refuse_unaligned_results_and_workspaces():
    L = _lib.load()
    one = (moe.MoeGrad * 1)(moe.MoeGrad(4096, None, 4, moe.MOE_F32))
    four = ctypes.c_void_p(4100)        # aligned for FP32, not for 64 bits
    for sumsq, norm, ws in ((four, NUL, P), (P, ODD, P), (P, NUL, four)):
        assert L.moe_grad_norm(one, 1, 0, sumsq, norm, ws, BIG, NUL) == INVALID
        assert L.moe_grad_clip_norm(one, 1, 1.0, sumsq, norm, NUL, ws, BIG, NUL) == INVALID
    assert L.moe_grad_clip_norm(one, 1, 1.0, P, NUL, ODD, P, BIG, NUL) == INVALID
    for sumsq, norm, coef in ((four, NUL, NUL), (P, ODD, NUL), (P, NUL, ODD)):
        assert L.moe_grad_clip(one, 1, sumsq, 1.0, norm, coef, NUL) == INVALID


def test_gradient_calls_refuse_a_list_of_another_device(monkeypatch):
    # the list holds addresses: those of another device must not reach a kernel on this one
    _lib._types()
    monkeypatch.setitem(_lib._TYPES, "device", lambda: -1)   # host tensors play device -1
    lst, none = moe.GradList([torch.zeros(4)]), moe.GradList([])
    monkeypatch.setitem(_lib._TYPES, "device", lambda: 0)
    ws = torch.zeros(8, dtype=torch.uint8)
    for call in (lambda g: moe.moe_grad_norm(g, 0, 16, None, ws, 0),
                 lambda g: moe.moe_grad_clip(g, torch.zeros(1), 1.0, None, None, 0),
                 lambda g: moe.moe_grad_clip_norm(g, 1.0, 16, None, None, ws, 0)):
        with pytest.raises(ValueError, match="gradients: on device -1, the current device is cuda:0"):
            call(lst)
        with pytest.raises(ValueError, match="ws: a contiguous|sumsq: torch.float32"):
            call(none)      # a list without tensors has no device: the next check answers


@pytest.mark.parametrize("d", [64, 320, 1024, 1088, 2048, 2112, 4096, 8256, 16384])
@pytest.mark.parametrize("L", [0, 130])
def test_norm_workspaces_grow_with_the_tokens(d, L):
    # one allocated for the most tokens of a run serves every smaller batch
    cfg = moe.MoeNormCfg.of(seq_len=L)
    sizes = [moe.moe_norm_workspace_size(moe.MoeDims.of(T, d, 8, 1, 0, 64, 64), cfg)
             for T in [*range(0, 3000), *range(16000, 16400), *range(1 << 20, (1 << 20) + 50)]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("L", [5, 1 << 40, (1 << 63) - 4, (1 << 63) - 1])
def test_sequences_longer_than_the_tokens_are_one_row(monkeypatch, L):
    # T + L - 1 would leave 64 bits
    for T in (1, 2, 5):
        dm = moe.MoeDims.of(T, 128, 8, 2, 0, 64, 64)
        size = lambda n: moe.moe_norm_workspace_size(dm, moe.MoeNormCfg.of(seq_len=n))  # noqa: E731
        assert size(L) == size(0)
    _lib._types()
    monkeypatch.setitem(_lib._TYPES, "device", lambda: -1)     # host tensors; no call is made
    x = torch.zeros(5, 8)
    with pytest.raises(ValueError, match="seq_grad: shape .* 8 needed"):
        moe.moe_route_bwd(dm, moe.MoeRouteCfg.of(), x, 16, 16, 16, torch.zeros(7), L, x, 0)
    with pytest.raises(ValueError, match="gate: shape .* 128 needed"):
        moe.moe_block_norm(dm, moe.MoeNormCfg.of(seq_len=L), 16, torch.zeros(5, 128), 16,
                           torch.zeros(1), 16, 16, 16, 0)


def test_first_calls_of_two_threads_find_a_whole_table(monkeypatch):
    # a second thread that comes in while the first fills the table must not find half of it
    class Table(dict):
        def update(self, *a, **kw):
            super().update(*a, **kw)
            assert {torch.float32, torch.bfloat16, torch.float16, "device", "stream"} <= set(self)

    monkeypatch.setattr(_lib, "_TYPES", Table())
    assert _lib._types()[torch.bfloat16] == moe.MOE_BF16 and _lib._TYPES


def _at(i, n=0):
    return ctypes.c_void_p((i << 20) + n)      # addresses a MB apart


def test_routing_refuses_outputs_over_what_other_tokens_read():
    L, cfg = _lib.load(), ctypes.byref(moe.MoeRouteCfg.of())
    T, E, k = 64, 8, 2
    dm = dims(T=T, E=E, k=k)
    sizes = dict(logits=T * E * 4, bias=E * 4, idx=T * k * 4, w=T * k * 4, probs=T * E * 4)
    names = list(sizes)
    for out in ("idx", "w", "probs"):
        for other in names:
            if other == out:
                continue
            for off in (0, sizes[other] - 4, 4 - sizes[out]):     # over it, its end, its start
                p = {n: _at(i + 1) for i, n in enumerate(names)}
                p[out] = _at(names.index(other) + 1, off)
                assert L.moe_route_topk(dm, cfg, 0, *(p[n] for n in names), NUL) == INVALID, \
                    (out, other, off)
    sizes = dict(logits=T * E * 4, idx=T * k * 4, w=T * k * 4, dw=T * k * 4, sg=8 * E * 4)
    names = list(sizes)
    for i, other in enumerate(names):
        for off in (0, sizes[other] - 4, 4 - T * E * 4):
            p = [_at(j + 1) for j in range(5)]
            assert L.moe_route_bwd(dm, cfg, 0, *p, 8, _at(i + 1, off), NUL) == INVALID, (other, off)


def test_norms_refuse_outputs_over_what_other_rows_read():
    L = _lib.load()
    T, d = 64, 128
    dm, cfg = dims(T=T, d=d), ctypes.byref(moe.MoeNormCfg.of(seq_len=8))
    rows, row = T * d * 2, d * 4
    f = dict(y=rows, res=rows, wp=row, g=8 * row, w=row, out=rows, n=rows)
    b = dict(dn=rows, du=rows, y=rows, u=rows, wp=row, g=8 * row, w=row, dy=rows, dres=rows,
             dwp=row, dg=8 * row, dw=row)
    for sizes, outs, call in (
            (f, ("out", "n"), lambda p: L.moe_block_norm(dm, cfg, 1, *p, NUL)),
            (b, ("dy", "dres", "dwp", "dg", "dw"),
             lambda p: L.moe_block_norm_bwd(dm, cfg, 1, *p, 0, _at(40), BIG, NUL))):
        names = list(sizes)
        for out in outs:
            for other in names:
                if other == out:
                    continue
                # an input of the same shape may be the output itself
                same = sizes[other] == sizes[out] == rows and other not in outs
                for off in (0, sizes[other] - 16, 16 - sizes[out])[1 if same else 0:]:
                    p = {n: _at(i + 1) for i, n in enumerate(names)}
                    p[out] = _at(names.index(other) + 1, off)
                    assert call(list(p.values())) == INVALID, (out, other, off)


def test_the_binding_is_built_again_for_another_torch_or_python(monkeypatch):
    from grouped_gemm_fp32_b200 import build
    assert not build.bind_stale()
    with monkeypatch.context() as m:
        m.setattr(build.importlib.metadata, "version", lambda name: "0.0.1+other")
        assert build.bind_stale()
    with monkeypatch.context() as m:
        m.setattr(build.sys.implementation, "cache_tag", "cpython-399")
        assert build.bind_stale()
    assert not build.bind_stale()


def test_token_counts_whose_picks_leave_64_bits():
    for T, k in (((1 << 62) + 4, 2), ((1 << 61) + 4, 8), (1 << 62, 4)):
        assert route(dm=dims(T=T, k=k)) == SHAPE
        assert route_bwd(dm=dims(T=T, k=k)) == SHAPE


def test_clipping_refuses_tensors_that_overlap_what_it_writes(monkeypatch):
    # a tensor in the list twice would be scaled once or twice, as the CTAs come
    _lib._types()
    monkeypatch.setitem(_lib._TYPES, "device", lambda: -1)     # host tensors; no call is made
    x, y = torch.zeros(100), torch.zeros(100)
    ws = torch.zeros(8, dtype=torch.uint8)
    bad = [([x, x], None), ([x, x[50:]], None), ([x[:60], y, x[59:]], None), ([x, y], [y, None]),
           ([x, y], [None, x]), ([x[:50], y[:50]], [y[50:], y[50:]]), ([x[1:50]], [x[:49]])]
    for grads, outs in bad:
        lst = moe.GradList(grads, outs)
        for call in (lambda: moe.moe_grad_clip(lst, 16, 1.0, None, None, 0),
                     lambda: moe.moe_grad_clip_norm(lst, 1.0, 16, None, None, ws, 0)):
            with pytest.raises(ValueError, match="gradients: .* overlap"):
                call()
        # a norm alone writes none of them: the next check answers
        with pytest.raises(ValueError, match="sumsq"):
            moe.moe_grad_norm(lst, 0, x, None, ws, 0)
    for grads, outs in (([x[:50], x[50:]], None), ([x, x], [y, torch.zeros(100)]),
                        ([x, y], [x, y]), ([x[:0], x], None), ([x, x[:0]], [y, y[10:10]])):
        with pytest.raises(ValueError, match="sumsq"):
            moe.moe_grad_clip(moe.GradList(grads, outs), x, 1.0, None, None, 0)


def test_gate_calls_refuse_outputs_over_their_operands():
    L = _lib.load()
    T, d, E = 64, 128, 8
    dm = dims(T=T, d=d, E=E)
    sizes = dict(x=T * d * 2, wg=E * d * 4, logits=T * E * 4)
    for other in ("x", "wg"):
        for off in (0, sizes[other] - 16, 16 - sizes["logits"]):
            p = [_at(1), _at(2), _at(1 + ("x", "wg").index(other), off)]
            assert L.moe_gate_logits(dm, *p, _at(9), BIG, NUL) == INVALID, (other, off)
    sizes = dict(x=T * d * 2, wg=E * d * 4, dl=T * E * 4, dx=T * d * 2, dwg=E * d * 4)
    names = list(sizes)
    for out in ("dx", "dwg"):
        for other in names:
            for off in (0, sizes[other] - 16, 16 - sizes[out]):
                if other == out:
                    continue
                p = [_at(i + 1) for i in range(5)]
                p[names.index(out)] = _at(names.index(other) + 1, off)
                assert L.moe_gate_bwd(dm, *p, 0, _at(9), BIG, NUL) == INVALID, (out, other, off)
