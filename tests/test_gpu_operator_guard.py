"""Every output and workspace of the operators around the layer stands between bands of a
known pattern: at odd sizes, on every path of the kernels, nothing is written beside them."""
import itertools

import pytest
import torch

import grouped_gemm_fp32_b200 as moe

pytestmark = pytest.mark.gpu
BAND = 4096      # bytes on either side
SM, SG = "softmax", "sigmoid"


class Guarded:
    def __init__(self):
        self.all = []

    def __call__(self, *shape, dt=torch.float32, like=None, off=0):
        """A tensor between two bands; off: elements that its address is past 16 bytes."""
        shape, dt = (like.shape, like.dtype) if like is not None else (shape, dt)
        n = dt.itemsize * torch.Size(shape).numel()
        lo = BAND + off * dt.itemsize
        raw = torch.full((lo + n + BAND + 16,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((raw, lo, n))
        t = raw[lo:lo + n].view(dt).view(shape)
        return t.copy_(like) if like is not None else t

    def check(self):
        torch.cuda.synchronize()
        for raw, lo, n in self.all:
            assert bool((raw[:lo] == 0xA5).all()) and bool((raw[lo + n:] == 0xA5).all())


@pytest.mark.parametrize("T", [1, 37, 2561])
@pytest.mark.parametrize("E,k,G,K", [(1, 1, 1, 1), (7, 3, 1, 1), (64, 6, 8, 3), (100, 5, 4, 2),
                                     (128, 6, 1, 1), (250, 9, 1, 1), (256, 8, 8, 4), (256, 40, 1, 1)])
def test_routing(T, E, k, G, K):
    if T > 2000 and k > 32:
        T = 300
    for score, dt, off in itertools.product((SM, SG), (torch.float32, torch.bfloat16), (0, 1)):
        g = Guarded()
        x = g(like=torch.randn(T, E, device="cuda").to(dt), off=off)
        bias = g(like=0.01 * torch.randn(E, device="cuda"), off=off)
        if T > 30:
            x[3], x[5, ::2], x[9, 0] = -torch.inf, -torch.inf, torch.nan
            x[11] = 0.0
        dm, rc = moe.MoeDims.of(T, 64, E, k, 0, 64, 64), moe.MoeRouteCfg.of(score, G, K, 1)
        idx, w, p = g(T, k, dt=torch.int32), g(T, k), g(T, E, off=off)
        moe.moe_route_topk(dm, rc, x, bias, idx, w, p)
        dl, sg = g(T, E, dt=dt, off=off), g(like=torch.randn(-(-T // 7), E, device="cuda"))
        moe.moe_route_bwd(dm, rc, x, idx, w, g(like=torch.randn(T, k, device="cuda")), sg, 7, dl)
        assert int(idx.min()) >= 0 and int(idx.max()) < E
        g.check()


@pytest.mark.parametrize("T,d", [(1, 64), (5, 192), (777, 1984), (300, 2112), (601, 4160),
                                 (20, 8256), (9, 16384)])
@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32])
def test_norms(T, d, rt):
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    for L in (0, 3, 130):
        g = Guarded()
        rows = -(-T // L) if L else 1
        dm, cfg = moe.MoeDims.of(T, d, 8, 1, 0, 64, 64), moe.MoeNormCfg.of(seq_len=L)
        y, res, gate = g(like=r(T, d).to(bf)), g(like=r(T, d).to(rt)), g(like=r(rows, d))
        w1, w2 = g(like=r(d)), g(like=r(d))
        u, n = g(T, d, dt=rt), g(T, d, dt=bf)
        moe.moe_block_norm(dm, cfg, None, res, None, None, w2, None, n)
        moe.moe_block_norm(dm, cfg, y, res, w1, gate, w2, u, n)
        dy, dres = g(T, d, dt=bf), g(T, d, dt=rt)
        dw1, dw2, dg = g(d), g(d), g(rows, d)
        ws = g(moe.moe_norm_workspace_size(dm, cfg), dt=torch.uint8)
        dn, du = g(like=r(T, d).to(bf)), g(like=r(T, d).to(rt))
        moe.moe_block_norm_bwd(dm, cfg, dn, du, y, u, w1, gate, w2, dy, dres, dw1, dg, dw2, 0, ws)
        moe.moe_block_norm_bwd(dm, cfg, dn, None, None, res, None, None, w2, None, dres, None, None,
                               dw2, 1, ws)
        assert dres.isfinite().all() and dw1.isfinite().all() and dg.isfinite().all()
        g.check()


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
def test_gradients(t):
    g = Guarded()
    sizes = [1, 7, 8, 9, 255, 2048, 2049, 32767, 32769, 70_001, 524_289]
    for a, b in itertools.product(range(0, 8, 3), range(8)):
        grads = [g(like=torch.randn(n, device="cuda").to(t), off=a) for n in sizes]
        outs = [g(n, dt=t, off=b) for n in sizes]
        lst = moe.GradList(grads, outs)
        sumsq, norm, coef = g(1, dt=torch.float64), g(1), g(1)
        ws = g(moe.moe_grad_workspace_size(len(lst)), dt=torch.uint8)
        moe.moe_grad_clip_norm(lst, 1.0, sumsq, norm, coef, ws)
        for x, o in zip(grads, outs):   # one rounding to t of an FP32 product, as torch makes it
            assert torch.equal(o, (x.float() * coef).to(t))
        g.check()
        g.all.clear()
