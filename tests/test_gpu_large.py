"""The operators around the layer on tensors of more than 2^31 elements: the last rows give
what they give alone (element offsets pass 32 bits)."""
import math

import pytest
import torch

import grouped_gemm_fp32_b200 as moe

pytestmark = pytest.mark.gpu


def test_routing():
    T, E, k, last = (1 << 31) // 256 + 5000, 256, 8, 3000
    x = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    some = torch.empty(4096, E, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    for t in range(0, T, 4096):
        x[t:t + 4096] = some[:min(4096, T - t)]
    x[-last:].normal_(generator=g)
    bias = 0.01 * torch.randn(E, generator=g, device="cuda")
    rc = moe.MoeRouteCfg.of("sigmoid", 8, 4, scale=2.5)

    def run(z, dw):
        t = z.shape[0]
        dm = moe.MoeDims.of(t, 64, E, k, 0, 64, 64)
        idx = torch.empty(t, k, dtype=torch.int32, device="cuda")
        w, dl = torch.empty(t, k, device="cuda"), torch.empty_like(z)
        moe.moe_route_topk(dm, rc, z, bias, idx, w, None)
        moe.moe_route_bwd(dm, rc, z, idx, w, dw, None, 0, dl)
        return idx, w, dl

    dw = torch.randn(T, k, generator=g, device="cuda")
    big = run(x, dw)
    for a, b in zip(big, run(x[-last:].contiguous(), dw[-last:].contiguous())):
        assert torch.equal(a[-last:], b)


def test_block_norms():
    T, d, last = (1 << 31) // 4096 + 300, 4096, 200
    g = torch.Generator(device="cuda").manual_seed(2)
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    res = torch.empty_like(y).normal_(generator=g)
    w1, w2 = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    cfg = moe.MoeNormCfg.of()

    def run(y, res):
        dm = moe.MoeDims.of(y.shape[0], d, 8, 1, 0, 64, 64)
        u, n = torch.empty_like(res), torch.empty_like(y)
        moe.moe_block_norm(dm, cfg, y, res, w1, None, w2, u, n)
        ws = torch.empty(moe.moe_norm_workspace_size(dm, cfg), dtype=torch.uint8, device="cuda")
        dy, dres = torch.empty_like(y), torch.empty_like(res)
        moe.moe_block_norm_bwd(dm, cfg, n, res, y, u, w1, None, w2, dy, dres, None, None, None, 0,
                               ws)
        return u, n, dy, dres

    for a, b in zip(run(y, res), run(y[-last:].contiguous(), res[-last:].contiguous())):
        assert torch.equal(a[-last:], b)


def test_gradient_of_more_than_2_31_elements():
    n = (1 << 31) + 12_345
    x = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    x[-1] = 3.0
    lst = moe.GradList([x])
    sumsq = torch.zeros(1, dtype=torch.float64, device="cuda")
    norm, coef = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    ws = torch.empty(moe.moe_grad_workspace_size(1), dtype=torch.uint8, device="cuda")
    moe.moe_grad_clip_norm(lst, 1024.0, sumsq, norm, coef, ws)
    want = (n - 1) * 0.25 + 9.0                 # every partial sum is exact in 64 bits
    assert float(sumsq) == want
    c = 1024.0 / (math.sqrt(want) + 1e-6)
    assert abs(float(coef) - c) <= 2.0 ** -23 * c
    got = torch.stack([x[0], x[1 << 30], x[-2], x[-1]]).double().cpu()
    ref = c * torch.tensor([0.5, 0.5, 0.5, 3.0], dtype=torch.float64)
    assert ((got - ref).abs() <= 2.0 ** -8 * ref).all()
    assert bool((x[:-1] == x[0]).all())
