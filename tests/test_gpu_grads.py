"""moe_grad_norm, moe_grad_clip and moe_grad_clip_norm against their 64-bit forms.

The norm is a 64-bit sum rounded once to FP32 (2^-24, twice that with its root); the
coefficient is rounded once, the clipped element once more to its type."""
import itertools
import math

import pytest
import torch

import grouped_gemm_fp32_b200 as moe
import ref64
from ref64 import HALF, TINY, U, within

pytestmark = pytest.mark.gpu
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16


def state(lst, n=None):
    n = len(lst) if n is None else n
    dev = dict(device="cuda")
    return dict(sumsq=torch.full((1,), 7.0, dtype=torch.float64, **dev),
                norm=torch.full((1,), 7.0, **dev), coef=torch.full((1,), 7.0, **dev),
                ws=torch.full((moe.moe_grad_workspace_size(n),), 0xFF, dtype=torch.uint8, **dev))


def check(grads, max_norm=1.0, outs=True):
    """Out of place into `outs` (made here when True), then in place."""
    norm, coef, ref = ref64.grad_clip(grads, max_norm)
    if outs is True:
        outs = [torch.full_like(g, 7.0) for g in grads]
    keep = [g.clone() for g in grads]
    lst = moe.GradList(grads, outs)
    s = state(lst)
    moe.moe_grad_clip_norm(lst, max_norm, s["sumsq"], s["norm"], s["coef"], s["ws"])
    within(s["norm"], torch.tensor([norm], dtype=torch.float64), 3 * U * norm, "norm")
    within(s["coef"], torch.tensor([coef], dtype=torch.float64), 3 * U * coef, "coef")
    within(s["sumsq"], torch.tensor([norm * norm], dtype=torch.float64), 1e-12 * norm * norm,
           "sumsq")
    for g, k, o, r in zip(grads, keep, outs, ref):
        assert torch.equal(g, k)
        within(o, r, (3 * U + HALF[o.dtype] * (1 + 3 * U)) * r.abs() + TINY[o.dtype], "clipped")
    moe.moe_grad_clip_norm(moe.GradList(keep), max_norm, s["sumsq"], s["norm"], s["coef"],
                           s["ws"])
    for k, o in zip(keep, outs):
        assert torch.equal(k, o)     # in place: the same bits


def rand(n, t, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + n)
    return (std * torch.randn(n, generator=g, device="cuda")).to(t)


@pytest.mark.parametrize("t", [F32, BF, F16])
@pytest.mark.parametrize("sizes", [[1], [7, 8, 9], [1, 0, 3, 5], [16384, 16385, 16383],
                                   [100_003], [3_000_001, 17], [1_000_000] * 3 + [1]])
def test_sizes(sizes, t):
    grads = [rand(n, t, i) for i, n in enumerate(sizes)]
    check(grads)
    check(grads, 1e6)                # below the clipping norm: copied, or left alone
    check(grads, 0.0)
    check(grads, math.inf)


@pytest.mark.parametrize("t", [F32, BF, F16])
def test_every_alignment_of_data_and_out(t):
    # data and out start at every element offset inside 16 bytes, and nothing around out
    # changes
    per = 16 // torch.empty(0, dtype=t).element_size()
    for n, (a, b) in itertools.product((1, 5, 37, 20_001), itertools.product(range(per), repeat=2)):
        src = rand(n + 2 * per, t, a)
        dst = torch.full((n + 2 * per,), 9.0, dtype=t, device="cuda")
        g, o = src[a:a + n], dst[b:b + n]
        check([g], 0.5, [o])
        assert (dst[:b] == 9).all() and (dst[b + n:] == 9).all()


def test_many_tensors_of_mixed_types_in_a_packed_buffer():
    # more tensors than one launch takes; odd sizes packed back to back
    for count in (511, 512, 513, 1300):
        sizes = [(i * 37) % 91 + (0 if i % 50 else 5000) for i in range(count)]
        types = [(F32, BF, F16)[i % 3] for i in range(count)]
        buf = {t: torch.full((sum(n for n, x in zip(sizes, types) if x is t),), 7.0, dtype=t,
                             device="cuda") for t in (F32, BF, F16)}
        at, grads, outs = dict.fromkeys(buf, 0), [], []
        for i, (n, t) in enumerate(zip(sizes, types)):
            grads.append(rand(n, t, i))
            outs.append(buf[t][at[t]:at[t] + n])
            at[t] += n
        check(grads, 3.0, outs)


def test_empty_lists():
    for grads in ([], [torch.empty(0, device="cuda")]):
        lst = moe.GradList(grads)
        s = state(lst)
        moe.moe_grad_clip_norm(lst, 1.0, s["sumsq"], s["norm"], s["coef"], s["ws"])
        assert float(s["norm"]) == 0 and float(s["coef"]) == 1 and float(s["sumsq"]) == 0


def test_large_and_small_values():
    # squares beyond FP32's range on both sides, and small ones next to large ones
    for v in (1e25, 3e37, 1e-30, 1e-38, 1e-42):
        g = torch.full((100_001,), v, device="cuda")
        lst = moe.GradList([g])
        s = state(lst)
        moe.moe_grad_norm(lst, 0, s["sumsq"], s["norm"], s["ws"])
        exact = float(g[0]) * math.sqrt(100_001)
        assert abs(float(s["sumsq"]) / exact ** 2 - 1) < 1e-12
        if exact < 3e38:
            # 1e-42 gives a norm of 3.2e-40: FP32 subnormals are 2^-149 apart
            assert abs(float(s["norm"]) - exact) <= 1e-6 * exact + 2.0 ** -150
    g = torch.cat([torch.full((1000,), 1e20, device="cuda"), rand(1000, F32, 1),
                   torch.zeros(4096, device="cuda"), torch.full((5000,), 1e-25, device="cuda")])
    check([g], 1.0)
    check([g[1000:2000], g[6100:]], 1.0)
    check([torch.zeros(100_000, device="cuda"), torch.zeros(33, device="cuda", dtype=BF)], 1.0)


@pytest.mark.parametrize("bad,coef", [(math.inf, 0.0), (-math.inf, 0.0), (math.nan, math.nan)])
def test_non_finite_gradients_follow_the_formula(bad, coef):
    for t in (F32, BF, F16):
        a, b = rand(5000, t, 1), rand(70_000, t, 2)
        b[31_337] = bad
        lst = moe.GradList([a, b], [torch.empty_like(a), torch.empty_like(b)])
        s = state(lst)
        moe.moe_grad_clip_norm(lst, 1.0, s["sumsq"], s["norm"], s["coef"], s["ws"])
        got = float(s["coef"])
        assert got == coef or (math.isnan(coef) and math.isnan(got))
        assert not math.isfinite(float(s["norm"]))
        for x, o in zip((a, b), lst.outs):
            ref = x.double() * coef
            assert torch.equal(o.double().isnan(), ref.isnan())
            assert (o[~ref.isnan()].double() == ref[~ref.isnan()]).all()


def test_shards_are_added_and_clipped_apart():
    grads = [rand(40_000, F32, 1), rand(1234, BF, 2), rand(777, F16, 3)]
    whole, s = state(grads), state(grads, 2)
    ref = [torch.empty_like(g) for g in grads]
    moe.moe_grad_clip_norm(moe.GradList(grads, ref), 2.0, whole["sumsq"], whole["norm"],
                           whole["coef"], whole["ws"])
    a, b = moe.GradList(grads[:1]), moe.GradList(grads[1:])
    moe.moe_grad_norm(a, 0, s["sumsq"], None, s["ws"])
    moe.moe_grad_norm(b, 1, s["sumsq"], s["norm"], s["ws"])
    within(s["sumsq"], whole["sumsq"], 1e-13 * whole["sumsq"], "sumsq")
    for lst in (a, b):
        moe.moe_grad_clip(lst, s["sumsq"], 2.0, None, s["coef"])
    within(s["coef"], whole["coef"], 2 * U, "coef")
    for g, r in zip(grads, ref):
        within(g, r, (2 * HALF[g.dtype] + 4 * U) * r.double().abs(), "clipped")


def test_streams_graphs_and_the_same_bits():
    grads = [rand(500_000, F32, 1), rand(123_457, BF, 2)]
    outs = [torch.zeros_like(g) for g in grads]
    lst = moe.GradList(grads, outs)
    s = state(lst)
    call = lambda st=None: moe.moe_grad_clip_norm(  # noqa: E731
        lst, 1.0, s["sumsq"], s["norm"], s["coef"], s["ws"], st)
    call()
    ref = [t.clone() for t in outs + [s["sumsq"], s["norm"], s["coef"]]]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call(st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in outs + [s["sumsq"], s["norm"], s["coef"]]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, r in zip(outs + [s["sumsq"], s["norm"], s["coef"]], ref):
            assert torch.equal(t, r)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16, torch.float32])
def test_runs_of_zeros_tiny_and_subnormal_elements(t):
    # long runs (whole vectors) whose squares are those of a type's smallest numbers, alone
    # and beside ordinary ones; a run of zeros gives exactly 0
    n = 40_000
    info = torch.finfo(t)
    least = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}[t]
    for v in (0.0, least, 5 * least, info.tiny, 3 * info.tiny, 2.0 ** -60 if t != torch.float16
              else 2.0 ** -14, 1.0):
        x = torch.full((n,), v, dtype=t, device="cuda")
        x[::2] *= -1
        s = state(moe.GradList([x]))
        moe.moe_grad_norm(moe.GradList([x]), 0, s["sumsq"], s["norm"], s["ws"])
        want = n * float(x[0].double()) ** 2
        # n sums of exact squares in 64 bits, each within 2^-53
        assert abs(float(s["sumsq"]) - want) <= n * 2.0 ** -53 * want, v
        y = torch.cat([x, torch.tensor([0.5], dtype=t, device="cuda")])
        moe.moe_grad_norm(moe.GradList([y]), 0, s["sumsq"], s["norm"], s["ws"])
        assert abs(float(s["sumsq"]) - want - 0.25) <= n * 2.0 ** -53 * (want + 0.25), v


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_one_non_finite_element_in_a_long_run(t, bad):
    for at in (0, 8, 12_345, 39_999):
        x = torch.ones(40_000, dtype=t, device="cuda")
        x[at] = bad
        s = state(moe.GradList([x]))
        moe.moe_grad_norm(moe.GradList([x]), 0, s["sumsq"], s["norm"], s["ws"])
        got = float(s["norm"])
        assert math.isnan(got) if math.isnan(bad) else got == math.inf


@pytest.mark.parametrize("t,v,max_norm", [(F32, 3e38, 1e-3), (BF, 3e38, 1e-3), (F32, 3e37, 1e-7),
                                          (F32, 1.5, 1e-37), (BF, 1.5, 1e-37), (F32, 2e30, 1e-38),
                                          (F32, 3e38, 1.2e-38)])
def test_a_factor_below_fp32_normal_range(t, v, max_norm):
    # max_norm / norm is a subnormal number of FP32, or 0 there; the clipped elements are
    # ordinary ones, rounded once
    for n in (7, 100_001):
        g = torch.full((n,), v, device="cuda").to(t)
        g[::3] *= -0.5
        norm = math.sqrt(float(g.double().square().sum()))
        q = max_norm / (norm + 1e-6)
        for out in (torch.full_like(g, 7.0), None):
            x = g.clone()
            lst = moe.GradList([x[:n // 2], x[n // 2:]],
                               None if out is None else [out[:n // 2], out[n // 2:]])
            s = state(lst)
            moe.moe_grad_clip_norm(lst, max_norm, s["sumsq"], s["norm"], s["coef"], s["ws"])
            r = g.double() * q
            within(x if out is None else out, r,
                   (4 * U + HALF[t] * (1 + 4 * U)) * r.abs() + TINY[t], "clipped")
            assert abs(float(s["coef"]) - q) <= 2 * U * q + 2.0 ** -150
        assert out is not None or torch.isfinite(x).all()


@pytest.mark.parametrize("t", [F32, BF, F16])
@pytest.mark.parametrize("bad", [math.inf, math.nan, 1.0])
def test_an_infinite_limit_never_clips(bad, t):
    x = rand(50_000, t, 3)
    x[777] = bad
    y = x.clone()
    for outs in ([torch.zeros_like(x)], None):
        lst = moe.GradList([x], outs)
        s = state(lst)
        moe.moe_grad_clip_norm(lst, math.inf, s["sumsq"], s["norm"], s["coef"], s["ws"])
        assert float(s["coef"]) == 1.0
        assert math.isfinite(float(s["norm"])) == (bad == 1.0)
        for got in (x, *(outs or [])):
            assert torch.equal(got.nan_to_num(-7.0, 9.0), y.nan_to_num(-7.0, 9.0))
