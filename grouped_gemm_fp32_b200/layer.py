"""One MoE FFN layer driven through the C ABI of libmoe.so.

``MoEBuffers`` owns the activations and workspace of one layer (torch device
tensors: torch is used for memory only); ``forward`` and ``backward`` issue the
C-ABI calls in the layer's order on one stream.  Every arithmetic step runs in
libmoe.so.

Layer (dots.llm1 Technical Report, §Architecture "Mixture of Experts layer"
and "Load balancing"; §3.2 "Efficient implementation of Grouped GEMM"):
    forward   moe_gate_topk -> moe_permute_align -> grouped_gemm_fwd[_gather] -> moe_combine
    backward  moe_combine_bwd -> grouped_gemm_bwd_dx(GEMM2) -> grouped_gemm_bwd_dw(GEMM2)
              -> grouped_gemm_bwd_dx(GEMM1) -> grouped_gemm_bwd_dw(GEMM1) [or _dw1_gather]
              -> moe_combine(weights = NULL)  (un-permute-sum of the dX rows)
              [-> moe_router_bwd (dlogits; gate term added into dX; dWg), or
                  moe_router_bwd_seqbal after forward's moe_seq_balance_loss]
              [-> moe_bias_update (next step's selection bias)]
The router backward runs when the gate weights are passed to ``backward``; the
bias step when an update speed ``gamma`` is.
With ``MoEBuffers(route=MoeRouteCfg...)`` the router is one of other kinds (sigmoid
scores, expert groups, a factor on the weights): moe_gate_logits -> moe_route_topk takes
the place of moe_gate_topk, and moe_route_bwd -> moe_gate_bwd that of moe_router_bwd.
``block_forward`` and ``block_backward`` run the layer between the norms of a
transformer block (moe_block_norm); ``GradClip`` clips the gradients by their global norm.
Under token data parallelism, ``dp_bias_step`` (the bias step on the whole batch's
loads) and ``dp_allreduce_grads`` (the weight gradients' sum) exchange what the
ranks share, over torch.distributed.
"""
from __future__ import annotations

from contextlib import nullcontext

import torch

from . import _lib as L


class MoEBuffers:
    def __init__(self, dims: L.MoeDims, device="cuda", train: bool = False,
                 gather: bool = False, experts: bool = True, route: L.MoeRouteCfg | None = None):
        """``gather``: the first GEMM (and dW1) read the routed x rows straight from x
        through ``sorted_ids`` (grouped_gemm_fwd_gather / grouped_gemm_bwd_dw1_gather)
        and no x_perm [Rr, d] is allocated; otherwise (the default, faster on B200:
        the row copy costs less than the four-row gather copies) they read the
        permuted copy ``x_perm`` that moe_permute_align writes.
        ``experts=False``: the buffers of a rank whose routed rows are computed
        elsewhere (expert parallelism): routing, permutation, combine and router
        buffers, with y, dy and dxp holding the routed rows only [Rr, d]; no
        expert activations (h, a1, da) and no expert weight gradients.
        ``route``: how the router scores and chooses (None: the layer's own, softmax over
        all experts); adds the logits [T, E] and, for training, their gradient."""
        self.dims = dims
        self.train = train
        self.gather = gather
        self.route = route
        T, d, E, k, S, I = dims.T, dims.d, dims.E, dims.k, dims.S, dims.I
        G = E + S
        self.Rr = L.moe_rows_routed(dims)
        self.Rt = L.moe_rows_total(dims)
        if self.Rr < 0:
            raise ValueError(f"invalid dims {dims}")
        dev = torch.device(device)
        i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
        e = lambda *s, dt=bf: torch.empty(*s, dtype=dt, device=dev)
        self.ws = torch.zeros(L.moe_workspace_size(dims), dtype=torch.uint8, device=dev)
        self.logits = e(T, E, dt=f32) if route is not None else None
        self.logits_valid = False      # the last forward's router wrote them
        self.topk_idx = e(T, k, dt=i32)
        self.topk_w = e(T, k, dt=f32)
        self.counts = e(E, dt=i32)
        self.offsets = e(E + 1, dt=i32)
        self.sorted_ids = e(self.Rr, dt=i32)
        self.row_of = e(T, k, dt=i32)
        self.x_perm = None if gather else e(self.Rr, d)
        rows = self.Rt if experts else self.Rr
        self.h = e(self.Rt, I) if experts else None
        self.a1 = e(self.Rt, 2 * I) if train and experts else None
        self.y = e(rows, d)
        self.out = e(T, d)
        if train:
            self.dy = e(self.Rr, d)
            self.dw_comb = e(T, k, dt=f32)
            self.da = e(self.Rt, 2 * I) if experts else None
            self.dxp = e(rows, d)
            self.dx = e(T, d)
            self.dw1 = e(G, 2 * I, d, dt=f32) if experts else None
            self.dw2 = e(G, d, I, dt=f32) if experts else None
            self.probs = e(T, E, dt=f32)
            self.dlogits = e(T, E, dt=f32) if route is not None else None
            self.dwg = e(E, d, dt=f32)
            self.bias_next = e(E, dt=f32)
            # sequence-wise balance loss: its value and dL/dp per sequence (sequences
            # of >= 128 tokens, so at most ceil(T / 128) of them)
            self.bal_loss = torch.zeros(1, dtype=f32, device=dev)
            self.bal_grad = e(max(1, -(-T // 128)), E, dt=f32)
            self.bal_seq_len = None

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in vars(self).values()
                   if isinstance(t, torch.Tensor))


def gate(b: MoEBuffers, x, wg, bias, stream=None):
    """The router's choice for x: b.topk_idx, b.topk_w and, for training, b.probs."""
    dm = b.dims
    probs = b.probs if b.train else None
    if b.route is None:
        L.moe_gate_topk(dm, x, wg, bias, b.topk_idx, b.topk_w, probs, b.ws, stream)
    else:
        L.moe_gate_logits(dm, x, wg, b.logits, b.ws, stream)
        L.moe_route_topk(dm, b.route, b.logits, bias, b.topk_idx, b.topk_w, probs, stream)
        b.logits_valid = True


def gate_backward(b: MoEBuffers, x, wg, stream=None):
    """The router's backward after the combine's: its term is added to b.dx, and b.dwg
    receives dL/dWg."""
    dm = b.dims
    seq_grad, seq_len = (b.bal_grad, b.bal_seq_len) if b.bal_seq_len is not None else (None, 0)
    if b.route is not None:
        if not b.logits_valid:
            raise ValueError("the router's backward needs a forward that ran the router")
        L.moe_route_bwd(dm, b.route, b.logits, b.topk_idx, b.topk_w, b.dw_comb, seq_grad, seq_len,
                        b.dlogits, stream)
        L.moe_gate_bwd(dm, x, wg, b.dlogits, b.dx, b.dwg, 0, b.ws, stream)
    elif seq_grad is not None:
        L.moe_router_bwd_seqbal(dm, x, wg, b.probs, b.topk_idx, b.topk_w, b.dw_comb, seq_grad,
                                seq_len, None, b.dx, b.dwg, 0, b.ws, stream)
    else:
        L.moe_router_bwd(dm, x, wg, b.probs, b.topk_idx, b.topk_w, b.dw_comb, None, b.dx, b.dwg,
                         0, b.ws, stream)


def forward(b: MoEBuffers, x, wg, bias, w1, w2, stream=None, routing=None, seq_balance=None):
    """out = MoE(x).  x [T, d] bf16, wg [E, d] f32, bias [E] f32, w1 [G, 2I, d], w2 [G, d, I].

    ``routing=(topk_idx, topk_w[, probs])`` (device int32 / f32 [T, k], f32 [T, E])
    replaces the gate's choice, e.g. to run the experts on a routing decided
    elsewhere.  With train buffers the gate also saves its affinities (probs) for
    the router backward.  ``seq_balance=(alpha, seq_len)`` (train buffers) also
    computes the sequence-wise balance loss into ``b.bal_loss``; ``backward``
    then adds its gradient to the router's."""
    dm = b.dims
    probs = b.probs if b.train else None
    if routing is None:
        gate(b, x, wg, bias, stream)
    else:
        b.logits_valid = False
        b.topk_idx.copy_(routing[0])
        b.topk_w.copy_(routing[1])
        if probs is not None and len(routing) > 2:
            probs.copy_(routing[2])
    L.moe_permute_align(dm, b.topk_idx, x, b.counts, b.offsets, b.sorted_ids, b.row_of, b.x_perm,
                        b.ws, stream)
    if b.gather:
        L.grouped_gemm_fwd_gather(dm, b.ws, b.sorted_ids, x, w1, w2, b.h, b.a1, b.y, stream)
    else:
        L.grouped_gemm_fwd(dm, b.ws, b.x_perm, x, w1, w2, b.h, b.a1, b.y, stream)
    L.moe_combine(dm, b.y, b.row_of, b.topk_w, b.out, stream)
    if b.train:
        b.bal_seq_len = None
        if seq_balance is not None:
            alpha, seq_len = seq_balance
            L.moe_seq_balance_loss(dm, seq_len, alpha, b.topk_idx, b.probs, b.bal_loss,
                                   b.bal_grad, b.ws, stream)
            b.bal_seq_len = int(seq_len)
    return b.out


def backward(b: MoEBuffers, x, dout, w1, w2, stream=None, wg=None, gamma=None, bias=None):
    """Gradients after ``forward``: dx [T, d], dw1, dw2 (f32) and the combine-weight
    gradient dw_comb [T, k].  dx holds the gradient through the experts, plus the
    router's (dlogit Wg) when ``wg`` is given; then ``b.dwg`` [E, d] f32 holds dL/dWg.
    With ``gamma`` (and the step's ``bias``) ``b.bias_next`` receives the
    aux-loss-free bias step."""
    if not b.train:
        raise ValueError("buffers were allocated without train=True")
    dm = b.dims
    L.moe_combine_bwd(dm, b.ws, dout, b.y, b.row_of, b.topk_w, b.dy, b.dw_comb, stream)
    L.grouped_gemm_bwd_dx(dm, b.ws, L.MOE_GEMM2, b.dy, dout, w2, b.a1, b.da, stream)
    L.grouped_gemm_bwd_dw(dm, b.ws, L.MOE_GEMM2, b.dy, dout, b.h, None, b.dw2, 0, stream)
    L.grouped_gemm_bwd_dx(dm, b.ws, L.MOE_GEMM1, b.da, None, w1, None, b.dxp, stream)
    if b.gather:
        L.grouped_gemm_bwd_dw1_gather(dm, b.ws, b.sorted_ids, b.da, x, b.dw1, 0, stream)
    else:
        L.grouped_gemm_bwd_dw(dm, b.ws, L.MOE_GEMM1, b.da, None, b.x_perm, x, b.dw1, 0, stream)
    L.moe_combine(dm, b.dxp, b.row_of, None, b.dx, stream)
    if wg is not None:
        gate_backward(b, x, wg, stream)
    if gamma is not None:
        L.moe_bias_update(dm, b.counts, gamma, bias, b.bias_next, stream)
    return b.dx, b.dw1, b.dw2, b.dw_comb


# ------------------------------------------------------------- data parallel --
# Token data parallelism: every rank holds the same weights and its own tokens.
# The layer's forward and backward need nothing from the other ranks; two steps
# do.  The bias step balances the loads of the whole batch, i.e. of all ranks'
# tokens (dots.llm1 Technical Report, §"Load balancing": the bias follows the
# experts' loads).  The weight gradients of the batch are the sums of the ranks'
# own.  Both are all-reduces over torch.distributed (NCCL between GPUs), issued
# on the layer's stream.

def on_stream(stream):
    """``torch.cuda.stream`` of a stream as the calls take it (a torch stream, or a handle as
    an integer: 0 is the default stream); no change of stream for None."""
    if stream is None:
        return nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def dp_load_counts(counts, group=None, stream=None):
    """Per-expert loads of the whole data-parallel batch: ``counts`` (int32 [E], this
    rank's tokens per expert, as moe_permute_align writes them) summed over the ranks
    of ``group``.  Returns a new tensor; ``counts`` itself is left as it is (the
    backward GEMMs still read it)."""
    import torch.distributed as dist
    with on_stream(stream):
        total = counts.clone()
        dist.all_reduce(total, op=dist.ReduceOp.SUM, group=group)
    return total


def dp_dims(dims: L.MoeDims, world: int) -> L.MoeDims:
    """The dims of the whole data-parallel batch: ``world`` ranks of ``dims.T`` tokens
    each (every rank must hold the same number of tokens)."""
    return L.MoeDims.of(dims.T * world, dims.d, dims.E, dims.k, dims.S, dims.I, dims.P,
                        dims.rows_cap)


def dp_bias_step(b: MoEBuffers, gamma, bias, group=None, stream=None):
    """The aux-loss-free bias step on the loads of the whole batch:
    ``b.bias_next = bias + gamma * sign(mean - load)`` with load = the experts' token
    counts summed over the ranks of ``group`` and mean = world·T·k/E.  Every rank
    gets the same ``b.bias_next``.  Returns the summed counts."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    total = dp_load_counts(b.counts, group, stream)
    L.moe_bias_update(dp_dims(b.dims, world), total, gamma, bias, b.bias_next, stream)
    return total


def dp_allreduce_grads(grads, group=None, stream=None):
    """Sum each gradient tensor (e.g. ``b.dw1``, ``b.dw2``, ``b.dwg``) over the ranks
    of ``group``, in place: the gradients of the whole data-parallel batch."""
    import torch.distributed as dist
    with on_stream(stream):
        for g in grads:
            dist.all_reduce(g, op=dist.ReduceOp.SUM, group=group)
    return grads


# -------------------------------------------------------------- global clipping --
class GradClip:
    """Clipping of gradients that stay where they are by their global norm, on the
    device: ``GradClip(grads)``, then ``clip(max_norm)`` every step.

    ``sharded``: tensors that this rank alone holds of the model's (under expert
    parallelism the routed experts' dW); their squares are added over ``group``.  Either
    every rank of ``group`` gives a list, which is empty on a rank that holds none, or
    none does (None): ``clip`` of a given list takes part in the group's sum.
    ``grads`` are whole on every rank (after ``dp_allreduce_grads``) and count once.
    ``outs`` / ``sharded_outs``: where the clipped gradients go (None: in place)."""

    def __init__(self, grads, outs=None, sharded=None, sharded_outs=None, group=None):
        self.whole = L.GradList(grads, outs)
        self.shards = None
        if sharded is not None:
            import torch.distributed as dist
            # an empty list without a process group: there is nobody to add to
            if len(sharded) or (dist.is_available() and dist.is_initialized()):
                self.shards = L.GradList(sharded, sharded_outs)
        self.group = group
        every = self.whole.grads + (self.shards.grads if self.shards is not None else [])
        if not every:
            raise ValueError("no gradients to clip")
        dev = every[0].device
        self.sumsq = torch.zeros(1, dtype=torch.float64, device=dev)
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)
        self.coef = torch.zeros(1, dtype=torch.float32, device=dev)
        n = max(len(self.whole), len(self.shards) if self.shards is not None else 0)
        self.ws = torch.empty(L.moe_grad_workspace_size(n), dtype=torch.uint8, device=dev)

    def clip(self, max_norm, stream=None):
        """Scales every gradient by min(1, max_norm / (norm + 1e-6)).  Returns ``norm`` [1]
        f32, the norm before; ``coef`` [1] holds the factor.  Nothing comes to the host."""
        if self.shards is None:
            L.moe_grad_clip_norm(self.whole, max_norm, self.sumsq, self.norm, self.coef, self.ws,
                                 stream)
            return self.norm
        import torch.distributed as dist
        L.moe_grad_norm(self.shards, 0, self.sumsq, None, self.ws, stream)
        with on_stream(stream):
            dist.all_reduce(self.sumsq, op=dist.ReduceOp.SUM, group=self.group)
        L.moe_grad_norm(self.whole, 1, self.sumsq, None, self.ws, stream)
        L.moe_grad_clip(self.shards, self.sumsq, max_norm, self.norm, self.coef, stream)
        L.moe_grad_clip(self.whole, self.sumsq, max_norm, None, None, stream)
        return self.norm


# ---------------------------------------------------------------- a block --
# The layer as a transformer block's second half:
#   n = RMSNorm(res) w_pre;  y = MoE(n);
#   res_out = alpha res + beta gate * (RMSNorm(y) w_post or y)
# and, where the next block's pre-norm weight is given, that block's n from the same pass.

class BlockBuffers:
    """Activations of one block: the layer's (``moe``, a MoEBuffers), the normed input
    ``n``, the residual stream after the block ``res_out`` and the next block's input
    ``n_next``; for training the gradients ``dres`` (of res), ``dy`` (of the layer's
    output), ``dw_pre``, ``dw_post``, ``dw_next`` [d] and ``dgate``.

    ``norm``: MoeNormCfg (eps, the factors alpha and beta, tokens per row of the gate).
    ``res_dtype``: type of the residual stream, torch.bfloat16 or torch.float32."""

    def __init__(self, dims: L.MoeDims, norm: L.MoeNormCfg, res_dtype=torch.bfloat16,
                 device="cuda", train: bool = False, gather: bool = False, route=None):
        self.dims, self.norm = dims, norm
        self.moe = MoEBuffers(dims, device=device, train=train, gather=gather, route=route)
        T, d = dims.T, dims.d
        dev = torch.device(device)
        e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=dev)
        self.n, self.n_next = e(T, d), e(T, d)
        self.res_out = e(T, d, dt=res_dtype)
        if train:
            f32 = torch.float32
            rows = max(1, -(-T // norm.seq_len)) if norm.seq_len > 0 else 1
            self.dy = e(T, d)
            self.dres = e(T, d, dt=res_dtype)
            self.dw_pre, self.dw_post, self.dw_next = (e(d, dt=f32) for _ in range(3))
            self.dgate = e(rows, d, dt=f32)
            self.ws = e(L.moe_norm_workspace_size(dims, norm), dt=torch.uint8)


def block_forward(bb: BlockBuffers, res, w_pre, wg, bias, w1, w2, w_post=None, gate=None,
                  w_next=None, n=None, stream=None, seq_balance=None):
    """res_out (and the next block's input) of a block on the residual stream res [T, d].

    w_pre [d] f32: the layer's pre-norm; with ``n`` [T, d] bf16, the normed input that the
    block before returned, it is not used.  w_post [d] f32, gate [rows, d] f32: the norm
    and the gate of the layer's output (None: without).  w_next [d] f32: the next block's
    pre-norm.  Returns (res_out, n_next), n_next None without w_next."""
    dm, cfg = bb.dims, bb.norm
    if bb.moe.train and res.data_ptr() == bb.res_out.data_ptr():
        raise ValueError("the backward reads res again: it cannot be this block's res_out")
    if bb.moe.train and n is not None and w_next is not None and \
            n.data_ptr() == bb.n_next.data_ptr():
        raise ValueError("the backward reads n again: it cannot be this block's n_next")
    if n is None:
        n = bb.n
        L.moe_block_norm(dm, cfg, None, res, None, None, w_pre, None, n, stream)
    y = forward(bb.moe, n, wg, bias, w1, w2, stream=stream, seq_balance=seq_balance)
    n_next = bb.n_next if w_next is not None else None
    L.moe_block_norm(dm, cfg, y, res, w_post, gate, w_next, bb.res_out, n_next, stream)
    return bb.res_out, n_next


def block_backward(bb: BlockBuffers, dres_out, res, w_pre, wg, w1, w2, w_post=None, gate=None,
                   w_next=None, n=None, dn_next=None, stream=None, gamma=None, bias=None):
    """Gradients after ``block_forward`` with the same arguments.  dres_out [T, d]: of
    res_out (None: zero, with w_next only); dn_next [T, d] bf16: of n_next, with w_next.

    Returns dres [T, d], the gradient of res; where the block was given ``n``, (dres, dn):
    the parts that reached res past the layer and n, for the block before.  Leaves the
    weights' gradients in bb.dw_pre, bb.dw_post, bb.dw_next, bb.dgate and bb.moe."""
    dm, cfg = bb.dims, bb.norm
    if (w_next is None) != (dn_next is None):
        raise ValueError("w_next and dn_next come together")
    moe = bb.moe
    L.moe_block_norm_bwd(dm, cfg, dn_next, dres_out, moe.out, bb.res_out, w_post, gate, w_next,
                         bb.dy, bb.dres, bb.dw_post if w_post is not None else None,
                         bb.dgate if gate is not None else None,
                         bb.dw_next if w_next is not None else None, 0, bb.ws, stream)
    dn, *_ = backward(moe, bb.n if n is None else n, bb.dy, w1, w2, stream=stream, wg=wg,
                      gamma=gamma, bias=bias)
    if n is not None:
        return bb.dres, dn
    L.moe_block_norm_bwd(dm, cfg, dn, bb.dres, None, res, None, None, w_pre, None, bb.dres, None,
                         None, bb.dw_pre, 0, bb.ws, stream)
    return bb.dres


class HostPipeline:
    """Forward (+ backward) steps fed from and returned to pinned host memory,
    with the copies of neighbouring steps overlapped with compute.

    Two device buffer sets alternate: while step i computes on set i % 2, the
    inputs of step i + 1 are copied in on an upload stream and the results of
    step i - 1 are copied out on a download stream.  Every step still moves its
    inputs host -> device and its results device -> host; only the overlap is
    added.  All arithmetic runs in libmoe.so; torch provides memory and streams.
    """

    def __init__(self, dims: L.MoeDims, w1, w2, wg, bias, train: bool, device="cuda",
                 gamma=None, graphs: bool = True, gather: bool = False, seq_balance=None,
                 route=None):
        self.dims, self.train, self.gamma = dims, train, gamma
        self.seq_balance = seq_balance if train else None
        self.w1, self.w2, self.wg, self.bias = w1, w2, wg, bias
        dev = torch.device(device)
        T, d = dims.T, dims.d
        self.bufs = [MoEBuffers(dims, device=dev, train=train, gather=gather, route=route)
                     for _ in range(2)]
        # zero-filled: with graphs, one step runs on them before the capture
        e = lambda: torch.zeros(T, d, dtype=torch.bfloat16, device=dev)
        self.x = [e(), e()]
        self.dout = [e(), e()] if train else [None, None]
        self.compute = torch.cuda.Stream(device=dev)
        self.up = torch.cuda.Stream(device=dev)
        self.down = torch.cuda.Stream(device=dev)
        self.uploaded = [torch.cuda.Event(), torch.cuda.Event()]
        self.computed = [torch.cuda.Event(), torch.cuda.Event()]
        self.downloaded = [torch.cuda.Event(), torch.cuda.Event()]
        self.consumed = [torch.cuda.Event(), torch.cuda.Event()]
        for ev in self.downloaded + self.consumed:
            ev.record(self.compute)
        # one captured step per buffer set (the graphs keep the sets' addresses)
        self.graphs = None
        if graphs:
            self.graphs = [GraphStep(self.bufs[j], self.x[j], wg, bias, w1, w2,
                                     dout=self.dout[j] if train else None,
                                     gamma=gamma if train else None,
                                     seq_balance=self.seq_balance) for j in range(2)]

    def _upload(self, j, hx, hd):
        with torch.cuda.stream(self.up):
            self.up.wait_event(self.consumed[j])      # step j-2 no longer reads set j
            self.x[j].copy_(hx, non_blocking=True)
            if self.train:
                self.dout[j].copy_(hd, non_blocking=True)
            self.uploaded[j].record(self.up)

    def run(self, host_x, host_dout, host_out, host_dx, steps: int):
        """``steps`` steps; step i reads host_x[i % n] (and host_dout) and writes
        host_out[i % n] (and host_dx).  Returns after all copies are issued;
        synchronise the streams (or ``self.down``) to wait for the results."""
        n = len(host_x)
        self._upload(0, host_x[0], host_dout[0] if self.train else None)
        for i in range(steps):
            j = i & 1
            if i + 1 < steps:
                self._upload(1 - j, host_x[(i + 1) % n],
                             host_dout[(i + 1) % n] if self.train else None)
            b = self.bufs[j]
            s = self.compute
            with torch.cuda.stream(s):
                s.wait_event(self.uploaded[j])
                s.wait_event(self.downloaded[j])  # results of step i-2 have left set j
                if self.graphs is not None:
                    self.graphs[j].replay()
                else:
                    forward(b, self.x[j], self.wg, self.bias, self.w1, self.w2, stream=s,
                            seq_balance=self.seq_balance)
                    if self.train:
                        backward(b, self.x[j], self.dout[j], self.w1, self.w2, stream=s,
                                 wg=self.wg, gamma=self.gamma, bias=self.bias)
                self.computed[j].record(s)
                self.consumed[j].record(s)
            with torch.cuda.stream(self.down):
                self.down.wait_event(self.computed[j])
                host_out[i % n].copy_(b.out, non_blocking=True)
                if self.train:
                    host_dx[i % n].copy_(b.dx, non_blocking=True)
                self.downloaded[j].record(self.down)

    def synchronize(self):
        for st in (self.up, self.compute, self.down):
            st.synchronize()


class GraphStep:
    """One layer step -- forward, and with ``dout`` the backward (router backward
    and bias step included when ``gamma`` is given, the sequence-wise balance loss
    when ``seq_balance=(alpha, seq_len)`` is) -- captured once as a CUDA
    graph and replayed.  Every node is one of the same C-ABI calls as in eager
    mode, on the captured stream; the graph keeps the buffers' addresses, so new
    inputs are written into ``x`` / ``dout`` in place before ``replay``.

    The step runs once eagerly before the capture: the library's first calls set
    kernel attributes and look up driver entry points, which must not happen
    inside a capture."""

    def __init__(self, b: MoEBuffers, x, wg, bias, w1, w2, dout=None, gamma=None,
                 seq_balance=None):
        self.b = b
        self.stream = torch.cuda.Stream(device=x.device)
        args = (b, x, wg, bias, w1, w2, dout, gamma, seq_balance)
        with torch.cuda.stream(self.stream):
            self._step(self.stream, *args)
        self.stream.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self.stream):
            self._step(self.stream, *args)
        self.stream.synchronize()

    @staticmethod
    def _step(s, b, x, wg, bias, w1, w2, dout, gamma, seq_balance):
        forward(b, x, wg, bias, w1, w2, stream=s,
                seq_balance=seq_balance if dout is not None else None)
        if dout is not None:
            backward(b, x, dout, w1, w2, stream=s, wg=wg, gamma=gamma,
                     bias=bias if gamma is not None else None)

    def replay(self):
        self.graph.replay()
