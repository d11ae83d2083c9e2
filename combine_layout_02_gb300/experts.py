"""What a model does with the rows between dispatch and combine, as PyTorch autograd functions over
the C ABI: rows into expert order and back (``ep_sort_*`` / ``ep_unsort_*``), the experts' products
(``ep_expert_gemm*``), the experts' gated feed-forward block in one function with the activations that its
backward pass needs kept in bf16, in 8 bits or not at all (``ep_expert_gated*``,
``ep_checkpoint_rows``), and a shared projection with each row's own low-rank adapter
(``ep_adapter_gemm``); and ``MoELayer``, a layer that runs all of it together with a ``Buffer``.

Like the rest of the package this module only allocates tensors and calls the library, on the
current stream. Tensors are bf16 unless stated. The library takes pointers, so each function first
checks its tensors' types and shapes and raises ValueError where they are others. The gradients are
the library's too and have no gradients of their own: differentiating them raises. What only the
device sees (ids out of range, rows beyond their buffer, a wait that gave up: EP_DEVERR_*) goes to
the error word that a call is given as ``err``, else to the module's own, which check_errors() reads.
"""
from __future__ import annotations

from typing import List, Optional

import torch
from torch.autograd.function import once_differentiable

from . import (_Address, EP_ACT_GELU_TANH, EP_ACT_SILU, EP_BF16, EP_CHECKPOINT_GROUP, EP_GEMM_MAX_FEATURES,
               ep_adapter_gemm, ep_adapter_shape, ep_adapter_workspace_size, ep_checkpoint_rows, ep_expert_gated,
               ep_expert_gated_dgrad, ep_expert_gemm, ep_expert_gemm_dgrad, ep_expert_gemm_wgrad, ep_expert_gemm_wgrad_checkpoint, ep_gemm_shape,
               ep_read_error_flags_sync, ep_restore_rows, ep_sort_layout, ep_sort_rows, ep_unsort_rows,
               ep_unsort_rows_backward, ep_wgrad_checkpoint_workspace_size, make_checkpoint, make_launch, make_shape)
from .api import Buffer
from .buffers import SortBuffers

__all__ = ["ExpertSort", "sort_rows", "unsort_rows", "expert_product", "expert_feed_forward", "checkpoint_rows",
           "restore_rows", "adapter_projection", "check_errors", "MoELayer"]


def _check(what: str, t: torch.Tensor, dtype: torch.dtype, *shape: Optional[int]) -> None:
    """t has to be a tensor of this type and shape (None: any length)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise ValueError(f"{what} has to be a tensor of {dtype}, not {getattr(t, 'dtype', type(t))}")
    has = t.shape
    if has == shape:
        return
    if len(has) != len(shape) or any(n is not None and n != m for n, m in zip(shape, has)):
        wants = ", ".join("any" if n is None else str(n) for n in shape)
        raise ValueError(f"{what} has to be [{wants}], not {list(has)}")


def _check_devices(*tensors: torch.Tensor) -> None:
    """The library launches on the current device's current stream."""
    at = tensors[0].device
    if any(t.device != at for t in tensors) or (at.type == "cuda" and at.index != torch.cuda.current_device()):
        raise ValueError(f"all tensors have to be on the current device, not on {[str(t.device) for t in tensors]}")


def _one_of(what: str, value, names) -> None:
    if value not in names:
        raise ValueError(f"{what} has to be one of {', '.join(map(repr, names))}, not {value!r}")


def _check_err(err: Optional[torch.Tensor]) -> None:
    if err is not None and (not isinstance(err, torch.Tensor) or err.dtype not in (torch.int32, torch.uint32) or
                            err.numel() < 1):
        raise ValueError("err has to be a tensor of one int32 error word")


_words: dict = {}           # device index -> the error word of calls without one


def _error_word(err: Optional[torch.Tensor], device: torch.device) -> Optional[torch.Tensor]:
    if err is not None or device.type != "cuda":
        return err
    if device.index not in _words and not torch.cuda.is_current_stream_capturing():
        word = torch.zeros(1, dtype=torch.int32, device=device)
        torch.cuda.current_stream(device).synchronize()            # any stream may use it from here on
        _words[device.index] = word
    return _words.get(device.index)          # none where a graph captures the very first call


def check_errors(device="cuda") -> int:
    """Waits for the device, then returns the EP_DEVERR_* bits that calls without an error word of
    their own have seen since the last check_errors."""
    device = torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    if index not in _words:
        return 0
    torch.cuda.synchronize(index)
    seen = ep_read_error_flags_sync(_words[index])
    if seen:
        _words[index].zero_()
        torch.cuda.synchronize(index)
    return seen


class ExpertSort:
    """The placement of rows by expert: ``topk_idx`` [N][k] int64, -1 masked, experts 0 to E - 1.
    ``rows``: how many sorted rows there are, where the caller knows (from the counts of a
    dispatch); otherwise it is read back (a CPU wait)."""

    def __init__(self, topk_idx: torch.Tensor, num_experts: int, hidden: int, rows: Optional[int] = None,
                 err: Optional[torch.Tensor] = None):
        _check("topk_idx", topk_idx, torch.int64, None, None)
        _check_err(err)
        self.N, self.k = topk_idx.shape
        self.E, self.H, self.err = num_experts, hidden, _error_word(err, topk_idx.device)
        self.shape = make_shape(1, self.N, hidden, num_experts, self.k)
        self.buffers = SortBuffers(self.shape, rows, topk_idx.device)
        ep_sort_layout(self.shape, topk_idx, self.buffers.handle(), self.buffers.workspace, self.launch())
        if rows is None:
            self.buffers.rows = int(self.buffers.expert_prefix[-1].item())      # what sorted rows are sized by
        self.rows = self.buffers.rows
        self.handle = self.buffers.handle()

    @property
    def expert_prefix(self) -> torch.Tensor:
        return self.buffers.expert_prefix

    def launch(self):
        return make_launch(error_flags=self.err)


class _SortRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, sort: ExpertSort):
        ctx.sort = sort
        out = torch.empty((sort.rows, sort.H), dtype=x.dtype, device=x.device)
        ep_sort_rows(sort.shape, x, EP_BF16, None, sort.handle, out, None, sort.launch())
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        sort = ctx.sort
        dx = torch.empty((sort.N, sort.H), dtype=grad.dtype, device=grad.device)
        ep_unsort_rows(sort.shape, grad.contiguous(), None, sort.handle, dx, sort.launch())
        return dx, None


class _UnsortRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, sort: ExpertSort):
        ctx.sort = sort
        ctx.save_for_backward(y, weights)
        out = torch.empty((sort.N, sort.H), dtype=y.dtype, device=y.device)
        ep_unsort_rows(sort.shape, y, weights, sort.handle, out, sort.launch())
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        sort, (y, weights) = ctx.sort, ctx.saved_tensors
        dy = torch.empty_like(y)
        dw = None if weights is None else torch.empty_like(weights)
        ep_unsort_rows_backward(sort.shape, grad.contiguous(), y, weights, sort.handle, dy, dw, sort.launch())
        return dy, dw, None


def _kept_width(features: int) -> int:
    return -(-features // EP_CHECKPOINT_GROUP) * EP_CHECKPOINT_GROUP


def _kept_bytes(rows: int, width: int) -> int:
    """Bytes of a checkpoint in 8 bits, values, then scales, to the next multiple of 16."""
    return (rows * width + rows * width // EP_CHECKPOINT_GROUP + 15) & ~15


def _kept_at(address: int, rows: int, width: int):
    return make_checkpoint(_Address(address), _Address(address + rows * width))


class _UnsortRowsKept(torch.autograd.Function):
    """_UnsortRows with y in 8 bits until the weights' gradient needs it."""

    @staticmethod
    def forward(ctx, y, weights, sort: ExpertSort):
        ctx.sort = sort
        kept = checkpoint_rows(y) if ctx.needs_input_grad[1] else (None, None)
        ctx.save_for_backward(weights, *kept)
        out = torch.empty((sort.N, sort.H), dtype=y.dtype, device=y.device)
        ep_unsort_rows(sort.shape, y, weights, sort.handle, out, sort.launch())
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        sort, (weights, values, scales) = ctx.sort, ctx.saved_tensors
        y, dw = None, None
        if ctx.needs_input_grad[1]:
            y, dw = restore_rows(values, scales, sort.H), torch.empty_like(weights)
        dy = y if y is not None else grad.new_empty((sort.rows, sort.H))          # in place: y is this call's own
        ep_unsort_rows_backward(sort.shape, grad.contiguous(), y, weights, sort.handle, dy, dw, sort.launch())
        return dy, dw, None


class _ExpertProduct(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, prefix, err):
        E, F, K = weight.shape
        ctx.save_for_backward(x, weight, prefix)
        ctx.shape, ctx.err = ep_gemm_shape(x.shape[0], E, K, F), err
        y = torch.empty((x.shape[0], F), dtype=x.dtype, device=x.device)
        ep_expert_gemm(ctx.shape, x, weight, prefix, y, make_launch(error_flags=err))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, weight, prefix = ctx.saved_tensors
        grad, launch, dx, dw = grad.contiguous(), make_launch(error_flags=ctx.err), None, None
        if ctx.needs_input_grad[0]:
            dx = torch.empty_like(x)
            ep_expert_gemm_dgrad(ctx.shape, grad, weight, prefix, dx, launch)
        if ctx.needs_input_grad[1]:
            dw = torch.empty_like(weight)
            ep_expert_gemm_wgrad(ctx.shape, grad, x, prefix, dw, launch)
        return dx, dw, None, None


class _FeedForward(torch.autograd.Function):
    # The host's part of a small call takes longer than the device's, so what is kept, and what only the
    # backward pass uses, is one allocation each.
    @staticmethod
    def forward(ctx, x, gate_up, down, prefix, act, checkpoint, err):
        (rows, K), (E, H, F) = x.shape, down.shape
        for_x, for_gate_up, for_down = ctx.needs_input_grad[:3]
        wanted = checkpoint is not None and (for_x or for_gate_up or for_down)
        if wanted and (for_x or for_gate_up) and 2 * F > EP_GEMM_MAX_FEATURES:          # one product of both, backward
            raise ValueError(f"gate_up has to be of {EP_GEMM_MAX_FEATURES // 2} features or fewer for gradients, not {F}")
        launch, new = make_launch(error_flags=err), x.new_empty
        h, y = new((rows, F)), new((rows, H))
        kept = rows_kept = keep = None
        if wanted and checkpoint == "bf16":
            kept, rows_kept = new((rows, 2 * F)), x if for_gate_up else None
            keep = make_checkpoint(kept)
        elif wanted and checkpoint == "e4m3":          # g and u, then the rows
            wide, width = 2 * _kept_width(F), _kept_width(K)
            own = _kept_bytes(rows, wide)
            kept = new(own + (_kept_bytes(rows, width) if for_gate_up else 0), dtype=torch.uint8)
            keep = _kept_at(kept.data_ptr(), rows, wide)
            if for_gate_up:
                ep_checkpoint_rows(rows, K, x, _kept_at(kept.data_ptr() + own, rows, width), launch)
        elif wanted:
            rows_kept = x
            if rows == 1:          # keeping nothing it would go another way than the backward pass does again
                spare = new((1, 2 * F))
                keep = make_checkpoint(spare)
        ep_expert_gated(ep_gemm_shape(rows, E, K, F), x, gate_up, prefix, act, h, keep, launch)
        ep_expert_gemm(ep_gemm_shape(rows, E, F, H), h, down, prefix, y, launch)
        if wanted:
            ctx.act, ctx.checkpoint, ctx.err = act, checkpoint, err
            ctx.save_for_backward(gate_up, down, prefix, kept, rows_kept)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        gate_up, down, prefix, kept, x = ctx.saved_tensors
        (rows, H), (E, _, F), K = grad.shape, down.shape, gate_up.shape[2]
        grad, launch, new = grad.contiguous(), make_launch(error_flags=ctx.err), grad.new_empty
        for_x, for_gate_up, for_down = ctx.needs_input_grad[:3]
        down_shape, up_shape = ep_gemm_shape(rows, E, F, H), ep_gemm_shape(rows, E, K, 2 * F)
        if ctx.checkpoint == "e4m3":
            wide, width = 2 * _kept_width(F), _kept_width(K)
            own = _kept_at(kept.data_ptr(), rows, wide)
        else:
            if ctx.checkpoint == "recompute":
                kept = new((rows, 2 * F))
                ep_expert_gated(ep_gemm_shape(rows, E, K, F), x, gate_up, prefix, ctx.act, None, make_checkpoint(kept), launch)
            own = make_checkpoint(kept)
        eight = ctx.checkpoint == "e4m3" and for_gate_up
        room = max(16, ep_wgrad_checkpoint_workspace_size(up_shape)) if eight else 0
        scratch = new(rows * F * (6 if for_down else 4) + room, dtype=torch.uint8)          # the workspace, dgu, h
        workspace = scratch[:room] if eight else None
        dgu = _Address(scratch.data_ptr() + room)
        h = _Address(dgu + rows * F * 4) if for_down else None
        ep_expert_gated_dgrad(down_shape, grad, down, prefix, ctx.act, own, dgu, h, launch)
        dx = dgate_up = ddown = None
        if for_down:
            ddown = torch.empty_like(down)
            ep_expert_gemm_wgrad(down_shape, grad, h, prefix, ddown, launch)
        if for_x:
            dx = new((rows, K))
            ep_expert_gemm_dgrad(up_shape, dgu, gate_up, prefix, dx, launch)
        if eight:
            dgate_up = torch.empty_like(gate_up)
            at = kept.data_ptr() + _kept_bytes(rows, wide)
            ep_expert_gemm_wgrad_checkpoint(up_shape, dgu, _kept_at(at, rows, width), prefix, dgate_up, workspace, launch)
        elif for_gate_up:
            dgate_up = torch.empty_like(gate_up)
            ep_expert_gemm_wgrad(up_shape, dgu, x, prefix, dgate_up, launch)
        return dx, dgate_up, ddown, None, None, None, None


class _NoGradient(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, *inputs):
        return y

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError("adapter_projection is for serving and has no gradient: call it under torch.no_grad(), or "
                           "detach its inputs where the gradient may leave it out")


def sort_rows(x: torch.Tensor, sort: ExpertSort) -> torch.Tensor:
    """x [N][H] -> [rows][H] in expert order; gradient to x. (Quantised rows: ``ep_sort_rows``.)"""
    _check("x", x, torch.bfloat16, sort.N, sort.H)
    return _SortRows.apply(x, sort)


def checkpoint_rows(x: torch.Tensor):
    """x [rows][features] bf16 -> (values, scales): the rows in 8 bits, uint8 [rows][features padded to
    16] of e4m3 and uint8 [rows][groups of 16], for a backward pass (see ep_checkpoint in ep.h)."""
    _check("x", x, torch.bfloat16, None, None)
    _check_devices(x)
    (rows, features), width = x.shape, _kept_width(x.shape[1])
    values, scales = (torch.empty((rows, n), dtype=torch.uint8, device=x.device) for n in (width, width // EP_CHECKPOINT_GROUP))
    ep_checkpoint_rows(rows, features, x, make_checkpoint(values, scales), make_launch())
    return values, scales


def restore_rows(values: torch.Tensor, scales: torch.Tensor, features: int) -> torch.Tensor:
    """The rows [rows][features] in bf16 that checkpoint_rows has kept."""
    width = _kept_width(features)
    _check("values", values, torch.uint8, None, width)
    _check("scales", scales, torch.uint8, values.shape[0], width // EP_CHECKPOINT_GROUP)
    _check_devices(values, scales)
    x = torch.empty((values.shape[0], features), dtype=torch.bfloat16, device=values.device)
    ep_restore_rows(*x.shape, make_checkpoint(values, scales), x, make_launch())
    return x


def unsort_rows(y: torch.Tensor, sort: ExpertSort, weights: Optional[torch.Tensor] = None,
                checkpoint: str = "bf16") -> torch.Tensor:
    """y [rows][H] -> [N][H], the sum of each row's entries, scaled by weights [N][k] fp32 if given;
    gradients to y and weights. The weights' gradient needs y: with checkpoint "e4m3" it is kept in
    8 bits until then."""
    _one_of("checkpoint", checkpoint, ("bf16", "e4m3"))
    _check("y", y, torch.bfloat16, sort.rows, sort.H)
    if weights is not None:
        _check("weights", weights, torch.float32, sort.N, sort.k)
        if checkpoint == "e4m3" and torch.is_grad_enabled():
            return _UnsortRowsKept.apply(y, weights, sort)
    return _UnsortRows.apply(y, weights, sort)


def expert_product(x: torch.Tensor, weight: torch.Tensor, expert_prefix: torch.Tensor,
                   err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [rows][in] in expert order, weight [E][out][in] -> [rows][out]; gradients to both. Every
    row has to belong to an expert (expert_prefix runs from 0 to rows)."""
    _check("weight", weight, torch.bfloat16, None, None, None)
    _check("x", x, torch.bfloat16, None, weight.shape[2])
    _check("expert_prefix", expert_prefix, torch.int32, weight.shape[0] + 1)
    _check_err(err)
    return _ExpertProduct.apply(x, weight, expert_prefix, _error_word(err, x.device))


_ACTIVATIONS = {"silu": EP_ACT_SILU, "gelu": EP_ACT_GELU_TANH}


def expert_feed_forward(x: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, expert_prefix: torch.Tensor,
                        activation: str = "silu", checkpoint: str = "bf16",
                        err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The experts' gated feed-forward block: x [rows][in] in expert order, gate_up [E][2 * features][in]
    (gate, then up), down [E][out][features] -> down (act(gate x) * (up x)) [rows][out]; gradients to
    all three. activation: "silu" or "gelu" (with a hyperbolic tangent). checkpoint: what is kept for
    the backward pass, which computes the product of activation and up again in any case:
      "bf16"       x and both projections' results, 2 bytes a value
      "e4m3"       the same in 8 bits (1.0625 bytes); the matrices' gradients and act' then go by
                   those values, the result and the gradient's way through down do not
      "recompute"  x; both projections run again
    The result is the same with all three. Where no gradient is wanted nothing is kept, and a single
    row then goes another way (ep_expert_gated), with its sums in another order.
    For gradients to x or gate_up there are EP_GEMM_MAX_FEATURES / 2 features at most.
    Every row has to belong to an expert (expert_prefix runs from 0 to rows)."""
    _check("down", down, torch.bfloat16, None, None, None)
    _check("gate_up", gate_up, torch.bfloat16, down.shape[0], 2 * down.shape[2], None)
    _check("x", x, torch.bfloat16, None, gate_up.shape[2])
    _check("expert_prefix", expert_prefix, torch.int32, gate_up.shape[0] + 1)
    _one_of("activation", activation, tuple(_ACTIVATIONS))
    _one_of("checkpoint", checkpoint, ("bf16", "e4m3", "recompute"))
    _check_err(err)
    _check_devices(x, gate_up, down, expert_prefix, *(() if err is None else (err,)))
    # (Under torch.no_grad() a function still sees which inputs want gradients.)
    return _FeedForward.apply(x, gate_up, down, expert_prefix, _ACTIVATIONS[activation],
                              checkpoint if torch.is_grad_enabled() else None, _error_word(err, x.device))


def adapter_projection(x: torch.Tensor, weight: torch.Tensor, a: Optional[torch.Tensor], b: Optional[torch.Tensor],
                       scales: Optional[torch.Tensor], adapter_idx: torch.Tensor,
                       err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [T][in], weight [out][in], a [L][r][in], b [L][out][r], scales [L] fp32, adapter_idx [T]
    int64 (-1 none) -> [T][out]. For serving: a backward pass that reaches it raises."""
    _check("x", x, torch.bfloat16, None, None)
    _check("weight", weight, torch.bfloat16, None, x.shape[1])
    (T, K), F = x.shape, weight.shape[0]
    L, r = 0, 8
    if a is not None:
        _check("a", a, torch.bfloat16, None, None, K)
        L, r = a.shape[0], a.shape[1]
        _check("b", b, torch.bfloat16, L, F, r)
        _check("scales", scales, torch.float32, L)
    _check("adapter_idx", adapter_idx, torch.int64, T)
    _check_err(err)
    shape = ep_adapter_shape(T, K, F, L, r)
    workspace = torch.empty(max(16, ep_adapter_workspace_size(shape)), dtype=torch.uint8, device=x.device)
    y = torch.empty((T, F), dtype=x.dtype, device=x.device)
    ep_adapter_gemm(shape, x, weight, a, b, scales, adapter_idx, y, workspace,
                    make_launch(error_flags=_error_word(err, x.device)))
    if torch.is_grad_enabled():
        inputs = [t for t in (x, weight, a, b, scales) if t is not None and t.requires_grad]
        if inputs:
            return _NoGradient.apply(y, *inputs)
    return y


class _Dispatch(torch.autograd.Function):
    """Buffer.dispatch of x and the routing weights; its gradient is Buffer.combine, which also adds
    up the weights' gradients ("DeepEP" README, dispatch_backward)."""

    @staticmethod
    def forward(ctx, x, topk_weights, topk_idx, buf: Buffer, out: dict):
        recv_x, recv_idx, recv_w, _, handle, _ = buf.dispatch(x, topk_idx=topk_idx, topk_weights=topk_weights)
        ctx.buf, ctx.handle = buf, handle
        off = handle.row_offset
        out["handle"], out["recv_idx"] = handle, buf._rows_tensor(recv_idx, off)
        rows = off[-1]
        return buf._rows_tensor(recv_x, off)[:rows], buf._rows_tensor(recv_w, off)[:rows]

    @staticmethod
    @once_differentiable
    def backward(ctx, dx, dw):
        gx, gw, _ = ctx.buf.combine(dx.contiguous(), ctx.handle, topk_weights=dw.contiguous())
        return gx, gw, None, None, None


class _Combine(torch.autograd.Function):
    """Buffer.combine (the sum over the ranks); its gradient is a dispatch with the same handle
    (combine_backward)."""

    @staticmethod
    def forward(ctx, y, buf: Buffer, handle):
        ctx.buf, ctx.handle = buf, handle
        return buf.combine(y, handle)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        recv_x = ctx.buf.dispatch(grad.contiguous(), handle=ctx.handle)[0]
        off = ctx.handle.row_offset
        return ctx.buf._rows_tensor(recv_x, off)[:off[-1]], None, None


class MoELayer(torch.nn.Module):
    """A mixture-of-experts layer over one virtual expert-parallel group: dispatch, rows into expert
    order, gate / up products, silu(gate) * up, down product, back with the routing weights,
    combine; plus a projection that every token passes, with each token's own adapter when
    serving. All ranks' experts live on this GPU, so one sort and one product cover all of
    them: rank d's local expert e is expert d * E_loc + e.

    checkpoint: None runs the experts product by product and keeps every step's result in bf16;
    "bf16", "e4m3" and "recompute" run them as expert_feed_forward does, the activation and the
    product in the projections' kernel, in serving too, where nothing is kept ("e4m3" keeps the
    experts' outputs in 8 bits too, for the routing weights' gradient). activation: "silu", or with a checkpoint "gelu"."""

    def __init__(self, buf: Buffer, features: int, device="cuda", checkpoint: Optional[str] = None,
                 activation: str = "silu"):
        super().__init__()
        _one_of("checkpoint", checkpoint, (None, "bf16", "e4m3", "recompute"))
        _one_of("activation", activation, tuple(_ACTIVATIONS) if checkpoint is not None else ("silu",))
        self.buf, self.checkpoint, self.activation = buf, checkpoint, activation
        H, E = buf.H, buf.E
        new = lambda *shape: torch.nn.Parameter(  # noqa: E731
            (torch.randn(*shape, device=device) * shape[-1] ** -0.5).bfloat16())
        self.gate_up, self.down, self.shared = new(E, 2 * features, H), new(E, H, features), new(H, H)

    def forward(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                adapters: Optional[tuple] = None) -> torch.Tensor:
        """x [R][T][H], topk_idx / topk_weights [R][T][k]; adapters: (a, b, scales, adapter_idx [R][T])
        of the shared projection (serving: under torch.no_grad(), a backward pass raises) or None
        -> [R][T][H]."""
        buf, out = self.buf, {}
        _check("x", x, torch.bfloat16, buf.R, None, buf.H)
        _check("topk_idx", topk_idx, torch.int64, buf.R, x.shape[1], buf.k)
        _check("topk_weights", topk_weights, torch.float32, buf.R, x.shape[1], buf.k)
        rows, weights = _Dispatch.apply(x, topk_weights, topk_idx, buf, out)
        off: List[int] = out["handle"].row_offset
        local = out["recv_idx"][:off[-1]]
        sizes = torch.tensor([off[d + 1] - off[d] for d in range(buf.R)], device=x.device)
        rank = torch.repeat_interleave(torch.arange(buf.R, device=x.device), sizes, output_size=off[-1])
        expert = torch.where(local >= 0, local + (rank * (buf.E // buf.R)).unsqueeze(1), local)
        sort = ExpertSort(expert, buf.E, buf.H, err=buf.err)
        if self.checkpoint is None:
            h = expert_product(sort_rows(rows, sort), self.gate_up, sort.expert_prefix, buf.err)
            gate, up = h.chunk(2, dim=1)
            y = expert_product(torch.nn.functional.silu(gate) * up, self.down, sort.expert_prefix, buf.err)
        else:
            y = expert_feed_forward(sort_rows(rows, sort), self.gate_up, self.down, sort.expert_prefix, self.activation,
                                    self.checkpoint, buf.err)
        back = unsort_rows(y, sort, weights, "e4m3" if self.checkpoint == "e4m3" else "bf16")
        routed = _Combine.apply(back, buf, out["handle"])
        flat = x.reshape(-1, buf.H)
        if adapters is None:
            one = torch.tensor([0, flat.shape[0]], dtype=torch.int32, device=x.device)
            common = expert_product(flat, self.shared.unsqueeze(0), one, buf.err)
        else:
            a, b, scales, idx = adapters
            common = adapter_projection(flat, self.shared, a, b, scales, idx.reshape(-1), buf.err)
        return routed + common.view_as(x)
