"""What a model does with the rows between dispatch and combine, as PyTorch autograd functions over
the C ABI: rows into expert order and back (``ep_sort_*`` / ``ep_unsort_*``), the experts' products
(``ep_expert_gemm*``) and a shared projection with each row's own low-rank adapter
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

from . import (EP_BF16, ep_adapter_gemm, ep_adapter_shape, ep_adapter_workspace_size, ep_expert_gemm,
               ep_expert_gemm_dgrad, ep_expert_gemm_wgrad, ep_gemm_shape, ep_read_error_flags_sync, ep_sort_layout, ep_sort_rows,
               ep_unsort_rows, ep_unsort_rows_backward, make_launch, make_shape)
from .api import Buffer
from .buffers import SortBuffers

__all__ = ["ExpertSort", "sort_rows", "unsort_rows", "expert_product", "adapter_projection", "check_errors",
           "MoELayer"]


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


def unsort_rows(y: torch.Tensor, sort: ExpertSort, weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [rows][H] -> [N][H], the sum of each row's entries, scaled by weights [N][k] fp32 if given;
    gradients to y and weights."""
    _check("y", y, torch.bfloat16, sort.rows, sort.H)
    if weights is not None:
        _check("weights", weights, torch.float32, sort.N, sort.k)
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
    them: rank d's local expert e is expert d * E_loc + e."""

    def __init__(self, buf: Buffer, features: int, device="cuda"):
        super().__init__()
        self.buf = buf
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
        h = expert_product(sort_rows(rows, sort), self.gate_up, sort.expert_prefix, buf.err)
        gate, up = h.chunk(2, dim=1)
        y = expert_product(torch.nn.functional.silu(gate) * up, self.down, sort.expert_prefix, buf.err)
        routed = _Combine.apply(unsort_rows(y, sort, weights), buf, out["handle"])
        flat = x.reshape(-1, buf.H)
        if adapters is None:
            one = torch.tensor([0, flat.shape[0]], dtype=torch.int32, device=x.device)
            common = expert_product(flat, self.shared.unsqueeze(0), one, buf.err)
        else:
            a, b, scales, idx = adapters
            common = adapter_projection(flat, self.shared, a, b, scales, idx.reshape(-1), buf.err)
        return routed + common.view_as(x)
