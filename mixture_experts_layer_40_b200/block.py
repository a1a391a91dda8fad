"""The Transformer block around an MoE layer, per-expert linear maps in 16
bits, and gradient clipping: thin holders of device memory over the C ABI, as
layer.MoELayer is. All compute is in the CUDA library.

A holder's buffers serve one call at a time: calls on several streams at once,
or two captured graphs replayed side by side, need holders of their own. A graph
that holds a call uses the holder's memory: keep the holder as long as the graph.
"""
from __future__ import annotations

import torch

from . import capi
from .layer import MoELayer


class MoEBlock:
    """r = x + alpha * scale * gate * N(layer(N(x; pre_weight)); post_weight):
    the norm before the MoE layer, the layer, and the norm after it with its
    gate and residual. post_weight, scale (weights [H], bf16 or float32 alike)
    and gate (float32 [T], or bf16 [T, H]) are optional. x is bf16 or float32;
    the layer runs on bf16. The block keeps the last forward's x, u and the
    layer's output (with next_weight also r) for the backward, and the layer its
    routing and rows: a backward after another pass of the same layer is refused
    (one inside a graph of the caller's cannot be seen)."""

    def __init__(self, layer: MoELayer, pre_weight: torch.Tensor,
                 post_weight: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                 alpha: float = 1.0, eps: float = 1e-6):
        self.layer, self.alpha, self.eps = layer, alpha, eps
        self.pre_weight, self.post_weight, self.scale = pre_weight, post_weight, scale
        shape = (layer.T, layer.H)
        self.u = torch.empty(shape, dtype=torch.bfloat16, device=layer.device)
        # the layer runs on the current device: made so in every call
        self._index = self.u.device.index if self.u.is_cuda else -1
        self.z = torch.empty(shape, dtype=torch.bfloat16, device=layer.device)
        self.x = self.gate = self.r = self.next_weight = self._ws = None

    def forward(self, x: torch.Tensor, bias: torch.Tensor, gate: torch.Tensor | None = None,
                r: torch.Tensor | None = None, next_weight: torch.Tensor | None = None,
                stream=None):
        """r [T, H] like x; with next_weight also u = N(r; next_weight), the
        normed input of what follows the block (an MoEBlock norms its own x),
        from the same pass: (r, u). r may be x, in place; there is no backward
        then, which reads x."""
        # the layer's state is a new forward's from here on
        self.x = self.gate = self.r = self.next_weight = None
        with torch.cuda.device(self._index), torch.cuda.stream(stream):  # None: the current one
            capi.moe_block_norm(x, self.eps, pre_weight=self.pre_weight, u=self.u, stream=stream)
            self.layer.forward(self.u, bias, self.z, stream)
            self._pass = getattr(self.layer, "passes", None)
            if r is None:
                r = torch.empty_like(x)
            u = None if next_weight is None else torch.empty_like(self.z)
            capi.moe_block_norm(x, self.eps, pre_weight=next_weight, u=u, z=self.z,
                                post_weight=self.post_weight, gate=gate, scale=self.scale,
                                alpha=self.alpha, r=r, stream=stream)
            if x.numel() == 0 or r.data_ptr() != x.data_ptr():  # (empty: both addresses are 0)
                self.x, self.gate = x, gate
                if next_weight is not None:
                    self.r, self.next_weight = r, next_weight
            self._keep(stream)
            return r if next_weight is None else (r, u)

    def backward(self, dr: torch.Tensor, weights: bool = True, stream=None,
                 du: torch.Tensor | None = None) -> dict:
        """Gradients of the last forward for the upstream gradients dr of r and,
        of a forward with next_weight, du of u (None: u was used for nothing
        that has a gradient), with the routing held fixed: a dict of dx (through
        the residual and the experts), gates (the layer's gate gradients,
        [T, K]), pre_weight, and as they were given post_weight, scale and gate;
        with du also next_weight; with `weights` also w13 and w2. With du the
        forward's r is read and must be as it was left."""
        if self.x is None:
            raise ValueError("backward needs a forward before it, and not one in place")
        if getattr(self.layer, "passes", None) != self._pass:
            raise ValueError("the layer has run since this block's forward; its state is another's")
        if du is not None and self.next_weight is None:
            raise ValueError("du needs a forward with next_weight before it")
        with torch.cuda.device(self._index), torch.cuda.stream(stream):  # None: the current one
            dev, H = self.layer.device, self.layer.H
            if self._ws is None:
                nbytes = capi.moe_block_norm_backward_workspace_size(H)
                self._ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)

            def column(w):
                return None if w is None else torch.empty(H, dtype=torch.float32, device=dev)

            out = {"pre_weight": column(self.pre_weight), "post_weight": column(self.post_weight),
                   "scale": column(self.scale),
                   "gate": None if self.gate is None else torch.empty_like(self.gate)}
            dz = torch.empty_like(self.z)
            # with du the norm of r joins in, and e is the whole gradient of r (to
            # dz unrounded, to dx rounded to x's type); without it r is not read
            e, r, norm = dr, dr, {}
            if du is not None:
                e, r, out["next_weight"] = torch.empty_like(dr), self.r, column(self.next_weight)
                norm = {"du": du, "pre_weight": self.next_weight, "dx": e, "dpre": out["next_weight"]}
            capi.moe_block_norm_backward(r, self.eps, self._ws, dr=dr, z=self.z,
                                         post_weight=self.post_weight, gate=self.gate,
                                         scale=self.scale, alpha=self.alpha, dz=dz,
                                         dgate=out["gate"], dscale=out["scale"],
                                         dpost=out["post_weight"], stream=stream, **norm)
            grads = self.layer.backward(dz, self.u if weights else None, stream)
            dx = torch.empty_like(self.x)
            capi.moe_block_norm_backward(self.x, self.eps, self._ws, dr=e, du=grads[0],
                                         pre_weight=self.pre_weight, dx=dx, dpre=out["pre_weight"],
                                         stream=stream)
            self._keep(stream)
            out.update(dx=dx, gates=grads[1])
            if weights:
                out.update(w13=grads[2], w2=grads[3])
            return {k: v for k, v in out.items() if v is not None}

    def _keep(self, stream):
        if self.u.is_cuda:
            capi.keep_until_done(self.u.device.index, stream, self.u, self.z, self._ws)


class GroupedLinear:
    """y[r] = x[r] W_g^T for the rows of each expert's group: weight [G, N, K],
    bf16 or fp16. The groups are device arrays (rows and first row of each),
    packed or with gaps, as MoELayer's workspace views "group_rows" and
    "row_start" hold them after a forward. A group table that fails the kernels'
    checks, or a wait that ran out, shows in status(), or in the status word
    that a call was given."""

    def __init__(self, weight: torch.Tensor):
        if weight.dim() != 3:
            raise ValueError("weight must be [groups, N, K]")
        self.weight = weight
        self._status = torch.zeros(1, dtype=torch.int32, device=weight.device)

    def status(self, stream=None) -> int:
        """MOE_OK, or the error code of the calls since the last status();
        waits for the stream."""
        return capi.moe_get_status(self._status, stream)

    def _keep(self, stream):
        capi.keep_until_done(self._status.device.index, stream, self._status)

    def forward(self, x, group_rows, group_start, y=None, status=None, stream=None):
        """y [R, N] like x; rows outside the groups stay as they are (zero in a
        new y)."""
        with torch.cuda.stream(stream):  # None: the current one
            if y is None:
                y = torch.zeros((x.shape[0], self.weight.shape[1]), dtype=x.dtype, device=x.device)
            capi.moe_grouped_matmul(x, self.weight, group_rows, group_start, y, True,
                                    self._status if status is None else status, stream)
            self._keep(stream)
            return y

    def backward(self, dy, x, group_rows, group_start, dw=None, accumulate=False, dx=None,
                 status=None, stream=None):
        """(dx [R, K] like dy, dw [G, N, K] float32); with accumulate the weight
        gradient is added to the dw given."""
        if accumulate and dw is None:
            raise ValueError("accumulate needs the dw to add to")
        if status is None:
            status = self._status
        with torch.cuda.stream(stream):  # None: the current one
            if dx is None:
                dx = torch.zeros((dy.shape[0], self.weight.shape[2]), dtype=dy.dtype, device=dy.device)
            if dw is None:
                dw = torch.empty(self.weight.shape, dtype=torch.float32, device=dy.device)
            capi.moe_grouped_matmul(dy, self.weight, group_rows, group_start, dx, False, status, stream)
            capi.moe_grouped_wgrad(dy, x, group_rows, group_start, dw, accumulate, status, stream)
            self._keep(stream)
            return dx, dw


class GradClip:
    """Clips a fixed set of gradient tensors by their global norm:

        clip = GradClip([grads["w13"], grads["w2"], ...])
        norm = clip(max_norm=1.0)

    In place, or into `out`. With the experts sharded over several GPUs the
    ranks' sums of squares have to meet first: call capi.moe_grad_sumsq and
    moe_grad_clip with an all-reduce of the partials between them."""

    def __init__(self, grads, out=None):
        self.list = capi.make_grad_list(grads, out)
        if self.list.device is None:
            raise ValueError("no gradients")
        dev = torch.device("cuda", self.list.device)
        self.partials = torch.empty(capi.GRAD_PARTIALS, dtype=torch.float64, device=dev)
        self.norm = torch.empty(1, dtype=torch.float32, device=dev)

    def __call__(self, max_norm: float, stream=None) -> torch.Tensor:
        """The norm before clipping, float32 [1] on the device (overwritten by
        the next call)."""
        capi.moe_grad_sumsq(self.list, self.partials, stream)
        capi.moe_grad_clip(self.list, self.partials, max_norm, self.norm, stream)
        capi.keep_until_done(self.list.device, stream, self.partials, self.norm)
        return self.norm
