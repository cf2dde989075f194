"""What surrounds the block in a decoder layer and in its training step: norms
fused with the combine, the gate and the scaled residual, their backward pass,
and the global gradient norm with clipping (bindings of include/moe.h), and
`MoESublayer`, which chains them with a `MoELayer`.

As in `moe.py`, PyTorch provides device memory and streams only.  A call runs
on `stream`, by default the current stream of its tensors' device; what it
allocates (outputs, a missing workspace) is allocated on that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import moe as _moe
from .moe import MOE_BF16, MOE_F32, MoELayer, Shape, _check, load_library

NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}
GATE_NONE, GATE_TOKEN, GATE_CHANNEL = 0, 1, 2


class MoENormSpec(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


@dataclass(frozen=True)
class Norm:
    """A norm over the hidden dimension: kind "rms", "layer" or "none";
    weight and bias [H] float32 (None: ones, zeros)."""
    kind: str = "rms"
    eps: float = 1e-5
    weight: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None

    def __post_init__(self):
        if self.kind not in NORM_KINDS:
            raise ValueError(f"unknown norm kind {self.kind!r}")
        if self.kind == "none" and (self.weight is not None or self.bias is not None):
            raise ValueError("a norm of kind 'none' has no weight or bias")

    def c(self) -> MoENormSpec:
        return MoENormSpec(NORM_KINDS[self.kind], self.eps,
                           None if self.weight is None else self.weight.data_ptr(),
                           None if self.bias is None else self.bias.data_ptr())


def _tensor(name, t, size, dtype, device):
    """`t` must be a dense tensor of this size, type and device."""
    if t.shape != size or t.dtype != dtype or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(size)} on "
                         f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}"
                         + ("" if t.is_contiguous() else " (not contiguous)"))


def _cuda(t):
    if not t.is_cuda:
        raise ValueError(f"expected CUDA tensors, got one on {t.device}")
    return t.device


def _addr(t):
    return None if t is None else t.data_ptr()


def _check_norm(name, n: Norm, H, device):
    for part in ("weight", "bias"):
        t = getattr(n, part)
        if t is not None:
            _tensor(f"{name}.{part}", t, (H,), torch.float32, device)


def _gate_kind(gate, shape: Shape, device) -> int:
    if gate is None:
        return GATE_NONE
    token = gate.dim() == 2 and gate.shape[1] == 1 and gate.shape[0] == shape.T
    channel = gate.shape in ((shape.H,), (1, shape.H))
    if not (token or channel):
        raise ValueError(f"gate must be [T, 1] = [{shape.T}, 1] or [H] = [{shape.H}], got "
                         f"{tuple(gate.shape)}")
    _tensor("gate", gate, gate.shape, torch.float32, device)
    return GATE_TOKEN if token else GATE_CHANNEL


# the raw handle alone where this PyTorch has the call (2 us less than through
# a Stream object, on calls of 15 us)
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(device) -> int:
    if _current_raw is not None:
        return _current_raw(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class _launch:
    """`with _launch(device, stream) as raw`: the raw stream of a call on
    `device`'s tensors, that device and (when one is given) `stream` being
    current inside."""
    __slots__ = ("device", "stream", "guard")

    def __init__(self, device, stream):
        self.device, self.stream, self.guard = device, stream, None

    def __enter__(self):
        if self.stream is not None:
            if self.stream.device != self.device:
                raise ValueError(f"stream is on {self.stream.device}, the tensors on {self.device}")
            self.guard = torch.cuda.stream(self.stream)
            self.guard.__enter__()
            return self.stream.cuda_stream
        if torch.cuda.current_device() != self.device.index:
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        return _raw_stream(self.device)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _on(device):
    """`device` current inside: what is sized by its SMs is sized by that device's."""
    device = torch.device(device)
    return torch.cuda.device(device) if device.type == "cuda" else contextlib.nullcontext()


def _check_workspace(t, device):
    """Kernels write the workspace as one run of bytes from its first."""
    if t is not None and t.device != device:
        raise ValueError(f"workspace is on {t.device}, the tensors on {device}")
    if t is not None and not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous, got strides {t.stride()}")


def _nbytes(t):
    return t.numel() * t.element_size()


def norm(shape: Shape, spec: Norm, x, out=None, stream=None):
    """N(x) [T, H] (dtype): the norm before the block."""
    lib, dev, size = load_library(), _cuda(x), (shape.T, shape.H)
    _tensor("x", x, size, shape.torch_dtype, dev)
    _check_norm("norm", spec, shape.H, dev)
    if out is not None:
        _tensor("out", out, size, shape.torch_dtype, dev)
    with _launch(dev, stream) as s:
        if out is None:
            out = torch.empty_like(x)
        _check(lib.moe_norm_forward(ctypes.byref(shape.c()), ctypes.byref(spec.c()), x.data_ptr(),
                                    out.data_ptr(), s), "moe_norm_forward")
    return out


def combine_norm(shape: Shape, y_slots, inv, residual=None, post: Optional[Norm] = None,
                 gate=None, scale: float = 1.0, next_norm: Optional[Norm] = None,
                 keep_y: bool = False, out=None, stream=None):
    """The combine, the norm after the block, its gate, the scaled residual and
    the next norm in one launch: (h, xn or None, y or None) with
    h = residual + scale * gate * N_post(y), xn = N_next(h), y = combine(y_slots).

    gate: [T, 1] (per token) or [H] (per channel) float32.  keep_y: also return
    y (rounded), which norm_backward reads.  out: optional dict of h, xn, y
    buffers, apart from one another (one of them may be `residual`)."""
    lib, dev, dt = load_library(), _cuda(y_slots), shape.torch_dtype
    size = (shape.T, shape.H)
    _tensor("y_slots", y_slots, (shape.slot_rows, shape.H), dt, dev)
    if inv.numel() != shape.T * shape.k:
        raise ValueError(f"inv must hold T*k = {shape.T * shape.k} indices, got {inv.numel()}")
    _tensor("inv", inv, inv.shape, torch.int32, dev)
    if residual is not None:
        _tensor("residual", residual, size, dt, dev)
    if post is not None:
        _check_norm("post", post, shape.H, dev)
    if next_norm is not None:
        _check_norm("next_norm", next_norm, shape.H, dev)
    kind = _gate_kind(gate, shape, dev)
    bufs = dict(out) if out else {}
    if not bufs.keys() <= {"h", "xn", "y"}:
        raise ValueError(f"out takes buffers named h, xn and y, got {sorted(bufs)}")
    for name, t in bufs.items():
        if t is not None:
            _tensor(name, t, size, dt, dev)
    with _launch(dev, stream) as s:
        h, xn, y = bufs.get("h"), None, None
        if h is None:
            h = y_slots.new_empty(size) if residual is None else torch.empty_like(residual)
        if next_norm is not None:
            xn = bufs.get("xn")
            if xn is None:
                xn = torch.empty_like(h)
        if keep_y:
            y = bufs.get("y")
            if y is None:
                y = torch.empty_like(h)
        _check(lib.moe_combine_norm(
            ctypes.byref(shape.c()), y_slots.data_ptr(), inv.data_ptr(), _addr(residual),
            None if post is None else ctypes.byref(post.c()), kind, _addr(gate), scale,
            None if next_norm is None else ctypes.byref(next_norm.c()), _addr(y), h.data_ptr(),
            _addr(xn), s), "moe_combine_norm")
    return h, xn, y


def norm_backward_workspace_size(shape: Shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_norm_backward_workspace_size(ctypes.byref(shape.c()),
                                                           ctypes.byref(n)),
           "moe_norm_backward_workspace_size")
    return n.value


def alloc_norm_backward_workspace(shape: Shape, device="cuda") -> torch.Tensor:
    with _on(device):
        return torch.empty(norm_backward_workspace_size(shape), dtype=torch.uint8, device=device)


def norm_backward(shape: Shape, spec: Norm, x, dout, gate=None, scale: float = 1.0, dadd=None,
                  workspace=None, dx=None, stream=None):
    """Gradients of scale * gate * N(x): dict of x (dtype, plus `dadd`, the
    gradient that reaches x past the norm), weight, bias and gate (float32;
    None where the norm or the call has none)."""
    lib, dev, dt = load_library(), _cuda(x), shape.torch_dtype
    size = (shape.T, shape.H)
    for name, t in (("x", x), ("dout", dout), ("dadd", dadd), ("dx", dx)):
        if t is not None:
            _tensor(name, t, size, dt, dev)
    _check_norm("norm", spec, shape.H, dev)
    kind = _gate_kind(gate, shape, dev)
    _check_workspace(workspace, dev)
    with _launch(dev, stream) as s:
        if workspace is None:
            workspace = alloc_norm_backward_workspace(shape, dev)
        g = {"x": torch.empty_like(x) if dx is None else dx,
             "weight": None if spec.weight is None else torch.empty_like(spec.weight),
             "bias": None if spec.bias is None else torch.empty_like(spec.bias),
             "gate": None if gate is None else torch.empty_like(gate)}
        _check(lib.moe_norm_backward(
            ctypes.byref(shape.c()), ctypes.byref(spec.c()), x.data_ptr(), dout.data_ptr(), kind,
            _addr(gate), scale, _addr(dadd), g["x"].data_ptr(), _addr(g["weight"]), _addr(g["bias"]),
            _addr(g["gate"]), workspace.data_ptr(), _nbytes(workspace), s),
            "moe_norm_backward")
    return g


# ------------------------------------------------------------- gradient norm, clipping
def alloc_grad_norm_workspace(device="cuda") -> torch.Tensor:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_grad_norm_workspace_size(ctypes.byref(n)),
           "moe_grad_norm_workspace_size")
    return torch.empty(n.value, dtype=torch.uint8, device=device)


_GRAD_TYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _grad_arrays(grads):
    """(device, n, pointers, sizes, types) of a list of dense gradients; None entries skipped."""
    grads = [g for g in grads if g is not None]
    n = len(grads)
    dev = grads[0].device if n else None
    types = (ctypes.c_int32 * n)()
    for i, g in enumerate(grads):
        kind = _GRAD_TYPES.get(g.dtype)
        if kind is None:
            raise ValueError(f"gradients must be float32 or bfloat16, got {g.dtype}")
        if g.device != dev:
            raise ValueError(f"gradients on {dev} and {g.device}: clip each device's alone, on "
                             "the all-reduced grad_square_sum")
        if not g.is_contiguous():
            raise ValueError(f"gradients must be contiguous, got strides {g.stride()}")
        types[i] = kind
    if n:
        _cuda(grads[0])
    return dev, n, (ctypes.c_void_p * n)(*[g.data_ptr() for g in grads]), \
        (ctypes.c_int64 * n)(*[g.numel() for g in grads]), types


def _check_clip(dev, workspace=None):
    if dev is None:
        raise ValueError("no gradients given")
    _check_workspace(workspace, dev)


def grad_square_sum(grads: Sequence[Optional[torch.Tensor]], workspace=None, stream=None):
    """[1] float64: the sum of squares over all tensors.  Ranks that hold
    different gradients sum it over their group before clip_grads."""
    lib = load_library()
    dev, n, ptrs, sizes, types = _grad_arrays(grads)
    _check_clip(dev, workspace)
    with _launch(dev, stream) as s:
        ws = alloc_grad_norm_workspace(dev) if workspace is None else workspace
        total = torch.empty(1, dtype=torch.float64, device=dev)
        _check(lib.moe_grad_square_sum(n, ptrs, sizes, types, total.data_ptr(), ws.data_ptr(),
                                       _nbytes(ws), s), "moe_grad_square_sum")
    return total


def clip_grads(grads, max_norm: float, square_sum, stream=None):
    """Scales the gradients in place to max_norm, given their square sum
    (float64 [1], from grad_square_sum); returns the norm, [1] float32."""
    lib = load_library()
    dev, n, ptrs, sizes, types = _grad_arrays(grads)
    _check_clip(dev)
    _tensor("square_sum", square_sum, (1,), torch.float64, dev)
    with _launch(dev, stream) as s:
        norm_out = torch.empty(1, dtype=torch.float32, device=dev)
        _check(lib.moe_clip_grads(n, ptrs, sizes, types, square_sum.data_ptr(), max_norm,
                                  norm_out.data_ptr(), s), "moe_clip_grads")
    return norm_out


def clip_grad_norm(grads, max_norm: float, workspace=None, stream=None):
    """Clips the gradients in place to a global norm of max_norm; returns the
    norm before clipping, [1] float32 on the device (nothing synchronises)."""
    lib = load_library()
    dev, n, ptrs, sizes, types = _grad_arrays(grads)
    _check_clip(dev, workspace)
    with _launch(dev, stream) as s:
        ws = alloc_grad_norm_workspace(dev) if workspace is None else workspace
        norm_out = torch.empty(1, dtype=torch.float32, device=dev)
        _check(lib.moe_clip_grad_norm(n, ptrs, sizes, types, max_norm, norm_out.data_ptr(),
                                      ws.data_ptr(), _nbytes(ws), s), "moe_clip_grad_norm")
    return norm_out


# ------------------------------------------------------------------ the whole sub-layer
class MoESublayer:
    """A decoder layer's sparse sub-layer around a MoELayer:

        h' = h + scale * gate * N_post(block(N_pre(h)))      (and N_next(h'))

    `gate` [T, 1] or [H] float32, or None; a gate that depends on the tokens is
    given to the call instead.  __call__ is the serving form;
    forward_train / backward the training form (bf16, more than 8 tokens).
    The weights may change in place from step to step.  Serving after such a
    change: layer.refresh_router() first.  A layer that merged its shared experts
    is trained on the merged layer.sh_gate_up and layer.sh_down, whose shapes
    their gradients have (merge_shared=False keeps them as given).
    """

    def __init__(self, layer: MoELayer, pre: Norm, post: Optional[Norm] = None, gate=None,
                 scale: float = 1.0, next_norm: Optional[Norm] = None):
        self.layer, self.pre, self.post = layer, pre, post
        self.gate, self.scale, self.next_norm = gate, float(scale), next_norm
        self.xn = torch.empty(layer.shape.T, layer.shape.H, dtype=layer.shape.torch_dtype,
                              device=layer.err_flag.device)

    def __call__(self, h, xn=None, out=None, stream=None, gate=None):
        """(h', N_next(h') or None).  `xn`: N_pre(h) when the previous layer's
        fused next norm has computed it already.  `out`: optional dict of h and
        xn buffers.  `gate`: this call's, in place of the sub-layer's."""
        layer = self.layer
        for name, t in (("h", h), ("xn", xn)):           # the block reads them unchecked
            if t is not None:
                _tensor(name, t, self.xn.shape, self.xn.dtype, self.xn.device)
        with _launch(layer.err_flag.device, stream):     # the block's calls follow it
            if xn is None:
                xn = norm(layer.shape, self.pre, h, out=self.xn, stream=stream)
            y_slots, inv = layer.slots(xn, stream=stream)
            return combine_norm(layer.shape, y_slots, inv, h, post=self.post,
                                gate=self.gate if gate is None else gate,
                                scale=self.scale, next_norm=self.next_norm, out=out,
                                stream=stream)[:2]

    def forward_train(self, h, gate=None):
        """(h', saved): the training forward; `saved` is what backward reads, the
        step's norms, gate and scale among it.  `gate` as in __call__."""
        with _launch(self.layer.err_flag.device, None):
            return self._forward_train(h, self.gate if gate is None else gate)

    def _forward_train(self, h, gate):
        layer, s = self.layer, self.layer.shape
        if layer.gate_up is None or layer.routing is not None:
            raise ValueError("training needs bf16 expert weights and the softmax routing")
        dev = h.device
        xn = norm(s, self.pre, h)
        layer.refresh_router()           # the last step changed the weight
        idx, w, logits = _moe.route(s, xn, layer.w_router, layer.router_bias, logits=True,
                                    err_flag=layer.err_flag, w_split=layer.w_split)
        counts, offsets, perm, inv = _moe.permute(s, idx, layer.workspace, layer.err_flag)
        state = torch.empty(_moe.train_state_size(s), dtype=torch.uint8, device=dev)
        y_slots = _moe.forward_train(s, xn, offsets, perm, w, layer.gate_up, layer.down,
                                     layer.sh_gate_up, layer.sh_down, layer.workspace, state,
                                     layer.err_flag)
        h2, _, y = combine_norm(s, y_slots, inv, h, post=self.post, gate=gate,
                                scale=self.scale, keep_y=True)
        return h2, dict(h=h, xn=xn, y=y, pre=self.pre, post=self.post, gate=gate,
                        scale=self.scale, topk_idx=idx, topk_w=w, logits=logits, counts=counts,
                        offsets=offsets, perm=perm, inv=inv, state=state)

    def backward(self, saved, dh, aux_coef: float = 0.0):
        """Gradients given dh = dL/dh': dict of h (dtype), the block's
        (moe.backward's names) and pre_weight, pre_bias, post_weight,
        post_bias, gate (float32; absent where there is none)."""
        with _launch(self.layer.err_flag.device, None):
            return self._backward(saved, dh, aux_coef)

    def _backward(self, saved, dh, aux_coef):
        layer, s = self.layer, self.layer.shape
        post = saved["post"] if saved["post"] is not None else Norm("none")
        gp = norm_backward(s, post, saved["y"], dh, gate=saved["gate"], scale=saved["scale"])
        ws = torch.empty(_moe.backward_workspace_size(s), dtype=torch.uint8, device=dh.device)
        g = _moe.backward(s, saved["xn"], layer.w_router, saved["topk_idx"], saved["topk_w"],
                          saved["counts"], saved["offsets"], saved["perm"], saved["inv"],
                          layer.gate_up, layer.down, layer.sh_gate_up, layer.sh_down,
                          saved["state"], gp["x"], ws, layer.err_flag, logits=saved["logits"],
                          aux_coef=aux_coef)
        # the residual's gradient joins in the norm's backward pass
        gn = norm_backward(s, saved["pre"], saved["h"], g.pop("x"), dadd=dh)
        g["h"] = gn["x"]
        for name, part in (("pre", gn), ("post", gp)):
            for p in ("weight", "bias"):
                if part[p] is not None:
                    g[f"{name}_{p}"] = part[p]
        if gp["gate"] is not None:
            g["gate"] = gp["gate"]
        return {n: t for n, t in g.items() if t is not None}
