"""Experts in 8-bit floating point (E4M3 codes, one float32 scale per 128 x 128
weight block, activations rounded per 128 columns): bindings of moe_fp8_quantize
and moe_forward_fp8.

An expert set is a dict of codes (float8_e4m3fn, or uint8 holding the same
bytes) and scales (float32):
    gate_up_q [E, 2I, H]   gate_up_s [E, 2, ceil(I/128), ceil(H/128)]
    down_q    [E, H, I]    down_s    [E, ceil(H/128), ceil(I/128)]
and with shared experts sh_gate_up_q, sh_gate_up_s, sh_down_q, sh_down_s alike.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .moe import MOE_BF16, MOE_F32, Shape, _check, load_library
from .sublayer import _addr, _check_workspace, _cuda, _launch, _nbytes, _on, _tensor

CODE_TYPES = (torch.float8_e4m3fn, torch.uint8)


def _blocks(n: int) -> int:
    return -(-n // 128)


def fp8_quantize(w, stream=None):
    """w [..., R, C] (float32 or bf16) -> (codes float8_e4m3fn, same shape;
    scales float32 [..., ceil(R/128), ceil(C/128)]): done once, at load time."""
    lib, dev = load_library(), _cuda(w)
    if w.dtype not in (torch.float32, torch.bfloat16) or w.dim() < 2 or not w.is_contiguous():
        raise ValueError("fp8_quantize takes contiguous float32 or bfloat16 matrices, got "
                         f"{w.dtype} {tuple(w.shape)}")
    *lead, R, C = w.shape
    n = 1
    for v in lead:
        n *= v
    with _launch(dev, stream) as st:
        q = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=dev)
        s = torch.empty(*lead, _blocks(R), _blocks(C), dtype=torch.float32, device=dev)
        _check(lib.moe_fp8_quantize(n, R, C, w.data_ptr(),
                                    MOE_BF16 if w.dtype == torch.bfloat16 else MOE_F32,
                                    q.data_ptr(), s.data_ptr(), st), "moe_fp8_quantize")
    return q, s


def fp8_experts(gate_up, down, sh_gate_up=None, sh_down=None, stream=None) -> dict:
    """The expert set of float32 or bf16 weights (gate_up [E, 2I, H], down [E, H, I]
    and the shared experts'), gate and up blocked separately."""
    out = {}
    for name, gu, dn in (("", gate_up, down), ("sh_", sh_gate_up, sh_down)):
        if gu is None:
            continue
        E, I2, H = gu.shape
        q, s = fp8_quantize(gu.view(E, 2, I2 // 2, H), stream=stream)
        out[f"{name}gate_up_q"], out[f"{name}gate_up_s"] = q.view(E, I2, H), s
        out[f"{name}down_q"], out[f"{name}down_s"] = fp8_quantize(dn, stream=stream)
    return out


def fp8_workspace_size(shape: Shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_fp8_workspace_size(ctypes.byref(shape.c()), ctypes.byref(n)),
           "moe_fp8_workspace_size")
    return n.value


def alloc_fp8_workspace(shape: Shape, device="cuda") -> torch.Tensor:
    with _on(device):
        return torch.empty(max(fp8_workspace_size(shape), 1), dtype=torch.uint8, device=device)


def _codes(name, t, size, dev):
    if t.dtype not in CODE_TYPES:
        raise ValueError(f"{name} must hold E4M3 codes (float8_e4m3fn or uint8), got {t.dtype}")
    _tensor(name, t, size, t.dtype, dev)


def check_fp8_experts(shape: Shape, fp8: dict, device) -> None:
    """Raises unless `fp8` is an expert set of `shape` on `device`."""
    H = shape.H
    sets = [("", shape.E, shape.I)]
    if shape.n_shared:
        sets.append(("sh_", shape.n_shared, shape.I_shared))
    for pre, E, I in sets:
        for name in ("gate_up_q", "gate_up_s", "down_q", "down_s"):
            if fp8.get(pre + name) is None:
                raise ValueError(f"{pre}{name} is missing")
        _codes(f"{pre}gate_up_q", fp8[f"{pre}gate_up_q"], (E, 2 * I, H), device)
        _codes(f"{pre}down_q", fp8[f"{pre}down_q"], (E, H, I), device)
        _tensor(f"{pre}gate_up_s", fp8[f"{pre}gate_up_s"], (E, 2, _blocks(I), _blocks(H)),
                torch.float32, device)
        _tensor(f"{pre}down_s", fp8[f"{pre}down_s"], (E, _blocks(H), _blocks(I)), torch.float32,
                device)


def forward_fp8(shape: Shape, x, offsets, perm, topk_w, fp8: dict, workspace=None, err_flag=None,
                y_slots: Optional[torch.Tensor] = None, stream=None):
    """moe_forward with the experts `fp8`: y_slots [T*k + S*T, H] (bf16)."""
    lib, dev = load_library(), _cuda(x)
    n = shape.T * shape.k
    _tensor("x", x, (shape.T, shape.H), shape.torch_dtype, dev)
    _tensor("offsets", offsets, (shape.E + 1,), torch.int32, dev)
    _tensor("perm", perm, (n,), torch.int32, dev)
    _tensor("topk_w", topk_w, (shape.T, shape.k), torch.float32, dev)
    check_fp8_experts(shape, fp8, dev)
    if y_slots is not None:
        _tensor("y_slots", y_slots, (shape.slot_rows, shape.H), shape.torch_dtype, dev)
    _check_workspace(workspace, dev)
    if err_flag is not None and (err_flag.device != dev or err_flag.dtype != torch.int32
                                 or err_flag.numel() < 1):
        raise ValueError(f"err_flag must be an int32 word on {dev}, got {err_flag.dtype} "
                         f"{tuple(err_flag.shape)} on {err_flag.device}")
    with _launch(dev, stream) as st:
        if workspace is None:
            workspace = alloc_fp8_workspace(shape, dev)
        if y_slots is None:
            y_slots = torch.empty(shape.slot_rows, shape.H, dtype=shape.torch_dtype, device=dev)
        sh = [_addr(fp8.get(f"sh_{k}") if shape.n_shared else None)
              for k in ("gate_up_q", "gate_up_s", "down_q", "down_s")]
        _check(lib.moe_forward_fp8(
            ctypes.byref(shape.c()), x.data_ptr(), offsets.data_ptr(), perm.data_ptr(),
            topk_w.data_ptr(), fp8["gate_up_q"].data_ptr(), fp8["gate_up_s"].data_ptr(),
            fp8["down_q"].data_ptr(), fp8["down_s"].data_ptr(), *sh, y_slots.data_ptr(),
            _addr(err_flag), workspace.data_ptr(), _nbytes(workspace), st), "moe_forward_fp8")
    return y_slots
