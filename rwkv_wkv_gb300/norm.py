"""Python binding of the gated norm of a layer's readout (wkv7_gated_norm of include/wkv7.h):
argument marshalling only."""
from __future__ import annotations

import torch

from .wkv7 import BF16, F32, NORM_ARGS, _check, _empty, _stream_handle, load_library, row_stride

_CODES = {torch.float32: F32, torch.bfloat16: BF16}
_KINDS = {"rms": 0, "layer": 1}
_GATES = {None: 0, "silu": 1, "sigmoid": 2}


def gated_norm(x: torch.Tensor, z: torch.Tensor | None = None, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, *, group_size: int | None = None, eps: float = 1e-5, kind: str = "rms",
               activation: str | None = "silu", gate_first: bool = False, out_dtype: torch.dtype | None = None,
               o: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Norm of each `group_size` consecutive columns (default: the whole row) of x [rows, width]
    with the gate z [rows, width]: norm(x act(z)) with gate_first, else norm(x) act(z).

    kind 'rms' or 'layer'; activation of the gate 'silu', 'sigmoid' or None (z itself).  weight
    and bias [width] share one type.  x, z and weight are float32 or bfloat16, each its own;
    rows of x and z may be any stride apart (column ranges of a projection).  A readout
    [rows, heads, size] is passed as readout.flatten(1).  The result has out_dtype (default x's)."""
    if kind not in _KINDS:
        raise ValueError("kind must be 'rms' or 'layer'")
    if activation not in _GATES:
        raise ValueError("activation must be 'silu', 'sigmoid' or None")
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a CUDA tensor [rows, width]")
    rows, width = x.shape
    for name, t, shape in (("z", z, (rows, width)), ("weight", weight, (width,)), ("bias", bias, (width,))):
        if t is None:
            continue
        if t.shape != shape or t.get_device() != x.get_device():
            raise ValueError(f"{name} must be {list(shape)} on {x.device}")
        if t.dtype not in _CODES:
            raise TypeError(f"{name} must be float32 or bfloat16")
    if x.dtype not in _CODES:
        raise TypeError("x must be float32 or bfloat16")
    if weight is not None and not weight.is_contiguous() or bias is not None and not bias.is_contiguous():
        raise ValueError("weight and bias must be contiguous")
    if weight is not None and bias is not None and weight.dtype is not bias.dtype:
        raise TypeError("weight and bias must share one type")
    out = x.dtype if out_dtype is None else out_dtype
    if o is not None:
        if o.shape != (rows, width) or not o.is_contiguous() or o.get_device() != x.get_device() or \
                out_dtype is not None and o.dtype is not out_dtype:
            raise ValueError(f"o must be a contiguous [{rows}, {width}] tensor on {x.device}")
        out = o.dtype
    if out not in _CODES:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if o is None:
        o = _empty((rows, width), out, x.device, stream)
    w = weight if weight is not None else bias
    args = NORM_ARGS.pack(rows, width, width if group_size is None else int(group_size), _CODES[x.dtype],
                          F32 if z is None else _CODES[z.dtype], F32 if w is None else _CODES[w.dtype], _CODES[out],
                          _KINDS[kind], _GATES[activation], int(bool(gate_first)), eps, x.data_ptr(),
                          row_stride("x", x.stride(), (rows,), (width,)), 0 if z is None else z.data_ptr(),
                          0 if z is None else row_stride("z", z.stride(), (rows,), (width,)),
                          0 if weight is None else weight.data_ptr(), 0 if bias is None else bias.data_ptr(), o.data_ptr())
    _check(load_library().wkv7_gated_norm(args, _stream_handle(stream, x.device)), "gated_norm")
    return o
