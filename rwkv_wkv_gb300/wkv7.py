"""Python binding of libwkv7 (ctypes).  Argument marshalling only: every step
of the recurrence and of the slot verbs runs in the library's CUDA kernels.
PyTorch supplies device memory (the pool buffer, the caller's tensors) and the
current CUDA stream; nothing here computes.

The C contract (layouts, ownership, errors) is documented in include/wkv7.h.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libwkv7.so")

F32, BF16 = 0, 1
DEV_OK, DEV_BAD_SLOT, DEV_BAD_SEQLENS, DEV_WAIT_TIMEOUT, DEV_DECAY_RANGE, DEV_DUP_SLOT = 0, 1, 2, 3, 4, 5
DEV_BAD_TOKEN = 6
TABLE_SLOTS, TABLE_SNAPSHOTS = 0, 1
HEAD_SIZE = 64
_HEADER_BYTES = 256

STATUS_NAMES = {
    0: "OK", 1: "ERR_INVALID_ARG", 2: "ERR_BAD_SLOT", 3: "ERR_DUP_SLOT", 4: "ERR_POOL_FULL",
    5: "ERR_BAD_SEQLENS", 6: "ERR_CUDA", 7: "ERR_UNSUPPORTED", 8: "ERR_DEVICE_STATUS",
    9: "ERR_TIMEOUT", 10: "ERR_NO_MEMORY",
}


class Wkv7Error(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))
        msg = f"{what}: {self.name}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


class PoolDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("head_size", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("n_snapshots", ctypes.c_int32), ("device_buffer", ctypes.c_void_p),
                ("buffer_bytes", ctypes.c_size_t), ("state_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class GdnPoolDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_k_heads", ctypes.c_int32),
                ("n_v_heads", ctypes.c_int32), ("head_k", ctypes.c_int32),
                ("head_v", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("n_snapshots", ctypes.c_int32), ("device_buffer", ctypes.c_void_p),
                ("buffer_bytes", ctypes.c_size_t), ("state_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class GdnTokens(ctypes.Structure):
    _fields_ = [("in_dtype", ctypes.c_int32), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("g_stride", ctypes.c_int64),
                ("beta_stride", ctypes.c_int64), ("scale", ctypes.c_float),
                ("l2norm_eps", ctypes.c_float), ("o", ctypes.c_void_p)]


class ConvDesc(ctypes.Structure):
    _fields_ = [("channels", ctypes.c_int32), ("width", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class SsmPoolDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_groups", ctypes.c_int32), ("head_p", ctypes.c_int32),
                ("d_state", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("n_snapshots", ctypes.c_int32), ("device_buffer", ctypes.c_void_p),
                ("buffer_bytes", ctypes.c_size_t), ("state_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("conv", ConvDesc)]


class SsmTokens(ctypes.Structure):
    _fields_ = [("in_dtype", ctypes.c_int32), ("dt_dtype", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("b", ctypes.c_void_p), ("c", ctypes.c_void_p),
                ("dt", ctypes.c_void_p), ("a", ctypes.c_void_p), ("d", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64),
                ("dt_stride", ctypes.c_int64), ("dt_softplus", ctypes.c_int32), ("all_or_none", ctypes.c_int32),
                ("o", ctypes.c_void_p)]


class ConvTokens(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("weight_dtype", ctypes.c_int32), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("activation", ctypes.c_int32), ("o", ctypes.c_void_p)]


class NormArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("width", ctypes.c_int32), ("group", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("z_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("o_dtype", ctypes.c_int32), ("kind", ctypes.c_int32), ("act", ctypes.c_int32),
                ("gate_first", ctypes.c_int32), ("eps", ctypes.c_float), ("x", ctypes.c_void_p),
                ("x_stride", ctypes.c_int64), ("z", ctypes.c_void_p), ("z_stride", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("o", ctypes.c_void_p)]


class DraftBatch(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("n_draft", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("prob_dtype", ctypes.c_int32), ("p", ctypes.c_void_p),
                ("p_batch_stride", ctypes.c_int64), ("p_row_stride", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("q_batch_stride", ctypes.c_int64),
                ("q_row_stride", ctypes.c_int64), ("draft_ids", ctypes.c_void_p),
                ("n_draft_rows", ctypes.c_void_p), ("uniforms", ctypes.c_void_p),
                ("noise", ctypes.c_void_p), ("noise_stride", ctypes.c_int64),
                ("step_snap_ids", ctypes.c_void_p), ("accepted", ctypes.c_void_p),
                ("tokens", ctypes.c_void_p), ("resume_ids", ctypes.c_void_p)]


# The call structures packed directly: a third of the time of filling the ctypes form.
GDN_TOKENS = struct.Struct("@i5P5qffP")
DRAFT_BATCH = struct.Struct("@4iPqqPqqPPPPqPPPP")
SSM_TOKENS = struct.Struct("@2i7P4q2iP")
CONV_TOKENS = struct.Struct("@PqiPPiP")
NORM_ARGS = struct.Struct("@10ifPqPqPPP")
assert GDN_TOKENS.size == ctypes.sizeof(GdnTokens) and DRAFT_BATCH.size == ctypes.sizeof(DraftBatch)
assert SSM_TOKENS.size == ctypes.sizeof(SsmTokens) and CONV_TOKENS.size == ctypes.sizeof(ConvTokens)
assert NORM_ARGS.size == ctypes.sizeof(NormArgs)

# name -> (restype, argtypes)
_P, _I32, _VP = ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p
_I32P = ctypes.POINTER(ctypes.c_int32)
_SIGS = {
    "wkv7_pool_required_bytes": (ctypes.c_size_t, [ctypes.POINTER(PoolDesc)]),
    "wkv7_pool_create": (ctypes.c_int, [ctypes.POINTER(PoolDesc), ctypes.POINTER(ctypes.c_void_p)]),
    "wkv7_pool_destroy": (ctypes.c_int, [_P]),
    "wkv7_pool_get_desc": (ctypes.c_int, [_P, ctypes.POINTER(PoolDesc)]),
    "wkv7_slot_bytes": (ctypes.c_size_t, [_P]),
    "wkv7_pool_state_ptr": (ctypes.c_int, [_P, _I32, _I32, ctypes.POINTER(ctypes.c_void_p)]),
    "wkv7_pool_snapshot_ptr": (ctypes.c_int, [_P, _I32, _I32, ctypes.POINTER(ctypes.c_void_p)]),
    "wkv7_slot_alloc": (ctypes.c_int, [_P, _I32, _I32P]),
    "wkv7_slot_free": (ctypes.c_int, [_P, _I32, _I32P]),
    "wkv7_snapshot_alloc": (ctypes.c_int, [_P, _I32, _I32P]),
    "wkv7_snapshot_free": (ctypes.c_int, [_P, _I32, _I32P]),
    "wkv7_slot_count_free": (ctypes.c_int32, [_P]),
    "wkv7_snapshot_count_free": (ctypes.c_int32, [_P]),
    "wkv7_slot_is_allocated": (ctypes.c_int, [_P, _I32, _I32P]),
    "wkv7_slot_create": (ctypes.c_int, [_P, _I32, _I32P, _VP]),
    "wkv7_slot_reset": (ctypes.c_int, [_P, _VP, _I32, _VP]),
    "wkv7_slot_snapshot": (ctypes.c_int, [_P, _VP, _VP, _I32, _VP]),
    "wkv7_slot_restore": (ctypes.c_int, [_P, _VP, _VP, _I32, _VP]),
    "wkv7_slot_fork": (ctypes.c_int, [_P, _VP, _VP, _I32, _VP]),
    "wkv7_slot_hibernate": (ctypes.c_int, [_P, _VP, _I32, _VP, ctypes.c_size_t, _VP]),
    "wkv7_slot_resume": (ctypes.c_int, [_P, _VP, ctypes.c_size_t, _VP, _I32, _VP]),
    "wkv7_decode_step": (ctypes.c_int, [_P, _I32, _VP, _I32, ctypes.c_int] + [_VP] * 7 + [_VP]),
    "wkv7_prefill": (ctypes.c_int, [_P, _I32, _VP, _VP, _I32, _I32, _I32, ctypes.c_int]
                     + [_VP] * 7 + [_VP]),
    "wkv7_prefill_sequential": (ctypes.c_int, [_P, _I32, _VP, _VP, _I32, _I32, _I32, ctypes.c_int]
                                + [_VP] * 7 + [_VP]),
    "wkv7_decode_multi": (ctypes.c_int, [_P, _I32, _VP, _I32, _I32, ctypes.c_int] + [_VP] * 7
                          + [_VP, _VP]),
    "wkv7_prefill_checkpointed": (ctypes.c_int, [_P, _I32, _VP, _VP, _I32, _I32, _I32, ctypes.c_int]
                                  + [_VP] * 7 + [_VP, _VP, _I32, _VP]),
    "wkv7_validate_ids": (ctypes.c_int, [_P, _I32, _VP, _I32, _VP, _I32, _VP]),
    "wkv7_validate_ids_noalloc": (ctypes.c_int, [_I32, _VP, _I32, _VP, _I32, _VP, _VP]),
    "wkv7_gdn_pool_required_bytes": (ctypes.c_size_t, [ctypes.POINTER(GdnPoolDesc)]),
    "wkv7_gdn_pool_create": (ctypes.c_int, [ctypes.POINTER(GdnPoolDesc), ctypes.POINTER(ctypes.c_void_p)]),
    "wkv7_gdn_pool_get_desc": (ctypes.c_int, [_P, ctypes.POINTER(GdnPoolDesc)]),
    "wkv7_gdn_decode_step": (ctypes.c_int, [_P, _I32, _VP, _I32, _VP, _VP]),
    "wkv7_gdn_decode_multi": (ctypes.c_int, [_P, _I32, _VP, _I32, _I32, _VP, _VP, _VP]),
    "wkv7_gdn_prefill": (ctypes.c_int, [_P, _I32, _VP, _VP, _I32, _I32, _I32, _VP,
                                        _VP, _VP, _VP, ctypes.c_size_t, _I32, _VP]),
    "wkv7_gdn_prefill_workspace_bytes": (ctypes.c_size_t, [_P, _I32, _I32]),
    "wkv7_pool_conv_desc": (ctypes.c_int, [_P, ctypes.POINTER(ConvDesc), ctypes.POINTER(ctypes.c_size_t)]),
    "wkv7_gdn_pool_conv_required_bytes": (ctypes.c_size_t, [ctypes.POINTER(GdnPoolDesc), ctypes.POINTER(ConvDesc)]),
    "wkv7_gdn_pool_create_conv": (ctypes.c_int, [ctypes.POINTER(GdnPoolDesc), ctypes.POINTER(ConvDesc),
                                                 ctypes.POINTER(ctypes.c_void_p)]),
    "wkv7_conv_step": (ctypes.c_int, [_P, _I32, _VP, _I32, _I32, _VP, _VP, _VP]),
    "wkv7_conv_prefill": (ctypes.c_int, [_P, _I32, _VP, _VP, _I32, _I32, _VP, _VP]),
    "wkv7_ssm_pool_required_bytes": (ctypes.c_size_t, [ctypes.POINTER(SsmPoolDesc)]),
    "wkv7_ssm_pool_create": (ctypes.c_int, [ctypes.POINTER(SsmPoolDesc), ctypes.POINTER(ctypes.c_void_p)]),
    "wkv7_ssm_pool_get_desc": (ctypes.c_int, [_P, ctypes.POINTER(SsmPoolDesc)]),
    "wkv7_ssm_decode_step": (ctypes.c_int, [_P, _I32, _VP, _I32, _VP, _VP]),
    "wkv7_ssm_decode_multi": (ctypes.c_int, [_P, _I32, _VP, _I32, _I32, _VP, _VP, _VP]),
    "wkv7_ssm_prefill": (ctypes.c_int, [_P, _I32, _VP, _VP, _I32, _I32, _I32, _VP, _VP, ctypes.c_size_t, _I32, _VP]),
    "wkv7_ssm_prefill_workspace_bytes": (ctypes.c_size_t, [_P, _I32, _I32]),
    "wkv7_gated_norm": (ctypes.c_int, [_VP, _VP]),
    "wkv7_verify_drafts": (ctypes.c_int, [_P, _VP, _VP]),
    "wkv7_get_device_status": (ctypes.c_int, [_P, _VP, _I32, _I32P]),
    "wkv7_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "wkv7_last_error": (ctypes.c_char_p, []),
    "wkv7_launch_count": (ctypes.c_uint64, []),
    "wkv7_version": (ctypes.c_int32, []),
    "wkv7_test_force_wait_timeout": (ctypes.c_int, [_I32]),
}

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libwkv7.so; raises if it has not been built.  There is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m rwkv_wkv_gb300.build` "
                          "(there is no fallback implementation)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def exported_symbols() -> list[str]:
    return list(_SIGS)


def _check(status: int, what: str):
    if status != 0:
        detail = ""
        if status == 6:
            detail = load_library().wkv7_last_error().decode(errors="replace")
        raise Wkv7Error(status, what, detail)


def launch_count() -> int:
    return int(load_library().wkv7_launch_count())


def _stream_handle(stream, device) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return int(stream.cuda_stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output tensor owned by the stream that will write it, so that its memory is not
    handed out again before that stream has passed the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def row_stride(name: str, st: tuple, lead: tuple, inner: tuple) -> int:
    """Elements between the rows of a tensor of strides st, whose own values must be contiguous;
    `lead` is its shape before a row's own `inner`."""
    if st[-1] != 1 and inner[-1] > 1 or len(inner) == 2 and st[-2] != inner[1] and inner[0] > 1:
        raise ValueError(f"{name}: a row's values must be contiguous")
    if len(lead) == 1:
        return st[0]
    if lead[1] == 1:
        return st[0]
    if lead[0] > 1 and st[0] != lead[1] * st[1]:
        raise ValueError(f"{name}: the rows of a batch must be one stride apart")
    return st[1]


def _ids_host(ids) -> ctypes.Array:
    vals = [int(x) for x in ids]
    return (ctypes.c_int32 * max(1, len(vals)))(*vals), len(vals)


def _dev_i32(t: torch.Tensor, name: str, device) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_cuda:
        raise TypeError(f"{name} must be an int32 CUDA tensor")
    if t.get_device() != device.index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous on {device}")
    return t.data_ptr()


class SlotPool:
    """What every pool of state slots has, whatever recurrence fills the slots: the slot
    table, the verbs, id validation, draft verification and the device status word.
    Subclasses create the library's pool (``_h``), its ``device`` and ``slot_bytes``, and
    add their recurrence."""

    def _adopt(self, prefix: str, desc, shape: tuple, n_slots: int, n_snapshots: int, state_dtype: str,
               conv=None) -> None:
        """Allocate the pool's buffer with torch, create the library's pool over it and
        expose its states and snapshots as tensors of per-slot shape `shape`.  `conv`, a
        ConvDesc, is passed on where the description does not hold it itself."""
        if self.device.index is None:  # "cuda": the current one
            self.device = torch.device(self.device.type, torch.cuda.current_device())
        self._index = self.device.index
        described = (ctypes.byref(desc),) if conv is None else (ctypes.byref(desc), ctypes.byref(conv))
        sized, made = ("_required_bytes", "_create") if conv is None else ("_conv_required_bytes", "_create_conv")
        nbytes = getattr(self._lib, prefix + sized)(*described)
        if nbytes == 0:
            raise Wkv7Error(1, type(self).__name__, "invalid description")
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.buffer[:_HEADER_BYTES].zero_()
        desc.device_buffer = self.buffer.data_ptr()
        desc.buffer_bytes = nbytes
        handle = ctypes.c_void_p()
        _check(getattr(self._lib, prefix + made)(*described, ctypes.byref(handle)), "pool_create")
        self._h = handle
        self.slot_bytes = int(self._lib.wkv7_slot_bytes(self._h))
        tdt = torch.bfloat16 if state_dtype == "bf16" else torch.float32
        slots = self.buffer[_HEADER_BYTES:_HEADER_BYTES + (n_slots + n_snapshots) * self.slot_bytes]
        slots = slots.view(n_slots + n_snapshots, self.slot_bytes)
        states = slots[:, :math.prod(shape) * tdt.itemsize].view(tdt).unflatten(1, shape)
        self.states, self.snapshots = states[:n_slots], states[n_slots:]
        got, at = ConvDesc(), ctypes.c_size_t()
        _check(self._lib.wkv7_pool_conv_desc(self._h, ctypes.byref(got), ctypes.byref(at)), "pool_conv_desc")
        self.conv_channels, self.conv_width = got.channels, got.width if got.channels else 0
        self.conv_tails = self.conv_snapshots = self._conv_torch_dtype = None
        if got.channels:
            cdt = self._conv_torch_dtype = torch.bfloat16 if got.dtype == BF16 else torch.float32
            inner = (shape[0], got.width - 1, got.channels)
            tails = slots[:, at.value:at.value + math.prod(inner) * cdt.itemsize].view(cdt).unflatten(1, inner)
            self.conv_tails, self.conv_snapshots = tails[:n_slots], tails[n_slots:]

    # -------------------------------------------------------------- lifetime
    def close(self):
        if getattr(self, "_h", None):
            _check(self._lib.wkv7_pool_destroy(self._h), "pool_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    # ------------------------------------------------------------ slot table
    def alloc(self, n: int) -> list[int]:
        arr = (ctypes.c_int32 * max(1, n))()
        _check(self._lib.wkv7_slot_alloc(self._h, n, arr), "slot_alloc")
        return list(arr[:n])

    def free(self, ids) -> None:
        arr, n = _ids_host(ids)
        _check(self._lib.wkv7_slot_free(self._h, n, arr), "slot_free")

    def snapshot_alloc(self, n: int) -> list[int]:
        arr = (ctypes.c_int32 * max(1, n))()
        _check(self._lib.wkv7_snapshot_alloc(self._h, n, arr), "snapshot_alloc")
        return list(arr[:n])

    def snapshot_free(self, ids) -> None:
        arr, n = _ids_host(ids)
        _check(self._lib.wkv7_snapshot_free(self._h, n, arr), "snapshot_free")

    def n_free(self) -> int:
        return int(self._lib.wkv7_slot_count_free(self._h))

    def n_snapshots_free(self) -> int:
        return int(self._lib.wkv7_snapshot_count_free(self._h))

    def is_allocated(self, slot: int) -> bool:
        out = ctypes.c_int32()
        _check(self._lib.wkv7_slot_is_allocated(self._h, slot, ctypes.byref(out)), "is_allocated")
        return bool(out.value)

    def state_ptr(self, slot: int, layer: int) -> int:
        p = ctypes.c_void_p()
        _check(self._lib.wkv7_pool_state_ptr(self._h, slot, layer, ctypes.byref(p)), "state_ptr")
        return int(p.value)

    # ----------------------------------------------------------------- verbs
    def create(self, n: int, stream=None) -> list[int]:
        arr = (ctypes.c_int32 * max(1, n))()
        _check(self._lib.wkv7_slot_create(self._h, n, arr, _stream_handle(stream, self.device)),
               "slot_create")
        return list(arr[:n])

    def reset(self, slot_ids: torch.Tensor, stream=None) -> None:
        _check(self._lib.wkv7_slot_reset(self._h, _dev_i32(slot_ids, "slot_ids", self.device),
                                         slot_ids.numel(), _stream_handle(stream, self.device)),
               "slot_reset")

    def snapshot(self, slot_ids: torch.Tensor, snap_ids: torch.Tensor, stream=None) -> None:
        self._pairs("wkv7_slot_snapshot", slot_ids, snap_ids, stream)

    def restore(self, snap_ids: torch.Tensor, slot_ids: torch.Tensor, stream=None) -> None:
        self._pairs("wkv7_slot_restore", snap_ids, slot_ids, stream)

    def fork(self, src_ids: torch.Tensor, dst_ids: torch.Tensor, stream=None) -> None:
        self._pairs("wkv7_slot_fork", src_ids, dst_ids, stream)

    def _host_buffer(self, host: torch.Tensor, n: int) -> tuple[int, int]:
        if not isinstance(host, torch.Tensor) or host.is_cuda or not host.is_contiguous():
            raise TypeError("host buffer must be a contiguous CPU tensor (pinned memory)")
        nbytes = host.numel() * host.element_size()
        if nbytes < n * self.slot_bytes:
            raise ValueError(f"host buffer holds {nbytes} bytes, {n} slots need {n * self.slot_bytes}")
        return host.data_ptr(), nbytes

    def hibernate(self, slot_ids: torch.Tensor, host: torch.Tensor, stream=None) -> None:
        """Copy the slots slot_ids[i] into pinned host memory `host`, packed slot after slot
        (asynchronous on the stream; see wkv7_slot_hibernate)."""
        n = slot_ids.numel()
        ptr, nbytes = self._host_buffer(host, n)
        _check(self._lib.wkv7_slot_hibernate(self._h, _dev_i32(slot_ids, "slot_ids", self.device), n,
                                             ptr, nbytes, _stream_handle(stream, self.device)),
               "slot_hibernate")

    def resume(self, host: torch.Tensor, slot_ids: torch.Tensor, stream=None) -> None:
        """Copy packed slot images from pinned host memory `host` into the slots slot_ids[i]."""
        n = slot_ids.numel()
        ptr, nbytes = self._host_buffer(host, n)
        _check(self._lib.wkv7_slot_resume(self._h, ptr, nbytes,
                                          _dev_i32(slot_ids, "slot_ids", self.device), n,
                                          _stream_handle(stream, self.device)), "slot_resume")

    def _pairs(self, fn, first, second, stream):
        if first.numel() != second.numel():
            raise ValueError("id arrays differ in length")
        _check(getattr(self._lib, fn)(self._h, _dev_i32(first, "ids", self.device),
                                      _dev_i32(second, "ids", self.device), first.numel(),
                                      _stream_handle(stream, self.device)), fn)

    # ------------------------------------------------------------ validation
    def validate_ids(self, ids_a: torch.Tensor, ids_b: torch.Tensor | None = None,
                     table: str = "slots", stream=None) -> None:
        """Debug pass (wkv7_validate_ids): every id of ids_a and ids_b (device int32)
        in the table and none twice; the verdict lands in the device status word
        (DEV_DUP_SLOT, DEV_BAD_SLOT), read with device_status()."""
        if table not in ("slots", "snapshots"):
            raise ValueError("table must be 'slots' or 'snapshots'")
        nb = 0 if ids_b is None else ids_b.numel()
        pb = _dev_i32(ids_b, "ids_b", self.device) if nb else None
        na = ids_a.numel()
        pa = _dev_i32(ids_a, "ids_a", self.device) if na else None
        _check(self._lib.wkv7_validate_ids(self._h, TABLE_SLOTS if table == "slots" else TABLE_SNAPSHOTS,
                                           pa, na, pb, nb, _stream_handle(stream, self.device)),
               "validate_ids")

    # ---------------------------------------------------------------- status
    def device_status(self, stream=None, timeout_ms: int = 10000) -> int:
        """Read and clear the device status word (a DEV_* code; 0 when clean)."""
        code = ctypes.c_int32()
        st = self._lib.wkv7_get_device_status(self._h, _stream_handle(stream, self.device),
                                              timeout_ms, ctypes.byref(code))
        if st not in (0, 3, 8):  # OK, ERR_DUP_SLOT and ERR_DEVICE_STATUS carry the code
            _check(st, "get_device_status")
        return int(code.value)

    # ----------------------------------------------------- short convolution
    def _conv(self, lead: tuple, x, weight, bias, activation, o, stream):
        """One convolution's tokens as the library takes them; `lead` is the shape before the
        channels ((rows,) or (n, K), whose rows must be one stride apart)."""
        dt, ch = self._conv_torch_dtype, self.conv_channels
        if dt is None:
            raise ValueError("the pool was made without conv_channels")
        if x.dtype is not dt:
            raise TypeError(f"x must be {dt}, as the pool's tails are")
        wdt = weight.dtype
        if wdt is torch.bfloat16:
            code = BF16
        elif wdt is torch.float32:
            code = F32
        else:
            raise TypeError("weight must be float32 or bfloat16")
        if bias is not None and bias.dtype is not wdt:
            raise TypeError("bias must have weight's type")
        at = self._index
        if not (x.get_device() == weight.get_device() == at and (bias is None or bias.get_device() == at)):
            raise TypeError(f"x, weight and bias must be on {self.device}")
        shape = lead + (ch,)
        if x.shape != shape or weight.shape not in ((ch, self.conv_width), (ch, 1, self.conv_width)) or \
                bias is not None and bias.shape != (ch,):
            raise ValueError(f"x must be {list(shape)}, weight [{ch}, {self.conv_width}] (or [{ch}, 1, {self.conv_width}]) "
                             f"and bias [{ch}]")
        if not weight.is_contiguous() or bias is not None and not bias.is_contiguous():
            raise ValueError("weight and bias must be contiguous")
        if activation not in ("silu", None):
            raise ValueError("activation must be 'silu' or None")
        stride = row_stride("x", x.stride(), lead, (ch,))
        if o is None:
            o = _empty(shape, dt, self.device, stream)
        elif o.dtype is not dt or o.get_device() != at or not o.is_contiguous() or o.shape != shape:
            raise ValueError(f"o must be a contiguous {dt} {list(shape)} tensor")
        return CONV_TOKENS.pack(x.data_ptr(), stride, code, weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
                                1 if activation else 0, o.data_ptr()), o

    def conv_step(self, layer: int, slot_ids: torch.Tensor, x, weight, bias=None, activation="silu", o=None,
                  stream=None) -> torch.Tensor:
        """The short causal convolution (wkv7_conv_step) for one token of each slot: x and o
        [n, conv_channels] in the pool's conv_dtype, weight [conv_channels, conv_width] (or
        [conv_channels, 1, conv_width]) and bias float32 or bfloat16, activation 'silu' or None.
        x may be a column range of a projection.  The slots' tails move on by a token."""
        n = slot_ids.numel()
        t, o = self._conv((n,), x, weight, bias, activation, o, stream)
        _check(self._lib.wkv7_conv_step(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device), n, 1, t, None,
                                        _stream_handle(stream, self.device)), "conv_step")
        return o

    def conv_multi(self, layer: int, slot_ids: torch.Tensor, x, weight, bias=None, activation="silu", o=None,
                   step_snap_ids: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """K consecutive tokens for each slot: x and o [n, K, conv_channels]; with step_snap_ids
        ([n, K] int32) the tail after every token also goes to those snapshots (this layer)."""
        n, K = slot_ids.numel(), int(x.shape[1])
        t, o = self._conv((n, K), x, weight, bias, activation, o, stream)
        snaps = None
        if step_snap_ids is not None:
            if step_snap_ids.numel() != n * K:
                raise ValueError("step_snap_ids must hold n * K ids")
            snaps = _dev_i32(step_snap_ids, "step_snap_ids", self.device)
        _check(self._lib.wkv7_conv_step(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device), n, K, t, snaps,
                                        _stream_handle(stream, self.device)), "conv_multi")
        return o

    def conv_prefill(self, layer: int, slot_ids: torch.Tensor, cu_seqlens: torch.Tensor, x, weight, bias=None,
                     activation="silu", o=None, stream=None) -> torch.Tensor:
        """Sequences packed back to back, each continuing its slot's tail: x and o [tokens,
        conv_channels].  Rows behind the last sequence are left as they were."""
        total = int(x.shape[0])
        t, o = self._conv((total,), x, weight, bias, activation, o, stream)
        if cu_seqlens.numel() != slot_ids.numel() + 1:
            raise ValueError("cu_seqlens must have n_seqs + 1 entries")
        _check(self._lib.wkv7_conv_prefill(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device),
                                           _dev_i32(cu_seqlens, "cu_seqlens", self.device), slot_ids.numel(), total, t,
                                           _stream_handle(stream, self.device)), "conv_prefill")
        return o

    # ---------------------------------------------------- draft verification
    def verify_drafts(self, draft_ids: torch.Tensor, target_probs: torch.Tensor,
                      draft_probs: torch.Tensor | None, uniforms: torch.Tensor, noise: torch.Tensor,
                      n_draft: torch.Tensor | None = None, step_snap_ids: torch.Tensor | None = None,
                      stream=None):
        """Accept or refuse drafted tokens (wkv7_verify_drafts).  draft_ids [n, K] int32;
        target_probs [n, K+1, vocab] and draft_probs [n, K, vocab] (or None) float32 or
        bfloat16, their rows contiguous and otherwise of any stride; uniforms [n, K] and
        noise [n, vocab] (exponential deviates) float32; n_draft [n] int32 for rows with
        fewer drafts; step_snap_ids [n, K+1] int32, the snapshots of decode_multi over
        [last token, drafts].  Returns (accepted [n], tokens [n, K+1], resume_ids [n] or
        None): tokens holds the accepted drafts, the next token, then -1; resume_ids the
        snapshot to restore."""
        n, K = draft_ids.shape
        dt, at = target_probs.dtype, self._index
        if dt is torch.float32:
            code = F32
        elif dt is torch.bfloat16:
            code = BF16
        else:
            raise TypeError("target_probs must be float32 or bfloat16")
        if not (noise.dtype is uniforms.dtype is torch.float32 and (draft_probs is None or draft_probs.dtype is dt)):
            raise TypeError("draft_probs must have target_probs' type, uniforms and noise must be float32")
        if not (target_probs.get_device() == noise.get_device() == uniforms.get_device() == at
                and (draft_probs is None or draft_probs.get_device() == at)):
            raise TypeError(f"every input must be on {self.device}")
        vocab = target_probs.shape[-1]
        if target_probs.shape != (n, K + 1, vocab) or noise.shape != (n, vocab) or uniforms.shape != (n, K) or \
                draft_probs is not None and draft_probs.shape != (n, K, vocab):
            raise ValueError(f"target_probs must be [{n}, {K + 1}, vocab], draft_probs [{n}, {K}, vocab], uniforms "
                             f"[{n}, {K}] and noise [{n}, vocab]")
        ps, ns = target_probs.stride(), noise.stride()
        qs, qp = (0, 0, 1), 0
        if draft_probs is not None:
            qs, qp = draft_probs.stride(), draft_probs.data_ptr()
        if vocab > 1 and not (ps[2] == ns[1] == qs[2] == 1) or not uniforms.is_contiguous():
            raise ValueError("rows of probabilities and noise must be contiguous, and uniforms")
        if n_draft is not None and n_draft.numel() != n:
            raise ValueError("n_draft must hold n counts")
        counts = 0 if n_draft is None else _dev_i32(n_draft, "n_draft", self.device)
        accepted = _empty((n,), torch.int32, self.device, stream)
        tokens = _empty((n, K + 1), torch.int32, self.device, stream)
        resume, snaps, to = None, 0, 0
        if step_snap_ids is not None:
            if step_snap_ids.numel() != n * (K + 1):
                raise ValueError("step_snap_ids must hold n * (K + 1) ids")
            snaps = _dev_i32(step_snap_ids, "step_snap_ids", self.device)
            resume = _empty((n,), torch.int32, self.device, stream)
            to = resume.data_ptr()
        d = DRAFT_BATCH.pack(n, K, vocab, code, target_probs.data_ptr(), ps[0], ps[1], qp, qs[0], qs[1],
                             _dev_i32(draft_ids, "draft_ids", self.device), counts, uniforms.data_ptr(),
                             noise.data_ptr(), ns[0], snaps, accepted.data_ptr(), tokens.data_ptr(), to)
        _check(self._lib.wkv7_verify_drafts(self._h, d, _stream_handle(stream, self.device)),
               "verify_drafts")
        return accepted, tokens, resume


class Pool(SlotPool):
    """A pool of fixed-size WKV-7 state slots on one GPU.

    States live in one torch-allocated device buffer: ``states`` is a float32
    (or, with state_dtype="bf16", bfloat16) view [n_slots, n_layers, n_heads,
    64, 64] and ``snapshots`` the same for the parked copies (S[i][j]: i =
    value row, j = key column).  Outputs o are float32, or bfloat16 with
    out_dtype="bf16" (the float32 readout rounded to nearest even).
    """

    def __init__(self, n_layers: int, n_heads: int, n_slots: int, n_snapshots: int = 0,
                 head_size: int = HEAD_SIZE, device=None, state_dtype: str = "f32",
                 out_dtype: str = "f32"):
        self._lib = load_library()
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.n_layers, self.n_heads, self.head_size = n_layers, n_heads, head_size
        self.n_slots, self.n_snapshots = n_slots, n_snapshots
        if state_dtype not in ("f32", "bf16"):
            raise ValueError("state_dtype must be 'f32' or 'bf16'")
        if out_dtype not in ("f32", "bf16"):
            raise ValueError("out_dtype must be 'f32' or 'bf16'")
        self.state_dtype, self.out_dtype = state_dtype, out_dtype
        self.o_torch_dtype = torch.bfloat16 if out_dtype == "bf16" else torch.float32
        desc = PoolDesc(n_layers, n_heads, head_size, n_slots, n_snapshots, None, 0,
                        BF16 if state_dtype == "bf16" else F32, BF16 if out_dtype == "bf16" else F32)
        self._adopt("wkv7_pool", desc, (n_layers, n_heads, head_size, head_size), n_slots, n_snapshots,
                    state_dtype)

    # ------------------------------------------------------------ recurrence
    def _inputs(self, xs, rows):
        dt = xs[0].dtype
        if dt not in (torch.float32, torch.bfloat16):
            raise TypeError("inputs must be float32 or bfloat16")
        for x in xs:
            if x.dtype != dt or x.device != self.device or not x.is_contiguous():
                raise ValueError("inputs must share one dtype and be contiguous on the pool device")
            if tuple(x.shape) != (rows, self.n_heads, self.head_size):
                raise ValueError(f"inputs must be [{rows}, {self.n_heads}, {self.head_size}]")
        return (BF16 if dt == torch.bfloat16 else F32), [x.data_ptr() for x in xs]

    def _out(self, o, rows):
        if o is None:
            return torch.empty(rows, self.n_heads, self.head_size, dtype=self.o_torch_dtype,
                               device=self.device)
        if (o.dtype != self.o_torch_dtype or o.device != self.device or not o.is_contiguous()
                or tuple(o.shape) != (rows, self.n_heads, self.head_size)):
            raise ValueError(f"o must be a contiguous {self.o_torch_dtype} [rows, n_heads, 64] tensor")
        return o

    def decode_step(self, layer: int, slot_ids: torch.Tensor, r, w, k, v, a, b, o=None,
                    stream=None) -> torch.Tensor:
        n = slot_ids.numel()
        dt, ptrs = self._inputs((r, w, k, v, a, b), n)
        o = self._out(o, n)
        _check(self._lib.wkv7_decode_step(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device),
                                          n, dt, *ptrs, o.data_ptr(),
                                          _stream_handle(stream, self.device)), "decode_step")
        return o

    def decode_multi(self, layer: int, slot_ids: torch.Tensor, r, w, k, v, a, b, o=None,
                     step_snap_ids: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """K consecutive tokens per slot: inputs [n, K, n_heads, 64] (one dtype), o the
        same shape in the pool's output dtype; with step_snap_ids ([n, K] device int32) the state after
        every token also goes to those snapshot ids (this layer)."""
        n = slot_ids.numel()
        if r.dim() != 4 or r.shape[0] != n:
            raise ValueError("decode_multi inputs must be [n, K, n_heads, 64]")
        K = int(r.shape[1])
        dt, ptrs = self._inputs(tuple(x.reshape(n * K, *x.shape[2:]) if x.dim() == 4 and
                                      tuple(x.shape[:2]) == (n, K) else x
                                      for x in (r, w, k, v, a, b)), n * K)
        if o is None:
            o = torch.empty(n, K, self.n_heads, self.head_size, dtype=self.o_torch_dtype,
                            device=self.device)
        self._out(o.reshape(n * K, *o.shape[2:]) if o.dim() == 4 else o, n * K)
        snaps = None
        if step_snap_ids is not None:
            if step_snap_ids.numel() != n * K:
                raise ValueError("step_snap_ids must hold n * K ids")
            snaps = _dev_i32(step_snap_ids, "step_snap_ids", self.device)
        _check(self._lib.wkv7_decode_multi(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device),
                                           n, K, dt, *ptrs, o.data_ptr(), snaps,
                                           _stream_handle(stream, self.device)), "decode_multi")
        return o

    def prefill(self, layer: int, slot_ids: torch.Tensor, cu_seqlens: torch.Tensor, r, w, k, v,
                a, b, o=None, max_seqlen: int | None = None, stream=None,
                sequential: bool = False, cu_ckpt: torch.Tensor | None = None,
                ckpt_ids: torch.Tensor | None = None) -> torch.Tensor:
        """Prefill; with cu_ckpt / ckpt_ids (device int32), also the state at every
        64-token boundary of each sequence into those snapshot ids (this layer)."""
        total = r.shape[0]
        dt, ptrs = self._inputs((r, w, k, v, a, b), total)
        o = self._out(o, total)
        if cu_seqlens.numel() != slot_ids.numel() + 1:
            raise ValueError("cu_seqlens must have n_seqs + 1 entries")
        if (cu_ckpt is None) != (ckpt_ids is None):
            raise ValueError("cu_ckpt and ckpt_ids go together")
        if cu_ckpt is not None:
            if cu_ckpt.numel() != slot_ids.numel() + 1:
                raise ValueError("cu_ckpt must have n_seqs + 1 entries")
            ids_ptr = _dev_i32(ckpt_ids, "ckpt_ids", self.device) if ckpt_ids.numel() else None
            if ids_ptr is None:  # no boundary anywhere: any non-null pointer will do
                ids_ptr = _dev_i32(cu_ckpt, "cu_ckpt", self.device)
            _check(self._lib.wkv7_prefill_checkpointed(
                self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device),
                _dev_i32(cu_seqlens, "cu_seqlens", self.device), slot_ids.numel(), total,
                total if max_seqlen is None else int(max_seqlen), dt, *ptrs, o.data_ptr(),
                _dev_i32(cu_ckpt, "cu_ckpt", self.device), ids_ptr, int(bool(sequential)),
                _stream_handle(stream, self.device)), "prefill_checkpointed")
            return o
        fn = self._lib.wkv7_prefill_sequential if sequential else self._lib.wkv7_prefill
        _check(fn(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device),
                  _dev_i32(cu_seqlens, "cu_seqlens", self.device), slot_ids.numel(), total,
                  total if max_seqlen is None else int(max_seqlen), dt, *ptrs, o.data_ptr(),
                  _stream_handle(stream, self.device)),
               "prefill_sequential" if sequential else "prefill")
        return o
