"""Python binding of the gated delta rule over state slots (the wkv7_gdn_* calls of
include/wkv7.h): argument marshalling only."""
from __future__ import annotations

import ctypes

import torch

from .wkv7 import (BF16, F32, GdnPoolDesc, GdnTokens, SlotPool, _check, _dev_i32, _empty, _stream_handle, load_library)


class GdnPool(SlotPool):
    """A pool of state slots for gated-delta-rule layers on one GPU.

    Per value head a state S [head_v, head_k]; a token does S <- exp(g) S,
    e = beta (v - S k), S <- S + e k^T, o = scale S q.  Value head h reads query/key head
    h // (n_v_heads // n_k_heads).  ``states`` is a float32 (or bfloat16) view
    [n_slots, n_layers, n_v_heads, head_v, head_k], ``snapshots`` the same for the parked
    copies; the slot table, the verbs and verify_drafts are SlotPool's.

    Every call takes q, k [rows, n_k_heads, head_k] and v [rows, n_v_heads, head_v]
    (float32 or bfloat16) and g (log decay, <= 0) and beta [rows, n_v_heads] (float32).
    A row's values are contiguous; rows may be any stride apart (q, k and v may be column
    ranges of one projection), for q, k and v a multiple of 16 bytes.  ``scale`` defaults
    to head_k ** -0.5; with ``l2norm_eps`` q and k are first divided by
    sqrt(sum x^2 + l2norm_eps) per head.
    """

    def __init__(self, n_layers: int, n_k_heads: int, n_v_heads: int, n_slots: int, n_snapshots: int = 0,
                 head_k: int = 128, head_v: int = 128, device=None, state_dtype: str = "f32",
                 out_dtype: str = "f32"):
        self._lib = load_library()
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.n_layers, self.n_k_heads, self.n_v_heads = n_layers, n_k_heads, n_v_heads
        self.head_k, self.head_v = head_k, head_v
        self.n_slots, self.n_snapshots = n_slots, n_snapshots
        for name, x in (("state_dtype", state_dtype), ("out_dtype", out_dtype)):
            if x not in ("f32", "bf16"):
                raise ValueError(f"{name} must be 'f32' or 'bf16'")
        self.state_dtype, self.out_dtype = state_dtype, out_dtype
        self.o_torch_dtype = torch.bfloat16 if out_dtype == "bf16" else torch.float32
        desc = GdnPoolDesc(n_layers, n_k_heads, n_v_heads, head_k, head_v, n_slots, n_snapshots, None, 0,
                           BF16 if state_dtype == "bf16" else F32, BF16 if out_dtype == "bf16" else F32)
        self._adopt("wkv7_gdn_pool", desc, (n_layers, n_v_heads, head_v, head_k), n_slots, n_snapshots, state_dtype)

    def _tokens(self, lead: tuple, q, k, v, g, beta, o, scale, l2norm_eps, stream):
        """The call's tokens as the library takes them; `lead` is the shape before the heads
        ((rows,) or (n, K), whose rows must be one stride apart)."""
        t = GdnTokens()
        if q.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("q, k and v must be float32 or bfloat16")
        t.in_dtype = BF16 if q.dtype == torch.bfloat16 else F32
        for name, x, dtype, inner in (("q", q, q.dtype, (self.n_k_heads, self.head_k)),
                                      ("k", k, q.dtype, (self.n_k_heads, self.head_k)),
                                      ("v", v, q.dtype, (self.n_v_heads, self.head_v)),
                                      ("g", g, torch.float32, (self.n_v_heads,)),
                                      ("beta", beta, torch.float32, (self.n_v_heads,))):
            if x.dtype != dtype or x.device != self.device:
                raise TypeError(f"{name} must be {dtype} on {self.device}")
            if tuple(x.shape) != (*lead, *inner):
                raise ValueError(f"{name} must be {[*lead, *inner]}")
            st = x.stride()
            tight = 1
            for size, s in zip(reversed(inner), reversed(st[len(lead):])):
                if size > 1 and s != tight:
                    raise ValueError(f"{name}: a row's heads must be contiguous")
                tight *= size
            row = st[len(lead) - 1]
            if len(lead) == 2:
                if lead[1] == 1:
                    row = st[0]
                elif lead[0] > 1 and st[0] != lead[1] * row:
                    raise ValueError(f"{name}: the rows of a batch must be one stride apart")
            setattr(t, name, x.data_ptr())
            setattr(t, name + "_stride", row)
        shape = (*lead, self.n_v_heads, self.head_v)
        if o is None:
            o = _empty(shape, self.o_torch_dtype, self.device, stream)
        elif o.dtype != self.o_torch_dtype or o.device != self.device or not o.is_contiguous() or \
                tuple(o.shape) != shape:
            raise ValueError(f"o must be a contiguous {self.o_torch_dtype} {list(shape)} tensor")
        t.o = o.data_ptr()
        t.scale = self.head_k ** -0.5 if scale is None else scale
        t.l2norm_eps = 0.0 if l2norm_eps is None else l2norm_eps
        return t, o

    def decode_step(self, layer: int, slot_ids: torch.Tensor, q, k, v, g, beta, o=None, scale=None,
                    l2norm_eps=None, stream=None) -> torch.Tensor:
        """One token for each slot; o [n, n_v_heads, head_v]."""
        n = slot_ids.numel()
        t, o = self._tokens((n,), q, k, v, g, beta, o, scale, l2norm_eps, stream)
        _check(self._lib.wkv7_gdn_decode_step(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device), n,
                                              ctypes.byref(t), _stream_handle(stream, self.device)),
               "gdn_decode_step")
        return o

    def decode_multi(self, layer: int, slot_ids: torch.Tensor, q, k, v, g, beta, o=None,
                     step_snap_ids: torch.Tensor | None = None, scale=None, l2norm_eps=None,
                     stream=None) -> torch.Tensor:
        """K consecutive tokens for each slot: inputs [n, K, ...], o [n, K, n_v_heads, head_v];
        with step_snap_ids ([n, K] int32) the state after every token also goes to those
        snapshots (this layer)."""
        n, K = slot_ids.numel(), int(q.shape[1])
        t, o = self._tokens((n, K), q, k, v, g, beta, o, scale, l2norm_eps, stream)
        snaps = None
        if step_snap_ids is not None:
            if step_snap_ids.numel() != n * K:
                raise ValueError("step_snap_ids must hold n * K ids")
            snaps = _dev_i32(step_snap_ids, "step_snap_ids", self.device)
        _check(self._lib.wkv7_gdn_decode_multi(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device), n, K,
                                               ctypes.byref(t), snaps, _stream_handle(stream, self.device)),
               "gdn_decode_multi")
        return o

    def prefill(self, layer: int, slot_ids: torch.Tensor, cu_seqlens: torch.Tensor, q, k, v, g, beta, o=None,
                max_seqlen: int | None = None, scale=None, l2norm_eps=None, stream=None,
                sequential: bool = False, cu_ckpt: torch.Tensor | None = None,
                ckpt_ids: torch.Tensor | None = None) -> torch.Tensor:
        """Sequences packed back to back, each continuing its slot's state; o [tokens, n_v_heads,
        head_v].  With cu_ckpt / ckpt_ids (int32) also the state at every 64-token boundary of
        each sequence into those snapshots (this layer)."""
        total = int(q.shape[0])
        t, o = self._tokens((total,), q, k, v, g, beta, o, scale, l2norm_eps, stream)
        if cu_seqlens.numel() != slot_ids.numel() + 1:
            raise ValueError("cu_seqlens must have n_seqs + 1 entries")
        if (cu_ckpt is None) != (ckpt_ids is None):
            raise ValueError("cu_ckpt and ckpt_ids go together")
        pc = pi = None
        if cu_ckpt is not None:
            if cu_ckpt.numel() != slot_ids.numel() + 1:
                raise ValueError("cu_ckpt must have n_seqs + 1 entries")
            pc = _dev_i32(cu_ckpt, "cu_ckpt", self.device)
            pi = _dev_i32(ckpt_ids, "ckpt_ids", self.device) if ckpt_ids.numel() else pc  # no boundary anywhere
        _check(self._lib.wkv7_gdn_prefill(
            self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device),
            _dev_i32(cu_seqlens, "cu_seqlens", self.device), slot_ids.numel(), total,
            total if max_seqlen is None else int(max_seqlen), ctypes.byref(t), pc, pi, int(bool(sequential)),
            _stream_handle(stream, self.device)), "gdn_prefill")
        return o
