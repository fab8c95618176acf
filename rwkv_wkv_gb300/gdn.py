"""Python binding of the gated delta rule over state slots (the wkv7_gdn_* calls of
include/wkv7.h): argument marshalling only."""
from __future__ import annotations

import torch

from .wkv7 import (BF16, F32, GDN_TOKENS, GdnPoolDesc, SlotPool, _check, _dev_i32, _empty, _stream_handle, load_library)


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
        self._k_inner, self._v_inner, self._g_inner = (n_k_heads, head_k), (n_v_heads, head_v), (n_v_heads,)
        self._k_tight, self._v_tight = (head_k, 1), (head_v, 1)
        self._scale = float(head_k) ** -0.5
        self._adopt("wkv7_gdn_pool", desc, (n_layers, n_v_heads, head_v, head_k), n_slots, n_snapshots, state_dtype)

    def _tokens(self, lead: tuple, q, k, v, g, beta, o, scale, l2norm_eps, stream):
        """The call's tokens as the library takes them; `lead` is the shape before the heads
        ((rows,) or (n, K), whose rows must be one stride apart)."""
        dt = q.dtype
        if dt is torch.bfloat16:
            code = BF16
        elif dt is torch.float32:
            code = F32
        else:
            raise TypeError("q, k and v must be float32 or bfloat16")
        if not (k.dtype is dt and v.dtype is dt and g.dtype is torch.float32 and beta.dtype is torch.float32):
            raise TypeError("q, k and v must share one type, g and beta must be float32")
        at = self._index
        if not (q.get_device() == k.get_device() == v.get_device() == g.get_device() == beta.get_device() == at):
            raise TypeError(f"q, k, v, g and beta must be on {self.device}")
        kshape, vshape, gshape = lead + self._k_inner, lead + self._v_inner, lead + self._g_inner
        if not (q.shape == kshape and k.shape == kshape and v.shape == vshape and g.shape == gshape
                and beta.shape == gshape):
            raise ValueError(f"q and k must be {list(kshape)}, v {list(vshape)}, g and beta {list(gshape)}")
        qs, ks, vs, gs, bs = q.stride(), k.stride(), v.stride(), g.stride(), beta.stride()
        if len(lead) == 1 and qs[1:] == self._k_tight == ks[1:] and vs[1:] == self._v_tight and gs[1] == bs[1] == 1:
            qs, ks, vs, gs, bs = qs[0], ks[0], vs[0], gs[0], bs[0]
        else:  # axes of length 1, or two leading ones
            qs, ks = self._row_stride("q", qs, lead, self._k_inner), self._row_stride("k", ks, lead, self._k_inner)
            vs = self._row_stride("v", vs, lead, self._v_inner)
            gs, bs = self._row_stride("g", gs, lead, self._g_inner), self._row_stride("beta", bs, lead, self._g_inner)
        if o is None:
            o = _empty(vshape, self.o_torch_dtype, self.device, stream)
        elif o.dtype is not self.o_torch_dtype or o.get_device() != at or not o.is_contiguous() or o.shape != vshape:
            raise ValueError(f"o must be a contiguous {self.o_torch_dtype} {list(vshape)} tensor")
        return GDN_TOKENS.pack(code, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), qs, ks, vs,
                               gs, bs, self._scale if scale is None else scale,
                               0.0 if l2norm_eps is None else l2norm_eps, o.data_ptr()), o

    @staticmethod
    def _row_stride(name: str, st: tuple, lead: tuple, inner: tuple) -> int:
        """Elements between the rows of a tensor of strides st, whose own values must be contiguous."""
        if st[-1] != 1 and inner[-1] > 1 or len(inner) == 2 and st[-2] != inner[1] and inner[0] > 1:
            raise ValueError(f"{name}: a row's values must be contiguous")
        if len(lead) == 1:
            return st[0]
        if lead[1] == 1:
            return st[0]
        if lead[0] > 1 and st[0] != lead[1] * st[1]:
            raise ValueError(f"{name}: the rows of a batch must be one stride apart")
        return st[1]

    def decode_step(self, layer: int, slot_ids: torch.Tensor, q, k, v, g, beta, o=None, scale=None,
                    l2norm_eps=None, stream=None) -> torch.Tensor:
        """One token for each slot; o [n, n_v_heads, head_v]."""
        n = slot_ids.numel()
        t, o = self._tokens((n,), q, k, v, g, beta, o, scale, l2norm_eps, stream)
        _check(self._lib.wkv7_gdn_decode_step(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device), n,
                                              t, _stream_handle(stream, self.device)),
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
                                               t, snaps, _stream_handle(stream, self.device)),
               "gdn_decode_multi")
        return o

    def prefill(self, layer: int, slot_ids: torch.Tensor, cu_seqlens: torch.Tensor, q, k, v, g, beta, o=None,
                max_seqlen: int | None = None, scale=None, l2norm_eps=None, stream=None,
                sequential: bool = False, cu_ckpt: torch.Tensor | None = None,
                ckpt_ids: torch.Tensor | None = None) -> torch.Tensor:
        """Sequences packed back to back, each continuing its slot's state; o [tokens, n_v_heads,
        head_v].  max_seqlen, the longest length, shapes the work: without it the total is taken
        for it, and several sequences may run slower.  In chunks (sequential=False, bfloat16 inputs)
        products take operands of 16 bits, errors about 3e-6 of the largest entry; sequential=True
        is float32 throughout and slower.  With cu_ckpt / ckpt_ids (int32) also the state at every 64-token boundary of
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
        n = slot_ids.numel()
        longest = total if max_seqlen is None else int(max_seqlen)
        need = 0 if sequential else self._lib.wkv7_gdn_prefill_workspace_bytes(self._h, n, longest)
        ws = _empty((need,), torch.uint8, self.device, stream) if need else None
        _check(self._lib.wkv7_gdn_prefill(
            self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device),
            _dev_i32(cu_seqlens, "cu_seqlens", self.device), n, total, longest, t, pc, pi,
            None if ws is None else ws.data_ptr(), need, int(bool(sequential)),
            _stream_handle(stream, self.device)), "gdn_prefill")
        return o
