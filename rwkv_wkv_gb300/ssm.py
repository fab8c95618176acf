"""Python binding of the selective scan over state slots (the wkv7_ssm_* calls of
include/wkv7.h): argument marshalling only."""
from __future__ import annotations

import torch

from .norm import gated_norm
from .wkv7 import (BF16, F32, SSM_TOKENS, ConvDesc, SlotPool, SsmPoolDesc, _check, _dev_i32, _empty, _stream_handle,
                   load_library, row_stride)


class SsmPool(SlotPool):
    """A pool of state slots for state space layers on one GPU.

    Per head a state S [head_p, d_state]; a token does S <- exp(dt A) S + (dt x) B^T,
    o = S C + D x.  Head h reads B and C of group h // (n_heads // n_groups).  ``states`` is
    a float32 (or bfloat16) view [n_slots, n_layers, n_heads, head_p, d_state], ``snapshots``
    the same for the parked copies.  With conv_channels each slot also keeps the tails of the
    layer's short convolution, viewed as ``conv_tails`` [n_slots, n_layers, conv_width - 1,
    conv_channels] and ``conv_snapshots``.  The slot table, the verbs, verify_drafts and the
    convolution's calls are SlotPool's.

    Every call takes x [rows, n_heads, head_p], B and C [rows, n_groups, d_state] (float32 or
    bfloat16, one type), dt [rows, n_heads] (float32 or bfloat16) and A, and optionally D and
    dt_bias, [n_heads] float32; with dt_softplus the step is softplus(dt + dt_bias), else
    dt + dt_bias.  A row's values are contiguous; rows may be any stride apart (x, B and C may
    be column ranges of the convolution's output), for x, B and C a multiple of 16 bytes.
    """

    def __init__(self, n_layers: int, n_heads: int, n_groups: int, n_slots: int, n_snapshots: int = 0,
                 head_p: int = 64, d_state: int = 128, device=None, state_dtype: str = "f32", out_dtype: str = "f32",
                 conv_channels: int = 0, conv_width: int = 4, conv_dtype: str = "bf16"):
        self._lib = load_library()
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.n_layers, self.n_heads, self.n_groups = n_layers, n_heads, n_groups
        self.head_p, self.d_state = head_p, d_state
        self.n_slots, self.n_snapshots = n_slots, n_snapshots
        for name, x in (("state_dtype", state_dtype), ("out_dtype", out_dtype), ("conv_dtype", conv_dtype)):
            if x not in ("f32", "bf16"):
                raise ValueError(f"{name} must be 'f32' or 'bf16'")
        self.state_dtype, self.out_dtype = state_dtype, out_dtype
        self.o_torch_dtype = torch.bfloat16 if out_dtype == "bf16" else torch.float32
        desc = SsmPoolDesc(n_layers, n_heads, n_groups, head_p, d_state, n_slots, n_snapshots, None, 0,
                           BF16 if state_dtype == "bf16" else F32, BF16 if out_dtype == "bf16" else F32,
                           ConvDesc(conv_channels, conv_width, BF16 if conv_dtype == "bf16" else F32))
        self._x_inner, self._b_inner, self._h_inner = (n_heads, head_p), (n_groups, d_state), (n_heads,)
        self._x_tight, self._b_tight = (head_p, 1), (d_state, 1)
        self._adopt("wkv7_ssm_pool", desc, (n_layers, n_heads, head_p, d_state), n_slots, n_snapshots, state_dtype)

    def _tokens(self, lead: tuple, x, dt, A, B, C, D, dt_bias, dt_softplus, o, stream, all_or_none=False):
        """The call's tokens as the library takes them; `lead` is the shape before the heads
        ((rows,) or (n, K), whose rows must be one stride apart)."""
        kind, step, at = x.dtype, dt.dtype, self._index
        if kind is torch.bfloat16:
            code = BF16
        elif kind is torch.float32:
            code = F32
        else:
            raise TypeError("x, B and C must be float32 or bfloat16")
        if step is torch.bfloat16:
            step_code = BF16
        elif step is torch.float32:
            step_code = F32
        else:
            raise TypeError("dt must be float32 or bfloat16")
        if not (B.dtype is kind and C.dtype is kind):
            raise TypeError("x, B and C must share one type")
        if not (x.get_device() == dt.get_device() == B.get_device() == C.get_device() == at):
            raise TypeError(f"x, dt, B and C must be on {self.device}")
        a = self._per_head("A", A)
        d = 0 if D is None else self._per_head("D", D)
        bias = 0 if dt_bias is None else self._per_head("dt_bias", dt_bias)
        xshape, bshape, hshape = lead + self._x_inner, lead + self._b_inner, lead + self._h_inner
        if not (x.shape == xshape and B.shape == bshape and C.shape == bshape and dt.shape == hshape):
            raise ValueError(f"x must be {list(xshape)}, B and C {list(bshape)}, dt {list(hshape)}")
        xs, bs, cs, ds = x.stride(), B.stride(), C.stride(), dt.stride()
        if len(lead) == 1 and xs[1:] == self._x_tight and bs[1:] == self._b_tight == cs[1:] and ds[1] == 1:
            xs, bs, cs, ds = xs[0], bs[0], cs[0], ds[0]
        else:  # axes of length 1, or two leading ones
            xs, ds = row_stride("x", xs, lead, self._x_inner), row_stride("dt", ds, lead, self._h_inner)
            bs, cs = row_stride("B", bs, lead, self._b_inner), row_stride("C", cs, lead, self._b_inner)
        if o is None:
            o = _empty(xshape, self.o_torch_dtype, self.device, stream)
        elif o.dtype is not self.o_torch_dtype or o.get_device() != at or not o.is_contiguous() or o.shape != xshape:
            raise ValueError(f"o must be a contiguous {self.o_torch_dtype} {list(xshape)} tensor")
        return SSM_TOKENS.pack(code, step_code, x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), a, d, bias,
                               xs, bs, cs, ds, 1 if dt_softplus else 0, 1 if all_or_none else 0, o.data_ptr()), o

    def _per_head(self, name: str, t: torch.Tensor) -> int:
        """The address of one float32 value a head."""
        if t.dtype is not torch.float32 or t.get_device() != self._index or t.shape != self._h_inner or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 [{self.n_heads}] tensor on {self.device}")
        return t.data_ptr()

    def decode_step(self, layer: int, slot_ids: torch.Tensor, x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False,
                    o=None, stream=None) -> torch.Tensor:
        """One token for each slot; o [n, n_heads, head_p]."""
        n = slot_ids.numel()
        t, o = self._tokens((n,), x, dt, A, B, C, D, dt_bias, dt_softplus, o, stream)
        _check(self._lib.wkv7_ssm_decode_step(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device), n, t,
                                              _stream_handle(stream, self.device)), "ssm_decode_step")
        return o

    def decode_multi(self, layer: int, slot_ids: torch.Tensor, x, dt, A, B, C, D=None, dt_bias=None, dt_softplus=False,
                     o=None, step_snap_ids: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """K consecutive tokens for each slot: inputs [n, K, ...], o [n, K, n_heads, head_p];
        with step_snap_ids ([n, K] int32) the state after every token also goes to those
        snapshots (this layer)."""
        n, K = slot_ids.numel(), int(x.shape[1])
        t, o = self._tokens((n, K), x, dt, A, B, C, D, dt_bias, dt_softplus, o, stream)
        snaps = None
        if step_snap_ids is not None:
            if step_snap_ids.numel() != n * K:
                raise ValueError("step_snap_ids must hold n * K ids")
            snaps = _dev_i32(step_snap_ids, "step_snap_ids", self.device)
        _check(self._lib.wkv7_ssm_decode_multi(self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device), n, K, t,
                                               snaps, _stream_handle(stream, self.device)), "ssm_decode_multi")
        return o

    def prefill(self, layer: int, slot_ids: torch.Tensor, cu_seqlens: torch.Tensor, x, dt, A, B, C, D=None, dt_bias=None,
                dt_softplus=False, o=None, max_seqlen: int | None = None, stream=None,
                sequential: bool = False, all_or_none: bool = False) -> torch.Tensor:
        """Sequences packed back to back, each continuing its slot's state; o [tokens, n_heads,
        head_p].  max_seqlen, the longest length, shapes the work: without it the total is taken
        for it, and several sequences may run slower.  A sequence that cu_seqlens gives no range
        of the tokens is skipped, with all_or_none the whole call (conv_prefill's rule)."""
        total = int(x.shape[0])
        t, o = self._tokens((total,), x, dt, A, B, C, D, dt_bias, dt_softplus, o, stream, all_or_none)
        if cu_seqlens.numel() != slot_ids.numel() + 1:
            raise ValueError("cu_seqlens must have n_seqs + 1 entries")
        n = slot_ids.numel()
        longest = total if max_seqlen is None else int(max_seqlen)
        need = 0 if sequential else self._lib.wkv7_ssm_prefill_workspace_bytes(self._h, n, longest)
        ws = _empty((need,), torch.uint8, self.device, stream) if need else None
        _check(self._lib.wkv7_ssm_prefill(
            self._h, layer, _dev_i32(slot_ids, "slot_ids", self.device), _dev_i32(cu_seqlens, "cu_seqlens", self.device),
            n, total, longest, t, None if ws is None else ws.data_ptr(), need, int(bool(sequential)),
            _stream_handle(stream, self.device)), "ssm_prefill")
        return o


class SsmLayer:
    """What a state space layer computes between its two projections, on one layer of a pool with
    conv_channels = n_heads * head_p + 2 * n_groups * d_state: the short convolution over x, B and
    C, the scan, and the gated norm of its readout.

    Every call takes the rows of the input projection, columns z [n_heads * head_p], x, B and C
    [conv_channels] and dt [n_heads] (any more columns are left alone: rows are a multiple of 16
    bytes), and returns the rows of the output projection's input, [.., n_heads * head_p], in the
    projection's type.  A, D and dt_bias are float32, the other weights float32 or bfloat16.
    With gate_first the norm is taken of the readout times silu(z), else the result is multiplied by
    it; the norm runs over norm_group columns (default: all of a row).
    """

    def __init__(self, pool: SsmPool, layer: int, conv_weight, conv_bias, A, D, dt_bias, norm_weight, eps: float = 1e-5,
                 gate_first: bool = True, norm_group: int | None = None):
        self.pool, self.layer = pool, layer
        self.inner, self.state = pool.n_heads * pool.head_p, pool.n_groups * pool.d_state
        if pool.conv_channels != self.inner + 2 * self.state:
            raise ValueError(f"the pool must have {self.inner + 2 * self.state} conv_channels")
        self.conv = (conv_weight, conv_bias)
        self.A, self.scan = A, {"D": D, "dt_bias": dt_bias, "dt_softplus": True}
        self.norm = (norm_weight,)
        self.norm_kw = {"eps": eps, "gate_first": gate_first, "group_size": norm_group}

    def _split(self, rows):
        """z, the convolution's inputs and dt."""
        last = self.inner + self.pool.conv_channels
        if rows.shape[-1] < last + self.pool.n_heads:
            raise ValueError(f"a row must hold at least {last + self.pool.n_heads} columns")
        return rows[..., :self.inner], rows[..., self.inner:last], rows[..., last:last + self.pool.n_heads]

    def _parts(self, y):
        """x, B and C of the convolution's outputs."""
        p, a = self.pool, self.inner + self.state
        return (y[..., :self.inner].unflatten(-1, (p.n_heads, p.head_p)),
                y[..., self.inner:a].unflatten(-1, (p.n_groups, p.d_state)), y[..., a:].unflatten(-1, (p.n_groups, p.d_state)))

    def _out(self, o, z, stream):
        o, z = o.reshape(-1, self.inner), z if z.dim() == 2 else z.flatten(0, 1)
        return gated_norm(o, z, *self.norm, out_dtype=z.dtype, stream=stream, **self.norm_kw)

    def step(self, slot_ids: torch.Tensor, rows, stream=None) -> torch.Tensor:
        """One token for each slot: rows [n, columns]."""
        z, u, dt = self._split(rows)
        x, B, C = self._parts(self.pool.conv_step(self.layer, slot_ids, u, *self.conv, stream=stream))
        return self._out(self.pool.decode_step(self.layer, slot_ids, x, dt, self.A, B, C, stream=stream, **self.scan), z, stream)

    def multi(self, slot_ids: torch.Tensor, rows, step_snap_ids: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """K tokens for each slot: rows [n, K, columns]; with step_snap_ids ([n, K] int32) what the
        slot holds after every token (state and tail of this layer) also goes to those snapshots."""
        z, u, dt = self._split(rows)
        y = self.pool.conv_multi(self.layer, slot_ids, u, *self.conv, step_snap_ids=step_snap_ids, stream=stream)
        x, B, C = self._parts(y)
        o = self.pool.decode_multi(self.layer, slot_ids, x, dt, self.A, B, C, step_snap_ids=step_snap_ids, stream=stream, **self.scan)
        return self._out(o, z, stream).unflatten(0, rows.shape[:2])

    def prefill(self, slot_ids: torch.Tensor, cu_seqlens: torch.Tensor, rows, max_seqlen: int | None = None,
                stream=None) -> torch.Tensor:
        """Sequences packed back to back, each going on from its slot: rows [tokens, columns].  Where
        cu_seqlens is not monotone or out of range no slot changes (device_status tells).  max_seqlen has
        to bound every length: a longer sequence is not scanned, but its tail moves on."""
        z, u, dt = self._split(rows)
        x, B, C = self._parts(self.pool.conv_prefill(self.layer, slot_ids, cu_seqlens, u, *self.conv, stream=stream))
        o = self.pool.prefill(self.layer, slot_ids, cu_seqlens, x, dt, self.A, B, C, max_seqlen=max_seqlen, stream=stream,
                              all_or_none=True, **self.scan)
        return self._out(o, z, stream)
