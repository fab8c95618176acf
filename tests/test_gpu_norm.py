"""The gated norm against the float64 formula, its edges and refusals."""
import numpy as np
import pytest
import torch

from oracle.ssm import gate, gated_norm as reference
from rwkv_wkv_gb300 import Wkv7Error, gated_norm
from ssm_helpers import EPS32, check, host

pytestmark = pytest.mark.gpu


def inputs(seed, rows, width, xt, zt, wt):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width + 16, generator=gen).to(xt).cuda()[:, 8:8 + width]
    z = (2 * torch.randn(rows, width + 8, generator=gen)).to(zt).cuda()[:, 8:]
    w, b = (torch.randn(width, generator=gen).to(wt).cuda() for _ in range(2))
    return x, z, w, b


def compare(o, x, z, w, b, group, eps, kind, activation, gate_first):
    """Relative roundings of: the gate (12 half steps, and 2^-24 |z| of its exponent), its product, the
    root of the mean square (sums of up to 16,384 squares in chains and trees of at most 32, the
    root to 2 ulp), weight and bias; and of a layer norm's mean, half steps of the largest deviation."""
    a = [None if t is None else host(t) for t in (x, z, w, b)]
    want = reference(*a, group, eps, kind, activation, gate_first)
    g = np.ones_like(a[0]) if z is None else np.abs(gate(a[1], activation))
    u = np.abs(a[0]) * g if gate_first else np.abs(a[0])
    shape = (len(u), -1, group)
    ug = u.reshape(shape)
    if kind == "layer":
        v = a[0] * gate(a[1], activation) if z is not None and gate_first else a[0]
        v = v.reshape(shape)
        dev = np.sqrt(((v - v.mean(-1, keepdims=True)) ** 2).mean(-1, keepdims=True) + eps)
        size = ((ug + ug.mean(-1, keepdims=True) * 2) / dev)
        size = size + np.abs((v - v.mean(-1, keepdims=True)) / dev) * (1 + (ug.max(-1, keepdims=True) / dev))
    else:
        size = ug / np.sqrt((ug ** 2).mean(-1, keepdims=True) + eps)
    size = size.reshape(u.shape) * (1 if w is None else np.abs(a[2])) + (0 if b is None else np.abs(a[3]))
    if not gate_first:
        size = size * g
    zmax = 0 if z is None else float(np.abs(a[1]).max())
    check(o, want, size, (60 + 4 * zmax) * EPS32, o.dtype)


TYPES = [(torch.bfloat16,) * 4, (torch.float32,) * 4, (torch.float32, torch.bfloat16, torch.float32, torch.bfloat16)]


@pytest.mark.parametrize("types", TYPES, ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("kind,activation,first", [("rms", "silu", True), ("rms", "silu", False), ("layer", None, False),
                                                   ("layer", "sigmoid", True)])
@pytest.mark.parametrize("rows,groups,group", [(1, 1, 8), (3, 5, 24), (67, 4, 64), (130, 2, 128), (5, 3, 256), (2, 2, 264),
                                               (9, 1, 1000), (4, 1, 4096), (3, 2, 16384)])
def test_values(rows, groups, group, kind, activation, first, types):
    xt, zt, wt, ot = types
    x, z, w, b = inputs(rows + group, rows, groups * group, xt, zt, wt)
    o = gated_norm(x, z, w, b, group_size=group, eps=1e-5, kind=kind, activation=activation, gate_first=first, out_dtype=ot)
    assert o.dtype is ot
    compare(o, x, z, w, b, group, 1e-5, kind, activation, first)


@pytest.mark.parametrize("have", ["x", "xw", "xb", "xz", "xzw"])
def test_optional_inputs(have):
    x, z, w, b = inputs(1, 33, 192, torch.bfloat16, torch.bfloat16, torch.float32)
    z, w, b = (t if n in have else None for n, t in (("z", z), ("w", w), ("b", b)))
    o = gated_norm(x, z, w, b, group_size=64)
    compare(o, x, z, w, b, 64, 1e-5, "rms", "silu", False)


def test_rows_do_not_meet():
    """A row that is not finite, one of zeros and one of the type's largest values leave the others as they are."""
    x, z, w, _ = inputs(2, 6, 128, torch.float32, torch.float32, torch.float32)
    clean = gated_norm(x, z, w, group_size=64)
    x = x.clone()
    x[1, 3], x[2, 70], x[3] = float("nan"), float("inf"), 0.0
    o = gated_norm(x, z, w, group_size=64)
    assert torch.equal(o[[0, 4, 5]], clean[[0, 4, 5]]) and torch.equal(o[1, 64:], clean[1, 64:]) and torch.equal(o[2, :64], clean[2, :64])
    assert torch.isnan(o[1, :64]).all() and (o[3] == 0).all()
    assert torch.equal(gated_norm(x[:1], torch.full_like(z[:1], -200.0), w, group_size=64), torch.zeros(1, 128, device="cuda"))


def test_same_row_for_all_and_nothing():
    x, z, w, _ = inputs(3, 1, 64, torch.bfloat16, torch.bfloat16, torch.bfloat16)
    o = gated_norm(x.expand(5, 64), z.expand(5, 64), w)
    assert torch.equal(o, gated_norm(x, z, w).expand(5, 64))
    assert gated_norm(x[:0], z[:0], w).shape == (0, 64)


def test_refusals():
    x, z, w, b = inputs(4, 4, 64, torch.bfloat16, torch.bfloat16, torch.bfloat16)
    for args, kw in (((x.double(), z), {}), ((x, z[:3]), {}), ((x, z, w.half()), {}), ((x, z, w, b.float()), {}), ((x[0],), {}),
                     ((x, z), dict(kind="l1")), ((x, z), dict(activation="relu")), ((x.t(),), {}), ((x, z, w[::2]), {}),
                     ((x, z), dict(out_dtype=torch.float16))):
        with pytest.raises((TypeError, ValueError)):
            gated_norm(*args, **kw)
    for kw, name in ((dict(group_size=24), "INVALID_ARG"), (dict(group_size=4), "UNSUPPORTED"), (dict(group_size=0), "INVALID_ARG"),
                     (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG")):
        with pytest.raises(Wkv7Error, match=name):
            gated_norm(x, z, w, **kw)
    whole = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(Wkv7Error, match="INVALID_ARG"):
        gated_norm(whole, z, o=whole)
    with pytest.raises(Wkv7Error, match="UNSUPPORTED"):
        gated_norm(torch.zeros(2, 16385 * 8, device="cuda"), group_size=16385 * 8)
    with pytest.raises(Wkv7Error, match="UNSUPPORTED"):
        gated_norm(torch.zeros(4, 68, device="cuda", dtype=torch.bfloat16)[:, 4:])


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("group", [64, 512])
@pytest.mark.parametrize("types", TYPES, ids=["bf16", "f32", "mixed"])
def test_gates_far_below_zero_close(types, group, first):
    """silu of a large negative z is 0 whatever it multiplies: x z alone would pass float32's range."""
    xt, zt, wt, ot = types
    x, z, w, b = inputs(5, 4, 2 * group, xt, zt, wt)
    x, z = x.clone(), z.clone()
    if first:
        x[0, 3], z[0, 3] = 3e30, -2e10
        x[1, group:], z[1, group:] = -1e38, -3e38
    else:
        x[0, 3], z[0, 3] = 50.0, -3e38
        z[1, group:] = -3e38
    o = gated_norm(x, z, w, b, group_size=group, gate_first=first, out_dtype=ot)
    assert torch.isfinite(o).all()
    closed = z < -200                               # (silu is 0 in float32 and in the formula's product)
    compare(o, x.masked_fill(closed, 0) if first else x, z.masked_fill(closed, 0), w, b, group, 1e-5, "rms", "silu", first)
