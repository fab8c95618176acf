"""Inputs and error bounds of the state space operators' GPU tests."""
import numpy as np
import torch

from oracle.ssm import scan_run, softplus

EPS32 = 2.0 ** -24   # half a step of float32, relative
EPS16 = 2.0 ** -8    # of bfloat16


def scan_inputs(seed, rows, h, g, p, n, dtype=torch.bfloat16, dt_dtype=None, decay=1.0):
    """x, B and C as column ranges of one buffer, dt of another; A, D, dt_bias.  On the GPU."""
    gen = torch.Generator().manual_seed(seed)
    wide = torch.nn.functional.silu(torch.randn(rows, h * p + 2 * g * n + 8, generator=gen)).to(dtype).cuda()
    x = wide[:, 8:8 + h * p].unflatten(1, (h, p))
    B = wide[:, 8 + h * p:8 + h * p + g * n].unflatten(1, (g, n))
    C = wide[:, 8 + h * p + g * n:].unflatten(1, (g, n))
    dt = (torch.randn(rows, 3 + h, generator=gen) * 0.7).to(dt_dtype or dtype).cuda()[:, 3:]
    A = -decay * (1 + 15 * torch.rand(h, generator=gen)).cuda()
    D = torch.randn(h, generator=gen).cuda()
    bias = (torch.randn(h, generator=gen) - 3).cuda()
    return dict(x=x, dt=dt, A=A, B=B, C=C, D=D, dt_bias=bias, dt_softplus=True)


def host(t):
    return t if t is None or isinstance(t, bool) else t.detach().double().cpu().numpy()


def rows_of(ins, a, b):
    return {k: (v[a:b] if k in ("x", "dt", "B", "C") else v) for k, v in ins.items()}


def scan_reference(S0, ins):
    """The oracle's outputs and final state, and the sizes their errors are measured by: the sums
    of the terms' absolute values, and a quarter of the same sums without any decay."""
    a = {k: host(v) for k, v in ins.items()}
    o, S, _ = scan_run(S0, **a)
    step = a["dt"] + (0 if a["dt_bias"] is None else a["dt_bias"])
    step = softplus(step) if a["dt_softplus"] else step
    big = dict(x=np.abs(a["x"]), dt=np.abs(step), B=np.abs(a["B"]), C=np.abs(a["C"]), D=None if a["D"] is None else np.abs(a["D"]))
    uo, us, _ = scan_run(np.abs(S0), A=a["A"], **big)
    vo, vs, _ = scan_run(np.abs(S0), A=np.zeros_like(a["A"]), **big)
    return o, S, uo + vo / 4, us + vs / 4


def step_bound(T):
    """Relative to those sums, token by token in float32.  A token rounds its decay factor (the
    exponential to 2 ulp, 4 half steps, and the product with the state), dt x and its product with
    B, and the sum: 8 half steps at most, each on a term that is there; the step itself comes from
    an exponential, a logarithm and two sums, 16 half steps, and multiplies every term once more
    through dt x.  A readout adds 128 products in trees and chains of at most 12 sums, and D x.
    An exponent e that a term's decays add up to is off by 16 half steps of itself, the term
    by as much times e exp(-e) <= 0.37 of its undecayed self: less than a quarter of 46 half steps."""
    return (8 * T + 16 + 8 + 14) * EPS32


# In chunks: the computed operands (the states, the masked scores and the steps' values) go into the
# products as two bf16 parts, which leave 2^-18 of each; a term of an output passes through two
# of them, one of a state through one.  An exponent is a pair of floats of terms rounded by 2^-23;
# 2^x is approximate, 2 ulp, at most three factors of it in a term (12 half steps).  Sums over a chunk
# are float32 in the tensor core, at most 128 terms that may be cut rather than rounded: 128 * 2^-23.
# From chunk to chunk a state is rounded as by one token.
def chunk_bound(T):
    return 3 * 2.0 ** -18 + 128 * 2.0 ** -23 + step_bound(T // 128 + 2)


def check(got, want, size, rel, out=torch.float32, floor=0.0):
    """|got - want| within rel * size, and half a step of the output's type."""
    got = host(got)
    half = EPS16 if out == torch.bfloat16 else EPS32
    allowed = rel * size * (1 + half) + half * np.abs(want) + floor
    bad = ~(np.abs(got - want) <= allowed)
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want)[bad].max()), float(allowed[bad].min()))
