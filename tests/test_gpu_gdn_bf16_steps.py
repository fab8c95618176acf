"""GPU tests of the bf16-state pools' single steps of the gated delta rule: a stored state is
rounded to bf16, so two float32 evaluations that differ in their last bit can leave neighbours
2^-8 apart, and from the second step on their float32 outputs differ by more than float32
rounding.  The step is therefore defined to the bit: every product, sum, quotient and root
rounded as the formulas are written, sums over columns of x_c + x_{c+32} (+ ...) first and then
over neighbours.  Here it is evaluated so by elementary float32 operations."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from rwkv_wkv_gb300 import GdnPool

pytestmark = pytest.mark.gpu

EPS = 1e-6
HEADS = [(2, 4, 128, 128), (3, 3, 64, 64), (1, 3, 128, 64), (2, 2, 64, 128)]
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# o: a sum of at most 128 products, each product and sum rounded: below 136 x 2^-24 < 1e-5 of the
# largest entry against the same sum in another order, with the factors' few roundings.
O_TOL = 1e-5


def tree_sum(x):
    p = x[..., :32]
    for m in range(32, x.shape[-1], 32):
        p = p + x[..., m:m + 32]
    while p.shape[-1] > 1:
        p = p[..., 0::2] + p[..., 1::2]
    return p[..., 0]


def plain_step(S, q, k, v, g, beta, scale, eps):
    """One token for each row in float32: S [n, hv, dv, dk] -> (new S in float32, o)."""
    share = S.shape[1] // q.shape[1]
    q, k, v = q.float(), k.float(), v.float()
    if eps:
        q, k = (x / torch.sqrt(tree_sum(x * x) + eps)[..., None] for x in (q, k))
    q, k = (x.repeat_interleave(share, 1) for x in (q, k))
    S = S * torch.exp(g)[..., None, None]
    e = beta[..., None] * (v - tree_sum(S * k[..., None, :]))
    S = S + e[..., None] * k[..., None, :]
    return S, scale * tree_sum(S * q[..., None, :])


def inputs(gen, rows, heads, dtype):
    hk, hv, dk, dv = heads
    x = [torch.randn(rows, hk, dk, device="cuda", generator=gen) * 0.7 + 0.15 for _ in range(2)]
    x.append(torch.randn(rows, hv, dv, device="cuda", generator=gen))
    x = [t.to(DT[dtype]) for t in x]
    x.append(-torch.rand(rows, hv, device="cuda", generator=gen))
    x.append(torch.rand(rows, hv, device="cuda", generator=gen))
    return x


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [EPS, 0.0])
def test_decode_steps_leave_the_formulas_bits(heads, dtype, eps):
    hk, hv, dk, dv = heads
    n, slots = 37, 41
    gen = torch.Generator(device="cuda").manual_seed(31)
    S = (torch.randn(slots, 1, hv, dv, dk, device="cuda", generator=gen) * 0.1).to(torch.bfloat16)
    ids = torch.randperm(slots, device="cuda", generator=gen)[:n]
    with GdnPool(1, hk, hv, slots, head_k=dk, head_v=dv, state_dtype="bf16") as pool:
        pool.states.copy_(S)
        for _ in range(6):
            x = inputs(gen, n, heads, dtype)
            if not eps:
                x[1] = x[1] * 0.125
            o = pool.decode_step(0, ids.to(torch.int32), *x, l2norm_eps=eps or None)
            new, ref = plain_step(S[ids, 0].float(), *x, float(dk) ** -0.5, eps)
            S[ids, 0] = new.to(torch.bfloat16)
            assert torch.equal(pool.states, S)
            assert float((o - ref).abs().max()) <= O_TOL * float(ref.abs().max())
        assert pool.device_status() == 0
