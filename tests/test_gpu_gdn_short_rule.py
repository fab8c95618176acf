"""GPU test of where short prefills of the gated delta rule change over from running token by token
to running in chunks, for heads of 64 x 128 and 128 x 64 that fill the SMs."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from rwkv_wkv_gb300 import GdnPool

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.mark.parametrize("heads,n", [((1, 3, 128, 64), 60), ((2, 2, 64, 128), 100)])
@pytest.mark.parametrize("T", [13, 24, 25])
def test_mixed_heads_change_over_after_24_tokens(heads, n, T):
    hk, hv, dk, dv = heads
    gen = torch.Generator(device="cuda").manual_seed(71)
    bf = torch.bfloat16
    x = [torch.randn(n * T, hk, dk, device="cuda", generator=gen).to(bf) for _ in range(2)]
    x.append(torch.randn(n * T, hv, dv, device="cuda", generator=gen).to(bf))
    x += [-torch.rand(n * T, hv, device="cuda", generator=gen), torch.rand(n * T, hv, device="cuda", generator=gen)]
    S0 = torch.randn(n, 1, hv, dv, dk, device="cuda", generator=gen) * 0.1
    ids, cu = i32(np.arange(n)), i32(np.arange(n + 1) * T)
    got = {}
    with GdnPool(1, hk, hv, n, n_snapshots=1, head_k=dk, head_v=dv) as pool:
        for name, kw in (("auto", {}), ("by token", {"sequential": True}),
                         ("in chunks", {"cu_ckpt": i32(np.zeros(n + 1)), "ckpt_ids": i32([])})):
            pool.states.copy_(S0)
            o = pool.prefill(0, ids, cu, *x, l2norm_eps=EPS, max_seqlen=T, **kw)
            assert pool.device_status() == 0
            got[name] = (o, pool.states.clone())
    same = got["by token" if T <= 24 else "in chunks"]
    assert torch.equal(got["auto"][0], same[0]) and torch.equal(got["auto"][1], same[1])
    assert not torch.equal(got["by token"][0], got["in chunks"][0])
