"""GPU tests that the gated delta rule's multi-token decode is K single steps, bit for bit:
outputs, every kept state and the state left in the slot, on both kinds of pool and for both
input types.  (A server that checks drafts with one pass must be left with the state that
single steps would have left.)"""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from rwkv_wkv_gb300 import GdnPool

pytestmark = pytest.mark.gpu

EPS = 1e-6
HEADS = [(2, 4, 128, 128), (3, 3, 64, 64), (1, 3, 128, 64), (2, 2, 64, 128)]
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("inputs", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("K,eps", [(1, EPS), (5, EPS), (37, EPS), (6, 0.0)])
def test_multi_is_k_steps(heads, state, inputs, out, K, eps):
    hk, hv, dk, dv = heads
    n, slots = 5, 7
    gen = torch.Generator(device="cuda").manual_seed(K)
    qkv = torch.randn(n, K, 2 * hk * dk + hv * dv, device="cuda", generator=gen) * (0.8 if eps else 0.1)
    qkv = qkv.to(DT[inputs])
    q = qkv[..., :hk * dk].unflatten(2, (hk, dk))
    k = qkv[..., hk * dk:2 * hk * dk].unflatten(2, (hk, dk))
    v = qkv[..., 2 * hk * dk:].unflatten(2, (hv, dv))
    g = -torch.rand(n, K, hv, device="cuda", generator=gen)
    beta = torch.rand(n, K, hv, device="cuda", generator=gen)
    S0 = (torch.randn(slots, 1, hv, dv, dk, device="cuda", generator=gen) * 0.3).to(DT[state])
    ids = torch.randperm(slots, device="cuda", generator=gen)[:n].to(torch.int32)
    with GdnPool(1, hk, hv, slots, n_snapshots=n * K, head_k=dk, head_v=dv, state_dtype=state, out_dtype=out) as pool:
        pool.states.copy_(S0)
        o = pool.decode_multi(0, ids, q, k, v, g, beta, l2norm_eps=eps or None,
                              step_snap_ids=i32(np.arange(n * K).reshape(n, K)))
        many, kept = pool.states.clone(), pool.snapshots.clone().unflatten(0, (n, K))
        pool.states.copy_(S0)
        bare = pool.decode_multi(0, ids, q, k, v, g, beta, l2norm_eps=eps or None)
        assert torch.equal(bare, o) and torch.equal(pool.states, many)
        pool.states.copy_(S0)
        for t in range(K):
            one = pool.decode_step(0, ids, q[:, t], k[:, t], v[:, t], g[:, t], beta[:, t], l2norm_eps=eps or None)
            assert torch.equal(one, o[:, t]), t
            assert torch.equal(pool.states[ids.long()], kept[:, t]), t
        assert torch.equal(pool.states, many)
        assert pool.device_status() == 0
