"""GPU tests of the gated delta rule's calls in forms that its other tests leave out: row strides
of 0, pools of several layers, weak decay over cut sequences, and prefill without max_seqlen."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import i32
from oracle.gdn import gdn_run
from rwkv_wkv_gb300 import GdnPool

pytestmark = pytest.mark.gpu

EPS = 1e-6
F32_TOL, CHUNK_TOL = 2e-5, 4e-5  # as derived in test_gpu_gdn.py
HEADS = [(2, 4, 128, 128), (3, 3, 64, 64), (1, 3, 128, 64), (2, 2, 64, 128)]
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(lead, heads, dtype="bf16", seed=61):
    hk, hv, dk, dv = heads
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = [torch.randn(*lead, hk, dk, device="cuda", generator=gen).to(DT[dtype]) for _ in range(2)]
    x.append(torch.randn(*lead, hv, dv, device="cuda", generator=gen).to(DT[dtype]))
    return x + [-torch.rand(*lead, hv, device="cuda", generator=gen), torch.rand(*lead, hv, device="cuda", generator=gen)]


def start(n, heads, layers=1, dtype="f32"):
    gen = torch.Generator(device="cuda").manual_seed(62)
    return (torch.randn(n, layers, heads[1], heads[3], heads[2], device="cuda", generator=gen) * 0.1).to(DT[dtype])


@pytest.mark.parametrize("heads", HEADS[:2])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("which", [(0,), (1,), (2,), (3,), (4,), (0, 1, 2, 3, 4)])
def test_one_row_for_all(heads, dtype, state, which):
    """A row stride of 0 gives what the repeated rows give, in every call."""
    n, K = 4, 20
    S0 = start(n, heads, dtype=state)
    ids, cu = i32(np.arange(n)), i32(np.arange(n + 1) * K)
    with GdnPool(1, heads[0], heads[1], n, head_k=heads[2], head_v=heads[3], state_dtype=state) as pool:
        for form in ("decode", "multi", "prefill"):
            lead = {"decode": (n,), "multi": (n, K), "prefill": (n * K,)}[form]
            x = inputs(lead, heads, dtype)
            x = [t[(0,) * len(lead)].expand_as(t) if i in which else t for i, t in enumerate(x)]
            got = []
            for y in (x, [t.contiguous() for t in x]):
                pool.states.copy_(S0)
                if form == "decode":
                    o = pool.decode_step(0, ids, *y, l2norm_eps=EPS)
                elif form == "multi":
                    o = pool.decode_multi(0, ids, *y, l2norm_eps=EPS)
                else:  # (strides of 0 of q, k or v run token by token)
                    o = pool.prefill(0, ids, cu, *y, l2norm_eps=EPS, max_seqlen=K, sequential=True)
                got.append((o, pool.states.clone()))
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]), form
            if form == "prefill":
                pool.states.copy_(S0)
                o = pool.prefill(0, ids, cu, *x, l2norm_eps=EPS, max_seqlen=K)
                tol = CHUNK_TOL if state == "f32" else 2.0 ** -8
                assert oracle.rel_err(o.double().cpu().numpy(), got[0][0].double().cpu().numpy()) < CHUNK_TOL + F32_TOL
                assert oracle.rel_err(pool.states.double().cpu().numpy(), got[0][1].double().cpu().numpy()) < tol + F32_TOL
        assert pool.device_status() == 0


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_layers_are_apart(heads, state):
    """Calls on one layer of a pool of three leave the others, and do what a pool of one layer does."""
    n, K, total = 3, 3, 200
    hk, hv, dk, dv = heads
    S0 = start(n, heads, 3, state)
    ids, cu = i32([2, 0, 1]), i32([0, 100, 130, 200])
    kw = dict(l2norm_eps=EPS)
    runs = []
    for layers, at in ((3, 1), (1, 0)):
        with GdnPool(layers, hk, hv, n, n_snapshots=n * K, head_k=dk, head_v=dv, state_dtype=state) as pool:
            pool.states.copy_(S0 if layers == 3 else S0[:, 1:2])
            pool.snapshots.fill_(3.0)
            o = [pool.prefill(at, ids, cu, *inputs((total,), heads), max_seqlen=100, cu_ckpt=i32([0, 1, 1, 2]),
                              ckpt_ids=i32([4, 7]), **kw),
                 pool.prefill(at, ids, cu, *inputs((total,), heads), max_seqlen=100, **kw),
                 pool.decode_step(at, ids, *inputs((n,), heads), **kw),
                 pool.decode_multi(at, ids, *inputs((n, K), heads), step_snap_ids=i32(np.arange(n * K).reshape(n, K)), **kw)]
            assert pool.device_status() == 0
            runs.append((o, pool.states[:, at].clone(), pool.snapshots[:, at].clone()))
            if layers == 3:
                for other in (0, 2):
                    assert torch.equal(pool.states[:, other], S0[:, other])
                    assert bool((pool.snapshots[:, other] == 3.0).all())
    (o, S, kept), (o1, S1, kept1) = runs
    assert all(torch.equal(a, b) for a, b in zip(o, o1)) and torch.equal(S, S1) and torch.equal(kept, kept1)


@pytest.mark.parametrize("g", [-0.02, -0.002])
@pytest.mark.parametrize("heads", HEADS)
def test_cut_prefill_with_even_weak_decay(g, heads):
    """Segments whose transition hardly contracts, with nothing that empties the state."""
    hk, hv, dk, dv = heads
    total = 2048 + 37
    x = inputs((total,), heads)
    x[3].fill_(g)
    S0 = start(1, heads)
    with GdnPool(1, hk, hv, 1, head_k=dk, head_v=dv) as pool:
        assert pool._lib.wkv7_gdn_prefill_workspace_bytes(pool._h, 1, total) > 0
        pool.states.copy_(S0)
        o = pool.prefill(0, i32([0]), i32([0, total]), *x, l2norm_eps=EPS)
        assert pool.device_status() == 0
        S = pool.states[0, 0].double().cpu().numpy()
    o_ref, S_ref, _ = gdn_run(S0[0, 0].double().cpu().numpy(), *[t.double().cpu().numpy() for t in x], dk ** -0.5, EPS)
    assert oracle.rel_err(o.double().cpu().numpy(), o_ref) < CHUNK_TOL and oracle.rel_err(S, S_ref) < CHUNK_TOL


@pytest.mark.parametrize("lens", [[40, 3, 0, 17], [700, 900, 5], [300] * 50])
def test_prefill_without_a_longest_length(lens):
    """The bound only shapes the work: without it the total stands for it, and results agree."""
    heads, n = HEADS[0], len(lens)
    x = inputs((sum(lens),), heads)
    S0 = start(n, heads)
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    got = []
    with GdnPool(1, heads[0], heads[1], n) as pool:
        for kw in ({}, {"max_seqlen": max(lens)}):
            pool.states.copy_(S0)
            o = pool.prefill(0, i32(np.arange(n)), cu, *x, l2norm_eps=EPS, **kw)
            assert pool.device_status() == 0
            got.append((o.double().cpu().numpy(), pool.states.double().cpu().numpy()))
    for a, b in zip(*got):
        assert oracle.rel_err(a, b) < 2 * CHUNK_TOL
