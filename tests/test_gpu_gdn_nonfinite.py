"""GPU tests that a value that is not finite reaches, in a chunked prefill of the gated delta rule,
only what the formulas let it reach: nothing before its token, no other sequence, head or (for
v) value row.  The token-by-token call says what is finite; where it is, both agree as ever."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from rwkv_wkv_gb300 import GdnPool

pytestmark = pytest.mark.gpu

EPS = 1e-6
# As derived in test_gpu_gdn.py, between a chunked and a token-by-token float32 result; bf16
# outputs add half a spacing on either side.
TOL = {"f32": 4e-5 + 2e-5, "bf16": 2.0 ** -8 + 2.0 ** -8}
NAN, INF = float("nan"), float("inf")


def inputs(heads, total, seed=51):
    hk, hv, dk, dv = heads
    gen = torch.Generator(device="cuda").manual_seed(seed)
    bf = torch.bfloat16
    x = [torch.randn(total, hk, dk, device="cuda", generator=gen).to(bf) for _ in range(2)]
    x.append(torch.randn(total, hv, dv, device="cuda", generator=gen).to(bf))
    x += [-torch.rand(total, hv, device="cuda", generator=gen), torch.rand(total, hv, device="cuda", generator=gen)]
    return x


def same_reach(a, b, tol):
    """Equal sets of finite values, and these within tol of the largest."""
    a, b = a.float(), b.float()
    fine = torch.isfinite(b)
    assert torch.equal(fine, torch.isfinite(a))
    if not bool(fine.any()):   # (a NaN key leaves nothing of the state of the heads that share it)
        return
    assert float((a[fine] - b[fine]).abs().max()) <= tol * float(b[fine].abs().max())


def both(heads, lens, poison, state="f32", out="f32", ckpt=False, S0=None, workspace=None):
    hk, hv, dk, dv = heads
    n, total = len(lens), int(sum(lens))
    x = inputs(heads, total)
    poison(x)
    cu = np.concatenate([[0], np.cumsum(lens)])
    cks = np.concatenate([[0], np.cumsum(np.asarray(lens) // 64)])
    gen = torch.Generator(device="cuda").manual_seed(52)
    if S0 is None:
        S0 = torch.randn(n, 1, hv, dv, dk, device="cuda", generator=gen) * 0.1
    got = []
    with GdnPool(1, hk, hv, n, n_snapshots=max(1, int(cks[-1])), head_k=dk, head_v=dv, state_dtype=state,
                 out_dtype=out) as pool:
        kw = dict(cu_ckpt=i32(cks), ckpt_ids=i32(np.arange(cks[-1]))) if ckpt else {}
        need = pool._lib.wkv7_gdn_prefill_workspace_bytes(pool._h, n, max(lens))
        assert workspace is None or (need > 0) == workspace
        for sequential in (False, True):
            pool.states.copy_(S0)
            pool.snapshots.zero_()
            o = pool.prefill(0, i32(np.arange(n)), i32(cu), *x, l2norm_eps=EPS, max_seqlen=max(lens),
                             sequential=sequential, **kw)
            assert pool.device_status() == 0
            got.append((o, pool.states.clone(), pool.snapshots.clone()))
    (o, S, kept), (o2, S2, kept2) = got
    tol = TOL["bf16"] if state == "bf16" and ckpt else TOL[out]
    assert bool(torch.isfinite(o2).any())
    same_reach(o, o2, tol)
    same_reach(S, S2, TOL[state])
    if ckpt:
        same_reach(kept, kept2, TOL[state])
    return o


def at(name, *where, value=NAN):
    def poison(x):
        x["qkvgb".index(name)][where] = value
    return poison


CASES = {
    "v": at("v", 150, 1, 5), "v infinite": at("v", 150, 0, 7, value=INF), "v at a chunk's last token": at("v", 191, 0, 0),
    "v at a chunk's first token": at("v", 128, 0, 0), "v at the first token": at("v", 0, 0, 3),
    "v from token 80 on": at("v", slice(80, 128), 0, 9), "k": at("k", 100, 0, 3), "k infinite": at("k", 229, 0, 3, value=-INF),
    "q": at("q", 90, 0, 1), "g": at("g", 75, 0), "beta": at("b", 200, 0), "beta at a chunk's last token": at("b", 127, 0),
    "beta infinite": at("b", 20, 0, value=INF), "v at the last token": at("v", 229, 0, 2),
}


@pytest.mark.parametrize("heads", [(2, 4, 128, 128), (3, 3, 64, 64), (1, 3, 128, 64), (2, 2, 64, 128)])
@pytest.mark.parametrize("what", list(CASES))
def test_reach(heads, what):
    both(heads, [230], CASES[what], workspace=False)


@pytest.mark.parametrize("state,out", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("what", ["v", "k", "beta"])
@pytest.mark.parametrize("ckpt", [False, True])
def test_reach_by_types_and_with_checkpoints(state, out, what, ckpt):
    both((2, 4, 128, 128), [230, 64, 20], CASES[what], state, out, ckpt)


@pytest.mark.parametrize("heads", [(2, 4, 128, 128), (1, 3, 128, 64), (2, 2, 64, 128)])
@pytest.mark.parametrize("where", [70, 1000, 1990])
@pytest.mark.parametrize("name", ["v", "k"])
def test_reach_in_segments(heads, where, name):
    both(heads, [2000], at(name, where, 0, 3), workspace=True)


@pytest.mark.parametrize("where", [70, 1400, 2000])
def test_reach_in_pieces(where):
    both((2, 4, 128, 128), [2070] * 40, at("v", 5 * 2070 + where, 2, 3), workspace=True)


def test_a_state_that_is_not_finite():
    """A row of the start state that is not finite stays so; its head's other rows are as ever."""
    heads = (2, 4, 128, 128)
    S0 = torch.randn(1, 1, 4, 128, 128, device="cuda") * 0.1
    S0[0, 0, 1, 17, 40] = NAN
    S0[0, 0, 3, 0, 0] = INF
    o = both(heads, [300], lambda x: None, S0=S0)
    assert not bool(torch.isfinite(o[:, 1, 17]).any())
    assert bool(torch.isfinite(o[:, [0, 2]]).all()) and bool(torch.isfinite(o[:, 1, :17]).all())


def test_resume_where_a_later_token_is_not_finite():
    """The checkpoints' promise holds: the path of the tail is the path of the whole."""
    heads, total = (2, 4, 128, 128), 300
    x = inputs(heads, total)
    x[2][250, 1, 5] = NAN
    with GdnPool(1, 2, 4, 2, n_snapshots=5) as pool:
        pool.states.zero_()
        o = pool.prefill(0, i32([0]), i32([0, total]), *x, l2norm_eps=EPS, cu_ckpt=i32([0, 4]), ckpt_ids=i32([0, 1, 2, 3]))
        pool.restore(i32([1]), i32([1]))
        tail = pool.prefill(0, i32([1]), i32([0, total - 128]), *[t[128:] for t in x], l2norm_eps=EPS, cu_ckpt=i32([0, 2]),
                            ckpt_ids=i32([4, 0]))
        assert torch.equal(tail.isnan(), o[128:].isnan())
        assert torch.equal(tail.nan_to_num(), o[128:].nan_to_num())
        assert torch.equal(pool.states[0].nan_to_num(), pool.states[1].nan_to_num())
