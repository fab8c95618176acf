"""GPU tests of what a chunked prefill of the gated delta rule leaves behind when a bounded wait
gives up (forced by the library's test hook: input loads that are not issued): the call reports
it, and neither a slot's state nor a checkpoint is written; the next call runs as ever."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import i32
from oracle.gdn import gdn_run
from rwkv_wkv_gb300 import DEV_WAIT_TIMEOUT, GdnPool, load_library

pytestmark = pytest.mark.gpu

EPS = 1e-6
CHUNK_TOL = 4e-5  # as derived in test_gpu_gdn.py


def run_both(heads, lens, hook, ckpt=False):
    """A call with the hook on, then one without; the pool after each, and the second's outputs."""
    lib = load_library()
    hk, hv, dk, dv = heads
    n, total = len(lens), int(sum(lens))
    gen = torch.Generator(device="cuda").manual_seed(41)
    bf = torch.bfloat16
    x = [torch.randn(total, hk, dk, device="cuda", generator=gen).to(bf) for _ in range(2)]
    x.append(torch.randn(total, hv, dv, device="cuda", generator=gen).to(bf))
    x += [-torch.rand(total, hv, device="cuda", generator=gen), torch.rand(total, hv, device="cuda", generator=gen)]
    S0 = torch.randn(n, 1, hv, dv, dk, device="cuda", generator=gen) * 0.1
    cu = np.concatenate([[0], np.cumsum(lens)])
    cks = np.concatenate([[0], np.cumsum(np.asarray(lens) // 64)])
    with GdnPool(1, hk, hv, n, n_snapshots=max(1, int(cks[-1])), head_k=dk, head_v=dv) as pool:
        kw = dict(cu_ckpt=i32(cks), ckpt_ids=i32(np.arange(cks[-1]))) if ckpt else {}
        pool.states.copy_(S0)
        pool.snapshots.fill_(7.0)
        assert lib.wkv7_test_force_wait_timeout(hook) == 0
        try:
            pool.prefill(0, i32(np.arange(n)), i32(cu), *x, l2norm_eps=EPS, max_seqlen=max(lens), **kw)
            assert pool.device_status() == DEV_WAIT_TIMEOUT
        finally:
            lib.wkv7_test_force_wait_timeout(0)
        assert torch.equal(pool.states, S0)
        assert bool((pool.snapshots == 7.0).all())
        o = pool.prefill(0, i32(np.arange(n)), i32(cu), *x, l2norm_eps=EPS, max_seqlen=max(lens), **kw)
        assert pool.device_status() == 0
        S = pool.states.double().cpu().numpy()
    for i in (0, n - 1):
        h = [t[cu[i]:cu[i + 1]].double().cpu().numpy() for t in x]
        o_ref, S_ref, _ = gdn_run(S0[i, 0].double().cpu().numpy(), *h, dk ** -0.5, EPS)
        assert oracle.rel_err(o[cu[i]:cu[i + 1]].double().cpu().numpy(), o_ref) < CHUNK_TOL
        assert oracle.rel_err(S[i, 0], S_ref) < CHUNK_TOL


def test_no_checkpoint_is_written_after_a_wait_gave_up():
    run_both((2, 4, 128, 128), [300, 64, 130], 1, ckpt=True)


@pytest.mark.parametrize("heads", [(2, 4, 128, 128), (1, 3, 128, 64), (2, 2, 64, 128)])
@pytest.mark.parametrize("lens", [[2000], [3000, 1500]])
def test_a_lost_transfer_leaves_the_slot_alone(heads, lens):
    """Only the first pass over the segments of cut sequences gives up: what it would have handed on
    is not in the workspace, and the last pass, whose own waits are met, must not use it."""
    hk, hv, dk, dv = heads
    with GdnPool(1, hk, hv, len(lens), head_k=dk, head_v=dv) as pool:
        assert pool._lib.wkv7_gdn_prefill_workspace_bytes(pool._h, len(lens), max(lens)) > 0
    run_both(heads, lens, 2)


@pytest.mark.parametrize("ckpt", [False, True])
def test_pieces_that_give_up(ckpt):
    """More units than SMs, in pieces: the wait for the piece before gives up too."""
    heads, n = (2, 4, 128, 128), 40
    with GdnPool(1, *heads[:2], n) as pool:
        assert pool._lib.wkv7_gdn_prefill_workspace_bytes(pool._h, n, 2070) == n * 4 * (128 * 128 + 1) * 4
    run_both(heads, [2070] * n, 1, ckpt)
