"""A state space layer's prefill where cu_seqlens does not fit its tokens: convolution and scan by one rule."""
import pytest
import torch

from gpu_helpers import i32
from rwkv_wkv_gb300 import DEV_BAD_SEQLENS, DEV_BAD_SLOT, SsmLayer
from test_gpu_ssm_layer import CH, G, H, N, P, build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu,longest", [([0, 12, 7, 20], 14), ([0, 300, 150, 600], 300), ([0, 200, 400, 601], 300), ([-1, 200, 400, 600], 300),
                                        ([0, 2500, 2400, 2600], 2600)], ids=str)
@pytest.mark.parametrize("odd", [[0, 1, 2], [0, 5, 2]], ids=["ids", "an id out of range"])
def test_lengths_that_do_not_fit_leave_every_slot(cu, longest, odd):
    """Token by token, in chunks, and where long sequences run in segments: the convolution writes nothing then, and
    the scan does not run on what it did not write."""
    pool, w, draw = build(3)
    with pool:
        pool.create(3)
        pool.states.normal_()
        pool.conv_tails.normal_()
        before = pool.states.clone(), pool.conv_tails.clone()
        rows = draw(max(cu[-1] // 100 * 100, 20), H * P + CH + 8)
        SsmLayer(pool, 1, *w).prefill(i32(odd), i32(cu), rows, max_seqlen=longest)
        assert pool.device_status() == DEV_BAD_SEQLENS
        assert torch.equal(pool.states, before[0]) and torch.equal(pool.conv_tails, before[1])


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("sequential", [True, False])
def test_scan_of_all_or_none(sequential, softplus):
    """With lengths that fit the same bits as without, a sequence of an odd id skipped alone; else nothing at all.
    (Without softplus some steps are negative and their states grow past float32: bits are compared.)"""
    pool, w, draw = build(3, layers=1)
    with pool:
        rows = torch.nn.functional.silu(draw(600, CH))
        x, B, C = rows[:, :H * P].unflatten(1, (H, P)), rows[:, H * P:H * P + G * N].unflatten(1, (G, N)), rows[:, H * P + G * N:].unflatten(1, (G, N))
        dt = draw(600, H)
        begin = torch.randn_like(pool.states)
        for cu, fits in (([0, 200, 400, 600], True), ([0, 300, 250, 600], False), ([0, 200, 400, 601], False), ([-5, 200, 400, 600], False)):
            got = []
            for whole in (False, True):
                pool.states.copy_(begin)
                o = torch.full((600, H, P), 7.0, device="cuda")
                pool.prefill(0, i32([2, 9, 1]), i32(cu), x, dt, w[2], B, C, dt_softplus=softplus, max_seqlen=400, sequential=sequential,
                             all_or_none=whole, o=o)
                code = pool.device_status()
                assert code == DEV_BAD_SLOT or not fits and code == DEV_BAD_SEQLENS
                got.append((o.view(torch.int32), pool.states.view(torch.int32).clone()))
            if fits:
                assert all(torch.equal(a, b) for a, b in zip(*got)) and not torch.equal(got[1][1], begin.view(torch.int32))
            else:
                assert (got[1][0].view(torch.float32) == 7).all() and torch.equal(got[1][1], begin.view(torch.int32))
                assert not torch.equal(got[0][1], begin.view(torch.int32))
