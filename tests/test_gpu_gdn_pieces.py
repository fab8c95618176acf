"""GPU tests of chunked prefills whose sequences are handed from CTA to CTA in pieces: each CTA
takes its piece from a count of the CTAs started, so nothing depends on the order in which they
start, on what else runs on the GPU, or on what an earlier call left in the workspace's memory."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from rwkv_wkv_gb300 import GdnPool

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.mark.parametrize("heads,lens", [((2, 4, 128, 128), [2070] * 39 + [1345]), ((2, 160, 64, 128), [1300]),
                                        ((1, 1, 64, 64), [4096, 2600, 0] * 11 + [70] * 480)])
def test_pieces_beside_other_work(heads, lens):
    """Few sequences, one sequence of many heads, more sequences than are put in order; repeated
    calls into one workspace while another stream keeps part of the SMs busy."""
    hk, hv, dk, dv = heads
    n, total = len(lens), sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(43)
    bf = torch.bfloat16
    x = [torch.randn(total, hk, dk, device="cuda", generator=gen).to(bf) for _ in range(2)]
    x.append(torch.randn(total, hv, dv, device="cuda", generator=gen).to(bf))
    x += [-torch.rand(total, hv, device="cuda", generator=gen), torch.rand(total, hv, device="cuda", generator=gen)]
    S0 = torch.randn(n, 1, hv, dv, dk, device="cuda", generator=gen) * 0.1
    ids, cu = i32(np.arange(n)), i32(np.concatenate([[0], np.cumsum(lens)]))
    a = torch.randn(2048, 2048, device="cuda", dtype=bf)
    with GdnPool(1, hk, hv, n, head_k=dk, head_v=dv) as pool:
        need = pool._lib.wkv7_gdn_prefill_workspace_bytes(pool._h, n, max(lens))
        assert need == n * hv * (dk * dv + 1) * 4

        def call(workspace):
            o = torch.empty(total, hv, dv, device="cuda")
            pool.states.copy_(S0)
            t, o = pool._tokens((total,), *x, o, None, EPS, None)
            assert pool._lib.wkv7_gdn_prefill(pool._h, 0, ids.data_ptr(), cu.data_ptr(), n, total, max(lens), t, None, None,
                                              None if workspace is None else workspace.data_ptr(),
                                              0 if workspace is None else need, 0,
                                              torch.cuda.current_stream().cuda_stream) == 0
            return o, pool.states.clone()

        whole = call(None)
        ws = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        for _ in range(3):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(20):
                    b = a @ a
            got = call(ws)
            assert pool.device_status() == 0
            assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])
        torch.cuda.current_stream().wait_stream(side)
        del b
