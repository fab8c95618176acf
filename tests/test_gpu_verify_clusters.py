"""GPU tests of draft verification where a row's cluster of CTAs has little to do: parts of a row
that are short or empty, rows that return early, call after call (whole numbers: equal)."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from oracle.gdn import verify_drafts
from rwkv_wkv_gb300 import DEV_BAD_SEQLENS, Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,vocab", [(1, 4097), (3, 5000), (37, 8200), (5, 16400), (2, 33000), (130, 4099)])
def test_short_parts_call_after_call(n, vocab):
    """1 to 8 CTAs a row; every call's rows hold their only entries in another place."""
    rng = np.random.default_rng(vocab)
    K = 2
    p = torch.zeros(n, K + 1, vocab, device="cuda")
    noise = torch.ones(n, vocab, device="cuda")
    u = torch.full((n, K), 0.5, device="cuda")
    ids = rng.integers(0, vocab, (n, K)).astype(np.int32)
    rows = torch.arange(n, device="cuda")
    with Pool(1, 1, 1) as pool:
        for turn in range(60):
            at = torch.from_numpy(rng.integers(0, vocab, n)).cuda()
            if turn % 4 == 0:
                at.fill_(vocab - 1 if turn % 8 else 0)
            p.zero_()
            p[rows, 0, at] = 0.25
            q = torch.zeros(n, K, vocab, device="cuda")
            q[rows, 0, torch.from_numpy(ids[:, 0]).long().cuda()] = 1.0
            counts = rng.integers(0, K + 1, n).astype(np.int32)
            bad = rng.random(n) < 0.3
            counts[bad] = K + 1
            accepted, tokens, _ = pool.verify_drafts(i32(ids), p, q, u, noise, n_draft=i32(counts))
            assert pool.device_status() == (DEV_BAD_SEQLENS if bad.any() else 0)
            a, t = verify_drafts(ids, p.cpu().numpy(), q.cpu().numpy(), u.cpu().numpy(), noise.cpu().numpy(),
                                 np.where(bad, 0, counts).astype(np.int32))
            assert np.array_equal(accepted.cpu().numpy(), np.where(bad, -1, a))
            assert np.array_equal(tokens.cpu().numpy(), np.where(bad[:, None], -1, t))
