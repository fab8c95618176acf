"""Draft verification refuses, before any launch, a base that is not aligned to its element, as
the header says: the ids, counts, uniforms and outputs too (a misaligned 4-byte access on the
device would be a fault).  Fake addresses, never dereferenced."""
import ctypes

import pytest

from test_gdn_abi import X, fake_pool, lib  # noqa: F401
from rwkv_wkv_gb300 import wkv7


@pytest.mark.parametrize("name", ["draft_ids", "n_draft_rows", "uniforms", "noise", "step_snap_ids", "accepted", "tokens",
                                  "resume_ids", "p", "q"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_bases_are_refused(lib, name, off):  # noqa: F811
    st, h = fake_pool(lib)
    assert st == 0
    args = dict(n=2, n_draft=3, vocab=100, prob_dtype=0, p=X, p_batch_stride=400, p_row_stride=100, q=X,
                q_batch_stride=300, q_row_stride=100, draft_ids=X, n_draft_rows=X, uniforms=X, noise=X,
                noise_stride=100, step_snap_ids=X, accepted=X, tokens=X, resume_ids=X)
    args[name] = X + off
    try:
        assert lib.wkv7_verify_drafts(h, ctypes.byref(wkv7.DraftBatch(**args)), None) == 7
    finally:
        lib.wkv7_pool_destroy(h)
