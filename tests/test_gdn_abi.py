"""The gated-delta-rule and draft-verification entry points without a GPU: pool sizes and
host-side refusals, each returned before any launch (fake, never dereferenced addresses)."""
import ctypes

import pytest

from rwkv_wkv_gb300 import build as wbuild
from rwkv_wkv_gb300 import wkv7

ADDR = 0x7F0000000000
X = ADDR


@pytest.fixture(scope="module")
def lib():
    wbuild.build()
    return wkv7.load_library()


def desc(**kw):
    d = dict(n_layers=2, n_k_heads=2, n_v_heads=4, head_k=128, head_v=64, n_slots=8, n_snapshots=4,
             device_buffer=None, buffer_bytes=0, state_dtype=0, out_dtype=0)
    d.update(kw)
    return wkv7.GdnPoolDesc(**d)


def fake_pool(lib, **kw):
    d = desc(**kw)
    d.buffer_bytes = lib.wkv7_gdn_pool_required_bytes(ctypes.byref(d))
    d.device_buffer = ADDR
    h = ctypes.c_void_p()
    return lib.wkv7_gdn_pool_create(ctypes.byref(d), ctypes.byref(h)), h


def test_pool_sizes_and_descriptions(lib):
    slot = 2 * 4 * 64 * 128 * 4
    assert lib.wkv7_gdn_pool_required_bytes(ctypes.byref(desc())) == 256 + 12 * slot + 256
    assert lib.wkv7_gdn_pool_required_bytes(ctypes.byref(desc(state_dtype=1))) == 256 + 6 * slot + 256
    for bad in (dict(n_v_heads=3), dict(n_layers=0), dict(n_k_heads=0), dict(state_dtype=2), dict(n_slots=0),
                dict(n_snapshots=-1), dict(out_dtype=-1)):
        assert lib.wkv7_gdn_pool_required_bytes(ctypes.byref(desc(**bad))) == 0
        assert fake_pool(lib, **bad)[0] == 1
    for bad in (dict(head_k=32), dict(head_v=256)):
        assert fake_pool(lib, **bad)[0] == 7
    st, h = fake_pool(lib)
    assert st == 0
    try:
        assert lib.wkv7_slot_bytes(h) == slot
        p = ctypes.c_void_p()
        assert lib.wkv7_pool_state_ptr(h, 3, 1, ctypes.byref(p)) == 0
        assert p.value == ADDR + 256 + 3 * slot + slot // 2
        got = wkv7.GdnPoolDesc()
        assert lib.wkv7_gdn_pool_get_desc(h, ctypes.byref(got)) == 0
        assert (got.n_v_heads, got.head_k, got.head_v, got.device_buffer) == (4, 128, 64, ADDR)
        assert lib.wkv7_pool_get_desc(h, ctypes.byref(wkv7.PoolDesc())) == 7
        ids = (ctypes.c_int32 * 8)()
        assert lib.wkv7_slot_alloc(h, 8, ids) == 0 and lib.wkv7_slot_count_free(h) == 0
    finally:
        assert lib.wkv7_pool_destroy(h) == 0


def tokens(**kw):
    d = dict(in_dtype=1, q=X, k=X, v=X, g=X, beta=X, q_stride=512, k_stride=512, v_stride=512, g_stride=4,
             beta_stride=4, scale=1.0, l2norm_eps=0.0, o=X)
    d.update(kw)
    return wkv7.GdnTokens(**d)


def test_gdn_host_checks(lib):
    st, h = fake_pool(lib)
    assert st == 0
    ref = ctypes.byref

    def decode(t, layer=0, ids=X, n=2, pool=h):
        return lib.wkv7_gdn_decode_step(pool, layer, ids, n, None if t is None else ref(t), None)

    def multi(t, n=2, K=2, snaps=None):
        return lib.wkv7_gdn_decode_multi(h, 0, X, n, K, ref(t), snaps, None)

    def prefill(t, ids=X, cu=X, n=1, total=10, longest=10, cks=None, cki=None, layer=0, ws=None):
        return lib.wkv7_gdn_prefill(h, layer, ids, cu, n, total, longest, ref(t), cks, cki, ws, 0, 0, None)

    try:
        assert decode(tokens(), layer=2) == 1 and decode(tokens(), n=9) == 1 and decode(tokens(), n=-1) == 1
        assert decode(tokens(), ids=None) == 1 and decode(None) == 1 and decode(tokens(), pool=None) == 1
        assert decode(tokens(), n=0) == 0
        for name in ("q", "k", "v", "g", "beta", "o"):
            assert decode(tokens(**{name: None})) == 1
            assert decode(tokens(**{name: X + 2})) == 7
        for name, low in (("q", 255), ("k", 255), ("v", 255), ("g", 3), ("beta", 3)):
            assert decode(tokens(**{name + "_stride": low})) == 1
        for name in ("q", "k", "v"):
            assert decode(tokens(**{name + "_stride": 516})) == 7      # 1,032 bytes
        assert decode(tokens(in_dtype=3)) == 1
        for eps in (-1.0, float("nan"), float("inf")):
            assert decode(tokens(l2norm_eps=eps)) == 1
        assert multi(tokens(), K=0) == 1 and multi(tokens(), n=9) == 1 and multi(tokens(q_stride=8)) == 1
        assert multi(tokens(), n=0) == 0 and multi(tokens(), n=8, K=1 << 29) == 1
        assert prefill(tokens(), longest=11) == 5 and prefill(tokens(), cu=None) == 1 and prefill(tokens(), n=9) == 1
        assert prefill(tokens(), ids=None) == 1 and prefill(tokens(), layer=-1) == 1
        assert prefill(tokens(), cks=X) == 1 and prefill(tokens(), cki=X) == 1
        assert prefill(tokens(k=X + 8)) == 7 and prefill(tokens(), n=0, total=0, longest=0) == 0
        assert prefill(tokens(), ws=X + 8) == 7
        # a few long sequences can use a workspace, and as many as fill part of a round of the SMs
        # (float32 states and a count each), but not short ones nor a full round
        size = lib.wkv7_gdn_prefill_workspace_bytes
        assert size(h, 1, 16384) > 0 and size(h, 1, 16384) % 16 == 0
        assert size(h, 1, 256) == size(h, 8, 0) == size(h, 0, 16384) == size(None, 1, 16384) == 0
        assert size(h, 40, 16384) == 40 * 4 * (128 * 64 + 1) * 4 and size(h, 38, 16384) == 0 == size(h, 40, 640)
        # the WKV-7 recurrence is not this pool's
        ins = [ctypes.c_void_p(X)] * 6
        assert lib.wkv7_decode_step(h, 0, X, 1, 1, *ins, X, None) == 7
        assert lib.wkv7_decode_multi(h, 0, X, 1, 1, 1, *ins, X, None, None) == 7
        assert lib.wkv7_prefill(h, 0, X, X, 1, 1, 1, 1, *ins, X, None) == 7
        assert lib.wkv7_prefill_sequential(h, 0, X, X, 1, 1, 1, 1, *ins, X, None) == 7
    finally:
        lib.wkv7_pool_destroy(h)
    st, h = fake_pool(lib, n_snapshots=0)
    try:
        assert multi(tokens(), snaps=X) == 1 and prefill(tokens(), cks=X, cki=X) == 1
    finally:
        lib.wkv7_pool_destroy(h)
    w = wkv7.PoolDesc(1, 1, 64, 1, 0, ADDR, 1 << 30, 0, 0)
    h = ctypes.c_void_p()
    assert lib.wkv7_pool_create(ref(w), ref(h)) == 0
    try:
        assert decode(tokens(), n=1, pool=h) == 7
        assert lib.wkv7_gdn_pool_get_desc(h, ref(desc())) == 7
    finally:
        lib.wkv7_pool_destroy(h)


def test_verify_host_checks(lib):
    st, h = fake_pool(lib)
    assert st == 0
    good = dict(n=2, n_draft=3, vocab=100, prob_dtype=0, p=X, p_batch_stride=400, p_row_stride=100, q=X,
                q_batch_stride=300, q_row_stride=100, draft_ids=X, n_draft_rows=None, uniforms=X, noise=X,
                noise_stride=100, step_snap_ids=X, accepted=X, tokens=X, resume_ids=X)

    def verify(**kw):
        return lib.wkv7_verify_drafts(h, ctypes.byref(wkv7.DraftBatch(**{**good, **kw})), None)

    try:
        for bad in (dict(n=-1), dict(n_draft=-1), dict(vocab=0), dict(prob_dtype=2), dict(p=None), dict(noise=None),
                    dict(accepted=None), dict(tokens=None), dict(draft_ids=None), dict(uniforms=None),
                    dict(step_snap_ids=None), dict(p_row_stride=99), dict(q_row_stride=99), dict(p_batch_stride=-400),
                    dict(q_batch_stride=50), dict(noise_stride=99)):
            assert verify(**bad) == 1, bad
        for bad in (dict(p=X + 2), dict(q=X + 1), dict(noise=X + 2), dict(vocab=(1 << 30) + 1)):
            assert verify(**bad) == 7, bad
        assert verify(n=0) == 0
        assert lib.wkv7_verify_drafts(None, ctypes.byref(wkv7.DraftBatch(**good)), None) == 1
        assert lib.wkv7_verify_drafts(h, None, None) == 1
    finally:
        lib.wkv7_pool_destroy(h)
