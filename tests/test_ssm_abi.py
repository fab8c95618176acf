"""The selective scan, short convolution and gated norm without a GPU: pool sizes and host-side
refusals, each returned before any launch (fake, never dereferenced addresses)."""
import ctypes

import numpy as np
import pytest

from oracle.ssm import conv_run, gated_norm, scan_run
from rwkv_wkv_gb300 import build as wbuild
from rwkv_wkv_gb300 import wkv7

X = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    wbuild.build()
    return wkv7.load_library()


def desc(conv=(40, 4, 1), **kw):
    d = dict(n_layers=2, n_heads=4, n_groups=2, head_p=64, d_state=128, n_slots=8, n_snapshots=4, device_buffer=None,
             buffer_bytes=0, state_dtype=0, out_dtype=0, conv=wkv7.ConvDesc(*conv))
    d.update(kw)
    return wkv7.SsmPoolDesc(**d)


def fake_pool(lib, **kw):
    d = desc(**kw)
    d.buffer_bytes = lib.wkv7_ssm_pool_required_bytes(ctypes.byref(d))
    d.device_buffer = X
    h = ctypes.c_void_p()
    return lib.wkv7_ssm_pool_create(ctypes.byref(d), ctypes.byref(h)), h


@pytest.fixture
def pool(lib):
    st, h = fake_pool(lib)
    assert st == 0
    yield h
    assert lib.wkv7_pool_destroy(h) == 0


def test_pool_sizes_and_descriptions(lib, pool):
    states = 2 * 4 * 64 * 128 * 4
    tails = 512  # 2 layers of 3 x 40 bf16 values, 480 bytes, in whole 256
    assert lib.wkv7_ssm_pool_required_bytes(ctypes.byref(desc())) == 256 + 12 * (states + tails) + 256
    assert lib.wkv7_ssm_pool_required_bytes(ctypes.byref(desc(conv=(0, 0, 0)))) == 256 + 12 * states + 256
    assert lib.wkv7_ssm_pool_required_bytes(ctypes.byref(desc(state_dtype=1, conv=(40, 2, 0)))) == 256 + 12 * (states // 2 + 512) + 256
    for bad in (dict(n_groups=3), dict(n_layers=0), dict(n_heads=0), dict(state_dtype=2), dict(n_slots=0), dict(n_snapshots=-1),
                dict(out_dtype=-1), dict(conv=(12, 4, 0)), dict(conv=(16, 5, 0)), dict(conv=(16, 1, 0)), dict(conv=(16, 4, 2)),
                dict(conv=(-8, 4, 0))):
        assert lib.wkv7_ssm_pool_required_bytes(ctypes.byref(desc(**bad))) == 0
        assert fake_pool(lib, **bad)[0] == 1
    for bad in (dict(head_p=32), dict(d_state=256)):
        assert fake_pool(lib, **bad)[0] == 7
    assert lib.wkv7_slot_bytes(pool) == states + tails
    p = ctypes.c_void_p()
    assert lib.wkv7_pool_state_ptr(pool, 3, 1, ctypes.byref(p)) == 0
    assert p.value == X + 256 + 3 * (states + tails) + states // 2
    got, conv, at = wkv7.SsmPoolDesc(), wkv7.ConvDesc(), ctypes.c_size_t()
    assert lib.wkv7_ssm_pool_get_desc(pool, ctypes.byref(got)) == 0
    assert (got.n_heads, got.n_groups, got.d_state, got.device_buffer, got.conv.width) == (4, 2, 128, X, 4)
    assert lib.wkv7_pool_conv_desc(pool, ctypes.byref(conv), ctypes.byref(at)) == 0
    assert (conv.channels, conv.dtype, at.value) == (40, 1, states)
    for call in (lib.wkv7_pool_get_desc, lib.wkv7_gdn_pool_get_desc):
        assert call(pool, (wkv7.PoolDesc if call is lib.wkv7_pool_get_desc else wkv7.GdnPoolDesc)()) == 7


def test_gdn_pools_take_tails(lib):
    d = wkv7.GdnPoolDesc(2, 1, 2, 64, 64, 4, 2, None, 0, 0, 0)
    plain = lib.wkv7_gdn_pool_required_bytes(ctypes.byref(d))
    conv = wkv7.ConvDesc(64, 4, 0)
    assert lib.wkv7_gdn_pool_conv_required_bytes(ctypes.byref(d), None) == plain
    assert lib.wkv7_gdn_pool_conv_required_bytes(ctypes.byref(d), ctypes.byref(conv)) == plain + 6 * 2 * 3 * 64 * 4
    bad = wkv7.ConvDesc(63, 4, 0)
    assert lib.wkv7_gdn_pool_conv_required_bytes(ctypes.byref(d), ctypes.byref(bad)) == 0
    h = ctypes.c_void_p()
    d.device_buffer, d.buffer_bytes = X, plain
    assert lib.wkv7_gdn_pool_create_conv(ctypes.byref(d), ctypes.byref(conv), ctypes.byref(h)) == 1
    assert lib.wkv7_gdn_pool_create_conv(ctypes.byref(d), ctypes.byref(bad), ctypes.byref(h)) == 1
    assert lib.wkv7_gdn_pool_create(ctypes.byref(d), ctypes.byref(h)) == 0
    t = wkv7.ConvTokens(X, 64, 0, X, X, 1, X + 4096)
    assert lib.wkv7_conv_step(h, 0, X, 1, 1, ctypes.byref(t), None, None) == 7  # no tails
    assert lib.wkv7_ssm_decode_step(h, 0, X, 0, ctypes.byref(wkv7.SsmTokens()), None) == 7
    assert lib.wkv7_pool_destroy(h) == 0


def tokens(**kw):
    t = dict(in_dtype=1, dt_dtype=1, x=X, b=X, c=X, dt=X, a=X, d=X, dt_bias=X, x_stride=256, b_stride=256, c_stride=256,
             dt_stride=4, dt_softplus=1, o=X + 4096)
    t.update(kw)
    return ctypes.byref(wkv7.SsmTokens(**t))


BAD_TOKENS = [(dict(in_dtype=2), 1), (dict(dt_dtype=-1), 1), (dict(x=0), 1), (dict(a=0), 1), (dict(o=0), 1), (dict(x_stride=248), 1),
              (dict(b_stride=128), 1), (dict(dt_stride=3), 1), (dict(x=X + 8), 7), (dict(c=X + 2), 7), (dict(o=X + 4100), 7),
              (dict(o=X), 1), (dict(o=X + 496), 1), (dict(x=X + 4096 + 3 * 256 * 4 // 2), 1), (dict(dt=X + 1), 7), (dict(d=X + 2), 7), (dict(x_stride=257), 7), (dict(c_stride=260), 7)]


@pytest.mark.parametrize("bad,status", BAD_TOKENS)
def test_scan_refuses_tokens(lib, pool, bad, status):
    assert lib.wkv7_ssm_decode_step(pool, 0, X, 2, tokens(**bad), None) == status
    assert lib.wkv7_ssm_decode_multi(pool, 0, X, 1, 2, tokens(**bad), None, None) == status
    assert lib.wkv7_ssm_prefill(pool, 0, X, X, 1, 2, 2, tokens(**bad), None, 0, 0, None) == status


def test_scan_refuses_calls(lib, pool):
    t = tokens()
    assert lib.wkv7_ssm_decode_step(None, 0, X, 1, t, None) == 1
    for layer, n in ((2, 1), (-1, 1), (0, -1), (0, 9)):
        assert lib.wkv7_ssm_decode_step(pool, layer, X, n, t, None) == 1
        assert lib.wkv7_ssm_decode_multi(pool, layer, X, n, 1, t, None, None) == 1
        assert lib.wkv7_ssm_prefill(pool, layer, X, X, n, 4, 4, t, None, 0, 0, None) == 1
    assert lib.wkv7_ssm_decode_step(pool, 0, None, 1, t, None) == 1
    assert lib.wkv7_ssm_decode_step(pool, 0, X, 1, None, None) == 1
    assert lib.wkv7_ssm_decode_step(pool, 0, None, 0, t, None) == 0
    assert lib.wkv7_ssm_decode_multi(pool, 0, X, 1, 0, t, None, None) == 1
    assert lib.wkv7_ssm_decode_multi(pool, 0, X, 8, 2 ** 30, t, None, None) == 1
    assert lib.wkv7_ssm_prefill(pool, 0, X, X, 1, 4, 5, t, None, 0, 0, None) == 5
    assert lib.wkv7_ssm_prefill(pool, 0, X, X, 1, 2 ** 31 - 1, 5, t, None, 0, 0, None) == 1
    assert lib.wkv7_ssm_prefill(pool, 0, X, None, 1, 4, 4, t, None, 0, 0, None) == 1
    assert lib.wkv7_ssm_prefill(pool, 0, X, X, 1, 4, 4, t, X + 8, 64, 0, None) == 7
    assert lib.wkv7_ssm_prefill(pool, 0, None, None, 0, 0, 0, t, None, 0, 0, None) == 0
    st, none = fake_pool(lib, n_snapshots=0)
    assert st == 0 and lib.wkv7_ssm_decode_multi(none, 0, X, 1, 1, t, X, None) == 1
    assert lib.wkv7_pool_destroy(none) == 0
    for name, args in (("wkv7_decode_step", (0, X, 1, 0) + (X,) * 7), ("wkv7_prefill", (0, X, X, 1, 4, 4, 1) + (X,) * 7)):
        assert getattr(lib, name)(pool, *args, None) == 7
    assert lib.wkv7_gdn_decode_step(pool, 0, X, 1, ctypes.byref(wkv7.GdnTokens()), None) == 7
    assert lib.wkv7_gdn_prefill_workspace_bytes(pool, 8, 4096) == 0


def conv_tokens(**kw):
    t = dict(x=X, x_stride=40, weight_dtype=1, weight=X, bias=X, activation=1, o=X + 4096)
    t.update(kw)
    return ctypes.byref(wkv7.ConvTokens(**t))


@pytest.mark.parametrize("bad,status", [(dict(weight_dtype=2), 1), (dict(activation=2), 1), (dict(x=0), 1), (dict(weight=0), 1),
                                        (dict(o=0), 1), (dict(x_stride=32), 1), (dict(x=X + 8), 7), (dict(weight=X + 8), 7),
                                        (dict(bias=X + 2), 7), (dict(o=X + 4104), 7), (dict(x_stride=44), 7), (dict(o=X), 1),
                                        (dict(o=X + 144), 1), (dict(x=X + 4096 + 144), 1), (dict(x_stride=4096, x=X - 8192 + 4096), 1)])
def test_conv_refuses_tokens(lib, pool, bad, status):
    assert lib.wkv7_conv_step(pool, 0, X, 2, 1, conv_tokens(**bad), None, None) == status
    assert lib.wkv7_conv_prefill(pool, 0, X, X, 1, 2, conv_tokens(**bad), None) == status


def test_conv_refuses_calls(lib, pool):
    t = conv_tokens()
    for layer, n in ((2, 1), (-1, 1), (0, -1), (0, 9)):
        assert lib.wkv7_conv_step(pool, layer, X, n, 1, t, None, None) == 1
        assert lib.wkv7_conv_prefill(pool, layer, X, X, n, 2, t, None) == 1
    assert lib.wkv7_conv_step(pool, 0, None, 1, 1, t, None, None) == 1
    assert lib.wkv7_conv_step(pool, 0, X, 1, 0, t, None, None) == 1
    assert lib.wkv7_conv_prefill(pool, 0, X, None, 1, 2, t, None) == 1
    assert lib.wkv7_conv_step(pool, 0, None, 0, 1, t, None, None) == 0
    assert lib.wkv7_conv_prefill(pool, 0, None, None, 3, 0, t, None) == 0


def norm_args(**kw):
    a = dict(rows=3, width=64, group=32, x_dtype=1, z_dtype=1, w_dtype=1, o_dtype=1, kind=0, act=1, gate_first=0, eps=1e-5, x=X,
             x_stride=64, z=X, z_stride=64, weight=X, bias=0, o=X + 4096)
    a.update(kw)
    return ctypes.byref(wkv7.NormArgs(**a))


@pytest.mark.parametrize("bad,status", [(dict(rows=-1), 1), (dict(group=24), 1), (dict(group=0), 1), (dict(width=0), 1), (dict(kind=2), 1),
                                        (dict(act=3), 1), (dict(x_dtype=2), 1), (dict(o_dtype=3), 1), (dict(eps=-1.0), 1),
                                        (dict(eps=float("inf")), 1), (dict(x=0), 1), (dict(o=0), 1), (dict(x_stride=56), 1),
                                        (dict(z_stride=1), 1), (dict(group=4), 7), (dict(width=32776, group=32776), 7),
                                        (dict(x=X + 2), 7), (dict(z=X + 4), 7), (dict(weight=X + 8), 7), (dict(x_stride=68), 7),
                                        (dict(o=X), 1), (dict(o=X + 368), 1)])
def test_norm_refuses(lib, bad, status):
    assert lib.wkv7_gated_norm(norm_args(**bad), None) == status


def test_norm_of_nothing(lib):
    assert lib.wkv7_gated_norm(None, None) == 1
    assert lib.wkv7_gated_norm(norm_args(rows=0), None) == 0


def test_oracle_agrees_with_other_forms():
    """The recurrence against its unrolled sum, the convolution against a direct sum, and tails and
    states that carry over a cut."""
    rng = np.random.default_rng(0)
    T, h, g, p, n = 9, 4, 2, 3, 5
    x, dt, B, C = rng.standard_normal((T, h, p)), rng.random((T, h)), rng.standard_normal((T, g, n)), rng.standard_normal((T, g, n))
    A, S0, D = -rng.random(h), rng.standard_normal((h, p, n)), rng.standard_normal(h)
    o, S, states = scan_run(S0, x, dt, A, B, C, D, keep=True)
    L = np.cumsum(dt * A, 0)
    for hh in range(h):
        gg = hh // 2
        for t in range(T):
            want = np.exp(L[t, hh]) * S0[hh] @ C[t, gg] + D[hh] * x[t, hh]
            for s in range(t + 1):
                want += np.exp(L[t, hh] - L[s, hh]) * dt[s, hh] * x[s, hh] * (B[s, gg] @ C[t, gg])
            assert np.allclose(o[t, hh], want)
    o2, S2, _ = scan_run(states[4], x[4:], dt[4:], A, B[4:], C[4:], D)
    assert np.allclose(o2, o[4:]) and np.allclose(S2, S)
    u, w, b, tail = rng.standard_normal((6, 8)), rng.standard_normal((8, 4)), rng.standard_normal(8), rng.standard_normal((3, 8))
    y, new = conv_run(tail, u, w, b, None)
    line = np.concatenate([tail, u])
    assert np.allclose(y[2], b + sum(w[:, j] * line[2 + j] for j in range(4))) and np.array_equal(new, u[3:])
    assert np.array_equal(conv_run(tail, u[:1], w, b)[1], np.concatenate([tail[1:], u[:1]]))
    r = gated_norm(u, group=4, eps=0.0, kind="layer")
    assert np.allclose(r.reshape(6, 2, 4).mean(-1), 0) and np.allclose((r.reshape(6, 2, 4) ** 2).mean(-1), 1)
