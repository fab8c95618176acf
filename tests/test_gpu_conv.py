"""The short causal convolution over state slots against the float64 formula, its edges and refusals."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from oracle.ssm import conv_run
from rwkv_wkv_gb300 import DEV_BAD_SEQLENS, DEV_BAD_SLOT, GdnPool, SsmPool, Wkv7Error
from ssm_helpers import EPS32, check, host

pytestmark = pytest.mark.gpu


def make(ch, width, slots, snaps=0, layers=2, dtype="bf16", kind="ssm"):
    more = dict(n_snapshots=snaps, conv_channels=ch, conv_width=width, conv_dtype=dtype)
    pool = SsmPool(layers, 1, 1, slots, d_state=64, **more) if kind == "ssm" else \
        GdnPool(layers, 1, 2, slots, head_k=64, head_v=64, state_dtype="bf16", **more)
    gen = torch.Generator(device="cuda").manual_seed(ch + width)
    pool.conv_tails.copy_(torch.randn(pool.conv_tails.shape, device="cuda", generator=gen))
    pool.states.fill_(2)
    return pool


def inputs(seed, rows, ch, width, dtype, wdtype=None, bias=True):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, ch + 24, generator=gen).to(dtype).cuda()[:, 16:16 + ch]
    w = torch.randn(ch, width, generator=gen).to(wdtype or dtype).cuda()
    b = torch.randn(ch, generator=gen).to(wdtype or dtype).cuda() if bias else None
    return x, w, b


def compare(o, tail, x, w, b, activation="silu"):
    """Sums of width + 1 terms, half a step each, then x / (1 + e^-x): of slope below 1.1, from a
    2^x and a reciprocal of a unit in the last place or two and an exponent rounded at most 2^-24 |x|."""
    want, _ = conv_run(host(tail), host(x), host(w), host(b), activation)
    size, _ = conv_run(np.abs(host(tail)), np.abs(host(x)), np.abs(host(w)), None if b is None else np.abs(host(b)), None)
    check(o, want, size, 1.1 * (w.shape[-1] + 1) * EPS32 + 12 * EPS32, o.dtype, floor=np.abs(want) * size * 2 * EPS32)


KINDS = [("bf16", torch.bfloat16, None), ("f32", torch.float32, None), ("bf16", torch.bfloat16, torch.float32)]


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("ch", [8, 72, 1100 * 8])
def test_step(ch, width, kind):
    name, dtype, wdtype = kind
    with make(ch, width, 5, dtype=name) as pool:
        tails = pool.conv_tails.clone()
        x, w, b = inputs(1, 3, ch, width, dtype, wdtype)
        o = pool.conv_step(1, i32([4, 0, 2]), x, w, b)
        for i, s in enumerate([4, 0, 2]):
            compare(o[i:i + 1], tails[s, 1], x[i:i + 1], w, b)
            assert torch.equal(pool.conv_tails[s, 1], torch.cat([tails[s, 1, 1:], x[i:i + 1]]))
        assert torch.equal(pool.conv_tails[:, 0], tails[:, 0]) and torch.equal(pool.conv_tails[[1, 3]], tails[[1, 3]])
        assert (pool.states == 2).all() and pool.device_status() == 0


LENGTHS = [[1], [2, 1, 3, 0, 1, 4], [7, 8, 9, 1, 1, 30], [33, 31, 32, 2, 64, 5], [0, 0, 100], [700]]


# (the wide ones take the long tiles: one type and the shorter batches are enough)
SIZES = [(72, kind, lens) for kind in KINDS[:2] for lens in LENGTHS] + [(152 * 1024, KINDS[0], lens) for lens in LENGTHS[:-2]]


@pytest.mark.parametrize("ch,kind,lens", SIZES, ids=str)
@pytest.mark.parametrize("width", [2, 3, 4])
def test_prefill_is_steps(ch, width, kind, lens):
    """Outputs and tails of single steps, bit for bit."""
    name, dtype, _ = kind
    n = len(lens)
    with make(ch, width, 2 * n, layers=1, dtype=name) as pool:
        pool.conv_tails[n:] = pool.conv_tails[:n]
        x, w, b = inputs(2, sum(lens) + 3, ch, width, dtype)
        cu = np.concatenate([[0], np.cumsum(lens)])
        o = torch.full((sum(lens) + 3, ch), 7.0, device="cuda", dtype=dtype)
        pool.conv_prefill(0, i32(range(n)), i32(cu), x, w, b, o=o)
        assert (o[cu[-1]:] == 7).all()
        for t in range(max(lens)):
            alive = [s for s in range(n) if lens[s] > t]
            rows = [int(cu[s]) + t for s in alive]
            ot = pool.conv_step(0, i32([n + s for s in alive]), x[rows], w, b)
            assert torch.equal(o[rows], ot)
        assert torch.equal(pool.conv_tails[:n], pool.conv_tails[n:])
        assert pool.device_status() == 0


@pytest.mark.parametrize("activation", ["silu", None])
@pytest.mark.parametrize("bias", [True, False])
def test_prefill_values(bias, activation):
    ch, width, lens = 136, 4, [5, 90, 2]
    with make(ch, width, 3) as pool:
        tails = pool.conv_tails.clone()
        x, w, b = inputs(3, sum(lens), ch, width, torch.bfloat16, bias=bias)
        o = pool.conv_prefill(0, i32([2, 0, 1]), i32([0, 5, 95, 97]), x, w[:, None], b, activation)
        for (a, e), s in zip(((0, 5), (5, 95), (95, 97)), (2, 0, 1)):
            compare(o[a:e], tails[s, 0], x[a:e], w, b, activation)


def test_multi_keeps_every_tail():
    ch, width, n, K = 264, 4, 3, 6
    with make(ch, width, 2 * n, snaps=n * K) as pool:
        pool.conv_tails[n:] = pool.conv_tails[:n]
        pool.snapshots.fill_(5)
        x, w, b = inputs(4, n * K, ch, width, torch.bfloat16)
        x = x.unflatten(0, (n, K))
        snaps = i32(np.random.default_rng(1).permutation(n * K).reshape(n, K))
        o = pool.conv_multi(1, i32(range(n)), x, w, b, step_snap_ids=snaps)
        for t in range(K):
            assert torch.equal(o[:, t], pool.conv_step(1, i32(range(n, 2 * n)), x[:, t], w, b))
            assert torch.equal(pool.conv_snapshots[snaps[:, t].long(), 1], pool.conv_tails[n:, 1])
        assert torch.equal(pool.conv_tails[:n], pool.conv_tails[n:])
        assert (pool.snapshots == 5).all()
        snaps[1, 2] = n * K
        pool.conv_multi(1, i32(range(n)), x, w, b, step_snap_ids=snaps)
        assert pool.device_status() == DEV_BAD_SLOT


@pytest.mark.parametrize("kind", ["ssm", "gdn"])
def test_verbs_move_tails_with_states(kind):
    with make(40, 3, 4, snaps=2, kind=kind) as pool:
        pool.states[2].fill_(9)
        pool.snapshot(i32([2]), i32([1]))
        assert torch.equal(pool.conv_snapshots[1], pool.conv_tails[2]) and (pool.snapshots[1] == 9).all()
        pool.fork(i32([2]), i32([0]))
        assert torch.equal(pool.conv_tails[0], pool.conv_tails[2]) and (pool.states[0] == 9).all()
        kept = pool.conv_tails[2].clone()
        image = torch.empty(pool.slot_bytes, dtype=torch.uint8).pin_memory()
        pool.hibernate(i32([2]), image)
        pool.reset(i32([2]))
        assert not pool.conv_tails[2].any() and not pool.states[2].any()
        pool.resume(image, i32([2]))
        assert torch.equal(pool.conv_tails[2], kept)
        pool.reset(i32([2]))
        pool.restore(i32([1]), i32([2]))
        assert torch.equal(pool.conv_tails[2], kept) and (pool.states[2] == 9).all()
        x, w, b = inputs(5, 2, 40, 3, torch.bfloat16)
        pool.conv_step(1, i32([1, 3]), x, w, b)
        assert (pool.states[1] == 2).all() and torch.equal(pool.conv_tails[1, 1, 1], x[0])
        assert pool.device_status() == 0


def test_gdn_with_tails_computes_what_it_did():
    """A pool with tails behind its states gives the bits of one without."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (torch.randn(150, h, 64, device="cuda", generator=gen).to(torch.bfloat16) for h in (1, 1, 2))
    g, beta = -torch.rand(150, 2, device="cuda", generator=gen), torch.rand(150, 2, device="cuda", generator=gen)
    got = []
    for ch in (0, 24):
        with GdnPool(2, 1, 2, 3, head_k=64, head_v=64, conv_channels=ch) as pool:
            pool.states.fill_(0.25)
            o = pool.prefill(1, i32([2, 0]), i32([0, 100, 149]), q, k, v, g, beta, max_seqlen=100, l2norm_eps=1e-6)
            o2 = pool.decode_step(0, i32([2]), q[149:], k[149:], v[149:], g[149:], beta[149:])
            got.append((o[:149].clone(), o2, pool.states.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_bad_ids_and_lengths():
    with make(32, 4, 3) as pool:
        before = pool.conv_tails.clone()
        x, w, b = inputs(7, 90, 32, 4, torch.bfloat16)
        for cu in ([0, 50, 40, 90], [0, 30, 60, 91], [-1, 30, 60, 90], [0, 95, 60, 90]):
            o = torch.full((90, 32), 7.0, device="cuda", dtype=torch.bfloat16)
            pool.conv_prefill(0, i32([0, 1, 2]), i32(cu), x, w, b, o=o)
            assert pool.device_status() == DEV_BAD_SEQLENS
            assert (o == 7).all() and torch.equal(pool.conv_tails, before)
        o = torch.full((90, 32), 7.0, device="cuda", dtype=torch.bfloat16)
        pool.conv_prefill(0, i32([0, 3, -1]), i32([0, 30, 60, 90]), x, w, b, o=o)
        assert pool.device_status() == DEV_BAD_SLOT
        assert (o[30:] == 7).all() and not (o[:30] == 7).all() and torch.equal(pool.conv_tails[1:], before[1:])
        pool.conv_step(0, i32([3]), x[:1], w, b)
        assert pool.device_status() == DEV_BAD_SLOT


def test_refusals():
    with make(32, 4, 3) as pool:
        x, w, b = inputs(8, 3, 32, 4, torch.bfloat16)
        ids = i32([0, 1, 2])
        for args in ((x.float(), w, b), (x, w[:, :3], b), (x, w, b.float()), (x[:2], w, b), (x, w.half(), b), (x, w.t().contiguous().t(), b)):
            with pytest.raises((TypeError, ValueError)):
                pool.conv_step(0, ids, *args)
        with pytest.raises(ValueError):
            pool.conv_step(0, ids, x, w, b, activation="relu")
        with pytest.raises(Wkv7Error, match="INVALID_ARG"):
            pool.conv_step(2, ids, x, w, b)
        whole = torch.zeros(3, 32, device="cuda", dtype=torch.bfloat16)
        with pytest.raises(Wkv7Error, match="INVALID_ARG"):
            pool.conv_step(0, ids, whole, w, b, o=whole)
        with pytest.raises(Wkv7Error, match="UNSUPPORTED"):
            pool.conv_step(0, ids, torch.zeros(3, 36, device="cuda", dtype=torch.bfloat16)[:, 4:], w, b)
    for bad in (dict(conv_channels=12), dict(conv_channels=16, conv_width=5), dict(conv_channels=-8), dict(conv_channels=16, conv_width=1)):
        with pytest.raises(Wkv7Error):
            SsmPool(1, 1, 1, 1, **bad)
