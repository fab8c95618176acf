"""GPU parity of the gated delta rule over state slots (wkv7_gdn_*) with the float64
oracle: decode, multi-token decode with rollback states, prefill by chunks and token by
token, over head sizes, shared heads, types, strides and lengths.

Tolerances, normwise-max relative to the oracle.  A float32 step of n = head_k terms has a
relative error of at most about (n + 8) 2^-24 < 1e-5 per token against the largest entry,
and the rule contracts earlier errors (exp(g) <= 1, beta <= 1, unit keys), so F32_TOL =
2e-5 covers the runs here.  The chunked path's operands carry 16 bits (two bf16 parts,
2^-17 each) through four products in a row: 4 x 2^-17 < CHUNK_TOL = 4e-5.  A bf16 value
adds half its spacing, 2^-9, to either: BF16_TOL = 2^-8.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import i32
from oracle.gdn import gdn_run
from rwkv_wkv_gb300 import (DEV_BAD_SEQLENS, DEV_BAD_SLOT, DEV_WAIT_TIMEOUT, GdnPool, Pool, Wkv7Error,
                            load_library)

pytestmark = pytest.mark.gpu

F32_TOL, CHUNK_TOL, BF16_TOL = 2e-5, 4e-5, 2.0 ** -8
EPS = 1e-6
HEADS = [(2, 4, 128, 128), (3, 3, 64, 64), (1, 3, 128, 64), (2, 2, 64, 128)]
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(rng, rows, heads, dtype="bf16", g=None, beta=None, scale_k=1.0):
    """Host values, exact in `dtype`, and device tensors that are column ranges of one buffer."""
    hk, hv, dk, dv = heads
    qkv = torch.from_numpy(rng.standard_normal((rows, 2 * hk * dk + hv * dv)).astype(np.float32) * 0.7 + 0.15)
    qkv[:, hk * dk:2 * hk * dk] *= scale_k
    qkv = qkv.to(DT[dtype]).cuda()
    q = qkv[:, :hk * dk].unflatten(1, (hk, dk))
    k = qkv[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk))
    v = qkv[:, 2 * hk * dk:].unflatten(1, (hv, dv))
    gb = torch.empty(rows, 2 * hv + 1, device="cuda")   # gates at an odd stride
    g = -np.exp(rng.standard_normal((rows, hv)) - 1.5) if g is None else np.broadcast_to(g, (rows, hv))
    beta = 1 / (1 + np.exp(-rng.standard_normal((rows, hv)))) if beta is None else np.broadcast_to(beta, (rows, hv))
    gb[:, :hv] = torch.from_numpy(np.ascontiguousarray(g, dtype=np.float32))
    gb[:, hv:2 * hv] = torch.from_numpy(np.ascontiguousarray(beta, dtype=np.float32))
    dev = [q, k, v, gb[:, :hv], gb[:, hv:2 * hv]]
    return dev, [x.float().cpu().numpy().astype(np.float64) for x in dev]


def start(rng, slots, heads, dtype="f32"):
    hk, hv, dk, dv = heads
    return torch.from_numpy(rng.standard_normal((slots, 1, hv, dv, dk)).astype(np.float32) * 0.1).to(DT[dtype])


def host(x):
    return x.float().cpu().numpy().astype(np.float64)


def err(x, ref):
    return oracle.rel_err(host(x), ref)


def tol_of(base, dtype):
    return BF16_TOL if dtype == "bf16" else base


def bf16_round(S):
    return torch.from_numpy(S).to(torch.float32).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("state,inputs,out", [("f32", "bf16", "f32"), ("f32", "f32", "bf16"), ("bf16", "bf16", "f32"),
                                              ("bf16", "f32", "bf16")])
@pytest.mark.parametrize("eps", [EPS, 0.0])
def test_decode(heads, state, inputs, out, eps):
    rng = np.random.default_rng(1)
    hk, hv, dk, dv = heads
    n, slots = 5, 9
    dev, hst = make(rng, n, heads, inputs, scale_k=1.0 if eps else 0.1)
    S0 = start(rng, slots, heads, state)
    ids = rng.permutation(slots)[:n]
    with GdnPool(1, hk, hv, slots, head_k=dk, head_v=dv, state_dtype=state, out_dtype=out) as pool:
        pool.states.copy_(S0)
        o = pool.decode_step(0, i32(ids), *dev, l2norm_eps=eps or None)
        assert pool.device_status() == 0
        assert o.dtype == DT[out]
        S = host(pool.states)
    rest = np.setdiff1d(np.arange(slots), ids)
    assert np.array_equal(S[rest], host(S0)[rest])
    for b in range(n):
        o_ref, S_ref, _ = gdn_run(host(S0)[ids[b], 0], *[x[b:b + 1] for x in hst], dk ** -0.5, eps)
        assert err(o[b], o_ref[0]) < tol_of(F32_TOL, out)
        assert oracle.rel_err(S[ids[b], 0], S_ref) < tol_of(F32_TOL, state)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 5, 16, 37])
@pytest.mark.parametrize("snaps", [False, True])
def test_decode_multi(heads, state, K, snaps):
    rng = np.random.default_rng(2)
    hk, hv, dk, dv = heads
    n, slots = 3, 4
    dev, hst = make(rng, n * K, heads)
    S0 = start(rng, slots, heads, state)
    ids = np.array([2, 0, 3])
    order = rng.permutation(n * K)
    with GdnPool(1, hk, hv, slots, n_snapshots=n * K, head_k=dk, head_v=dv, state_dtype=state) as pool:
        pool.states.copy_(S0)
        o = pool.decode_multi(0, i32(ids), *[x.unflatten(0, (n, K)) for x in dev], l2norm_eps=EPS, scale=0.3,
                              step_snap_ids=i32(order.reshape(n, K)) if snaps else None)
        assert pool.device_status() == 0
        S, kept = host(pool.states), host(pool.snapshots)
    for b in range(n):
        o_ref, S_ref, every = gdn_run(host(S0)[ids[b], 0], *[x[b * K:(b + 1) * K] for x in hst], 0.3, EPS, True,
                                      bf16_round if state == "bf16" else None)
        # a bf16 pool rounds after every token: one spacing of each step's rounding may fall the other way
        assert err(o[b], o_ref) < (BF16_TOL if state == "bf16" else F32_TOL)
        assert oracle.rel_err(S[ids[b], 0], S_ref) < (BF16_TOL if state == "bf16" else F32_TOL)
        if snaps:
            got = kept[order.reshape(n, K)[b], 0]
            assert oracle.rel_err(got, every) < (BF16_TOL if state == "bf16" else F32_TOL)
            assert np.array_equal(got[-1], S[ids[b], 0])


def run_prefill(heads, lens, state="f32", out="f32", inputs="bf16", sequential=False, eps=EPS, seed=3, ckpt=False, **kw):
    rng = np.random.default_rng(seed)
    hk, hv, dk, dv = heads
    lens = np.asarray(lens)
    n, slots = len(lens), len(lens) + 2
    cu = np.concatenate([[0], np.cumsum(lens)])
    dev, hst = make(rng, int(cu[-1]), heads, inputs, **kw)
    S0 = start(rng, slots, heads, state)
    ids = rng.permutation(slots)[:n]
    cks = np.concatenate([[0], np.cumsum(lens // 64)])
    with GdnPool(1, hk, hv, slots, n_snapshots=max(1, int(cks[-1])), head_k=dk, head_v=dv, state_dtype=state,
                 out_dtype=out) as pool:
        pool.states.copy_(S0)
        pool.snapshots.zero_()
        o = pool.prefill(0, i32(ids), i32(cu), *dev, l2norm_eps=eps or None, sequential=sequential,
                         max_seqlen=int(lens.max()) if n else 0,
                         **(dict(cu_ckpt=i32(cks), ckpt_ids=i32(np.arange(cks[-1])[::-1].copy())) if ckpt else {}))
        assert pool.device_status() == 0
        S, kept = host(pool.states), host(pool.snapshots)
    rest = np.setdiff1d(np.arange(slots), ids)
    assert np.array_equal(S[rest], host(S0)[rest])
    ref = [gdn_run(host(S0)[ids[i], 0], *[x[cu[i]:cu[i + 1]] for x in hst], dk ** -0.5, eps, ckpt) for i in range(n)]
    return o, S[ids, 0], ref, cu, host(S0)[ids, 0], kept, cks


def check_prefill(got, base, state="f32", out="f32"):
    o, S, ref, cu, S0 = got[:5]
    for i, (o_ref, S_ref, _) in enumerate(ref):
        if cu[i] == cu[i + 1]:
            assert np.array_equal(S[i], S0[i])
            continue
        assert err(o[cu[i]:cu[i + 1]], o_ref) < tol_of(base, out), i
        assert oracle.rel_err(S[i], S_ref) < tol_of(base, state), i


LENS = [[1], [0, 2, 0], [63, 64, 65], [128, 1, 200, 0, 17], [257]]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("state,out", [("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("sequential", [False, True])
def test_prefill(heads, lens, state, out, sequential):
    got = run_prefill(heads, lens, state, out, sequential=sequential)
    check_prefill(got, F32_TOL if sequential else CHUNK_TOL, state, out)


@pytest.mark.parametrize("heads", HEADS[:2])
def test_prefill_f32_inputs(heads):
    check_prefill(run_prefill(heads, [70, 3], inputs="f32"), F32_TOL)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("what", ["no decay", "strong decay", "emptied state", "beta 0", "beta 1", "raw keys"])
def test_prefill_gates(heads, what):
    """Gates at the ends of their range, over lengths of several chunks and a ragged end."""
    hv, kw, eps = heads[1], {}, EPS
    total = 64 * 3 + 5
    if what == "no decay":
        kw["g"] = 0.0
    elif what == "strong decay":  # a chunk's total far beyond float32's range, with weak tokens after it
        g = np.full((total, hv), -0.01)
        g[10:40] = -30.0
        g[100] = -700.0
        kw["g"] = g
    elif what == "emptied state":  # exp(g) = 0 at a chunk's start, inside one, twice in a row, and at its end
        g = np.full((total, hv), -0.05)
        g[[0, 20, 21, 64, 127, 150]] = -np.inf
        kw["g"] = g
    elif what == "beta 0":
        kw["beta"] = 0.0
    elif what == "beta 1":
        kw["beta"] = 1.0
    else:
        eps, kw["scale_k"] = 0.0, 0.08
    with np.errstate(invalid="ignore"):
        got = run_prefill(heads, [total], eps=eps, **kw)
    check_prefill(got, CHUNK_TOL)


def test_prefill_like_keys():
    """Keys that hardly differ: the chunk's triangular system at its worst conditioning."""
    rng = np.random.default_rng(9)
    hk, hv, dk, dv = heads = (1, 2, 128, 128)
    dev, _ = make(rng, 200, heads, g=-0.001, beta=0.9)
    dev[1].copy_((1.0 + 0.02 * torch.randn(200, hk, dk, device="cuda")).to(torch.bfloat16))
    hst = [host(x) for x in dev]
    S0 = start(rng, 1, heads)
    with GdnPool(1, hk, hv, 1) as pool:
        pool.states.copy_(S0)
        o = pool.prefill(0, i32([0]), i32([0, 200]), *dev, l2norm_eps=EPS)
        S = host(pool.states[0, 0])
    o_ref, S_ref, _ = gdn_run(host(S0)[0, 0], *hst, dk ** -0.5, EPS)
    assert err(o, o_ref) < CHUNK_TOL and oracle.rel_err(S, S_ref) < CHUNK_TOL


def test_prefill_zero_and_empty_rows():
    """Keys and queries of zeros (a padded row): no NaN, and the state only decays."""
    heads = (1, 1, 64, 64)
    rng = np.random.default_rng(10)
    for sequential in (False, True):
        dev, _ = make(rng, 70, heads)
        dev[0].zero_()
        dev[1].zero_()
        S0 = start(rng, 1, heads)
        with GdnPool(1, 1, 1, 1, head_k=64, head_v=64) as pool:
            pool.states.copy_(S0)
            o = pool.prefill(0, i32([0]), i32([0, 70]), *dev, l2norm_eps=EPS, sequential=sequential)
            S = host(pool.states[0, 0])
        assert torch.equal(o, torch.zeros_like(o))
        assert oracle.rel_err(S, host(S0)[0, 0] * np.exp(host(dev[3]).sum())) < F32_TOL


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("sequential", [False, True])
@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_checkpoints_resume_bit_for_bit(heads, sequential, state):
    lens = [130, 64, 20, 250]
    o, S, ref, cu, S0, kept, cks = run_prefill(heads, lens, state, sequential=sequential, ckpt=True)
    for i in range(len(lens)):
        for m in range(cks[i], cks[i + 1]):
            at = 64 * (m - cks[i] + 1)
            got = kept[cks[-1] - 1 - m, 0]
            assert oracle.rel_err(got, ref[i][2][at - 1]) < tol_of(CHUNK_TOL, state)
            if at == lens[i]:
                assert np.array_equal(got, S[i])
    # resume sequence 3 after 128 tokens
    hk, hv, dk, dv = heads
    rng = np.random.default_rng(3)
    dev, _ = make(rng, int(cu[-1]), heads)
    tail = [x[cu[3] + 128:cu[4]] for x in dev]
    tail = [x.clone() if j < 3 else x for j, x in enumerate(tail)]  # q, k, v at another stride
    with GdnPool(1, hk, hv, 1, n_snapshots=1, head_k=dk, head_v=dv, state_dtype=state) as pool:
        pool.snapshots[0, 0].copy_(torch.from_numpy(kept[cks[-1] - 1 - (cks[3] + 1), 0]))
        pool.restore(i32([0]), i32([0]))
        o2 = pool.prefill(0, i32([0]), i32([0, 122]), *tail, l2norm_eps=EPS, sequential=sequential,
                          cu_ckpt=i32([0, 1]), ckpt_ids=i32([0]))
        assert pool.device_status() == 0
        assert torch.equal(o2, o[cu[3] + 128:cu[4]])
        assert np.array_equal(host(pool.states[0, 0]), S[3])


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", [[3000], [2500, 1, 0, 64 * 23, 700]])
@pytest.mark.parametrize("state,out", [("f32", "f32"), ("bf16", "bf16")])
def test_prefill_cut_into_segments(heads, lens, state, out):
    """Long sequences of few heads: the library cuts them and joins the states in float32 (one
    more product in a row than the uncut path's four: CHUNK_TOL holds for the start of each
    segment, and the rule contracts it)."""
    hk, hv, dk, dv = heads
    with GdnPool(1, hk, hv, len(lens), head_k=dk, head_v=dv) as pool:
        assert pool._lib.wkv7_gdn_prefill_workspace_bytes(pool._h, len(lens), max(lens)) > 0
    check_prefill(run_prefill(heads, lens, state, out, seed=12), CHUNK_TOL, state, out)


def test_cut_prefill_with_weak_and_strong_decay():
    """Segments whose transition hardly contracts, and segments that empty the state."""
    heads = (1, 2, 128, 128)
    total = 2048 + 37
    for g in (np.full((total, 2), -1e-4), np.full((total, 2), -0.02), np.full((total, 2), -0.02)):
        if g[0, 0] == -0.02:
            g[700:702] = -np.inf
            g[1500] = -300.0
        with np.errstate(invalid="ignore"):
            check_prefill(run_prefill(heads, [total], g=g, seed=13), CHUNK_TOL)


@pytest.mark.parametrize("heads,n,state,out", [(HEADS[0], 40, "f32", "bf16"), (HEADS[1], 60, "bf16", "f32"),
                                               (HEADS[3], 100, "f32", "f32")])
def test_pieces_change_no_bit(heads, n, state, out):
    """More units than SMs: sequences that CTAs hand on to later ones, against the same call
    without a workspace; lengths of every piece, at and beside its ends, with checkpoints."""
    hk, hv, dk, dv = heads
    rng = np.random.default_rng(18)
    lens = rng.choice([2070, 2070, 2070, 1344, 1345, 1280, 1856, 1857, 1984, 64, 0, 1], n)  # pieces end at 1,344 and 1,856
    lens[:3] = [2070, 1345, 0]
    cu = np.concatenate([[0], np.cumsum(lens)])
    cks = np.concatenate([[0], np.cumsum(lens // 64)])
    total = int(cu[-1])
    dev, hst = make(rng, total, heads)
    S0 = start(rng, n, heads, state)
    ids = rng.permutation(n)
    with GdnPool(1, hk, hv, n, n_snapshots=int(cks[-1]), head_k=dk, head_v=dv, state_dtype=state, out_dtype=out) as pool:
        assert pool._lib.wkv7_gdn_prefill_workspace_bytes(pool._h, n, 2070) == n * hv * (dk * dv + 1) * 4
        for ckpt in (False, True):
            kw = dict(cu_ckpt=i32(cks), ckpt_ids=i32(np.arange(cks[-1]))) if ckpt else {}
            got = []
            for bare in (False, True):
                pool.states.copy_(S0)
                pool.snapshots.zero_()
                if bare:
                    t, o = pool._tokens((total,), *dev, None, None, EPS, None)
                    ptrs = [kw[k].data_ptr() if ckpt else None for k in ("cu_ckpt", "ckpt_ids")]
                    at, cut = i32(ids), i32(cu)
                    assert pool._lib.wkv7_gdn_prefill(pool._h, 0, at.data_ptr(), cut.data_ptr(), n, total, 2070, t, *ptrs,
                                                      None, 0, 0, torch.cuda.current_stream().cuda_stream) == 0
                else:
                    o = pool.prefill(0, i32(ids), i32(cu), *dev, l2norm_eps=EPS, max_seqlen=2070, **kw)
                assert pool.device_status() == 0
                got.append((o, pool.states.clone(), pool.snapshots.clone()))
            assert all(torch.equal(x, y) for x, y in zip(*got))
        o, S = got[0][0], host(got[0][1])
    for i in range(2):
        o_ref, S_ref, _ = gdn_run(host(S0)[ids[i], 0], *[x[cu[i]:cu[i + 1]] for x in hst], dk ** -0.5, EPS)
        if state == "f32":  # (with bf16 states a checkpointed carry goes on from the rounded state)
            assert err(o[cu[i]:cu[i + 1]], o_ref) < tol_of(CHUNK_TOL, out)
            assert oracle.rel_err(S[ids[i], 0], S_ref) < CHUNK_TOL
    assert np.array_equal(S[ids[2]], host(S0)[ids[2]])


@pytest.mark.parametrize("n", [512, 600])   # as many as are put in order, and more
def test_many_sequences(n):
    heads = HEADS[1]
    lens = np.random.default_rng(19).integers(0, 90, n)
    lens[5] = 90
    check_prefill(run_prefill(heads, lens, seed=20), CHUNK_TOL)


def test_cut_and_uncut_agree():
    heads = (2, 4, 128, 128)
    rng = np.random.default_rng(14)
    dev, _ = make(rng, 4000, heads)
    S0 = start(rng, 2, heads).cuda()
    with GdnPool(1, 2, 4, 2, n_snapshots=100) as pool:
        pool.states.copy_(S0)
        a = pool.prefill(0, i32([0]), i32([0, 4000]), *dev, l2norm_eps=EPS)
        sa = pool.states.clone()
        pool.states.copy_(S0)
        b = pool.prefill(0, i32([0]), i32([0, 4000]), *dev, l2norm_eps=EPS, cu_ckpt=i32([0, 62]),
                         ckpt_ids=i32(np.arange(62)))   # checkpointed: not cut
        assert err(a, host(b)) < CHUNK_TOL and err(sa, host(pool.states)) < CHUNK_TOL
        pool.states.copy_(S0)
        assert torch.equal(a, pool.prefill(0, i32([0]), i32([0, 4000]), *dev, l2norm_eps=EPS))


@pytest.mark.parametrize("heads,n,longest", [(HEADS[0], 1, 16), (HEADS[1], 2, 16), (HEADS[1], 60, 32),
                                             (HEADS[0], 40, 12)])
def test_short_prefill_runs_token_by_token(heads, n, longest):
    """Up to the rule's length a call is the token-by-token one, bit for bit; above it, and
    at any length in a checkpointed call, it is the chunked one.  All agree with the oracle."""
    for T in (longest - 1, longest, longest + 1):
        auto = run_prefill(heads, [T] * n, "bf16", out="f32", seed=15)
        by_token = run_prefill(heads, [T] * n, "bf16", out="f32", seed=15, sequential=True)
        in_chunks = run_prefill(heads, [T] * n, "bf16", out="f32", seed=15, ckpt=True)
        check_prefill(auto, CHUNK_TOL, "bf16")
        same = by_token if T <= longest else in_chunks
        assert torch.equal(auto[0], same[0]) and np.array_equal(auto[1], same[1])
        assert not torch.equal(by_token[0], in_chunks[0])


def test_short_tail_resumes_bit_for_bit():
    """A checkpointed call of a few tokens repeats the path of the long one it goes on from."""
    heads, total = HEADS[0], 64 + 5
    o, S, _, _, _, kept, _ = run_prefill(heads, [total], seed=16, ckpt=True)
    dev, _ = make(np.random.default_rng(16), total, heads)
    with GdnPool(1, heads[0], heads[1], 1, n_snapshots=1) as pool:
        pool.snapshots[0, 0].copy_(torch.from_numpy(kept[0, 0]))
        pool.restore(i32([0]), i32([0]))
        o2 = pool.prefill(0, i32([0]), i32([0, 5]), *[x[64:] for x in dev], l2norm_eps=EPS, cu_ckpt=i32([0, 0]),
                          ckpt_ids=i32([0]))
        assert pool.device_status() == 0
        assert torch.equal(o2, o[64:]) and np.array_equal(host(pool.states[0, 0]), S[0])


@pytest.mark.parametrize("total", [150, 2000])   # uncut, and cut into segments
def test_bounded_waits_of_the_chunked_prefill(total):
    """With the test hook on no input is loaded: every wait gives up, the call reports it, and
    the next call runs as ever."""
    lib = load_library()
    heads = HEADS[0]
    rng = np.random.default_rng(17)
    dev, hst = make(rng, total, heads)
    S0 = start(rng, 1, heads)
    with GdnPool(1, heads[0], heads[1], 1) as pool:
        pool.states.copy_(S0)
        assert lib.wkv7_test_force_wait_timeout(1) == 0
        try:
            pool.prefill(0, i32([0]), i32([0, total]), *dev, l2norm_eps=EPS)
            assert pool.device_status() == DEV_WAIT_TIMEOUT
        finally:
            lib.wkv7_test_force_wait_timeout(0)
        pool.states.copy_(S0)
        o = pool.prefill(0, i32([0]), i32([0, total]), *dev, l2norm_eps=EPS)
        assert pool.device_status() == 0
        S = host(pool.states[0, 0])
    o_ref, S_ref, _ = gdn_run(host(S0)[0, 0], *hst, heads[2] ** -0.5, EPS)
    assert err(o, o_ref) < CHUNK_TOL and oracle.rel_err(S, S_ref) < CHUNK_TOL


def test_prefill_equals_decode_steps():
    heads = (2, 4, 128, 128)
    rng = np.random.default_rng(4)
    dev, _ = make(rng, 40, heads)
    with GdnPool(1, 2, 4, 2) as pool:
        pool.create(2)
        a = pool.prefill(0, i32([0]), i32([0, 40]), *dev, l2norm_eps=EPS, sequential=True)
        b = torch.cat([pool.decode_step(0, i32([1]), *[x[t:t + 1] for x in dev], l2norm_eps=EPS) for t in range(40)])
        assert err(a, host(b)) < F32_TOL and err(pool.states[0], host(pool.states[1])) < F32_TOL


def test_another_stream_graph_and_repeat():
    """The same bits on another stream, from a captured graph, and for a second run."""
    heads = (2, 4, 128, 128)
    rng = np.random.default_rng(5)
    dev, _ = make(rng, 300, heads)
    S0 = start(rng, 2, heads).cuda()
    with GdnPool(1, 2, 4, 2) as pool:
        args = (0, i32([1, 0]), i32([0, 170, 300]), *dev)
        pool.states.copy_(S0)
        o = pool.prefill(*args, l2norm_eps=EPS, max_seqlen=170)
        S = pool.states.clone()
        side = torch.cuda.Stream()
        pool.states.copy_(S0)
        side.wait_stream(torch.cuda.current_stream())
        o2 = pool.prefill(*args, l2norm_eps=EPS, max_seqlen=170, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, o2) and torch.equal(S, pool.states)
        out = torch.empty_like(o)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pool.prefill(*args, o=out, l2norm_eps=EPS, max_seqlen=170)
        pool.states.copy_(S0)
        graph.replay()
        assert torch.equal(o, out) and torch.equal(S, pool.states)


def test_verbs_on_a_gdn_pool():
    heads = (1, 2, 128, 64)
    rng = np.random.default_rng(6)
    S0 = start(rng, 4, heads).cuda()
    with GdnPool(1, 1, 2, 4, n_snapshots=2, head_v=64) as pool:
        assert pool.slot_bytes == 2 * 64 * 128 * 4
        pool.states.copy_(S0)
        pool.snapshot(i32([3]), i32([1]))
        pool.fork(i32([0]), i32([3]))
        pool.restore(i32([1]), i32([2]))
        assert torch.equal(pool.states[3], S0[0]) and torch.equal(pool.states[2], S0[3])
        pinned = torch.empty(pool.slot_bytes, dtype=torch.uint8).pin_memory()
        pool.hibernate(i32([2]), pinned)
        pool.reset(i32([2]))
        assert not pool.states[2].any()
        pool.resume(pinned, i32([2]))
        assert torch.equal(pool.states[2], S0[3])
        pool.validate_ids(i32([0, 1, 0]))
        assert pool.device_status() == 5


def test_device_faults_leave_the_rest_alone():
    heads = (1, 2, 64, 64)
    rng = np.random.default_rng(7)
    S0 = start(rng, 3, heads).cuda()
    dev, _ = make(rng, 4, heads)
    with GdnPool(1, 1, 2, 3, n_snapshots=1, head_k=64, head_v=64) as pool:
        pool.states.copy_(S0)
        o = torch.full((2, 2, 64), 7.0, device="cuda")
        pool.decode_step(0, i32([1, 3]), *[x[:2] for x in dev], o=o, l2norm_eps=EPS)
        assert pool.device_status() == DEV_BAD_SLOT
        assert (o[1] == 7).all() and not (o[0] == 7).any()
        assert torch.equal(pool.states[[0, 2]], S0[[0, 2]])
        pool.states.copy_(S0)
        pool.decode_multi(0, i32([1, -1]), *[x.unflatten(0, (2, 2)) for x in dev], l2norm_eps=EPS,
                          step_snap_ids=i32([[0, 1], [0, 0]]))
        assert pool.device_status() == DEV_BAD_SLOT
        for sequential in (False, True):
            pool.states.copy_(S0)
            o = torch.full((4, 2, 64), 7.0, device="cuda")
            pool.prefill(0, i32([0, 1]), i32([0, 3, 2]), *dev, o=o, l2norm_eps=EPS, max_seqlen=3,
                         sequential=sequential)
            assert pool.device_status() == DEV_BAD_SEQLENS
            assert torch.equal(pool.states[1], S0[1]) and not torch.equal(pool.states[0], S0[0])
            assert (o[3] == 7).all()


def test_refusals():
    heads = (2, 4, 64, 64)
    rng = np.random.default_rng(8)
    dev, _ = make(rng, 2, heads)
    ids = i32([0, 1])
    with pytest.raises(Wkv7Error, match="UNSUPPORTED"):
        GdnPool(1, 1, 1, 1, head_k=32, head_v=64)
    with pytest.raises(Wkv7Error, match="INVALID_ARG"):
        GdnPool(1, 2, 3, 1)
    with pytest.raises(ValueError):
        GdnPool(1, 1, 1, 1, state_dtype="f16")
    with GdnPool(1, 2, 4, 2, head_k=64, head_v=64) as pool, Pool(1, 4, 2) as wkv:
        with pytest.raises(TypeError):
            pool.decode_step(0, ids, dev[0].half(), dev[1].half(), dev[2].half(), *dev[3:])
        with pytest.raises(TypeError):
            pool.decode_step(0, ids, dev[0].float(), *dev[1:])
        with pytest.raises(TypeError):
            pool.decode_step(0, ids, *dev[:3], dev[3].to(torch.bfloat16), dev[4])
        with pytest.raises(ValueError):
            pool.decode_step(0, ids, dev[0][:1], *dev[1:])
        with pytest.raises(ValueError):
            pool.decode_step(0, ids, dev[0].transpose(1, 2).contiguous().transpose(1, 2), *dev[1:])
        with pytest.raises(ValueError):
            pool.decode_step(0, ids, *dev, o=torch.empty(2, 4, 64, dtype=torch.bfloat16, device="cuda"))
        with pytest.raises(Wkv7Error, match="INVALID_ARG"):
            pool.decode_step(1, ids, *dev)
        with pytest.raises(Wkv7Error, match="INVALID_ARG"):
            pool.decode_step(0, ids, *dev, l2norm_eps=-1.0)
        with pytest.raises(Wkv7Error, match="INVALID_ARG"):
            pool.decode_multi(0, ids, *[x.unsqueeze(1) for x in dev], step_snap_ids=i32([[0], [0]]))
        odd = torch.empty(2, 2 * 64 * 2 + 4 * 64 + 4, device="cuda", dtype=torch.bfloat16)[:, 4:4 + 128]
        with pytest.raises(Wkv7Error, match="UNSUPPORTED"):   # base and stride not multiples of 16 bytes
            pool.decode_step(0, ids, odd.unflatten(1, (2, 64)), *dev[1:])
        with pytest.raises(Wkv7Error, match="BAD_SEQLENS"):
            pool.prefill(0, ids, i32([0, 1, 2]), *dev, max_seqlen=3)
        x = torch.zeros(2, 4, 64, device="cuda")
        lib = pool._lib
        assert lib.wkv7_decode_step(pool._h, 0, ids.data_ptr(), 2, 0, *[x.data_ptr()] * 6, x.data_ptr(), None) == 7
        import ctypes
        from rwkv_wkv_gb300.wkv7 import GdnTokens
        assert lib.wkv7_gdn_decode_step(wkv._h, 0, ids.data_ptr(), 2, ctypes.byref(GdnTokens()), None) == 7
