"""The chunked selective scan from unit to unit: marks of values that are not finite, outputs that are written again,
more sequences than a CTA has threads, lengths that one call is planned by."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from rwkv_wkv_gb300 import DEV_BAD_SLOT, SsmPool
from ssm_helpers import EPS32, check, chunk_bound, host, rows_of, scan_inputs, scan_reference
from test_gpu_ssm_chunks import WithoutWorkspace

pytestmark = pytest.mark.gpu


def make(shape, slots, **kw):
    h, g, p, n = shape
    pool = SsmPool(1, h, g, slots, head_p=p, d_state=n, **kw)
    gen = torch.Generator(device="cuda").manual_seed(slots)
    pool.states.copy_((torch.randn(pool.states.shape, device="cuda", generator=gen) * 0.3).to(pool.states.dtype))
    return pool


def both(shape, lens, ins, **kw):
    """Outputs and states of the call, and of the same token by token."""
    got = []
    cu = i32([0] + np.cumsum(lens).tolist())
    for sequential in (False, True):
        with make(shape, len(lens), **kw) as pool:
            o = torch.zeros(sum(lens), shape[0], shape[2], device="cuda", dtype=pool.o_torch_dtype)
            pool.prefill(0, i32(range(len(lens))), cu, **ins, o=o, max_seqlen=max(lens), sequential=sequential)
            assert pool.device_status() == 0
            got.append((o, pool.states.clone()))
    return got


def same_where_odd(got, ref):
    """The same NaNs and infinities, and elsewhere 1e-4 of the largest value: chunks and tokens each within 1e-5."""
    assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(torch.isinf(got), torch.isinf(ref))
    fine = torch.isfinite(ref)
    assert (got[fine] - ref[fine]).abs().max() < 1e-4 * ref[fine].abs().max()


@pytest.mark.parametrize("shape", [(8, 1, 64, 128), (6, 2, 128, 64)], ids=str)
def test_units_of_one_chunk_with_values_that_are_not_finite(shape):
    """A thousand units and more, a third of the sequences with a NaN or an infinity in some row or all: each unit's
    rows are marked for itself, whatever the units before and behind it on the same SM left."""
    rng = np.random.default_rng(shape[0])
    lens = rng.integers(25, 129, 240).tolist()
    lens[0] = 128
    ins = scan_inputs(shape[1], sum(lens), *shape, decay=0.05)
    starts = np.cumsum([0] + lens)
    for s in range(0, 240, 3):
        at = int(starts[s]) + lens[s] - 1 - int(rng.integers(0, 20))
        h, row = int(rng.integers(0, shape[0])), int(rng.integers(0, shape[2]))
        kind = s // 3 % 4
        if kind == 0:
            ins["x"][at, h, row] = float("nan")
        elif kind == 1:
            ins["x"][at, :, row] = float("-inf")
        elif kind == 2:
            ins["B"][at, 0, int(rng.integers(0, shape[3]))] = float("nan")
        else:
            ins["dt"][at, h] = float("nan")
    (o, S), (want, ref) = both(shape, lens, ins)
    same_where_odd(o, want)
    same_where_odd(S, ref)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("last", [1, 31, 33, 127])
def test_rows_run_again_behind_a_short_last_chunk(last, out):
    """The last chunk ends before the rows of some of the warps that stored the chunks before it: what they
    stored is replaced in every chunk."""
    shape, lens = (16, 1, 64, 64), [128 * k + last for k in (1, 2, 3, 1, 2, 1, 1, 2, 1, 3)]
    ins = scan_inputs(last, sum(lens), *shape, decay=0.05)
    for end in np.cumsum(lens):
        ins["B"][int(end) - 1, 0, 5] = float("nan")    # (each row of each unit, at its last token)
    (o, S), (want, ref) = both(shape, lens, ins, out_dtype=out)
    if out == "bf16":   # both rounded: a step of bf16 apart at most
        assert torch.equal(torch.isnan(o), torch.isnan(want))
        fine = torch.isfinite(want)
        assert ((o[fine].float() - want[fine].float()).abs() <= 2.0 ** -7 * want[fine].float().abs() + 1e-4).all()
    else:
        same_where_odd(o, want)
    assert torch.isnan(S).any(-1).all() and torch.equal(torch.isnan(S), torch.isnan(ref))
    for end, n in zip(np.cumsum(lens), lens):
        assert torch.isfinite(o[int(end) - n:int(end) - 1]).all() and torch.isnan(o[int(end) - 1]).all()


def test_long_runs_again_are_waited_for():
    """A sequence whose every part runs again token by token, a few us each: its parts follow each other on as many SMs
    for more than the two seconds that a wait of a short call has, and end as the formulas say; the others as ever."""
    shape, T, n = (1, 1, 64, 64), 400000, 200
    lens = [T] + [100] * (n - 1)
    ins = scan_inputs(7, sum(lens), *shape, decay=0.05)
    ins["B"][5, 0, 3] = float("nan")
    with make(shape, n) as pool:
        before = pool.states.clone()
        o = pool.prefill(0, i32(range(n)), i32([0] + np.cumsum(lens).tolist()), **ins, max_seqlen=T)
        assert pool.device_status() == 0
        S = pool.states.clone()
        pool.states.copy_(before)
        some = {k: (v[T:] if k in ("x", "dt", "B", "C") else v) for k, v in ins.items()}
        want = pool.prefill(0, i32(range(1, n)), i32([100 * k for k in range(n)]), **some, max_seqlen=100)
        assert torch.equal(o[T:], want) and torch.equal(S[1:], pool.states[1:])
    assert torch.isnan(S[0, 0, 0, :, 3]).all() and torch.isfinite(S[0, 0, 0, :, [2, 4]]).all()
    assert torch.isfinite(o[:5]).all() and torch.isnan(o[5:T]).all()


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("n", [897, 2000])
def test_more_sequences_than_threads(n, workspace):
    """Each thread adds up a run of sequences, among them empty ones, whole runs of empty ones and ones of ids out of range:
    the bits of calls of fifty sequences, whose units stay whole."""
    shape, rng = (2, 1, 64, 64), np.random.default_rng(n)
    lens = np.where(rng.random(n) < 0.6, 0, rng.integers(1, 150, n))
    lens[[5, n // 2, n - 2]] = 700, 530, 641
    lens[n // 3:n // 3 + 40] = 0
    ids = rng.permutation(n)
    lost = rng.choice(n, 25, replace=False)
    ids[lost] = np.where(np.arange(25) % 2, -1, n + np.arange(25))
    cu = np.concatenate([[0], np.cumsum(lens)])
    ins = scan_inputs(n, int(cu[-1]) + 4, *shape, decay=0.05)
    with make(shape, n) as pool:
        before = pool.states.clone()
        assert pool._lib.wkv7_ssm_prefill_workspace_bytes(pool._h, n, 700) > 0
        lib = pool._lib
        if not workspace:
            pool._lib = WithoutWorkspace(lib)
        o = torch.full((int(cu[-1]) + 4, 2, 64), 7.0, device="cuda")
        pool.prefill(0, i32(ids), i32(cu), **ins, max_seqlen=700, o=o)
        assert pool.device_status() == DEV_BAD_SLOT
        S = pool.states.clone()
        pool._lib = lib
        pool.states.copy_(before)
        want = torch.full_like(o, 7.0)
        for a in range(0, n, 50):
            b = min(a + 50, n)
            part = want[cu[a]:cu[b]]
            pool.prefill(0, i32(ids[a:b]), i32(cu[a:b + 1] - cu[a]), **rows_of(ins, int(cu[a]), int(cu[b])), max_seqlen=min(700, len(part)), o=part)
        assert pool.device_status() in (0, DEV_BAD_SLOT)
    assert torch.equal(o, want) and torch.equal(S, pool.states)
    for s in lost:
        assert (o[cu[s]:cu[s + 1]] == 7).all()
    assert (o[cu[-1]:] == 7).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[333], [128, 77, 260], [2500]], ids=str)
def test_d_times_x_is_added_in_float32(lens, state, out):
    """D of 24 bits, up to 2^11: D x and its sum round by half a step of float32 each, beside what an output without D
    is off by.  (As an entry of two bf16 parts D alone would be off by up to 2^-18.)"""
    shape = (2, 1, 64, 128)
    cu = np.cumsum([0] + lens)
    ins = scan_inputs(11, int(cu[-1]), *shape, decay=0.05)
    ins["D"] = torch.tensor([1234.5677, -876.54321], device="cuda")
    with make(shape, len(lens), state_dtype=state, out_dtype=out) as pool:
        before = pool.states.clone()
        o = pool.prefill(0, i32(range(len(lens))), i32(cu), **ins, max_seqlen=max(lens))
        assert pool.device_status() == 0
    for s, n in enumerate(lens):
        one = rows_of(ins, int(cu[s]), int(cu[s + 1]))
        want, _, size, _ = scan_reference(host(before[s, 0]), dict(one, D=None))
        skip = host(ins["D"])[:, None] * host(one["x"])
        check(o[cu[s]:cu[s + 1]], want + skip, size, chunk_bound(n), o.dtype, floor=2 * EPS32 * (np.abs(skip) + np.abs(want + skip)))


def test_infinite_d():
    """D x as the formula has it: infinities, and NaN of a zero of x, in that head alone."""
    shape, T = (2, 1, 64, 64), 300
    ins = scan_inputs(12, T, *shape)
    ins["D"][1] = float("-inf")
    ins["x"][200, :, 5] = 0
    (o, S), (want, ref) = both(shape, [T], ins)
    same_where_odd(o, want)
    assert torch.isnan(o[200, 1, 5]) and torch.isfinite(o[:, 0]).all() and torch.isfinite(S).all() and torch.isfinite(ref).all()
