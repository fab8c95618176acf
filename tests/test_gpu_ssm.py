"""Selective scan over state slots: decode, multi-token decode and prefill against the float64
recurrence, their edges and refusals."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from oracle.ssm import scan_run
from rwkv_wkv_gb300 import DEV_BAD_SEQLENS, DEV_BAD_SLOT, SsmPool, Wkv7Error
from ssm_helpers import check, chunk_bound, host, rows_of, scan_inputs, scan_reference, step_bound

pytestmark = pytest.mark.gpu

SHAPES = [(4, 2, 64, 128), (3, 1, 64, 64), (2, 2, 128, 128), (6, 3, 128, 64)]


def fill(pool, seed, scale=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pool.states.copy_((torch.randn(pool.states.shape, device="cuda", generator=gen) * scale).to(pool.states.dtype))


def make(shape, slots, snaps=0, layers=2, **kw):
    h, g, p, n = shape
    return SsmPool(layers, h, g, slots, n_snapshots=snaps, head_p=p, d_state=n, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_decode_step(shape, out, dtype):
    n = 7
    with make(shape, n + 2, out_dtype=out) as pool:
        fill(pool, 1)
        before = pool.states.clone()
        ids = [8, 0, 3, 1, 7, 2, 5]
        ins = scan_inputs(2, n, *shape, dtype=dtype)
        o = pool.decode_step(1, i32(ids), **ins)
        for b, s in enumerate(ids):
            want, S, uo, us = scan_reference(host(before[s, 1]), rows_of(ins, b, b + 1))
            check(o[b:b + 1], want, uo, step_bound(1), o.dtype)
            check(pool.states[s, 1], S, us, step_bound(1))
        others = [s for s in range(n + 2) if s not in ids]
        assert torch.equal(pool.states[:, 0], before[:, 0]) and torch.equal(pool.states[others], before[others])
        assert pool.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_decode_of_bf16_states_stores_the_rounded_formula(shape, dtype):
    """The stored state against the same float32 products and sums in torch: a neighbour of the
    exact value (the exponential may differ in its last bit, which moves a rounding border)."""
    n = 5
    with make(shape, n, state_dtype="bf16") as pool:
        fill(pool, 3)
        before = pool.states.clone()
        ins = scan_inputs(4, n, *shape, dtype=dtype)
        o = pool.decode_step(0, i32(range(n)), **ins)
        for b in range(n):
            want, S, uo, us = scan_reference(host(before[b, 0]), rows_of(ins, b, b + 1))
            check(o[b:b + 1], want, uo, step_bound(1))
            check(pool.states[b, 0], S, us, step_bound(1), torch.bfloat16)
        step = torch.nn.functional.softplus(ins["dt"].float() + ins["dt_bias"])
        a = torch.exp(step * ins["A"])[:, :, None, None]
        B = ins["B"].float().repeat_interleave(shape[0] // shape[1], 1)
        u = (step[..., None] * ins["x"].float())[..., None] * B[:, :, None, :]
        same = (a * before[:, 0].float() + u).to(torch.bfloat16) == pool.states[:, 0]
        assert same.float().mean() > 0.999


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_decode_multi_is_single_steps(shape, dtype, state):
    """Outputs, every kept state and the final one, bit for bit, over more tokens than one pass stages."""
    n, K = 3, 19
    with make(shape, 2 * n, snaps=n * K, state_dtype=state) as pool:
        fill(pool, 5)
        pool.states[n:] = pool.states[:n]
        ins = scan_inputs(6, n * K, *shape, dtype=dtype)
        multi = {k: (v.unflatten(0, (n, K)) if k in ("x", "dt", "B", "C") else v) for k, v in ins.items()}
        snaps = i32(np.random.default_rng(0).permutation(n * K).reshape(n, K))
        o = pool.decode_multi(1, i32(range(n)), **multi, step_snap_ids=snaps)
        for t in range(K):
            one = {k: (v[:, t] if k in ("x", "dt", "B", "C") else v) for k, v in multi.items()}
            ot = pool.decode_step(1, i32(range(n, 2 * n)), **one)
            assert torch.equal(o[:, t], ot)
            assert torch.equal(pool.snapshots[snaps[:, t].long(), 1], pool.states[n:, 1])
        assert torch.equal(pool.states[:n], pool.states[n:])
        assert pool.device_status() == 0


LENGTHS = [[1], [0, 1, 0, 5], [63, 64, 65], [127, 128, 129, 1], [300, 17, 513]]


@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("sequential", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_prefill(shape, sequential, lens):
    with make(shape, len(lens) + 1) as pool:
        fill(pool, 7)
        before = pool.states.clone()
        total = sum(lens)
        ins = scan_inputs(8, total, *shape)
        cu = np.concatenate([[0], np.cumsum(lens)])
        ids = list(range(len(lens), 0, -1))
        o = pool.prefill(1, i32(ids), i32(cu), **ins, max_seqlen=max(lens), sequential=sequential)
        assert pool.device_status() == 0
        for s, slot in enumerate(ids):
            want, S, uo, us = scan_reference(host(before[slot, 1]), rows_of(ins, cu[s], cu[s + 1]))
            rel = step_bound(lens[s]) if sequential else max(chunk_bound(lens[s]), step_bound(lens[s]))
            check(o[cu[s]:cu[s + 1]], want, uo, rel)
            check(pool.states[slot, 1], S, us, rel)
        assert torch.equal(pool.states[:, 0], before[:, 0]) and torch.equal(pool.states[0], before[0])


@pytest.mark.parametrize("kind", ["f32 inputs", "bf16 states", "bf16 outputs", "f32 dt"])
def test_prefill_types(kind):
    shape, lens = (4, 2, 64, 128), [200, 131]
    kw = {"state_dtype": "bf16"} if kind == "bf16 states" else {"out_dtype": "bf16"} if kind == "bf16 outputs" else {}
    with make(shape, 2, **kw) as pool:
        fill(pool, 9)
        before = pool.states.clone()
        ins = scan_inputs(10, sum(lens), *shape, dtype=torch.float32 if kind == "f32 inputs" else torch.bfloat16,
                          dt_dtype=torch.float32 if kind == "f32 dt" else None)
        o = pool.prefill(0, i32([0, 1]), i32([0, 200, 331]), **ins, max_seqlen=200)
        for s, (a, b) in enumerate(((0, 200), (200, 331))):
            want, S, uo, us = scan_reference(host(before[s, 0]), rows_of(ins, a, b))
            check(o[a:b], want, uo, chunk_bound(b - a), o.dtype)
            check(pool.states[s, 0], S, us, chunk_bound(b - a), pool.states.dtype)


@pytest.mark.parametrize("sequential", [True, False])
def test_optional_inputs_and_plain_steps(sequential):
    """No D, no bias, no softplus: dt as given, zeros and a step that empties the state among them."""
    shape = (4, 2, 64, 128)
    with make(shape, 1) as pool:
        fill(pool, 11)
        before = host(pool.states[0, 0])
        ins = scan_inputs(12, 150, *shape, dt_dtype=torch.float32)
        dt = ins["dt"].abs().clone()
        dt[::7] = 0
        dt[40, 1] = 1000.0
        dt[90:92, 2] = 30.0
        ins.update(D=None, dt_bias=None, dt_softplus=False, dt=dt)
        o = pool.prefill(0, i32([0]), i32([0, 150]), **ins, sequential=sequential)
        want, S, uo, us = scan_reference(before, ins)
        check(o, want, uo, chunk_bound(150))
        check(pool.states[0, 0], S, us, chunk_bound(150))


def test_rows_of_stride_zero_and_single_heads():
    """The same x, B, C and dt for every row, from one row of each."""
    shape = (1, 1, 64, 128)
    with make(shape, 5) as pool:
        fill(pool, 13)
        before = pool.states.clone()
        one = scan_inputs(14, 1, *shape)
        ins = {k: (v.expand(5, *v.shape[1:]) if k in ("x", "dt", "B", "C") else v) for k, v in one.items()}
        o = pool.decode_step(0, i32(range(5)), **ins)
        for b in range(5):
            want, S, uo, us = scan_reference(host(before[b, 0]), one)
            check(o[b:b + 1], want, uo, step_bound(1))
            check(pool.states[b, 0], S, us, step_bound(1))
        ins = {k: (v.expand(140, *v.shape[1:]) if k in ("x", "dt", "B", "C") else v) for k, v in one.items()}
        before = host(pool.states[0, 0])
        o = pool.prefill(0, i32([0]), i32([0, 140]), **ins)
        want, S, uo, us = scan_reference(before, ins)
        check(o, want, uo, chunk_bound(140) + step_bound(140))


def test_bad_ids_and_lengths_are_skipped_and_flagged():
    shape = (2, 1, 64, 64)
    with make(shape, 3, snaps=2) as pool:
        fill(pool, 15)
        before = pool.states.clone()
        ins = scan_inputs(16, 3, *shape)
        o = torch.full((3, 2, 64), 7.0, device="cuda")
        pool.decode_step(0, i32([0, 3, -1]), **ins, o=o)
        assert pool.device_status() == DEV_BAD_SLOT
        assert torch.equal(o[1:], torch.full_like(o[1:], 7.0)) and not torch.equal(o[0], torch.full_like(o[0], 7.0))
        assert torch.equal(pool.states[1:], before[1:])
        multi = {k: (v[None] if k in ("x", "dt", "B", "C") else v) for k, v in ins.items()}
        pool.snapshots.zero_()
        pool.decode_multi(0, i32([1]), **multi, step_snap_ids=i32([[0, 2, 1]]))
        assert pool.device_status() == DEV_BAD_SLOT
        assert torch.equal(pool.snapshots[1, 0], pool.states[1, 0]) and pool.snapshots[0, 0].any()
        ins = scan_inputs(17, 300, *shape)
        for sequential in (True, False):
            for cu, ids, code, done in (([0, 100, 50, 300], [0, 1, 2], DEV_BAD_SEQLENS, [0, 2]),
                                        ([0, 100, 200, 301], [0, 1, 2], DEV_BAD_SEQLENS, [0, 1]),
                                        ([0, 100, 200, 300], [0, 5, 2], DEV_BAD_SLOT, [0, 2]),
                                        ([-1, 100, 200, 300], [0, 1, 2], DEV_BAD_SEQLENS, [1, 2])):
                fill(pool, 16)  # (a state that has forgotten its start would end as it began)
                before = pool.states.clone()
                pool.prefill(0, i32(ids), i32(cu), **ins, max_seqlen=260, sequential=sequential)
                assert pool.device_status() == code
                for s in range(3):
                    assert torch.equal(pool.states[s], before[s]) == (s not in done)


def test_rows_behind_the_last_sequence_are_left():
    shape = (2, 1, 64, 128)
    ins = scan_inputs(18, 300, *shape)
    for sequential in (True, False):
        with make(shape, 1) as pool:
            pool.states.zero_()
            o = torch.full((300, 2, 64), 7.0, device="cuda")
            pool.prefill(0, i32([0]), i32([0, 201]), **ins, o=o, max_seqlen=201, sequential=sequential)
            assert torch.equal(o[201:], torch.full_like(o[201:], 7.0)) and (o[200] != 7).any()


def test_refusals():
    shape = (2, 1, 64, 64)
    ins = scan_inputs(19, 4, *shape)
    with make(shape, 4) as pool:
        ids, cu = i32(range(4)), i32([0, 4])
        for bad in (dict(x=ins["x"][:3]), dict(x=ins["x"].float()), dict(A=ins["A"].double()), dict(A=ins["A"][:1]),
                    dict(dt=ins["dt"].half()), dict(B=ins["B"][:, :, :32]), dict(D=ins["D"].cpu()),
                    dict(x=ins["x"].transpose(1, 2)), dict(o=torch.empty(4, 2, 64, device="cuda", dtype=torch.bfloat16))):
            with pytest.raises((TypeError, ValueError)):
                pool.decode_step(0, ids, **{**ins, **bad})
        for bad in (dict(layer=2), dict(layer=-1)):
            with pytest.raises(Wkv7Error, match="INVALID_ARG"):
                pool.decode_step(bad["layer"], ids, **ins)
        odd = torch.zeros(4, 2 * 64 + 4, device="cuda", dtype=torch.bfloat16)[:, 4:].unflatten(1, (2, 64))
        with pytest.raises(Wkv7Error, match="UNSUPPORTED"):
            pool.decode_step(0, ids, **{**ins, "x": odd})
        with pytest.raises(Wkv7Error, match="INVALID_ARG"):
            pool.decode_multi(0, i32([0]), **{k: (v[None] if k in ("x", "dt", "B", "C") else v) for k, v in ins.items()},
                              step_snap_ids=i32([[0, 0, 0, 0]]))
        with pytest.raises(Wkv7Error, match="BAD_SEQLENS"):
            pool.prefill(0, i32([0]), cu, **ins, max_seqlen=5)
        with pytest.raises(ValueError):
            pool.conv_step(0, ids, torch.zeros(4, 8, device="cuda"), torch.zeros(8, 4, device="cuda"))
        assert pool.device_status() == 0


def test_nothing_to_do():
    shape = (2, 1, 64, 64)
    with make(shape, 2) as pool:
        pool.states.fill_(3)
        none = {k: (v[:0] if k in ("x", "dt", "B", "C") else v) for k, v in scan_inputs(20, 1, *shape).items()}
        assert pool.decode_step(0, i32([]), **none).shape == (0, 2, 64)
        assert pool.prefill(0, i32([]), i32([0]), **none).shape == (0, 2, 64)
        pool.prefill(0, i32([0, 1]), i32([0, 0, 0]), **none)
        assert pool.device_status() == 0 and (pool.states == 3).all()


def test_slots_far_into_a_large_pool():
    """State offsets past 2^31 entries."""
    shape, layers = (64, 1, 64, 128), 8
    slots = 2 ** 31 // (layers * 64 * 64 * 128) + 2
    with make(shape, slots, layers=layers) as pool:
        last = slots - 1
        assert last * layers * 64 * 64 * 128 >= 2 ** 31
        pool.states[last].zero_()
        ins = scan_inputs(21, 130, *shape)
        o = pool.prefill(7, i32([last]), i32([0, 129]), **{k: (v[:129] if k in ("x", "dt", "B", "C") else v) for k, v in ins.items()})
        o1 = pool.decode_step(7, i32([last]), **rows_of(ins, 129, 130))
        heads = [0, 63]
        a = {k: host(v) for k, v in ins.items()}
        part = dict(a, x=a["x"][:, heads], dt=a["dt"][:, heads], A=a["A"][heads], D=a["D"][heads], dt_bias=a["dt_bias"][heads])
        want, S, _ = scan_run(np.zeros((2, 64, 128)), **part)
        assert np.abs(host(torch.cat([o, o1])[:, heads]) - want).max() < 1e-4 * np.abs(want).max()
        assert np.abs(host(pool.states[last, 7, heads]) - S).max() < 1e-4 * np.abs(S).max()
