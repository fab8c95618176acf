"""Selective scan prefill in chunks: long sequences cut into segments, values that are not finite,
waits that give up, captured and concurrent calls, many sequences."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from oracle.ssm import scan_run
from rwkv_wkv_gb300 import DEV_WAIT_TIMEOUT, SsmPool, gated_norm, load_library
from oracle.ssm import conv_run, gated_norm as norm_reference
from ssm_helpers import check, chunk_bound, host, rows_of, scan_inputs, scan_reference, step_bound

pytestmark = pytest.mark.gpu


def make(shape, slots, snaps=0, layers=1, **kw):
    h, g, p, n = shape
    pool = SsmPool(layers, h, g, slots, n_snapshots=snaps, head_p=p, d_state=n, **kw)
    gen = torch.Generator(device="cuda").manual_seed(slots)
    pool.states.copy_((torch.randn(pool.states.shape, device="cuda", generator=gen) * 0.3).to(pool.states.dtype))
    return pool


@pytest.mark.parametrize("lens", [[2500], [1024, 3000, 5, 0, 1153]], ids=str)
@pytest.mark.parametrize("shape,kw", [((2, 1, 64, 128), {}), ((1, 1, 128, 64), dict(state_dtype="bf16")),
                                      ((3, 3, 64, 64), dict(out_dtype="bf16"))], ids=str)
def test_cut_sequences(shape, kw, lens):
    with make(shape, len(lens), **kw) as pool:
        assert pool._lib.wkv7_ssm_prefill_workspace_bytes(pool._h, len(lens), max(lens)) > 0
        before = pool.states.clone()
        ins = scan_inputs(1, sum(lens), *shape, decay=0.05)  # (slow decays: segments see each other)
        cu = np.concatenate([[0], np.cumsum(lens)])
        o = pool.prefill(0, i32(range(len(lens))), i32(cu), **ins, max_seqlen=max(lens))
        assert pool.device_status() == 0
        for s in range(len(lens)):
            want, S, uo, us = scan_reference(host(before[s, 0]), rows_of(ins, cu[s], cu[s + 1]))
            check(o[cu[s]:cu[s + 1]], want, uo, chunk_bound(lens[s]), o.dtype)
            check(pool.states[s, 0], S, us, chunk_bound(lens[s]), pool.states.dtype)


@pytest.mark.parametrize("shape,T", [((8, 2, 64, 128), 700), ((8, 2, 128, 64), 700), ((4, 1, 128, 128), 1500)], ids=str)
def test_stored_bf16_states_are_the_rounded_formula_but_for_a_few(shape, T):
    """What goes into a bf16 state is off by about r = 2^-22 of the state's size (its weights' approximate 2^x, 2
    ulp): then an entry v, a step of 2^-8 |v| or more apart from the next value, is rounded the other way
    with a chance of r 2^8 size / |v| at most.  Over normally distributed v that is 0.8 r 2^8 log(1 / (r 2^8))
    = 4.7e-4.  (Errors of 2^-18 / 3 in each product, as of two parts, give four times that.)"""
    with make(shape, 1, state_dtype="bf16") as pool:
        before = host(pool.states[0, 0])
        ins = scan_inputs(6, T, *shape, decay=0.2)
        pool.prefill(0, i32([0]), i32([0, T]), **ins, max_seqlen=T)
        _, S, _ = scan_run(before, **{k: host(v) for k, v in ins.items()})
        other = pool.states[0, 0].cpu() != torch.from_numpy(S).to(torch.bfloat16)
        assert float(other.double().mean()) < 4.7e-4


def test_many_ragged_sequences():
    """More sequences than are put in order, of 0 to 300 tokens, in one call."""
    shape, n = (2, 1, 64, 128), 530
    lens = np.random.default_rng(2).integers(0, 300, n)
    lens[7] = 290
    cu = np.concatenate([[0], np.cumsum(lens)])
    with make(shape, n) as pool:
        before = pool.states.clone()
        ins = scan_inputs(3, int(cu[-1]), *shape)
        o = pool.prefill(0, i32(range(n)), i32(cu), **ins, max_seqlen=300)
        for s in range(0, n, 23):
            want, S, uo, us = scan_reference(host(before[s, 0]), rows_of(ins, int(cu[s]), int(cu[s + 1])))
            check(o[cu[s]:cu[s + 1]], want, uo, chunk_bound(300))
            check(pool.states[s, 0], S, us, chunk_bound(300))
        few = 40
        pool.states.copy_(before)
        o2 = pool.prefill(0, i32(range(few)), i32(cu[:few + 1]), **rows_of(ins, 0, int(cu[few])), max_seqlen=300)
        assert torch.equal(o2, o[:cu[few]])


@pytest.mark.parametrize("decay", [1e-4, 30.0])
def test_weak_and_steep_decays(decay):
    """Sums of hundreds of terms that hardly decay, and decays that leave nothing after a token or two."""
    shape = (4, 1, 64, 128)
    with make(shape, 1) as pool:
        before = host(pool.states[0, 0])
        ins = scan_inputs(4, 900, *shape, decay=decay)
        o = pool.prefill(0, i32([0]), i32([0, 900]), **ins)
        want, S, uo, us = scan_reference(before, ins)
        check(o, want, uo, chunk_bound(900))
        check(pool.states[0, 0], S, us, chunk_bound(900))


def compare_nonfinite(got, want, size, rel):
    got = host(got)
    odd = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)])
    check(torch.from_numpy(np.where(odd, 0, got)), np.where(odd, 0, want), size, rel)


CASES = ["x nan", "x inf", "B nan", "C nan", "dt nan", "state inf", "two rows"]


@pytest.mark.parametrize("where", CASES)
@pytest.mark.parametrize("mode", ["whole", "cut", "sequential"])
def test_values_that_are_not_finite_reach_what_the_formulas_let_them(mode, where):
    """(dt A is no -inf here: with it the formula's 0 * inf depends on which products are 0.)"""
    shape, T = (2, 1, 64, 128), 1300 if mode == "cut" else 400
    with make(shape, 1) as pool:
        ins = scan_inputs(5, T + 20, *shape, decay=0.05)
        clean = scan_reference(host(pool.states[0, 0]), rows_of(ins, 0, T))
        at = 1100 if mode == "cut" else 300
        nan, inf = float("nan"), float("inf")
        if where == "x nan":
            ins["x"][at, 1, 5] = nan
        elif where == "x inf":
            ins["x"][at, 0, 63] = -inf
        elif where == "B nan":
            ins["B"][at, 0, 100] = nan
        elif where == "C nan":
            ins["C"][at, 0, 3] = nan
        elif where == "dt nan":
            ins["dt"][at, 1] = nan
        elif where == "state inf":
            pool.states[0, 0, 1, 7, 9] = inf
        else:
            ins["x"][200, 0, 1], ins["x"][at, 0, 40] = nan, inf
        ins["x"][T:], ins["B"][T:] = nan, inf   # behind the sequence
        before = host(pool.states[0, 0])
        o = pool.prefill(0, i32([0]), i32([0, T]), **ins, max_seqlen=T, sequential=mode == "sequential")
        assert pool.device_status() == 0
        a = {k: host(v) for k, v in rows_of(ins, 0, T).items()}
        want, S, _ = scan_run(before, **a)
        rel = max(chunk_bound(T), step_bound(T))
        compare_nonfinite(o[:T], want, clean[2] + 1, rel)
        compare_nonfinite(pool.states[0, 0], S, clean[3] + 1, rel)


@pytest.mark.parametrize("hook,lens", [(1, [300, 64, 130]), (1, [2500]), (2, [2500])])
def test_waits_that_give_up(hook, lens):
    """The call reports it and leaves every slot as it was; the next one runs as ever."""
    shape, lib = (2, 1, 64, 128), load_library()
    with make(shape, len(lens)) as pool:
        before = pool.states.clone()
        ins = scan_inputs(6, sum(lens), *shape)
        cu = np.concatenate([[0], np.cumsum(lens)])
        args = (0, i32(range(len(lens))), i32(cu))
        assert lib.wkv7_test_force_wait_timeout(hook) == 0
        try:
            pool.prefill(*args, **ins, max_seqlen=max(lens))
            assert pool.device_status() == DEV_WAIT_TIMEOUT
        finally:
            lib.wkv7_test_force_wait_timeout(0)
        assert torch.equal(pool.states, before)
        o = pool.prefill(*args, **ins, max_seqlen=max(lens))
        assert pool.device_status() == 0
        want, S, uo, us = scan_reference(host(before[0, 0]), rows_of(ins, 0, lens[0]))
        check(o[:lens[0]], want, uo, chunk_bound(lens[0]))
        check(pool.states[0, 0], S, us, chunk_bound(lens[0]))


def layer_inputs(seed, rows, h, g, p, n):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ch = h * p + 2 * g * n
    wide = torch.randn(rows, h * p + ch + (h + 7) // 8 * 8, device="cuda", generator=gen).to(torch.bfloat16)  # (rows of whole 16 bytes)
    z, u, dt = wide[:, :h * p], wide[:, h * p:h * p + ch], wide[:, h * p + ch:h * p + ch + h]
    w = torch.randn(ch, 4, device="cuda", generator=gen).to(torch.bfloat16) * 0.3
    bias = torch.randn(ch, device="cuda", generator=gen).to(torch.bfloat16) * 0.1
    A, D, dt_bias = -1 - 9 * torch.rand(h, device="cuda", generator=gen), torch.ones(h, device="cuda"), torch.full((h,), -3.0, device="cuda")
    nw = torch.rand(h * p, device="cuda", generator=gen).to(torch.bfloat16)
    return z, u, dt, w, bias, A, D, dt_bias, nw


def layer(pool, ids, cu, lens, ins, shape, step):
    """Convolution, scan and gated norm of one layer, for a prompt or for one token a slot."""
    h, g, p, n = shape
    z, u, dt, w, bias, A, D, dt_bias, nw = ins
    y = pool.conv_step(0, ids, u, w, bias) if step else pool.conv_prefill(0, ids, cu, u, w, bias)
    x, B, C = y[:, :h * p].unflatten(1, (h, p)), y[:, h * p:h * p + g * n].unflatten(1, (g, n)), y[:, h * p + g * n:].unflatten(1, (g, n))
    more = dict(D=D, dt_bias=dt_bias, dt_softplus=True)
    o = pool.decode_step(0, ids, x, dt, A, B, C, **more) if step else pool.prefill(0, ids, cu, x, dt, A, B, C, max_seqlen=max(lens), **more)
    return gated_norm(o.flatten(1), z, nw, gate_first=True, out_dtype=torch.float32)


def test_a_layer_prompt_then_tokens():
    """The three operators together against float64: a ragged prefill, then four tokens of each slot."""
    shape, lens, K = (4, 2, 64, 64), [150, 3, 40], 4
    h, g, p, n = shape
    ch = h * p + 2 * g * n
    total, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    whole = layer_inputs(8, total + 3 * K, *shape)
    cut = lambda a, b: tuple(t[a:b] if i < 3 else t for i, t in enumerate(whole))  # noqa: E731
    with make(shape, 3, conv_channels=ch) as pool:
        pool.states.zero_()
        pool.conv_tails.zero_()
        ids = i32(pool.create(3))
        got = [layer(pool, ids, i32(cu), lens, cut(0, total), shape, False)]
        for k in range(K):
            got.append(layer(pool, ids, None, None, cut(total + 3 * k, total + 3 * k + 3), shape, True))
        assert pool.device_status() == 0
        z, u, dt, w, bias, A, D, dt_bias, nw = (host(t) for t in whole)
        for s in range(3):
            rows = list(range(cu[s], cu[s + 1])) + [total + 3 * k + s for k in range(K)]
            y, tail = conv_run(np.zeros((3, ch)), u[rows], w, bias)
            y = torch.from_numpy(y).to(torch.bfloat16).double().numpy()
            x, B, C = y[:, :h * p].reshape(-1, h, p), y[:, h * p:h * p + g * n].reshape(-1, g, n), y[:, h * p + g * n:].reshape(-1, g, n)
            o, S, _ = scan_run(np.zeros((h, p, n)), x, dt[rows], A, B, C, D, dt_bias, True)
            want = norm_reference(o.reshape(len(rows), -1), z[rows], nw, gate_first=True)
            mine = host(torch.cat([got[0][cu[s]:cu[s + 1]]] + [t[s:s + 1] for t in got[1:]]))
            # a convolution's output near a rounding border may round the other way: half a step of
            # bf16 more in x, B and C of some terms of a sum
            assert np.abs(mine - want).max() < 2.0 ** -7 * np.abs(want).max()
            assert np.array_equal(host(pool.conv_tails[int(ids[s]), 0]), tail)
            assert np.abs(host(pool.states[int(ids[s]), 0]) - S).max() < 2.0 ** -7 * np.abs(S).max()


def test_captured_calls_replay_to_the_same_bits():
    shape, lens = (2, 1, 64, 128), [1300, 200]
    ch = 2 * 64 + 2 * 128
    total, cu = sum(lens), i32([0, 1300, 1500])
    pre, one = layer_inputs(9, total, *shape), layer_inputs(10, 2, *shape)
    got = {}
    with make(shape, 2, conv_channels=ch) as pool:
        ids = i32([1, 0])
        begin = pool.states.clone()

        def calls():
            a = layer(pool, ids, cu, lens, pre, shape, False)
            return a, layer(pool, ids, None, None, one, shape, True)

        for mode in ("eager", "graph"):
            pool.states.copy_(begin)
            pool.conv_tails.zero_()
            if mode == "eager":
                out = calls()
            else:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    out = calls()
                pool.states.copy_(begin)
                pool.conv_tails.zero_()
                graph.replay()
            torch.cuda.synchronize()
            assert pool.device_status() == 0
            got[mode] = [t.clone() for t in out] + [pool.states.clone(), pool.conv_tails.clone()]
    assert all(torch.equal(a, b) for a, b in zip(got["eager"], got["graph"]))


def test_calls_on_two_streams():
    """Two pools' calls on two streams at once, each with a workspace of its own."""
    shape = (2, 1, 64, 128)
    ins = scan_inputs(11, 2500, *shape)
    with make(shape, 1) as a, make(shape, 1) as b:
        b.states.copy_(a.states)
        begin = a.states.clone()
        want = a.prefill(0, i32([0]), i32([0, 2500]), **ins)
        end = a.states.clone()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(3):
            a.states.copy_(begin)
            b.states.copy_(begin)
            torch.cuda.synchronize()
            ids, cu = i32([0]), i32([0, 2500])
            torch.cuda.synchronize()
            got = [pool.prefill(0, ids, cu, **ins, stream=s) for pool, s in zip((a, b), streams)]
            torch.cuda.synchronize()
            for pool, o in zip((a, b), got):
                assert pool.device_status() == 0 and torch.equal(o, want) and torch.equal(pool.states, end)


class WithoutWorkspace:
    """The library, but for the workspace it asks for."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        return (lambda *_: 0) if name == "wkv7_ssm_prefill_workspace_bytes" else getattr(self.lib, name)


def with_and_without(shape, lens, ins, poison=None, **kw):
    """A call whose units are cut where an SM's share ends, and one whose units stay whole."""
    got = []
    cu = np.concatenate([[0], np.cumsum(lens)])
    for whole in (False, True):
        with make(shape, len(lens), **kw) as pool:
            need = pool._lib.wkv7_ssm_prefill_workspace_bytes(pool._h, len(lens), max(lens))
            assert need > 0
            if whole:
                pool._lib = WithoutWorkspace(pool._lib)
            if poison is not None:
                poison(pool)
            o = pool.prefill(0, i32(range(len(lens))), i32(cu), **ins, max_seqlen=max(lens))
            assert pool.device_status() == 0
            got.append((o, pool.states.clone()))
    return got


@pytest.mark.parametrize("lens", [[900, 0, 513, 128, 700], [2600] * 4, [520] + [0] * 30 + [1], [517, 5, 5, 5, 1030] * 9],
                         ids=["mixed", "long", "mostly empty", "many"])
@pytest.mark.parametrize("kw", [{}, dict(state_dtype="bf16", out_dtype="bf16")], ids=str)
def test_units_cut_at_any_chunk_have_the_bits_of_whole_ones(lens, kw):
    shape = (40, 1, 64, 64)
    assert 40 * len(lens) >= 152
    ins = scan_inputs(21, sum(lens), *shape, decay=0.05)
    cut, whole = with_and_without(shape, lens, ins, **kw)
    assert all(torch.equal(a, b) for a, b in zip(cut, whole))
    with make(shape, len(lens), **kw) as pool:
        before = host(pool.states[0, 0])
        few = [0, 39]
        one = {k: (v[:lens[0]] if k in ("x", "dt", "B", "C") else v) for k, v in ins.items()}
        part = dict(one, x=one["x"][:, few], dt=one["dt"][:, few], **{k: one[k][few] for k in ("A", "D", "dt_bias")})
        want, S, uo, us = scan_reference(before[few], part)
        check(cut[0][:lens[0], few], want, uo, chunk_bound(lens[0]), cut[0].dtype)
        check(cut[1][0, 0, few], S, us, chunk_bound(lens[0]), cut[1].dtype)


def test_values_that_are_not_finite_across_cuts():
    """In three heads of units that are cut, in their first part, their second, and the start state."""
    shape, lens = (40, 1, 64, 64), [2600] * 4
    ins = scan_inputs(22, sum(lens), *shape, decay=0.05)
    ins["x"][50, 3, 7], ins["x"][2600 + 2500, 20, 60], ins["x"][5200 + 1300, :, 11] = float("nan"), float("inf"), float("-inf")

    def poison(pool):
        pool.states[3, 0, 5, 9, 10] = float("inf")

    (o, S), _ = with_and_without(shape, lens, ins, poison)
    with make(shape, 4) as pool:
        poison(pool)
        want = pool.prefill(0, i32(range(4)), i32([0, 2600, 5200, 7800, 10400]), **ins, max_seqlen=2600, sequential=True)
        for got, ref in ((o, want), (S, pool.states)):
            assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(torch.isinf(got), torch.isinf(ref))
            fine = torch.isfinite(ref)
            assert (got[fine] - ref[fine]).abs().max() < 1e-4 * ref[fine].abs().max()
        assert torch.isnan(o[50:2600, 3, 7]).all() and torch.isfinite(o[:50]).all()
