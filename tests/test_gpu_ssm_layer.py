"""A state space layer's three operators in one call: the same bits as call after call, drafts that are
rolled back, and its refusals."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from rwkv_wkv_gb300 import SsmLayer, SsmPool, gated_norm

pytestmark = pytest.mark.gpu

H, G, P, N = 4, 2, 64, 128
CH = H * P + 2 * G * N


def build(slots, snaps=0, layers=2, **kw):
    pool = SsmPool(layers, H, G, slots, n_snapshots=snaps, head_p=P, d_state=N, conv_channels=CH, **kw)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def draw(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, device="cuda", generator=gen).to(dtype)

    w = (draw(CH, 4) * 0.4, draw(CH) * 0.1, -1 - 5 * torch.rand(H, device="cuda", generator=gen),
         draw(H, dtype=torch.float32), draw(H, dtype=torch.float32) - 3, draw(H * P))
    return pool, w, draw


@pytest.mark.parametrize("first,group", [(True, None), (False, 64)])
def test_is_its_calls(first, group):
    pool, w, draw = build(6)
    with pool:
        pool.create(6)
        lens = [140, 0, 9]
        cu, rows = i32([0, 140, 140, 149]), draw(149, H * P + CH + 8)
        got = SsmLayer(pool, 1, *w, gate_first=first, norm_group=group).prefill(i32([0, 1, 2]), cu, rows, max_seqlen=max(lens))
        one = draw(3, H * P + CH + 8)
        step = SsmLayer(pool, 1, *w, gate_first=first, norm_group=group).step(i32([0, 1, 2]), one)
        more = dict(D=w[3], dt_bias=w[4], dt_softplus=True)
        for r, want, prompt in ((rows, got, True), (one, step, False)):
            z, u, dt = r[:, :H * P], r[:, H * P:H * P + CH], r[:, H * P + CH:H * P + CH + H]
            ids = i32([3, 4, 5])
            y = pool.conv_prefill(1, ids, cu, u, w[0], w[1]) if prompt else pool.conv_step(1, ids, u, w[0], w[1])
            x, B, C = y[:, :H * P].unflatten(1, (H, P)), y[:, H * P:H * P + G * N].unflatten(1, (G, N)), y[:, H * P + G * N:].unflatten(1, (G, N))
            o = pool.prefill(1, ids, cu, x, dt, w[2], B, C, max_seqlen=140, **more) if prompt else \
                pool.decode_step(1, ids, x, dt, w[2], B, C, **more)
            o = gated_norm(o.flatten(1), z, w[5], gate_first=first, group_size=group, out_dtype=torch.bfloat16)
            assert torch.equal(o, want)
        assert torch.equal(pool.states[:3], pool.states[3:]) and torch.equal(pool.conv_tails[:3], pool.conv_tails[3:])
        assert pool.device_status() == 0


@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_refused_drafts_are_rolled_back(state):
    """After a pass over K drafts and the restore of the state after m of them, the next token's row is the
    one that m single tokens would have been followed by; states and tails of every layer go back together."""
    n, K = 3, 4
    pool, w, draw = build(2 * n, snaps=n * K, state_dtype=state, out_dtype="bf16")
    with pool:
        pool.create(2 * n)
        layers = [SsmLayer(pool, i, *w) for i in range(2)]
        a, b = i32(range(n)), i32(range(n, 2 * n))
        rows, following = draw(n, K, H * P + CH + 8), draw(n, H * P + CH + 8)
        snaps = i32(np.arange(n * K).reshape(n, K))
        multi = [layer.multi(a, rows, step_snap_ids=snaps) for layer in layers]
        taken = [0, 2, 3]  # the last token that stands, of each row
        pool.restore(snaps[torch.arange(n), torch.tensor(taken)].contiguous(), a)
        after = [layer.step(a, following) for layer in layers]
        for t in range(K):
            some = [s for s in range(n) if taken[s] >= t]
            for layer, m in zip(layers, multi):
                assert torch.equal(layer.step(i32([n + s for s in some]), rows[some, t]), m[some, t])
        for layer, o in zip(layers, after):
            assert torch.equal(layer.step(b, following), o)
        assert torch.equal(pool.states[:n], pool.states[n:]) and torch.equal(pool.conv_tails[:n], pool.conv_tails[n:])
        assert pool.device_status() == 0


def test_on_another_stream():
    pool, w, draw = build(2, layers=1)
    with pool:
        pool.create(2)
        layer = SsmLayer(pool, 0, *w)
        rows = draw(300, H * P + CH + 8)
        cu = i32([0, 300])
        want = layer.prefill(i32([0]), cu, rows)
        ids = i32([1])
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = layer.prefill(ids, cu, rows, stream=side)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(pool.states[0], pool.states[1])


def test_refusals():
    pool, w, draw = build(2)
    with pool:
        pool.create(2)
        layer = SsmLayer(pool, 0, *w)
        with pytest.raises(ValueError):
            layer.step(i32([0]), draw(1, H * P + CH))
        with pytest.raises(ValueError):
            layer.step(i32([0, 1]), draw(1, H * P + CH + 8))
        with SsmPool(1, H, G, 1, head_p=P, d_state=N) as bare:
            with pytest.raises(ValueError):
                SsmLayer(bare, 0, *w)
