"""The convolution's prefill in its long tiles, of few and of many channels, against single steps bit for bit."""
import numpy as np
import pytest
import torch

from conv_sizes import TILED
from gpu_helpers import i32
from rwkv_wkv_gb300 import SsmPool

pytestmark = pytest.mark.gpu


def lengths(seed, total, tile, width):
    """Sequences of 0 to 4 tokens, such as end near a tile's border, and longer ones, in turn."""
    rng, lens, at = np.random.default_rng(seed), [], 0
    while True:
        pick = rng.integers(0, 4)
        n = int(rng.integers(0, 5)) if pick < 2 else int(rng.integers(0, 4 * tile)) if pick == 2 else \
            tile * int(rng.integers(1, 4)) - at % tile + int(rng.integers(-width, 2))
        if at + max(0, n) > total:
            return lens
        lens.append(max(0, n))
        at += max(0, n)


def windows(x, tails, seq, first, rows, width):
    """The width - 1 inputs before each of `rows`, of a sequence `seq` that starts at `first`: [rows, width - 1, ch]."""
    at = rows[:, None] + torch.arange(1 - width, 0, device=x.device)
    inside = at >= first[:, None]
    old = tails[seq[:, None], (at - first[:, None] + width - 1).clamp(0, width - 2)]
    return torch.where(inside[..., None], x[at.clamp(0)], old)


@pytest.mark.parametrize("ch,total,tile", TILED, ids=str)
@pytest.mark.parametrize("width,name", [(2, "bf16"), (3, "f32"), (4, "bf16")])
def test_long_tiles_are_steps(ch, total, tile, width, name):
    dtype = torch.bfloat16 if name == "bf16" else torch.float32
    unused = 5                                           # rows behind the last sequence
    lens = lengths(ch + total + width, total - unused, tile, width)
    lens[-1] += total - unused - sum(lens)
    n, used = len(lens), sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randn(total, ch + 8, device="cuda", generator=gen).to(dtype)[:, :ch]
    w, b = (torch.randn(*s, device="cuda", generator=gen).to(dtype) for s in ((ch, width), (ch,)))
    begin = torch.randn(n, width - 1, ch, device="cuda", generator=gen).to(dtype)
    ids = torch.randperm(n, device="cuda", generator=gen)
    size = torch.tensor(lens, device="cuda")
    first = size.cumsum(0) - size
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), size, output_size=used)
    more = dict(d_state=64, state_dtype="bf16", conv_channels=ch, conv_width=width, conv_dtype=name)
    with SsmPool(1, 1, 1, n, **more) as pool:
        pool.conv_tails[ids, 0] = begin
        o = torch.full((total, ch), 7.0, device="cuda", dtype=dtype)
        pool.conv_prefill(0, ids.to(torch.int32), i32([0] + np.cumsum(lens).tolist()), x, w, b, o=o)
        assert pool.device_status() == 0
        tails = pool.conv_tails[ids, 0].clone()
    with SsmPool(1, 1, 1, used, **more) as pool:         # a slot for each token
        pool.conv_tails[:, 0] = windows(x, begin, seq, first[seq], torch.arange(used, device="cuda"), width)
        want = pool.conv_step(0, torch.arange(used, device="cuda", dtype=torch.int32), x[:used], w, b)
        assert pool.device_status() == 0
    assert torch.equal(o[:used], want) and (o[used:] == 7).all()
    assert torch.equal(tails, windows(x, begin, torch.arange(n, device="cuda"), first, first + size, width))
