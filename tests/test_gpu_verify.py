"""GPU tests of draft verification (wkv7_verify_drafts) against the oracle's entry-by-entry
rule.  Every value compared is a single correctly rounded float32 operation, so the
results, whole numbers, must be equal."""
import numpy as np
import pytest
import torch

from gpu_helpers import i32
from oracle.gdn import verify_drafts
from rwkv_wkv_gb300 import DEV_BAD_SEQLENS, DEV_BAD_SLOT, DEV_BAD_TOKEN, GdnPool, Pool, Wkv7Error

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rows(rng, n, r, vocab, pad, dtype):
    z = rng.standard_normal((n, r, vocab)) * 2.5
    p = np.exp(z - z.max(-1, keepdims=True))
    x = torch.zeros(n, r, vocab + pad, dtype=DT[dtype], device="cuda")[..., :vocab]
    x.copy_(torch.from_numpy((p / p.sum(-1, keepdims=True)).astype(np.float32)))
    return x


def case(seed, n, K, vocab, pad=0, dtype="f32", draft=True, ragged=False):
    rng = np.random.default_rng(seed)
    p = rows(rng, n, K + 1, vocab, pad, dtype)
    q = None
    if draft:
        q = torch.zeros(n, K, vocab + pad, dtype=DT[dtype], device="cuda")[..., :vocab]
        mix = rows(rng, n, K, vocab, 0, "f32")
        q.copy_(0.8 * p[:, :K].float() + 0.2 * mix)
    src = (q if draft else p[:, :K]).float().cpu().numpy()
    ids = (src / rng.exponential(size=src.shape)).argmax(-1).astype(np.int32)
    noise = torch.zeros(n, vocab + pad, device="cuda")[:, :vocab]
    noise.copy_(torch.from_numpy(rng.exponential(size=(n, vocab)).astype(np.float32)))
    u = torch.from_numpy(rng.random((n, K)).astype(np.float32)).cuda()
    nd = i32(rng.integers(0, K + 1, n)) if ragged else None
    return ids, p, q, u, noise, nd


def expect(ids, p, q, u, noise, nd):
    f = lambda x: None if x is None else x.float().cpu().numpy()  # noqa: E731
    return verify_drafts(ids, f(p), f(q), f(u), f(noise), None if nd is None else nd.cpu().numpy())


def check(pool, ids, p, q, u, noise, nd, snaps=None):
    accepted, tokens, resume = pool.verify_drafts(i32(ids), p, q, u, noise, n_draft=nd, step_snap_ids=snaps)
    assert pool.device_status() == 0
    a, t = expect(ids, p, q, u, noise, nd)
    assert np.array_equal(accepted.cpu().numpy(), a)
    assert np.array_equal(tokens.cpu().numpy(), t)
    if snaps is not None:
        assert torch.equal(resume, snaps[torch.arange(len(a)), torch.from_numpy(a).long()])
    else:
        assert resume is None
    return a


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("n,K,vocab,pad", [(1, 1, 1, 0), (1, 0, 37, 0), (3, 2, 2, 1), (7, 4, 1001, 3), (5, 40, 300, 4),
                                           (2, 3, 65529, 0), (1, 4, 65536, 0), (400, 2, 5000, 8), (9, 1, 40000, 1)])
def test_matches_the_rule(dtype, draft, n, K, vocab, pad):
    with Pool(1, 1, 1, n_snapshots=n * (K + 1)) as pool:
        snaps = i32(np.random.default_rng(1).permutation(n * (K + 1)).reshape(n, K + 1))
        for ragged in (False, True):
            check(pool, *case(n * 31 + K, n, K, vocab, pad, dtype, draft, ragged), snaps=snaps)


def test_accepts_and_refuses_in_every_place():
    ids, p, q, u, noise, _ = case(5, 64, 4, 500)
    with GdnPool(1, 1, 1, 1) as pool:
        for m in range(5):
            v = torch.zeros_like(u)
            p2 = p.clone()
            if m < 4:  # the m-th draft is impossible
                p2[torch.arange(64), m, torch.from_numpy(ids[:, m]).long()] = 0
            assert (check(pool, ids, p2, q, v, noise, None) == m).all()


def test_ties_empty_residuals_and_odd_values():
    vocab, K = 4097, 2
    ids, p, q, u, noise, _ = case(6, 8, K, vocab)
    u.fill_(0.999)
    noise.fill_(1.0)
    p.zero_(), q.zero_()
    p[0, 0, [5, 4000, 17]] = 0.25            # equal scores: the lowest index
    q[1, 0, 9] = 1.0                         # p empty everywhere, draft refused: no token
    ids[1, 0] = 9
    p[2] = 1 / vocab                         # q = p and a draft outside p: the residual is empty, p decides
    q[2] = 1 / vocab
    p[2, 0, 3], q[2, 0, 3] = 0.0, 0.5
    ids[2, 0] = 3
    noise[3, 11] = 0.0                       # an infinite score
    p[3, 0, [2, 11, 12]] = 0.3
    noise[3, 12] = 0.0
    p[4, 0] = float("nan")                   # nothing is larger than NaN
    p[5, 0, 100], p[5, 0, 200] = float("nan"), 1e-42
    p[6, 0, 7], q[6, 0, 7] = float("inf"), 0.5
    p[7, 0, vocab - 1] = 1e-30
    with Pool(1, 1, 1) as pool:
        accepted, tokens, _ = pool.verify_drafts(i32(ids), p, q, u, noise)
        assert pool.device_status() == 0
        a, t = expect(ids, p, q, u, noise, None)
        assert np.array_equal(accepted.cpu().numpy(), a) and np.array_equal(tokens.cpu().numpy(), t)
        first = tokens[:, 0].tolist()
        assert first[0] == 5 and first[1] == -1 and first[2] == 0 and first[3] == 11 and first[4] == -1
        assert first[5] == 200 and first[7] == vocab - 1


def test_sampled_tokens_follow_the_target():
    """Over many rows the first token's distribution is the target's, whatever the draft's."""
    vocab, n = 8, 200_000
    gen = torch.Generator(device="cuda").manual_seed(3)
    p = torch.tensor([0.3, 0.05, 0.15, 0.0, 0.2, 0.1, 0.15, 0.05], device="cuda")
    q = torch.tensor([0.05, 0.3, 0.1, 0.2, 0.0, 0.1, 0.05, 0.2], device="cuda")
    ids = torch.multinomial(q, n, replacement=True, generator=gen).to(torch.int32).view(n, 1)
    u = torch.rand(n, 1, device="cuda", generator=gen)
    noise = torch.empty(n, vocab, device="cuda").exponential_(generator=gen)
    with Pool(1, 1, 1) as pool:
        _, tokens, _ = pool.verify_drafts(ids, p.expand(n, 2, vocab), q.expand(n, 1, vocab), u, noise)
    share = torch.bincount(tokens[:, 0].long(), minlength=vocab).double().cpu() / n
    # five standard deviations of a share of n draws
    assert bool(((share - p.double().cpu()).abs() <= 5 * (p.double().cpu() * (1 - p.double().cpu()) / n).sqrt()).all())


def test_device_faults():
    ids, p, q, u, noise, _ = case(7, 4, 3, 1000)
    snaps = i32(np.arange(16).reshape(4, 4))
    bad = ids.copy()
    bad[1, 2] = 1000
    with Pool(1, 1, 1, n_snapshots=16) as pool:
        a, t, r = pool.verify_drafts(i32(bad), p, q, u, noise, step_snap_ids=snaps)
        assert pool.device_status() == DEV_BAD_TOKEN
        assert a[1] == -1 and (t[1] == -1).all() and r[1] == -1
        ra, rt = expect(ids, p, q, u, noise, None)
        assert np.array_equal(a.cpu().numpy()[[0, 2, 3]], ra[[0, 2, 3]])
        assert np.array_equal(t.cpu().numpy()[[0, 2, 3]], rt[[0, 2, 3]])
        a, t, _ = pool.verify_drafts(i32(ids), p, q, u, noise, n_draft=i32([3, 4, -1, 0]))
        assert pool.device_status() == DEV_BAD_SEQLENS
        assert a.tolist()[1:3] == [-1, -1] and a[3] == 0
        a, t, r = pool.verify_drafts(i32(ids), p, q, u, noise, step_snap_ids=snaps + 16)
        assert pool.device_status() == DEV_BAD_SLOT
        assert (r == -1).all() and np.array_equal(a.cpu().numpy(), ra)


def test_refusals():
    ids, p, q, u, noise, _ = case(8, 2, 2, 64)
    ids = i32(ids)
    with Pool(1, 1, 1) as pool:
        for args in ((ids, p.half(), q, u, noise), (ids, p, q.to(torch.bfloat16), u, noise),
                     (ids.long(), p, q, u, noise), (ids, p, q, u, noise.double())):
            with pytest.raises(TypeError):
                pool.verify_drafts(*args)
        for args in ((ids, p[:, :2], q, u, noise), (ids, p, q, u[:, :1], noise), (ids, p, q, u, noise[:1]),
                     (ids, p.transpose(1, 2).contiguous().transpose(1, 2), q, u, noise)):
            with pytest.raises(ValueError):
                pool.verify_drafts(*args)
        with pytest.raises(ValueError):
            pool.verify_drafts(ids, p, q, u, noise, step_snap_ids=i32([0, 1]))
        with pytest.raises(Wkv7Error, match="INVALID_ARG"):   # rows that overlap
            pool.verify_drafts(ids, torch.as_strided(p, (2, 3, 64), (192, 8, 1)), q, u, noise)


def test_chosen_ids_are_there_for_the_next_call():
    """A decode call reads its slot ids before earlier kernels end; ids that verify_drafts chose
    (here among candidate slots) must be there all the same.  In a graph, where the second
    kernel is ready while the first one runs."""
    n, vocab, heads = 64, 130001, 4
    rng = np.random.default_rng(23)
    p = torch.rand(n, 2, vocab, device="cuda")
    noise = torch.rand(n, vocab, device="cuda") + 0.1
    uniforms = torch.zeros(n, 1, device="cuda")
    drafts = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    ids = torch.zeros(n, 2, dtype=torch.int32, device="cuda")
    with GdnPool(1, heads, heads, 2 * n, n_snapshots=2 * n, head_k=64, head_v=64) as pool:
        x = [torch.randn(n, heads, 64, device="cuda") for _ in range(3)]
        gates = [torch.zeros(n, heads, device="cuda"), torch.ones(n, heads, device="cuda")]
        o = torch.empty(n, heads, 64, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            accepted, _, slots = pool.verify_drafts(drafts, p, None, uniforms, noise, step_snap_ids=ids)
            pool.decode_step(0, slots, *x, *gates, o=o)
        for turn in range(20):
            refused = torch.from_numpy(rng.integers(0, 2, n).astype(np.int32)).cuda()
            p[:, 0, 0] = 1.0 - refused        # u q < p: accepted unless p = 0
            ids.copy_(i32(rng.permutation(2 * n)).view(n, 2))
            pool.states.zero_()
            graph.replay()
            assert pool.device_status() == 0
            assert torch.equal(accepted, 1 - refused)
            touched = pool.states.flatten(1).abs().amax(1) > 0
            want = torch.zeros(2 * n, dtype=torch.bool, device="cuda")
            want[ids.gather(1, accepted.long()[:, None])[:, 0].long()] = True
            assert torch.equal(touched, want), turn
