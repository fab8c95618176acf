"""The operators together: examples/speculative_gdn.py."""
import os
import sys

import numpy as np
import pytest
import torch
from scipy import stats

import oracle
from gpu_helpers import i32

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from speculative_gdn import Model, generate  # noqa: E402

pytestmark = pytest.mark.gpu


def models(vocab, same=False):
    target = Model(1, 2, 2, 4, 128, vocab)
    draft = Model(1 if same else 2, 2 if same else 1, 2, 4, 128, vocab, target.embedding)
    draft.head = target.head
    return target, draft


@pytest.mark.parametrize("n_draft", [1, 3])
def test_rolled_back_states_are_those_of_the_accepted_tokens(n_draft):
    """After many accepted and refused drafts the target's first layer, whose inputs are the
    tokens' embeddings alone, holds the state that a prefill of the tokens leaves.

    The projections of another batch shape may add up in another order, so that a bf16 k or v
    rounds the other way, by 2^-8 each; twice that for what tokens add to one entry, 2^-6.  A
    state after one token too many or too few is off by its update, of the state's own size."""
    target, draft = models(50)
    prompts = [[3], [1, 2, 3, 4], list(range(40)), [9] * 70]
    rows, accepted, states = generate(target, draft, prompts, 30, n_draft)
    assert 0 < accepted < n_draft and all(len(r) >= len(p) + 30 for r, p in zip(rows, prompts))
    lens = [len(r) - 1 for r in rows]
    with target.pool(len(rows), 0) as pool:
        ids = i32(pool.create(len(rows)))
        cu = i32(np.concatenate([[0], np.cumsum(lens)]))
        target.probs(i32(np.concatenate([r[:-1] for r in rows])),
                     lambda layer, *x: pool.prefill(layer, ids, cu, *x, max_seqlen=max(lens), l2norm_eps=1e-6))
        assert pool.device_status() == 0
        for i in range(len(rows)):
            assert oracle.rel_err(states[i, 0].cpu().numpy(), pool.states[i, 0].cpu().numpy()) < 2.0 ** -6


def test_a_model_accepts_its_own_drafts():
    """Draft = target: p and q differ by rounding alone, and few drafts are refused."""
    target, draft = models(50, same=True)
    _, accepted, _ = generate(target, draft, [[5, 6]] * 64, 20, 3)
    assert accepted > 2.8


def test_first_tokens_have_the_targets_distribution():
    """Of 8,192 rows with one prompt, the first new token against the target's probabilities:
    a chi-square test that a right sampler fails once in 10^6 seeds."""
    target, draft = models(12)
    n = 8192
    rows, accepted, _ = generate(target, draft, [[3, 1, 4, 1, 5]] * n, 1, 2, seed=5)
    got = np.bincount([r[5] for r in rows], minlength=12)
    with target.pool(1, 0) as pool:
        ids = i32(pool.create(1))
        p = target.probs(i32([3, 1, 4, 1, 5]), lambda layer, *x: pool.prefill(layer, ids, i32([0, 5]), *x, l2norm_eps=1e-6))
    p = p[-1].double().cpu().numpy()
    assert stats.chisquare(got, p / p.sum() * n).pvalue > 1e-6
    assert 0 < accepted < 2
