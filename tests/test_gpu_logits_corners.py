"""Corners of the logit operators' definitions, against the float64 oracle or
against values worked by hand."""

import numpy as np
import pytest

from tests._helpers import announce, host, require_gpu
from tests.test_gpu_logits import check_distill, check_logprobs, dev, make, put, teacher_of

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


# ---------------------------------------------------------------------------
# Unmasked logits just above the bound of -1e8
# ---------------------------------------------------------------------------

ABOVE = np.float32(-99999992.0)  # the float32 next to -1e8


def equal_tolerance(vocab):
    """How far L - s may be off for equal logits: their exponents' errors are the
    same and cancel, so of the bound in test_gpu_logits.py what a sum adds is left."""
    return 2 * U * (vocab / 128 + 24)


def rows_above_the_bound(vocab):
    """float32 rows whose unmasked logits lie within 7000 of the bound, alone, far
    from masked ones, and beside ordinary logits."""
    rng = np.random.default_rng(vocab)
    z = np.full((7, vocab), -1e9, np.float32)
    z[0, vocab // 2] = ABOVE                       # one alone
    z[1, ::3] = ABOVE                              # equal ones
    z[2, ::2] = -99995000.0
    z[3, 1::2] = -99993500.0
    z[4] = ABOVE                                   # ordinary logits beside
    z[4, ::5] = rng.normal(size=z[4, ::5].shape)
    z[5] = rng.choice(np.array([ABOVE, -99996000.0, -99993400.0, -2e8], np.float32), vocab)
    z[6, -1] = ABOVE
    return z


@pytest.mark.parametrize("vocab", [3, 40, 2500, 20000, 140001])
def test_logits_just_above_the_mask_bound(vocab):
    """In float32 an additive mask of -1e8 puts a logit of 5 there."""
    torch = require_gpu()
    announce(f"logits above the bound {vocab}")
    z = rows_above_the_bound(vocab)
    tokens = np.full(len(z), vocab // 2, np.int64)
    r = check_logprobs(torch, z, "f32", tokens, min(vocab, 4), pad=3)
    n = len(range(0, vocab, 3))
    lse = equal_tolerance(vocab)
    assert abs(host(r.entropy)[1] - np.log(n)) <= 2 * lse * (10 + np.log(n))
    top = host(r.top_logp)[1][:min(n, min(vocab, 4))]
    assert (np.abs(top + np.log(n)) <= 2 * lse + U * np.log(n)).all()
    ids, a = teacher_of(make(len(z), vocab, "f32", 2), min(vocab, 3), 3, ragged=False)
    ids[:, 0] = vocab // 2
    for j in range(1, ids.shape[1]):
        ids[:, j] = (vocab // 2 + j) % vocab
    for tail in (True, False):
        check_distill(torch, z, "f32", ids, a, tokens, tail, 1.0, None, None)
