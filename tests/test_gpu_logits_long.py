"""The logit operators on rows longer than a workgroup's registers or 16 vectors
of a span hold: vocabularies above 131072 bf16 or 65536 float32 columns."""

import numpy as np
import pytest

import oracle as o
from tests._helpers import announce, host, require_gpu
from tests.test_gpu_logits import (check_distill, check_logprobs, dev, make, near, put, teacher_of, tokens_of,
                                   tol_lse)

pytestmark = pytest.mark.gpu
L = o.logits
U = 2.0 ** -24


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("rows,vocab,dtype,off", [
    (2, 70001, "f32", 0), (2, 70001, "f32", 33), (2, 65540, "f32", 1),        # whole rows, few of them
    (64, 150001, "bf16", 33), (64, 131080, "bf16", 0), (64, 140003, "f32", 1),  # the same, from 64 rows on
    (2, 150001, "bf16", 1), (2, 140007, "f32", 0)])                           # forward and gradient apart
def test_step_of_long_rows(rows, vocab, dtype, off, tail):
    """Alternatives and labels in what the registers hold, beyond it, on both sides
    of the border and at the row's ends; in place too (check_distill)."""
    torch = require_gpu()
    announce(f"step of long rows {rows}x{vocab} {dtype} tail={tail} off={off}")
    border = 1024 * 16 * (8 if dtype == "bf16" else 4)
    z = make(rows, vocab, dtype, vocab)
    ids, a = teacher_of(z, 12, 5, ragged=False)
    lead = -off % (64 if dtype == "bf16" else 32)  # columns up to the row's first whole line
    fixed = [0, 1, 7, border - 9, border - 1, border + 1, vocab - 9, vocab - 1, vocab - 2, min(vocab - 3, border + lead)]
    for i in range(rows):
        rest = [v for v in ids[i] if v not in fixed]
        ids[i] = (fixed + rest)[:12]
    labels = np.where(np.arange(rows) % 2 == 0, vocab - 1, border + 3).astype(np.int64)
    g = np.linspace(1.0, -0.5, rows).astype(np.float32)
    z[1, border // 2:border // 2 + 3000] = -np.inf
    check_distill(torch, z, dtype, ids, a, labels, tail, 1.0, g, -g, pad=5, off=off)
    if rows == 2:
        labels = np.array([2, vocab - 3], np.int64)
        check_distill(torch, z, dtype, None, None, labels, tail, 1.0, None, g, pad=0, off=off)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 140003), ("f32", 70003)])
def test_step_of_many_long_rows(dtype, vocab):
    """The copies of two rows all get the same bits, in place or not."""
    torch = require_gpu()
    import bit_block_scaled_bf16_amd as nv

    announce(f"step of many long rows {vocab} {dtype}")
    many = 65
    ld = vocab + (-vocab) % 64  # every row starts on a line
    z = make(2, vocab, dtype, 3)
    ids, a = teacher_of(z, 20, 5)
    g = np.array([0.5, -1.5], np.float32)
    t = [dev(torch, np.concatenate([v] * many)) for v in (ids, a, np.array([5, vocab - 1], np.int64), g, -g)]
    zz = put(torch, np.concatenate([z] * many), dtype, ld - vocab)
    want = L.distill(z, ids, a)
    first = None
    for out in (None, zz):
        r, d = nv.distill_step(zz, *t[:3], d_loss=t[3], d_logp=t[4], out=out)
        got = [v.reshape(many, 2, -1) for v in (*r, d)]
        near(host(r.lse)[:2], want["lse"], tol_lse(z, 1.0, want["lse"]), "lse")
        first = first or [v[:1].clone() for v in got]
        for x, y in zip(got, first):
            assert torch.equal(x, y.expand_as(x))


@pytest.mark.parametrize("k", [1, 20, 128])
@pytest.mark.parametrize("dtype,vocab", [("bf16", 140001), ("bf16", 290001), ("f32", 100001), ("f32", 150001)])
def test_alternatives_of_many_long_rows(dtype, vocab, k):
    """A workgroup takes whole rows of more than 8 tiles: spans of 2 tiles (one
    vector each is read again) and of 3 and more (all of the span is)."""
    torch = require_gpu()
    import bit_block_scaled_bf16_amd as nv

    announce(f"alternatives of many long rows {vocab} {dtype} k={k}")
    rows, many = 8, 128
    z = make(rows, vocab, dtype, vocab + k)
    z[1] = np.sort(z[1])
    z[2] = z[2, 0]
    z[3, 10000:] = -np.inf
    z[4, :] = -1e9
    z[4, vocab // 2:vocab // 2 + 60] = make(1, 60, dtype, 1)
    z[5, -200:] += 40.0 if dtype == "bf16" else 40.5
    z[6, ::2500] += 64.0
    z = z if dtype == "f32" else host(torch.from_numpy(z).bfloat16().float())
    tokens = tokens_of(rows, vocab, 2)
    want = L.token_logprobs(z, tokens, k)
    check_logprobs(torch, z, dtype, tokens, k, pad=3)
    for pad in (0, 3):
        zz = put(torch, z, dtype, pad)
        zz = torch.cat([torch.cat([zz, zz.new_zeros(rows, pad)], 1)] * many)[:, :vocab]
        r = nv.token_logprobs(zz, dev(torch, np.tile(tokens, many)), top_k=k)
        assert np.array_equal(host(r.top_ids), np.tile(want["top_ids"], (many, 1)))
        # and the same log probabilities as the check of the few rows has, up to the sums' order: both
        # within 2 (2 u (1.45 S + V / 128 + 24) + u |L|) of the truth, S the largest unmasked |s|
        got, alone = host(r.top_logp)[:rows], host(nv.token_logprobs(put(torch, z, dtype, pad), top_k=k).top_logp)
        assert np.array_equal(np.isneginf(got), np.isneginf(alone))
        fine = np.isfinite(alone)
        bound = 4 * tol_lse(z, 1.0, want["lse"])[:, None] + 2 * U * np.where(fine, np.abs(alone), 0)
        assert (np.abs(got - alone) <= bound)[fine].all()
