"""Corners of the logit operators' definitions, against the float64 oracle or
against values worked by hand."""

import numpy as np
import pytest

import oracle as o
from tests._helpers import announce, host, require_gpu
from tests.test_gpu_logits import (LOW, bf16, check_distill, check_gradient, check_logprobs, dev, make, near, put,
                                   teacher_of, tol_lse)

pytestmark = pytest.mark.gpu
L = o.logits
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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [7, 300, 20000, 140001])
def test_masked_logits_close_to_the_unmasked(vocab, dtype):
    """Columns at or just below the bound count nothing, also beside unmasked
    ones a few units away. n equal unmasked logits: H = -ln p = ln n. bf16: the
    scale puts neighbouring values on both sides."""
    torch = require_gpu()
    import bit_block_scaled_bf16_amd as nv

    announce(f"masked logits close by {vocab} {dtype}")
    if dtype == "f32":
        scale, live_z, masked_z = 1.0, ABOVE, [-1e8, -100000008.0, -100000080.0]
    else:
        # -1e8 / scale lies between two neighbours of bf16, right below the upper
        live_z, masked_z = np.float32(-99614720.0), [-100139008.0, -100663296.0]
        scale = float(np.float32(1e8 * (1.0 - 2.0 ** -22) / 99614720.0))
    masked_z = np.array(masked_z, np.float32)
    scaled = lambda v: v.astype(np.float64) * np.float64(np.float32(scale))  # noqa: E731
    assert scaled(live_z) > -1e8 and (scaled(masked_z) <= -1e8).all()
    rng = np.random.default_rng(vocab)
    z = rng.choice(masked_z, (4, vocab))
    z[0, vocab // 2] = live_z
    z[1, ::3] = live_z
    z[2, : vocab // 2] = live_z
    z[3, vocab - 1] = z[3, 0] = live_z
    n = (z == live_z).sum(1)
    tokens = np.array([0, 1, vocab - 1, 1], np.int64)  # masked ones
    r = nv.token_logprobs(put(torch, z, dtype, 3, 1), dev(torch, tokens), top_k=2, scale=scale)
    tol = 2 * equal_tolerance(vocab) + U * np.log(n)
    assert np.isneginf(host(r.logp)).all()
    assert (np.abs(host(r.entropy) - np.log(n)) <= tol * (10 + np.log(n))).all(), host(r.entropy)
    assert (np.abs(host(r.top_logp)[:, 0] + np.log(n)) <= tol).all()
    assert (host(r.top_ids)[0] == [vocab // 2, -1]).all()
    ids = np.full((4, 1), -1, np.int32)
    ids[1:, 0] = [0, 0, 0]
    a = np.zeros((4, 1), np.float32)
    d = nv.distill(put(torch, z, dtype, 3, 1), dev(torch, ids), dev(torch, a), dev(torch, (z == live_z).argmax(1)), scale=scale)
    assert (np.abs(host(d.logp) + np.log(n)) <= tol).all()
    assert (np.abs(host(d.loss)[1:] - np.log(n)[1:]) <= 4 * tol[1:]).all()
    if vocab >= 300:  # alternatives at every place of a vector, in a row of enough unmasked logits
        ids = np.tile(np.arange(8, dtype=np.int32), (4, 1))
        d8 = nv.distill(put(torch, z, dtype, 3, 1), dev(torch, ids), dev(torch, np.full((4, 8), -np.log(8), np.float32)), tail=False,
                        scale=scale)
        assert abs(host(d8.loss)[2] - np.log(n[2] / 8)) <= 4 * tol[2] + 8 * U * np.log(8)
    lse = scaled(z).max(1) + np.log(n)
    near(host(d.lse), lse, 4 * U * 1e8, "lse")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [7, 300, 20000, 140001])
def test_gradient_of_masked_logits_close_to_the_unmasked(vocab, dtype):
    """It is 0, whatever the neighbours."""
    torch = require_gpu()
    import bit_block_scaled_bf16_amd as nv

    announce(f"gradient of masked logits close by {vocab} {dtype}")
    if dtype == "f32":
        scale, live_z, masked_z = 1.0, ABOVE, [-1e8, -100000008.0, -100000080.0]
    else:
        live_z, masked_z = np.float32(-99614720.0), [-100139008.0, -100663296.0]
        scale = float(np.float32(1e8 * (1.0 - 2.0 ** -22) / 99614720.0))
    rng = np.random.default_rng(vocab)
    z = rng.choice(np.array(masked_z, np.float32), (5, vocab))
    z[0, vocab // 2] = live_z
    z[1, ::3] = live_z
    z[2, : vocab // 2] = live_z
    z[3, vocab - 1] = z[3, 0] = live_z
    z[4, ::2] = live_z
    live = z == live_z
    # an lse right on the unmasked logits (float32 steps there are 8 wide), as the forward call may round it
    lse = np.full(5, np.float32(-99999992.0), np.float32) if dtype == "f32" else np.float32(live_z * np.float32(scale)) * np.ones(5, np.float32)
    one = torch.ones(5, device="cuda")
    zt = put(torch, z, dtype, 3, 1)
    tokens = dev(torch, live.argmax(1))
    off = lambda t: host(t.float())[~live]  # noqa: E731
    on = lambda t: host(t.float())[live]  # noqa: E731
    d = nv.token_logprobs_backward(zt, tokens, dev(torch, lse), one, one, one, scale)
    ones, label = np.ones(5, np.float32), live.argmax(1)
    check_gradient(host(d.float()), L.token_logprobs_backward(z, label, lse, ones, ones, ones, scale), z, scale, lse,
                   3 * ones, dtype)
    assert (off(d) == 0).all() and (on(d) != 0).any()
    ids = label.astype(np.int32)[:, None]
    a = np.full((5, 1), -0.5, np.float32)
    t = (dev(torch, ids), dev(torch, a), tokens)
    for tail in (True, False):
        d = nv.distill_backward(zt, *t, dev(torch, lse), dev(torch, lse), one, one, tail, scale)
        ref = L.distill_backward(z, ids, a, label, lse, lse, ones, ones, tail, scale)
        check_gradient(host(d.float()), ref, z, scale, lse, 3 * ones, dtype, 2 * live)
        assert (off(d) == 0).all(), tail
        d = nv.distill_step(zt, *t, d_loss=one, d_logp=one, tail=tail, scale=scale)[1]
        assert (off(d) == 0).all() and np.isfinite(on(d)).all(), tail
        same = zt.clone()
        nv.distill_step(same, *t, d_loss=one, d_logp=one, tail=tail, scale=scale, out=same)
        assert (off(same) == 0).all() and np.isfinite(on(same)).all(), tail


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_do_not_depend_on_the_alignment(dtype):
    """Their bits, the zeros' signs of masked columns among them, where columns
    move from a vector to a single thread."""
    torch = require_gpu()
    import bit_block_scaled_bf16_amd as nv

    announce(f"gradient bits at other alignments {dtype}")
    z = make(4, 333, dtype, 6)
    z[0, ::3], z[1, 1::2], z[2, 5:], z[3, :7] = -np.inf, LOW[dtype], -1e9, -2e8
    z = bf16(z) if dtype == "bf16" else z
    f = L.token_logprobs(z, np.zeros(4, np.int64))
    lse, ent = dev(torch, f["lse"].astype(np.float32)), dev(torch, f["entropy"].astype(np.float32))
    ids, a = teacher_of(z, 4, 1, ragged=False)
    tok = dev(torch, np.array([1, 0, 2, 9], np.int64))
    one = torch.ones(4, device="cuda")
    bits = lambda t: t.contiguous().view(torch.int16 if dtype == "bf16" else torch.int32)  # noqa: E731
    first = None
    for off in range(9):
        zt = put(torch, z, dtype, 1, off)
        out = put(torch, z, dtype, 3, off)
        got = [nv.token_logprobs_backward(zt, tok, lse, ent, one, -one, out=out).clone(),
               nv.token_logprobs_backward(zt, tok, lse, None, one, None, out=out).clone(),
               nv.distill_backward(zt, dev(torch, ids), dev(torch, a), tok, lse, lse, one, -one, out=out).clone()]
        first = first or got
        for x, y in zip(got, first):
            assert torch.equal(bits(x), bits(y)), off


# ---------------------------------------------------------------------------
# Nothing unmasked outside the alternatives
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("scale", [1.0, 0.125])
@pytest.mark.parametrize("mask", [-1e8, -1.2e8, -1.38e8, -1.5e8, -1e9])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [40, 3000, 40001, 140001])
def test_step_with_masks_of_finite_values_outside_the_alternatives(vocab, dtype, mask, scale):
    """A grammar that leaves fewer choices than the teacher names, masked by a
    number as a user writes it: no gradient outside, in the step as in the
    backward call."""
    torch = require_gpu()
    announce(f"no tail {vocab} {dtype} mask {mask} scale {scale}")
    mask = mask / scale
    rows, k = 3, 6
    z = make(rows, vocab, dtype, 4)
    ids, a = teacher_of(z, k, 3, ragged=False)
    out = np.ones(z.shape, bool)
    np.put_along_axis(out, ids, False, 1)
    z[out] = mask
    z[1, ids[1, 2:]] = mask                        # some of the alternatives too
    z = bf16(z) if dtype == "bf16" else z
    a[2] -= np.log(np.exp(a[2].astype(np.float64)).sum()).astype(np.float32)
    labels = np.array([ids[0, 0], ids[1, 1], (ids[2, 0] + 1) % vocab], np.int64)
    g = np.array([0.5, 1.0, 1.5], np.float32)
    for tail in (True, False):
        check_distill(torch, z, dtype, ids, a, labels, tail, scale, g, -g)


# ---------------------------------------------------------------------------
# Rows that take no gradient from their teacher
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("vocab", [50, 20000])
def test_a_teacher_without_weight_is_not_looked_at(vocab, tail):
    """d_loss 0 beside a label's gradient: what the teacher holds is no matter."""
    torch = require_gpu()
    import bit_block_scaled_bf16_amd as nv

    announce(f"a teacher without weight {vocab} tail={tail}")
    rows = 3
    z = make(rows, vocab, "f32", 6)
    ids, a = teacher_of(z, 5, 3, ragged=False)
    a[0, 2], a[1, 3] = np.nan, np.inf
    labels = np.array([1, ids[1, 3], ids[2, 0]], np.int64)
    gl, zero = np.array([1.0, -2.0, 0.5], np.float32), np.zeros(rows, np.float32)
    f = L.distill(z, None, None, labels)
    lse = f["lse"].astype(np.float32)
    ref = L.distill_backward(z, None, None, labels, lse, lse, None, gl)
    zt = put(torch, z, "f32")
    t = (dev(torch, ids), dev(torch, a), dev(torch, labels))
    one = np.zeros(z.shape)
    one[np.arange(rows), labels] = np.abs(gl)
    for weight in (None, dev(torch, zero)):
        d = nv.distill_backward(zt, *t, dev(torch, lse), dev(torch, lse), weight, dev(torch, gl), tail)
        check_gradient(host(d), ref, z, 1.0, lse, np.abs(gl), "f32", one)
        d = nv.distill_step(zt, *t, d_loss=weight, d_logp=dev(torch, gl), tail=tail)[1]
        # its own L: off by at most the forward's tolerance, and u |L| from its rounding to float32
        p = np.exp(z.astype(np.float64) - f["lse"][:, None])
        slack = p * np.abs(gl)[:, None] * (2 * tol_lse(z, 1.0, f["lse"]) + 2 * U * np.abs(f["lse"]))[:, None] * 2 / (8 * U)
        check_gradient(host(d), ref, z, 1.0, lse, np.abs(gl), "f32", one + slack)


# ---------------------------------------------------------------------------
# No teacher
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("vocab", [9, 3000, 40001])
def test_without_a_teacher_there_is_no_divergence(vocab, tail):
    """Also in a row with nothing unmasked (a padded position of a cross entropy
    step): its loss is 0 and not in the way of a mean."""
    torch = require_gpu()
    import bit_block_scaled_bf16_amd as nv

    announce(f"no teacher {vocab} tail={tail}")
    z = make(4, vocab, "f32", 8)
    z[1], z[2] = -np.inf, LOW["f32"]
    labels = np.array([1, -1, 2, 0], np.int64)
    want = L.distill(z, None, None, labels, tail)
    assert (want["loss"] == 0).all()
    zt = put(torch, z, "f32")
    w = torch.ones(4, device="cuda")
    r = nv.distill(zt, None, None, dev(torch, labels), tail=tail)
    s, d = nv.distill_step(zt, None, None, dev(torch, labels), d_loss=w, d_logp=-w, tail=tail)
    for x in (r, s):
        assert (host(x.loss) == 0).all(), host(x.loss)
        assert np.isneginf(host(x.lse)[1:3]).all() and host(x.logp)[1] == 0 and np.isneginf(host(x.logp)[2])
    assert (host(d)[1:3] == 0).all()
    z[3, 4] = np.nan  # still told
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = nv.distill(put(torch, z, "f32"), None, None, dev(torch, labels), tail=tail, dev_status=flag)
    assert np.isnan(host(r.loss)[3]) and (host(r.loss)[:3] == 0).all() and int(flag.item()) == 1
