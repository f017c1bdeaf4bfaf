"""The divergence of a student near its teacher, against the float64 oracle and
relative to its own size (u = 2^-24).

The kernel sums terms q (ln(q / p) - 1) + p >= 0, which vanish with (q - p)^2. So
an error e_t of a term's ln p changes the loss by |q_t - p_t| e_t, and an error
E of L, which all terms share, by |Q - P| E only (Q the teacher's mass on the
terms, P the student's; both are 1 where the remaining masses are a term too).

* e_j of an alternative: 2 u S (c is rounded twice; S the largest |s|),
  u (1.45 |s_j - L| + 25) for the exponent's own rounding (the sum's reference is
  at most 25 powers of two from L), and 2 u each of |ln p|, |ln q| and 1 for the
  products, logarithms and differences that follow: u (2 S + 4 |s_j - L| +
  2 |ln q| + 40).
* E of a sum: its terms' exponentials as above, a thread adds at most V / 64 terms
  in a row and the joining tree 16: u (2 S + V / 64 + 60). The remaining mass's
  term takes this and 4 u (|ln p_r| + |ln q_r|).
* second order: (e + E)^2. The terms' own rounding, and the tree that adds
  them: 24 u of their sum (a term with |ln(q / p)| just above 1 takes 7).
"""

import numpy as np
import pytest

import oracle as o
from tests._helpers import announce, host, require_gpu
from tests.test_gpu_logits import bf16, dev, put

pytestmark = pytest.mark.gpu
L = o.logits
U = 2.0 ** -24


def pair(rows, vocab, k, noise, dtype, scale, kind, seed):
    """Student logits and a teacher that differs from them by `noise`. kind
    "top": the teacher's k most probable tokens, as they are; "whole": they hold
    all of its mass, and nearly all of the student's."""
    rng = np.random.default_rng(seed)
    z = rng.normal(0.0, 2.0, (rows, vocab))
    z[np.arange(rows)[:, None], rng.integers(0, vocab, (rows, 8))] += 6.0
    if kind == "whole":
        out = np.ones(z.shape, bool)
        np.put_along_axis(out, np.argpartition(-z, k - 1, 1)[:, :k], False, 1)
        z[out] -= 45.0
    z = (bf16(z.astype(np.float32)) if dtype == "bf16" else z.astype(np.float32))
    t = (z.astype(np.float64) + noise * rng.normal(size=z.shape)) * scale
    ids = np.argpartition(-t, k - 1, 1)[:, :k] if k < vocab else np.tile(np.arange(vocab), (rows, 1))
    top = t.max(1, keepdims=True)
    t -= top + np.log(np.exp(t - top).sum(1, keepdims=True))
    a = np.take_along_axis(t, ids, 1)
    if kind == "whole":
        a -= np.log(np.exp(a).sum(1, keepdims=True))
    return z, ids.astype(np.int32), a.astype(np.float32)


def loss_bound(z, ids, a, tail, scale):
    rows, vocab = z.shape
    tol = np.zeros(rows)
    for i in range(rows):
        s = z[i].astype(np.float64) * scale
        lse = L._lse(s)
        q, rest = L.teacher(ids[i], a[i], tail)
        x = s[ids[i]] - lse
        p = np.exp(x)
        big = np.abs(s).max()
        ln_q = np.log(np.where(q > 0, q, 1.0))
        e = U * (2 * big + 4 * np.abs(x) + 2 * np.abs(ln_q) + 40)
        e_sum = U * (2 * big + vocab / 64 + 60)
        out = np.ones(vocab, bool)
        out[ids[i]] = False
        p_rest = np.exp(L._lse(s[out]) - lse) if out.any() else 0.0
        terms = (q * (ln_q - x) - q + p)[q > 0].sum()
        first = (np.abs(q - p) * e)[q > 0].sum()
        total_q, total_p = q.sum(), p[q > 0].sum()
        if rest > 0:
            ln = np.abs(np.log(rest)) + np.abs(np.log(p_rest))
            first += abs(rest - p_rest) * (e_sum + 4 * U * ln)
            terms += rest * (np.log(rest) - np.log(p_rest)) - rest + p_rest
            total_q, total_p = total_q + rest, total_p + p_rest
        apart = abs(total_q - total_p)
        tol[i] = first + apart * (e_sum + e.max()) + (e.max() + e_sum) ** 2 + 24 * U * (abs(terms) + apart)
    return tol


NEAR = [(48, 3000, 64, "f32"), (48, 3000, 64, "bf16"), (40, 20011, 32, "f32"), (40, 20011, 32, "bf16"),
        (48, 5000, 1, "f32"), (3, 140001, 64, "f32"), (1100, 777, 100, "f32")]


@pytest.mark.parametrize("kind", ["top", "whole"])
@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("noise", [0.7, 0.02, 0.002])
@pytest.mark.parametrize("rows,vocab,k,dtype", NEAR)
def test_loss_near_the_teacher(rows, vocab, k, dtype, noise, tail, kind):
    torch = require_gpu()
    import bit_block_scaled_bf16_amd as nv

    announce(f"loss near the teacher {rows}x{vocab} k={k} {dtype} noise {noise} tail={tail} {kind}")
    scale = [1.0, 0.7][vocab % 2]
    z, ids, a = pair(rows, vocab, k, noise, dtype, scale, kind, vocab + k)
    want = L.distill(z, ids, a, None, tail, scale)["loss"]
    tol = loss_bound(z, ids, a, tail, scale)
    zt, t = put(torch, z, dtype, 3, 1), (dev(torch, ids), dev(torch, a))
    weights = torch.ones(rows, device="cuda")
    for name, r in (("distill", nv.distill(zt, *t, tail=tail, scale=scale)),
                    ("step", nv.distill_step(zt, *t, d_loss=weights, tail=tail, scale=scale)[0])):
        off = np.abs(host(r.loss).astype(np.float64) - want)
        assert (off <= tol).all(), (name, (off / tol).max(), off.max(), want.min())


@pytest.mark.parametrize("tail", [True, False])
def test_loss_with_doubled_absent_and_massless_alternatives(tail):
    """The student's mass counts once a term: ids named twice or three times, ids
    without mass, absent ones, and the teacher's masses a little over 1."""
    torch = require_gpu()
    import bit_block_scaled_bf16_amd as nv

    announce(f"loss with doubled alternatives tail={tail}")
    rows, vocab, k = 6, 900, 70
    z, ids, a = pair(rows, vocab, k, 0.3, "f32", 1.0, "top", 5)
    ids[0, 3] = ids[0, 1]
    ids[1, 69] = ids[1, 2] = ids[1, 66]
    a[2, 4:9] = -np.inf
    ids[3, 20:] = -1
    a[4] += np.float32(0.01) - np.log(np.exp(a[4].astype(np.float64)).sum()).astype(np.float32)
    a[5, 1:] = -np.inf
    ids[5, 2] = ids[5, 0]
    a[0, 2] = -200.0  # no mass in float32
    want = L.distill(z, ids, a, None, tail, 1.0)["loss"]
    # the terms are not all of one sign here: u of each, 64 times, and e as above
    tol = np.zeros(rows)
    for i in range(rows):
        q, rest = L.teacher(ids[i], a[i], tail)
        s = z[i].astype(np.float64)
        x = s[ids[i]] - L._lse(s)
        tol[i] = 64 * U * (1 + (q * np.abs(np.log(np.where(q > 0, q, 1)) - x)).sum()) + U * (2 * np.abs(s).max() + vocab / 64 + 60)
    got = nv.distill(put(torch, z, "f32"), dev(torch, ids), dev(torch, a), tail=tail)
    off = np.abs(host(got.loss).astype(np.float64) - want)
    assert (off <= tol).all(), (off, tol)
