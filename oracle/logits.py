"""Operators on a vocabulary's logits, row by row in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages judge the recipe by the validation loss of the trained model
(gist.science summary, Resumen técnico §4) and give no formula for it; these
are the textbook definitions. With s_v = scale * z_v over the unmasked columns
(s_v > -1e8): L = ln sum e^s, p = e^(s - L).

* log probability of token t: s_t - L; -inf if t is masked; 0 if t < 0.
* entropy: -sum p (s - L).
* alternatives: the k largest unmasked z, equal ones by rising column; -1 and
  -inf where no more are left.
* teacher masses from log probabilities a_j of the present ids: q_j = e^(a_j)
  with the rest q_r = 1 - sum q (0 below 1e-6), or q = softmax(a), q_r = 0.
* divergence: sum q_j (ln q_j - ln p_id_j) + q_r (ln q_r - ln p_r), p_r the
  student's mass on the columns that are no alternative. 0 without a teacher.

A row that holds NaN or an s_v > 1e8 (+inf), or an index beyond the vocabulary, gives
NaN in what depends on it.
"""

from __future__ import annotations

import numpy as np

MASKED = -1e8
MOST = 1e8
LEAST_TAIL = 1e-6


def _lse(s: np.ndarray) -> float:
    top = s.max() if s.size else -np.inf
    if not np.isfinite(top):
        return top if top == -np.inf else np.nan
    return float(top + np.log(np.exp(s - top).sum()))


def _scaled(z: np.ndarray, scale: float) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        return np.where(z * scale <= MASKED, -np.inf, z * scale)


def _row_lse(s: np.ndarray) -> float:
    return np.nan if np.isnan(s).any() or (s > MOST).any() else _lse(s)


def _logp(s: np.ndarray, lse: float, token: int) -> float:
    if token < 0:
        return 0.0
    if token >= s.size or np.isnan(lse):
        return np.nan
    return -np.inf if s[token] == -np.inf else float(s[token] - lse)


def token_logprobs(z, tokens=None, k: int = 0, scale: float = 1.0):
    """dict of logp, entropy, lse, top_ids, top_logp."""
    rows, vocab = z.shape
    out = {"logp": np.zeros(rows), "entropy": np.zeros(rows), "lse": np.zeros(rows),
           "top_ids": np.full((rows, k), -1, np.int32), "top_logp": np.full((rows, k), -np.inf)}
    for i in range(rows):
        s = _scaled(z[i], scale)
        lse = _row_lse(s)
        out["lse"][i] = lse
        if tokens is not None:
            out["logp"][i] = _logp(s, lse, int(tokens[i]))
        if np.isnan(lse):
            out["entropy"][i] = np.nan
            out["top_logp"][i] = np.nan
            continue
        live = np.flatnonzero(s > -np.inf)
        if live.size:
            x = s[live] - lse
            out["entropy"][i] = -(np.exp(x) * x).sum()
        best = live[np.lexsort((live, -np.asarray(z[i], np.float64)[live]))][:k]
        out["top_ids"][i, :best.size] = best
        out["top_logp"][i, :best.size] = s[best] - lse
    return out


def token_logprobs_backward(z, tokens, lse, entropy=None, d_logp=None, d_entropy=None,
                            scale: float = 1.0) -> np.ndarray:
    rows, vocab = z.shape
    out = np.zeros((rows, vocab))
    for i in range(rows):
        s = _scaled(z[i], scale)
        t = int(tokens[i]) if d_logp is not None else -1
        g = float(d_logp[i]) if t >= 0 else 0.0
        h = float(d_entropy[i]) if d_entropy is not None else 0.0
        if g == 0.0 and h == 0.0:
            continue
        live = ~(s == -np.inf)
        x = s[live] - float(lse[i])
        p = np.exp(x)
        d = -g * p
        if h != 0.0:
            d = d - h * p * (x + float(entropy[i]))
        out[i, live] = d
        if t >= vocab:
            if g != 0.0:
                out[i, live] = np.nan
        elif t >= 0 and live[t]:
            out[i, t] += g
        out[i] *= scale
    return out


def teacher(ids, logp, tail: bool):
    """(masses q of one row's entries, remaining mass)."""
    there = np.asarray(ids) >= 0
    a = np.where(there, np.asarray(logp, np.float64), -np.inf)
    if tail:
        q = np.exp(a)
        rest = 1.0 - q.sum()
        return q, 0.0 if rest < LEAST_TAIL else float(rest)
    if not there.any() or a.max() == -np.inf:
        return np.zeros(len(a)), 0.0
    q = np.exp(a - a.max())
    return q / q.sum(), 0.0


def _members(ids, vocab: int) -> np.ndarray:
    m = np.zeros(vocab, bool)
    for j in ids:
        if 0 <= j < vocab:
            m[j] = True
    return m


def distill(z, ids=None, logp=None, labels=None, tail: bool = True, scale: float = 1.0):
    """dict of loss, logp, lse, lse_tail."""
    rows, vocab = z.shape
    out = {n: np.zeros(rows) for n in ("loss", "logp", "lse", "lse_tail")}
    for i in range(rows):
        s = _scaled(z[i], scale)
        lse = _row_lse(s)
        row_ids = ids[i] if ids is not None else []
        member = _members(row_ids, vocab)
        lse_tail = _row_lse(s[~member])
        out["lse"][i], out["lse_tail"][i] = lse, lse_tail
        if labels is not None:
            out["logp"][i] = _logp(s, lse, int(labels[i]))
        q, rest = teacher(row_ids, logp[i], tail) if ids is not None else (np.zeros(0), 0.0)
        if np.isnan(lse) or any(j >= vocab for j in row_ids):
            out["loss"][i] = np.nan
            continue
        loss = 0.0
        for j, m in zip(row_ids, q):
            if m > 0.0:
                loss += np.inf if s[j] == -np.inf else m * (np.log(m) - (s[j] - lse))
        if rest > 0.0:
            loss += np.inf if lse_tail == -np.inf else rest * (np.log(rest) - (lse_tail - lse))
        out["loss"][i] = loss
    return out


def distill_backward(z, ids, logp, labels, lse, lse_tail, d_loss=None, d_logp=None,
                     tail: bool = True, scale: float = 1.0) -> np.ndarray:
    rows, vocab = z.shape
    out = np.zeros((rows, vocab))
    for i in range(rows):
        s = _scaled(z[i], scale)
        label = int(labels[i]) if d_logp is not None else -1
        gl = float(d_logp[i]) if label >= 0 else 0.0
        gk = float(d_loss[i]) if d_loss is not None else 0.0
        if gl == 0.0 and gk == 0.0:
            continue
        live = ~(s == -np.inf)
        row_ids = ids[i] if ids is not None else []
        member = _members(row_ids, vocab)
        q, rest = (teacher(row_ids, logp[i], tail) if ids is not None
                   else (np.zeros(0), 1.0 if tail else 0.0))
        p = np.where(live, np.exp(np.where(live, s, 0.0) - float(lse[i])), 0.0)
        d = np.zeros(vocab)
        if gk != 0.0:
            d += gk * (q.sum() + rest) * p
            for j, m in zip(row_ids, q):
                if 0 <= j < vocab:
                    d[j] -= gk * m
            gone = live & ~member
            if rest > 0.0 and gone.any():
                d[gone] -= gk * rest * np.exp(s[gone] - float(lse_tail[i]))
            if any(j >= vocab for j in row_ids):
                d[:] = np.nan
        if gl != 0.0:
            d -= gl * p
            if label >= vocab:
                d[:] = np.nan
            else:
                d[label] += gl
        out[i] = np.where(live, d * scale, 0.0)
    return out
