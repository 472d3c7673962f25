"""Plain 64-bit forms of the vocabulary operators (highest logits, distillation,
beam selection and reordering) on numpy arrays, written from their definitions
in include/dspark.h, and the tolerances that the library's 32-bit sums allow."""

from __future__ import annotations

import math

import numpy as np

# A mass sum exp(x / T) is a tree of fp32 sums: at most 32 terms in a group, 32
# groups in a thread, 6 + 3 levels over the workgroup and 64 segments' worth of
# levels over a row, under 128 roundings of 2^-24 with each term's own: its
# exponential (1 ulp), the argument's rounding and that of log2(e) / T, whose
# effect |a| 2^-24 2^a is under 2^-24 for an exponent a <= 0.  Its logarithm is
# then off by 2^-17 at most, and the output is rounded once.
MASS_TOL = 2.0 ** -17
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def near(got, want, tol=MASS_TOL):
    """Whether float32 outputs are within tol and their own rounding of 64-bit values."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        return bool(np.all(same | (np.abs(got - want) <= tol + HALF["f32"] * np.abs(want))))


def lse(z):
    z = np.asarray(z, np.float64)
    m = np.max(z, axis=-1, keepdims=True, initial=-np.inf)
    m = np.where(np.isinf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        return (m + np.log(np.sum(np.exp(z - m), axis=-1, keepdims=True)))[..., 0]


def top_logits(x, K, T=1.0):
    """(values, ids, rest, lse) of rows without NaN or +inf."""
    x = np.asarray(x, np.float64)
    R, V = x.shape
    values = np.full((R, K), -np.inf)
    ids = np.full((R, K), -1, np.int64)
    rest = np.empty(R)
    for r in range(R):
        order = np.argsort(-x[r], kind="stable")[:K]
        order = order[x[r][order] > -np.inf]
        values[r, :len(order)] = x[r][order]
        ids[r, :len(order)] = order
        rest[r] = lse(np.delete(x[r], order) / T) if len(order) < V else -np.inf
    return values, ids, rest, lse(x / T)


def outcomes(x, values, ids, teacher_rest, T, rest=None):
    """One row's (log t, log s, the entries' tokens, log Zs, rest): the listed
    entries, then everything else."""
    V = len(x)
    x = np.asarray(x, np.float64)
    ok = (ids >= 0) & (ids < V)
    listed = np.unique(ids[ok])
    if rest is None:
        rest = lse(np.delete(x, listed) / T) if len(listed) < V else -np.inf
    zt = np.append(np.where(ok, np.asarray(values, np.float64) / T, -np.inf),
                   -np.inf if teacher_rest is None else teacher_rest)
    zs = np.append(np.where(ok, x[np.where(ok, ids, 0)] / T, -np.inf), rest)
    big = lse(np.append(x[listed] / T, rest))
    with np.errstate(invalid="ignore"):
        return zt - lse(zt), zs - big, np.where(ok, ids, -1), big, rest


def distill(draft, values, ids, teacher_rest=None, mask=None, T=1.0, weight=1.0):
    N, G, V = draft.shape
    kl, big, rest = np.zeros((N, G)), np.zeros((N, G)), np.zeros((N, G))
    for b in range(N):
        for k in range(G):
            lt, ls, _, big[b, k], rest[b, k] = outcomes(draft[b, k], values[b, k], ids[b, k],
                                                        None if teacher_rest is None else teacher_rest[b, k], T)
            t = np.exp(lt)
            on = t > 0
            kl[b, k] = np.sum(t[on] * (lt[on] - ls[on])) if np.isfinite(big[b, k]) else 0.0
    on = np.ones(N) if mask is None else (np.asarray(mask) != 0).astype(np.float64)
    w = np.exp(-np.arange(1, G + 1) / G)
    with np.errstate(invalid="ignore"):
        part = np.where(on[:, None] > 0, kl, 0.0)
    return dict(kl=kl, lse=big, rest=rest,
                sums=np.array([weight * np.sum(part * w), on.sum() * G, part.sum(), on.sum() * G]))


def distill_grad(draft, values, ids, teacher_rest=None, mask=None, T=1.0, weight=1.0, scale=1.0, rest=None):
    """The gradient into the draft logits; rest: the value the row's normaliser is
    formed with (None: the row's own)."""
    N, G, V = draft.shape
    g = np.zeros((N, G, V))
    for b in range(N):
        if mask is not None and not mask[b]:
            continue
        for k in range(G):
            lt, ls, tok, big, r = outcomes(draft[b, k], values[b, k], ids[b, k],
                                           None if teacher_rest is None else float(teacher_rest[b, k]), T,
                                           None if rest is None else float(rest[b, k]))
            t, s = np.exp(lt), np.exp(ls)
            if not np.isfinite(big) or not np.sum(t) > 0:
                continue
            z = np.asarray(draft[b, k], np.float64) / T
            with np.errstate(over="ignore", invalid="ignore"):  # at listed tokens, replaced below
                d = (s[-1] - t[-1]) * np.exp(z - r) if r > -np.inf else np.zeros(V)
            for v in np.unique(tok[tok >= 0]):
                d[v] = math.exp(z[v] - big) - t[:-1][tok == v].sum()
            g[b, k] = scale * weight * math.exp(-(k + 1) / G) / T * d
    return g


def grad_tol(draft, rest, g, T, dtype):
    """Bound of a gradient element's error: A exp2(fma(x, c, -r)) has the roundings
    of c, of the argument (each 2^-24 of |x| c or of the argument, and the
    argument's effect is ln 2 of it) and three more 2^-24 (exponential 2, factor
    1), and is then rounded to its type; results below the smallest normal number
    may be flushed."""
    xc = np.abs(np.asarray(draft, np.float64)) / T * 1.4427
    arg = np.abs(np.asarray(draft, np.float64) / T - np.where(np.isfinite(rest), rest, 0.0)[..., None]) * 1.4427
    with np.errstate(invalid="ignore"):
        rel = np.abs(g) * (2.0 ** -24 * (xc + arg + 6.0) + HALF[dtype])
    return np.where(g == 0, 0.0, rel) + 2.0 ** -126  # a zero has no relative error, whatever the argument


def beam_scores(x, scores, finished=None, eos=0):
    """One request's candidate scores [W, V] in 64 bits (-inf: none)."""
    W, V = x.shape
    out = np.full((W, V), -np.inf)
    for w in range(W):
        if not scores[w] > -np.inf:
            continue
        if finished is not None and finished[w]:
            out[w, eos] = scores[w]
        elif np.max(x[w]) > -np.inf:
            out[w] = float(scores[w]) + (np.asarray(x[w], np.float64) - lse(x[w]))
    return out


def reorder(state, parents, batch_dim=0, lengths=None, length_dim=None, out=None):
    shape = list(state.shape)
    shape[batch_dim + 1] = parents.shape[1]
    got = np.zeros(shape, state.dtype) if out is None else out.copy()
    s = np.moveaxis(state, (batch_dim, batch_dim + 1), (0, 1))
    g = np.moveaxis(got, (batch_dim, batch_dim + 1), (0, 1))
    for b in range(parents.shape[0]):
        for j in range(parents.shape[1]):
            p = parents[b, j]
            if not 0 <= p < s.shape[1]:
                continue
            if lengths is None:
                g[b, j] = s[b, p]
            else:
                axis = length_dim - 2
                n = max(0, min(int(lengths[b]), state.shape[length_dim]))
                at = (slice(None),) * axis + (slice(0, n),)
                g[b, j][at] = s[b, p][at]
    return got
