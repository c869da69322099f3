"""Plain 64-bit implementations (numpy, one row or request at a time) of the
calls that follow a verification: token_logprobs, distill_topk with its
gradient, advance_blocks; and the error bounds of their 32-bit results."""

from __future__ import annotations

import numpy as np

EPS = 2.0 ** -24  # unit roundoff of fp32
DEVERR_TOKEN, DEVERR_NONFINITE, DEVERR_LENGTH, DEVERR_CAPACITY = 1, 2, 8, 32


def sum_bound(V):
    """Relative error bound of a sum of V positive fp32 exponentials: one
    thread of 256 adds V / 256 of them one after another (at most EPS each),
    the rest is a tree; an exponential is off by at most 2^-22 and, through
    the rounding of its argument, EPS per unit of it (weights below 2^-30 of
    the maximum do not matter): 64 EPS cover both."""
    return EPS * (V / 256 + 64)


def bad_row(x):
    """NaN or +inf somewhere, or nothing finite."""
    return bool(np.isnan(x).any() or (x == np.inf).any() or not np.isfinite(x).any())


def log_softmax(x, T):
    with np.errstate(all="ignore"):
        y = x.astype(np.float64) / T
        m = y.max()
        return (y - m) - np.log(np.exp(y - m).sum())


def order(x):
    """Indices in (value descending, index ascending) order."""
    return np.lexsort((np.arange(len(x)), -x.astype(np.float64)))


def token_logprobs(x, tokens, T, K):
    """x [R, V] float32 values; tokens [R] or None."""
    R, V = x.shape
    out = dict(logprob=np.zeros(R), rank=np.full(R, -1), entropy=np.zeros(R), top_ids=np.full((R, K), -1),
               top_logprobs=np.full((R, K), -np.inf))
    err = 0
    for r in range(R):
        t = None if tokens is None else int(tokens[r])
        if t == -1:
            continue
        e = 0
        if t is not None and not 0 <= t < V:
            e = DEVERR_TOKEN
        elif bad_row(x[r]):
            e = DEVERR_NONFINITE
        if e:
            err |= e
            out["logprob"][r] = 0.0 if t is None else -np.inf
            continue
        lp = log_softmax(x[r], T)
        p = np.exp(lp)
        out["entropy"][r] = -(p[p > 0] * lp[p > 0]).sum()
        lp[lp < -np.finfo(np.float32).max] = -np.inf  # past the range of 32 bits
        o = order(x[r])[:max(K, 0)]
        out["top_ids"][r], out["top_logprobs"][r] = o, lp[o]
        if t is not None:
            out["logprob"][r] = lp[t]
            out["rank"][r] = 1 + int(((x[r] > x[r][t]) | ((x[r] == x[r][t]) & (np.arange(V) < t))).sum())
    return out, err


def distill_row(s, ids, l, T, bucket):
    """(loss, gradient, scale, error) of one row: scale bounds |gradient's
    terms| for the error bound."""
    V = len(s)
    s = s.astype(np.float64)
    listed = ids[ids != -1]
    zero = np.zeros(V)
    if ((listed < 0) | (listed >= V)).any() or len(set(listed.tolist())) != len(listed):
        return 0.0, zero, zero, DEVERR_TOKEN
    lj = l[ids != -1].astype(np.float64)
    if bad_row(s) or np.isnan(lj).any() or (lj == np.inf).any():
        return 0.0, zero, zero, DEVERR_NONFINITE
    with np.errstate(all="ignore"):
        if not bucket:
            if not (lj > -np.inf).any():
                return 0.0, zero, zero, 0
            lj = lj - lj.max()
            lj = lj - np.log(np.exp(lj).sum())
        t = np.exp(lj)
        lq = log_softmax(s, T)
        q = np.exp(lq)
        tail = np.ones(V, bool)
        tail[listed] = False
        sT = s[tail]
        has_tail = len(sT) > 0 and bool(np.isfinite(sT).any())
        if has_tail:
            y = sT / T
            in_tail = np.exp(y - y.max())
            log_qT = (y.max() - s.max() / T) + np.log(in_tail.sum()) - np.log(np.exp((s - s.max()) / T).sum())
        else:
            log_qT = -np.inf
        tT = max(0.0, 1.0 - t.sum()) if bucket else 0.0
        if not has_tail and tT <= 2.0 ** -16:
            tT = 0.0
        on = t > 0
        loss = (t[on] * (lj[on] - lq[listed][on])).sum()
        if tT > 0:
            loss += tT * (np.log(tT) - log_qT)
        S = t.sum() + tT
        spread = np.zeros(V)
        if has_tail:
            spread[tail] = in_tail / in_tail.sum()
        g = spread * (S * np.exp(log_qT) - tT) / T
        scale = spread * (S * np.exp(log_qT) + tT) / T
        g[listed] = (S * q[listed] - t) / T
        scale[listed] = (S * q[listed] + t) / T
        if bucket:  # t_T = 1 - sum t is off by roundings of the whole sum
            scale[tail] += spread[tail] * t.sum() / T
    return loss, g, scale, 0


def distill_loss_bound(s, ids, l, T):
    """Bound of the 32-bit loss.  ln Z carries the sums' bound.  Each t, and
    t_T = 1 - sum t with the roundings of K of them, is off by a few EPS of
    the teacher's mass, times the log ratio it multiplies: at most `far`."""
    with np.errstate(all="ignore"):
        lq = log_softmax(s, T)
        parts = [np.abs(lq), np.abs(l)]
        far = max(float(p[np.isfinite(p)].max(initial=0.0)) for p in parts)
    return sum_bound(len(s)) + EPS * 8 * (len(ids) + 1) * (1 + far)


def advance_blocks(seq_lens, accepted, new, page, table, held, free, free_count, max_tokens):
    """Python integers throughout; table is copied."""
    B, M = table.shape
    table = table.copy()
    out_len, out_held, cu = [], [], [0]
    slots = np.full(max_tokens, -1, np.int64)
    positions = np.zeros(max_tokens, np.int32)
    err = 0
    if not 0 <= free_count <= len(free):
        err |= DEVERR_LENGTH
        free_count = 0
    lacking = taken = 0
    for b in range(B):
        L, n, h = int(seq_lens[b]), int(new[b]), int(held[b])
        a = -1 if accepted is None else int(accepted[b])
        length = L + a + 1
        bad = L < 0 or a < -1 or n < 0 or h < 0 or h > M or length > h * page or length + n > 2**31 - 1
        count = max(n, 0)
        served = not bad
        if bad:
            err |= DEVERR_LENGTH
            length = L
        else:
            need = -(-(length + n) // page)
            if need > M:
                served = False
            else:
                lacks = max(need - h, 0)
                lacking += lacks
                served = lacks == 0 or lacking <= free_count
                if served:
                    for j in range(lacks):
                        table[b, h + j] = free[free_count - 1 - (lacking - lacks + j)]
                    taken += lacks
                    h += lacks
            if not served:
                err |= DEVERR_CAPACITY
        out_len.append(length)
        out_held.append(h)
        for i in range(min(count, max_tokens - cu[-1])):
            at = cu[-1] + i
            if not bad:
                p = length + i
                positions[at] = p
                if served:
                    slots[at] = int(table[b, p // page]) * page + p % page
        cu.append(cu[-1] + count)
    if cu[-1] > max_tokens:
        err |= DEVERR_LENGTH
    return dict(seq_lens=np.array(out_len), held=np.array(out_held), free_count=free_count - taken,
                cu_tokens=np.array(cu), slots=slots, positions=positions, table=table), err
