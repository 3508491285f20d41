"""The operations on an LM head's logits in fp64, straight from their definitions (numpy; test infrastructure)."""
import numpy as np


def lse(x):
    """log sum exp over the last axis; -inf where it is empty or all -inf."""
    if x.shape[-1] == 0:
        return np.full(x.shape[:-1], -np.inf)
    m = x.max(-1, keepdims=True)
    m = np.where(m > -np.inf, m, 0.0)
    with np.errstate(divide="ignore"):
        return m[..., 0] + np.log(np.exp(x - m).sum(-1))


def order(row):
    """Columns of a row from best to worst: descending, lowest first among equals, NaN last."""
    nan = np.isnan(row)
    return np.lexsort((np.arange(len(row)), -np.where(nan, 0.0, row), nan))


def topk(z, k, T):
    idx = np.stack([order(r)[:k] for r in z])
    vals = np.take_along_axis(z, idx, 1)
    left = z / T
    taken = np.zeros(z.shape, bool)
    np.put_along_axis(taken, idx, True, 1)
    tail = np.array([lse(left[i][~taken[i]]) for i in range(len(z))])
    return vals, idx, lse(left), tail


def distill(z, tv, ti, tail=None, labels=None, weights=None, T=1.0, a=0.0, b=1.0, g=1.0):
    """(loss rows, dz, bad rows): one row after another, one entry after another."""
    B, C = z.shape
    loss, dz, bad = np.zeros(B), np.zeros((B, C)), np.zeros(B, bool)
    for i in range(B):
        w = 1.0 if weights is None else float(weights[i])
        if w == 0.0:
            continue
        used = [j for j in range(ti.shape[1]) if ti[i, j] != -1]
        cols = [int(ti[i, j]) for j in used]
        y = int(labels[i]) if labels is not None and a != 0.0 else None
        if any(c < 0 or c >= C for c in cols) or len(set(cols)) < len(cols) or (y is not None and not 0 <= y < C):
            bad[i] = True
            continue
        x = z[i] / T
        lq = x - lse(x)
        q = np.exp(lq)
        d = np.zeros(C)
        t = np.array([tv[i, j] / T for j in used] + [-np.inf if tail is None else float(tail[i])])
        kd = 0.0
        if t.max() > -np.inf:
            p = np.exp(t - lse(t))
            d = q.copy()
            others = np.ones(C, bool)
            others[cols] = False
            for pj, tj, c in zip(p, t, cols):
                if pj > 0:
                    kd += pj * (tj - lse(t) - lq[c])
                d[c] -= pj
            if p[-1] > 0:
                left = lse(x[others])
                kd += p[-1] * (t[-1] - lse(t) - (left - lse(x)))
                if left > -np.inf:   # (shares from differences: log-sums of masks of the lowest value lose the counts)
                    e = np.exp(x[others] - x[others].max())
                    d[others] -= p[-1] * e / e.sum()
        loss[i] = b * kd
        d *= b / T
        if y is not None:
            ls = z[i] - lse(z[i])
            loss[i] -= a * ls[y]
            d += a * np.exp(ls)
            d[y] -= a
        loss[i] *= w
        dz[i] = d * (w * g)
    return loss, dz, bad


def beam_totals(z, scores, done=None, eos=-1):
    """Totals [beams, C] of one batch entry."""
    W, C = z.shape
    out = np.full((W, C), np.nan)
    for w in range(W):
        s = float(scores[w])
        if s == -np.inf:
            out[w] = -np.inf
        elif np.isfinite(s) and done is not None and done[w]:
            out[w] = -np.inf
            out[w, eos] = s
        elif np.isfinite(s) and not np.isnan(z[w]).any() and z[w].max() < np.inf:
            out[w] = -np.inf if z[w].max() == -np.inf else s + (z[w] - lse(z[w]))
    return out


def beam_select(z, scores, m, done=None, eos=-1):
    """(totals, beams, tokens, done) of the m best pairs of one batch entry."""
    tot = beam_totals(z, scores, done, eos)
    W, C = z.shape
    beam, tok = np.repeat(np.arange(W), C), np.tile(np.arange(C), W)
    flat = tot.ravel()
    nan = np.isnan(flat)
    # (the logit decides between equals of a beam that its logits rank)
    alive = np.array([np.isfinite(tot[w]).any() and not (done is not None and done[w]) for w in range(W)])
    lg = np.where(alive[beam], z.ravel(), 0.0)
    o = np.lexsort((tok, -lg, beam, -np.where(nan, 0.0, flat), nan))[:m]
    ended = tok[o] == eos
    if done is not None:
        ended |= np.asarray(done)[beam[o]] != 0
    return flat[o], beam[o], tok[o], ended
