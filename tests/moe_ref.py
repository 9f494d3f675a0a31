"""Binary64 numpy forms of the mixture-of-experts training operators, from
their definitions, each with a bound on what fp32 sums may differ from it."""
import numpy as np

U = 2.0 ** -24   # half a step of fp32, relative
B = 2.0 ** -8    # half a step of bf16, relative
TINY = 1e-37     # below the smallest normal numbers a rounding is not relative


def softmax(z, live):
    """Rows of probabilities; rows that are not live, or hold -inf only, are zeros."""
    z = np.where(live[:, None], z, -np.inf)
    top = z.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        x = np.where(z == -np.inf, 0.0, np.exp(z - np.where(top == -np.inf, 0.0, top)))
    s = x.sum(1, keepdims=True)
    return x / np.where(s > 0, s, 1.0)


def spread(z, live):
    """The largest top - z of finite logits: the rounding of that difference, times e^x's slope, is relative."""
    z = z[live]
    z = np.where(np.isfinite(z), z, np.nan)
    if not np.isfinite(z).any():
        return 0.0
    keep = z[np.isfinite(z).any(1)]
    return min(104.0, float(np.nanmax(np.nanmax(keep, 1) - np.nanmin(keep, 1))))  # e^-104 is 0 in fp32


def route(z, k, mask=None, renorm=True, coef=0.0):
    z = np.asarray(z, np.float64)
    T, E = z.shape
    live = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    zz = np.where(live[:, None], z, -np.inf)
    p = softmax(zz, live)
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-zz[t, e], e))[:k]
        chosen = [e for e in order if zz[t, e] > -np.inf]
        ids[t, :len(chosen)] = chosen
        if chosen:
            v = np.exp(zz[t, chosen] - zz[t, chosen].max())
            w[t, :len(chosen)] = v / v.sum() if renorm else p[t, chosen]
    entries = sorted((ids[t, j], t, j) for t in range(T) for j in range(k) if ids[t, j] >= 0)
    rows = np.full((T, k), -1, np.int64)
    row_index = np.zeros(T * k, np.int64)
    for r, (_, t, j) in enumerate(entries):
        rows[t, j] = r
        row_index[r] = t
    row_index[len(entries):] = entries[0][1] if entries else 0
    count = np.bincount(ids[ids >= 0], minlength=E)
    n = int((ids[:, 0] >= 0).sum())
    psum = p.sum(0)
    loss = coef * E * float((count / (k * max(n, 1)) * psum / max(n, 1)).sum()) if n else 0.0
    off = np.concatenate([[0], np.cumsum(count)])
    sfo = np.concatenate([[0], np.cumsum((count + 127) // 128 * 128)])
    return dict(expert_ids=ids, weights=w, rows=rows, row_index=row_index, row_offsets=off, sf_row_offsets=sfo,
                counts=np.concatenate([count, [n]]), prob_sums=psum, loss=loss, p=p, live=live)


def route_bwd(z, ids, w, a, counts, dloss, coef, renorm):
    """(dlogits, the sum of the magnitudes that were added up for each)."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    k = ids.shape[1]
    live = (ids >= 0).any(1)
    p = softmax(np.where(live[:, None], z, -np.inf), live)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    if a is not None:
        full, q = np.zeros((T, E)), np.zeros((T, E))
        t, j = np.nonzero(ids >= 0)
        full[t, ids[t, j]] = a[t, j]
        q[t, ids[t, j]] = w[t, j]
        q = q if renorm else p
        d += q * (full - (q * full).sum(1, keepdims=True))
        mag += q * (abs(full) + (q * abs(full)).sum(1, keepdims=True))
    if dloss is not None:
        n = max(int(counts[E]), 1)
        b = dloss * coef * E / n * counts[:E] / (k * n)
        d += p * (b - (p * b).sum(1, keepdims=True))
        mag += p * (abs(b) + (p * abs(b)).sum(1, keepdims=True))
    return d, mag


def combine(y, rows, w):
    T, k = rows.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for j in range(k):
        t = np.nonzero((rows[:, j] >= 0) & (rows[:, j] < y.shape[0]))[0]
        x = (1.0 if w is None else w[t, j, None]) * y[rows[t, j]]
        out[t] += x
        mag[t] += abs(x)
    return out, mag


def combine_bwd(dout, y, rows, w, dy):
    """dy is filled in place; returns (dweights, the sum of |products| in each)."""
    T, k = rows.shape
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        t = np.nonzero((rows[:, j] >= 0) & (rows[:, j] < y.shape[0]))[0]
        dw[t, j] = (dout[t] * y[rows[t, j]]).sum(1)
        mag[t, j] = abs(dout[t] * y[rows[t, j]]).sum(1)
        dy[rows[t, j]] = w[t, j, None] * dout[t]
    return dw, mag


def sigmoid(g):
    e = np.exp(-abs(g))
    return np.where(g >= 0, 1 / (1 + e), e / (1 + e))


def swiglu(u):
    F = u.shape[1] // 2
    g, v = u[:, :F], u[:, F:]
    return g * sigmoid(g) * v


def swiglu_bwd(dh, u):
    """(du, the magnitude that its rounding errors are relative to)."""
    F = u.shape[1] // 2
    g, v = u[:, :F], u[:, F:]
    s = sigmoid(g)
    rest = sigmoid(-g)  # 1 - s
    du = np.concatenate([dh * v * s * (1 + g * rest), dh * g * s], 1)
    mag = np.concatenate([abs(dh * v * s) * (1 + abs(g)), abs(dh * g * s)], 1)
    return du, mag


def within(got, want, tol, what):
    got = np.asarray(got, np.float64)
    bad = np.argwhere(~(abs(got - want) <= tol))
    assert bad.size == 0, (f"{what}: {len(bad)} of {got.size} outside; first {bad[0].tolist()}: got "
                           f"{got[tuple(bad[0])]} want {np.asarray(want)[tuple(bad[0])]} "
                           f"tol {np.broadcast_to(tol, got.shape)[tuple(bad[0])]}")
