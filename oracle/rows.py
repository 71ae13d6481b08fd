"""4-bit rows, their products, the routing of vectors to lists, and what sorted
rows are multiplied and summed with, by definition, in numpy and 64-bit floats (sharing no code with the library).

4-bit rows follow the OCP Microscaling specification (MXFP4): blocks of 32
values, e2m1 codes and one power-of-two scale a block.
"""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes [n, 16 kb] uint8, scales [n, kb] uint8) of rows x [n, d] (float64
    holding float32, bfloat16 or binary16 values)."""
    x = np.asarray(x, dtype=np.float64)
    n, d = x.shape
    kb = -(-d // 32)
    codes = np.zeros((n, kb, 32), np.uint8)
    scales = np.zeros((n, kb), np.uint8)
    for i in range(n):
        for b in range(kb):
            v = x[i, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                scales[i, b] = 255
                continue
            top = np.abs(v).max()
            s = 0 if top == 0 else int(np.clip(np.frexp(top)[1] - 1 - 2 + 127, 0, 252))
            scales[i, b] = s
            y = v / 2.0 ** (s - 127)
            gap = np.abs(np.abs(y)[:, None] - MAGNITUDES[None, :])
            # nearest; of two equally near codes the even one
            gap[:, 1::2] *= 1 + 1e-12
            c = gap.argmin(axis=1)
            codes[i, b, :len(v)] = c | np.where(np.signbit(v), 8, 0)
    codes = codes.reshape(n, -1)
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)), scales


def values(codes, scales, d):
    """What 4-bit rows stand for, [..., d] float64 (NaN for scale 255)."""
    n = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = MAGNITUDES[n & 7] * np.where(n & 8, -1.0, 1.0)
    f = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * np.repeat(f, 32, axis=-1))[..., :d]


def list_product(a, b, offsets, order, k, rows):
    """Rows p of list e: a[order[p] // k] (or a[p]) times b[e]^T; the rest zero.
    a [arows, d], b [nlist, n, d].  Also the sums of the products' magnitudes."""
    out = np.zeros((rows, b.shape[1]))
    mag = np.zeros_like(out)
    for e in range(len(b)):
        for p in range(offsets[e], offsets[e + 1]):
            r = a[p if order is None else order[p] // k]
            out[p] = b[e] @ r
            mag[p] = np.abs(b[e]) @ np.abs(r)
    return out, mag


def route_sort(lists, nlist):
    nvec, k = lists.shape
    flat = lists.reshape(-1)
    order = np.full(nvec * k, -1, np.int32)
    pos = np.full(nvec * k, -1, np.int32)
    offsets = np.zeros(nlist + 1, np.int32)
    p = 0
    groups = {}
    for u, l in enumerate(flat.tolist()):
        groups.setdefault(l, []).append(u)
    for l in range(nlist):
        offsets[l] = p
        for u in groups.get(l, ()):
            order[p], pos[u] = u, p
            p += 1
    offsets[nlist] = p
    return offsets, order, pos.reshape(nvec, k)


def gather(x, order, k, weights=None):
    rows = np.zeros((len(order), x.shape[1]))
    for p, u in enumerate(order):
        if u >= 0:
            rows[p] = x[u // k] * (1.0 if weights is None else float(weights.reshape(-1)[u]))
    return rows


def combine(rows, pos, weights=None):
    """The weighted sums and the sums of their terms' magnitudes."""
    y = np.zeros((pos.shape[0], rows.shape[1]))
    mag = np.zeros_like(y)
    for t in range(pos.shape[0]):
        for j, p in enumerate(pos[t]):
            if p >= 0:
                term = rows[p] * (1.0 if weights is None else float(weights[t, j]))
                y[t] += term
                mag[t] += np.abs(term)
    return y, mag


def combine_grad(grad, rows, pos, weights):
    """d_rows, d_weights and the sums of magnitudes behind d_weights."""
    d_rows = np.zeros_like(rows)
    d_w = np.zeros(pos.shape)
    mag = np.zeros(pos.shape)
    for t in range(pos.shape[0]):
        for j, p in enumerate(pos[t]):
            if p >= 0:
                d_rows[p] = grad[t] * float(weights[t, j])
                d_w[t, j] = grad[t] @ rows[p]
                mag[t, j] = np.abs(grad[t]) @ np.abs(rows[p])
    return d_rows, d_w, mag


def list_gradient(grad, x, offsets, order, k, nlist):
    """Per list the sum of grad[p] (outer) x[order[p] // k] (or x[p]), and the sums of
    the terms' magnitudes."""
    out = np.zeros((nlist, grad.shape[1], x.shape[1]))
    mag = np.zeros_like(out)
    for e in range(nlist):
        for p in range(offsets[e], offsets[e + 1]):
            r = x[p if order is None else order[p] // k]
            out[e] += np.outer(grad[p], r)
            mag[e] += np.outer(np.abs(grad[p]), np.abs(r))
    return out, mag


def adapter(x, w, down, up, lists, scales=None):
    """W x + s U (D x) for each row x with the D, U and s of its list (W x where the
    list is masked), and the sums of the terms' magnitudes."""
    out, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    for i, e in enumerate(lists.tolist()):
        if 0 <= e < len(down):
            s = 1.0 if scales is None else float(scales[e])
            out[i] += s * (up[e] @ (down[e] @ x[i]))
            mag[i] += abs(s) * (np.abs(up[e]) @ (np.abs(down[e]) @ np.abs(x[i])))
    return out, mag


def table_lookup(table, ids, scale):
    out = np.zeros((len(ids), table.shape[1]))
    for i, e in enumerate(ids.tolist()):
        if 0 <= e < len(table):
            out[i] = table[e] * scale
    return out


def table_gradient(grad, ids, rows, scale):
    """Sums of the rows of grad with the same number (ids [nvec, k]), and of their
    magnitudes."""
    out, mag = np.zeros((rows, grad.shape[1])), np.zeros((rows, grad.shape[1]))
    for i, row in enumerate(ids.tolist()):
        for e in row:
            if 0 <= e < rows:
                out[e] += grad[i] * scale
                mag[e] += np.abs(grad[i] * scale)
    return out, mag
