"""Float64 statements of the latent attention and of the norm in front of a layer, for the tests.

Everything is written from the definition, one sequence and one head at a time, in numpy; arrays are
the values the kernels read (already rounded to their type). Each function also returns what the tests'
error bounds need: sums of absolute values along the same contractions.
"""
import numpy as np


def spans(cu_q, cu_k):
    return [(int(cu_q[n]), int(cu_q[n + 1]), int(cu_k[n]), int(cu_k[n + 1])) for n in range(len(cu_q) - 1)]


def _softmax(x):
    """Rows of scores (-inf: not visible) -> probabilities, log of the sum; zeros and -inf for empty rows."""
    lse = np.full(x.shape[0], -np.inf)
    p = np.zeros_like(x)
    for i in range(x.shape[0]):
        seen = x[i] > -np.inf
        if seen.any():
            m = x[i, seen].max()
            e = np.exp(x[i, seen] - m)
            lse[i] = m + np.log(e.sum())
            p[i, seen] = e / e.sum()
    return p, lse


def scores(q, k, r, scale, causal):
    """q [n, 128+R], k [m, 128], r [m, R] or None -> masked scores [n, m]."""
    n, m = q.shape[0], k.shape[0]
    key = k if r is None else np.concatenate([k, r], axis=1)
    x = scale * (q @ key.T)
    if causal:
        for i in range(n):
            x[i, max(0, i + m - n + 1):] = -np.inf
    return x, key


def forward(q, k, v, r, cu_q, cu_k, scale, causal):
    """q [T,H,W], k, v [Tk,H,128], r [Tk,R] or None. Returns out [T,H,128], lse [T,H], P|V| [T,H,128] and
    the largest scale |q|.|k| of each row [T,H]."""
    T, H, _ = q.shape
    out, lse = np.zeros((T, H, v.shape[2])), np.full((T, H), -np.inf)
    wide, big = np.zeros_like(out), np.zeros((T, H))
    for q0, q1, k0, k1 in spans(cu_q, cu_k):
        for h in range(H):
            if q1 == q0 or k1 == k0:
                continue
            x, key = scores(q[q0:q1, h], k[k0:k1, h], None if r is None else r[k0:k1], scale, causal)
            p, lse[q0:q1, h] = _softmax(x)
            out[q0:q1, h] = p @ v[k0:k1, h]
            wide[q0:q1, h] = p @ np.abs(v[k0:k1, h])
            big[q0:q1, h] = scale * (np.abs(q[q0:q1, h]) @ np.abs(key).T).max(axis=1)
    return out, lse, wide, big


def backward(q, k, v, r, dout, cu_q, cu_k, scale, causal, rounding=2.0 ** -8):
    """Gradients of sum(dout * out): dict dq, dk, dv, dr, and under ``<name>_bound`` how far a result may be
    off whose P and dS are rounded by at most ``rounding`` of their values before the second products and
    whose D = dout . out uses an ``out`` that is itself rounded once."""
    T, H, W = q.shape
    Tk, R = k.shape[0], 0 if r is None else r.shape[1]
    g = {"dq": np.zeros((T, H, W)), "dk": np.zeros((Tk, H, 128)), "dv": np.zeros((Tk, H, 128)), "dr": np.zeros((Tk, R))}
    bound = {key: np.zeros_like(x) for key, x in g.items()}
    for q0, q1, k0, k1 in spans(cu_q, cu_k):
        for h in range(H):
            if q1 == q0 or k1 == k0:
                continue
            qh, vh, do = q[q0:q1, h], v[k0:k1, h], dout[q0:q1, h]
            x, key = scores(qh, k[k0:k1, h], None if r is None else r[k0:k1], scale, causal)
            p, _ = _softmax(x)
            o = p @ vh
            dp = do @ vh.T
            ds = p * (dp - (p * dp).sum(1, keepdims=True)) * scale
            g["dv"][k0:k1, h] = p.T @ do
            g["dq"][q0:q1, h] = ds @ key
            g["dk"][k0:k1, h] = ds.T @ qh[:, :128]
            # fp32 sums: W products in a score, 128 in dP; the score's error is relative in P
            d_s = (W + 8) * 2.0 ** -24 * 2 * scale * (np.abs(qh) @ np.abs(key).T).max() + 2.0 ** -18
            d_p = (128 + 8) * 2.0 ** -24 * (np.abs(do) @ np.abs(vh).T)
            d_d = rounding * (np.abs(do) * np.abs(o)).sum(1, keepdims=True) + d_p.max(1, keepdims=True)
            e_p = p * (rounding + d_s)
            e_s = rounding * np.abs(ds) + p * scale * (d_p + d_d) + d_s * np.abs(ds)
            bound["dv"][k0:k1, h] = e_p.T @ np.abs(do)
            bound["dq"][q0:q1, h] = e_s @ np.abs(key)
            bound["dk"][k0:k1, h] = e_s.T @ np.abs(qh[:, :128])
            if R:
                g["dr"][k0:k1] += ds.T @ qh[:, 128:]
                bound["dr"][k0:k1] += e_s.T @ np.abs(qh[:, 128:])
    g.update({key + "_bound": x for key, x in bound.items()})
    return g


def decode(q, cache, table, lens, scale):
    """q [N,Tq,H,W], cache [pages,page,W], table [N,max], lens [N]. Returns out [N,Tq,H,512], lse, P|C| and
    the largest scale |q|.|c| of each row."""
    N, Tq, H, W = q.shape
    page = cache.shape[1]
    out, lse = np.zeros((N, Tq, H, 512)), np.full((N, Tq, H), -np.inf)
    wide, big = np.zeros_like(out), np.zeros((N, Tq, H))
    for n in range(N):
        rows = [cache[table[n, j // page], j % page] for j in range(int(lens[n]))]
        for t in range(Tq):
            seen = int(lens[n]) - Tq + t + 1
            if seen <= 0:
                continue
            c = np.stack(rows[:seen])
            x = scale * (q[n, t] @ c.T)
            p, lse[n, t] = _softmax(x)
            out[n, t] = p @ c[:, :512]
            wide[n, t] = p @ np.abs(c[:, :512])
            big[n, t] = scale * (np.abs(q[n, t]) @ np.abs(c).T).max(axis=1)
    return out, lse, wide, big


def rms_norm(h, w, eps):
    return h / np.sqrt((h * h).mean(axis=-1, keepdims=True) + eps) * w


def rms_norm_backward(dy, h, w, eps):
    """(dx, dw) of rms_norm at h, and the sums of absolute values along dw's rows."""
    rms = np.sqrt((h * h).mean(axis=-1, keepdims=True) + eps)
    unit = h / rms
    g = dy * w
    dx = (g - unit * (g * unit).mean(axis=-1, keepdims=True)) / rms
    return dx, (dy * unit).sum(axis=0), np.abs(dy * unit).sum(axis=0)


def round_e4m3(x):
    """Nearest e4m3 value (4 significant bits, smallest normal exponent -6, largest 448), ties to even."""
    x = np.asarray(x, dtype=np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.clip(np.round(x / step) * step, -448.0, 448.0)
