"""CPU oracle of token log probabilities, entropy, likeliest tokens and their gradient
(numpy, float64). Test infrastructure only: it shares no code with the GPU path."""
import numpy as np


def forward(x, targets, temperature=1.0, top=0):
    """x: float64 [rows, vocab]. Returns a dict of logprob, entropy, stats, top_logprob,
    top_id as mxfp8_token_logprobs defines them (rows with a NaN or +inf: NaN, id -1)."""
    rows, vocab = x.shape
    got = dict(logprob=np.zeros(rows), entropy=np.zeros(rows), stats=np.zeros((rows, 2)),
               top_logprob=np.full((rows, top), -np.inf), top_id=np.full((rows, top), -1, np.int64))
    for r in range(rows):
        z, t = x[r], int(targets[r])
        m = np.max(z)
        if np.isnan(m) or m == np.inf:
            for key in ("logprob", "entropy", "stats", "top_logprob"):
                got[key][r] = np.nan
            continue
        if m == -np.inf:
            got["logprob"][r] = 0.0 if t < 0 else -np.inf
            got["stats"][r] = (-np.inf, 0.0)
            continue
        d = (z - m) / temperature
        e = np.exp(d)
        s = e.sum()
        got["stats"][r] = (m, np.log(s))
        if t >= 0:
            got["logprob"][r] = d[t] - np.log(s)
        live = e > 0
        got["entropy"][r] = np.log(s) - np.sum(e[live] * d[live]) / s
        order = np.lexsort((np.arange(vocab), -(z + 0.0)))[:top]
        order = order[z[order] > -np.inf]
        got["top_id"][r, :len(order)] = order
        got["top_logprob"][r, :len(order)] = d[order] - np.log(s)
    for v in got.values():   # the results are FP32: beyond its range lies infinity
        if v.dtype == np.float64:
            v[np.abs(v) > np.finfo(np.float32).max] = -np.inf
    return got


def backward(x, targets, temperature, g, h=None, top_id=None, g_top=None):
    """Gradient of sum(g logprob + h entropy + g_top top_logprob) with respect to x."""
    rows, vocab = x.shape
    dx = np.zeros((rows, vocab))
    for r in range(rows):
        z, t = x[r], int(targets[r])
        m = np.max(z)
        if m == -np.inf:
            continue
        d = (z - m) / temperature
        p = np.exp(d) / np.exp(d).sum()
        logp = np.where(p > 0, d - np.log(np.exp(d).sum()), 0.0)
        gr = 0.0 if t < 0 else float(g[r])
        dz = np.zeros(vocab)
        if t >= 0:
            dz[t] += gr
        mass = gr
        if g_top is not None:
            for i, w in zip(top_id[r], g_top[r]):
                if i >= 0:
                    dz[int(i)] += w
                    mass += w
        hr = 0.0 if h is None else float(h[r])
        ent = -np.sum(p * logp)
        dx[r] = (dz - p * (mass + hr * (logp + ent))) / temperature
    return dx
