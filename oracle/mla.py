"""The latent-attention operators in float64 (numpy), written from their formulas and apart from the kernels.

``append``: norm, rotation, cache write.  ``decode``: absorbed attention over the paged
cache.  ``prefill`` and ``backward``: expanded attention over packed sequences and its
gradients.  Rows that see no key give o = 0 and lse = -inf.
"""
import numpy as np


def rotate(x, pos, inv_freq, interleaved):
    """x [T, ..., dr] turned by pos [T] times inv_freq [dr/2]."""
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    ang = ang.reshape(ang.shape[0], *([1] * (x.ndim - 2)), ang.shape[1])
    z = np.exp(1j * ang)
    h = x.shape[-1] // 2
    w = (x[..., 0::2] + 1j * x[..., 1::2] if interleaved else x[..., :h] + 1j * x[..., h:]) * z
    y = np.empty_like(x, dtype=np.float64)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = w.real, w.imag
    else:
        y[..., :h], y[..., h:] = w.real, w.imag
    return y


def append(c, k_rope, cache, page_table, past, cu, norm_weight=None, eps=1e-6, inv_freq=None, interleaved=False,
           q_rope=None):
    """(cache after, c', kr', q'); cache is copied.  kr' and q' are None where the inputs are."""
    cache = np.array(cache, np.float64)
    pages, page, _ = cache.shape
    c = np.array(c, np.float64)
    used = int(cu[-1])
    if norm_weight is not None:
        c[:used] = c[:used] / np.sqrt((c[:used] ** 2).mean(1, keepdims=True) + eps) * norm_weight
    kr = None if k_rope is None else np.array(k_rope, np.float64)
    q = None if q_rope is None else np.array(q_rope, np.float64)
    for b in range(len(cu) - 1):
        for t in range(cu[b], cu[b + 1]):
            p = int(past[b]) + t - cu[b]
            if inv_freq is not None:
                if kr is not None:
                    kr[t] = rotate(kr[t:t + 1], [p], inv_freq, interleaved)[0]
                if q is not None:
                    q[t] = rotate(q[t:t + 1], [p], inv_freq, interleaved)[0]
            if 0 <= p < page_table.shape[1] * page:
                at = int(page_table[b, p // page])
                if 0 <= at < pages:
                    cache[at, p % page] = c[t] if kr is None else np.concatenate([c[t], kr[t]])
    return cache, c, kr, q


def _softmax(s):
    """Softmax over the last axis with -inf for unseen places, and lse; a row without any is zero."""
    with np.errstate(invalid="ignore", divide="ignore"):
        m = s.max(-1, keepdims=True, initial=-np.inf)
        e = np.exp(s - np.where(np.isneginf(m), 0.0, m))
        z = e.sum(-1, keepdims=True)
        lse = (np.log(z) + np.where(np.isneginf(m), 0.0, m))[..., 0]
        return np.divide(e, z, out=np.zeros_like(e), where=z != 0), lse


def decode(q, cache, page_table, seq_lens, d_latent, scale):
    """(o [B,n,H,d_latent], lse [B,n,H])."""
    B, n, H, W = q.shape
    pages, page, _ = cache.shape
    o, lse = np.zeros((B, n, H, d_latent)), np.full((B, n, H), -np.inf)
    for b in range(B):
        L = max(0, min(int(seq_lens[b]), page_table.shape[1] * page))
        pos = np.arange(L)
        at = page_table[b][pos // page].astype(np.int64)
        here = (at >= 0) & (at < pages)
        rows = np.where(here[:, None], cache[np.where(here, at, 0), pos % page], 0.0)
        for i in range(n):
            end = max(0, L - (n - 1) + i)
            ok = here & (pos < end)
            if not ok.any():
                continue
            p, lse[b, i] = _softmax(q[b, i] @ rows[ok].T * scale)
            o[b, i] = p @ rows[ok, :d_latent]
    return o, lse


def _seen(lq, lk, causal):
    return (np.arange(lk)[None, :] <= np.arange(lq)[:, None] + lk - lq) if causal else np.ones((lq, lk), bool)


def _full_k(k, k_rope, ks, h):
    return k[ks, h] if k_rope is None else np.concatenate([k[ks, h], k_rope[ks]], 1)


def prefill(q, k, v, cu_q, cu_k, k_rope=None, scale=None, causal=True):
    """(o [Tq,H,dv], lse [Tq,H]); rows outside the sequences are 0 and -inf."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    o, lse = np.zeros((q.shape[0], q.shape[1], v.shape[2])), np.full(q.shape[:2], -np.inf)
    for b in range(len(cu_q) - 1):
        qs, ks = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        seen = _seen(cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b], causal)
        for h in range(q.shape[1]):
            p, lse[qs, h] = _softmax(np.where(seen, q[qs, h] @ _full_k(k, k_rope, ks, h).T * scale, -np.inf))
            o[qs, h] = p @ v[ks, h]
    return o, lse


def backward(q, k, v, cu_q, cu_k, dO, k_rope=None, scale=None, causal=True):
    """dict dq, dk, dv and, with k_rope, dk_rope."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    g = dict(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape))
    if k_rope is not None:
        g["dk_rope"] = np.zeros(k_rope.shape)
    dn = k.shape[2]
    for b in range(len(cu_q) - 1):
        qs, ks = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        seen = _seen(cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b], causal)
        for h in range(q.shape[1]):
            kf = _full_k(k, k_rope, ks, h)
            p, _ = _softmax(np.where(seen, q[qs, h] @ kf.T * scale, -np.inf))
            dp = dO[qs, h] @ v[ks, h].T
            ds = p * (dp - (p * dp).sum(1, keepdims=True)) * scale
            g["dq"][qs, h] = ds @ kf
            dk = ds.T @ q[qs, h]
            g["dk"][ks, h] = dk[:, :dn]
            if k_rope is not None:
                g["dk_rope"][ks] += dk[:, dn:]
            g["dv"][ks, h] = p.T @ dO[qs, h]
    return g
