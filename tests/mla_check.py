"""Inputs and error bounds shared by the latent-attention GPU tests.

Bounds follow from the roundings, u = finfo(dtype).eps / 2 (2^-8 for bf16, 2^-24 for f32).
The kernels multiply exactly or in float32 and sum in float32; on the bf16 path the
probabilities P and dS are rounded to bf16 (u each) before their products, and every output
is rounded once.  So, element by element, with |.| taken inside the sums,

    |o  - ref| <= u |ref| + u sum_j P |v|                      + f
    |dv - ref| <= u |ref| + u sum_i P |dO|                     + f
    |dq - ref| <= u |ref| + sum_j (u |dS| + |scale| P E) |k|     + f      E = error of delta = sum_c |dO| |o - ref|
    |dk - ref| <= the same with q

f is float32's share: products of d terms are off by about sqrt(d) 2^-23 of their absolute
sums (d <= 576: 3e-6), which through exp gives relative errors of P up to 4e-5 at the scores'
size here; f = 4e-5 of the absolute sums covers it for either dtype.
"""
import numpy as np
import torch

from oracle import mla

F = 4e-5
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def host(t):
    return t.detach().double().cpu().numpy()


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64).tolist()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def packed(q_lens, k_lens, H, dn, dr, dv, dtype, seed=0):
    """Tensors of one mla_prefill / mla_backward call; k and v are slices of one expansion."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    cq, ck = offsets(q_lens), offsets(k_lens)
    kv = r(ck[-1], H, dn + dv)
    return dict(q=r(cq[-1], H, dn + dr), k=kv[..., :dn], v=kv[..., dn:], k_rope=r(ck[-1], dr) if dr else None,
                cu_q=i32(cq), cu_k=i32(ck), cu_q_host=cq, cu_k_host=ck), r(cq[-1], H, dv)


def close(x, ref, bound, what):
    x = host(x)
    assert x.shape == ref.shape, what
    assert np.isfinite(x).all(), f"{what}: not finite"
    off = np.abs(x - ref) - bound
    assert x.size == 0 or off.max() <= 0, f"{what}: {np.abs(x - ref).max():.3e} off, {off.max():.3e} over its bound"


def check_lse(lse, ref, what="lse"):
    """Scores of up to 576 products: sqrt(576) 2^-23 times absolute sums of about 26 gives 7e-5; 2e-4 asked."""
    x = host(lse)
    assert (np.isneginf(x) == np.isneginf(ref)).all(), what
    ok = np.isfinite(ref)
    x, ref = x[ok], ref[ok]
    assert (np.abs(x - ref) <= 2e-4).all(), f"{what}: {np.abs(x - ref).max():.3e}"


def check_prefill(a, o, lse, causal=True, scale=None):
    h = {n: None if a[n] is None else host(a[n]) for n in ("q", "k", "v", "k_rope")}
    run = lambda v: mla.prefill(h["q"], h["k"], v, a["cu_q_host"], a["cu_k_host"], k_rope=h["k_rope"], scale=scale,
                                causal=causal)
    (ref, ref_lse), (mag, _) = run(h["v"]), run(np.abs(h["v"]))
    u = U[o.dtype]
    close(o, ref, u * np.abs(ref) + (u + F) * mag, "o")
    if lse is not None:
        check_lse(lse, ref_lse)
    return ref


def check_backward(a, dO, g, causal=True, scale=None):
    h = {n: None if a[n] is None else host(a[n]) for n in ("q", "k", "v", "k_rope")}
    scale = h["q"].shape[2] ** -0.5 if scale is None else scale
    cq, ck, D, u = a["cu_q_host"], a["cu_k_host"], host(dO), U[dO.dtype]
    ref = mla.backward(h["q"], h["k"], h["v"], cq, ck, D, k_rope=h["k_rope"], scale=scale, causal=causal)
    bound = {n: u * np.abs(r) for n, r in ref.items()}
    dn = h["k"].shape[2]
    for b in range(len(cq) - 1):
        qs, ks = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        seen = mla._seen(cq[b + 1] - cq[b], ck[b + 1] - ck[b], causal)
        for n in range(h["q"].shape[1]):
            k = mla._full_k(h["k"], h["k_rope"], ks, n)
            q, v, d = h["q"][qs, n], h["v"][ks, n], D[qs, n]
            p, _ = mla._softmax(np.where(seen, q @ k.T * scale, -np.inf))
            dp = d @ v.T
            ds = np.abs(p * (dp - (p * dp).sum(1, keepdims=True)) * scale)
            o_err = u * np.abs(p @ v) + (u + F) * (p @ np.abs(v))
            E = (np.abs(d) * o_err).sum(1, keepdims=True)
            size = abs(scale)  # an error is at most the sum of absolute terms, scale's sign apart
            wide = p * size * (np.abs(d) @ np.abs(v).T + (p * (np.abs(d) @ np.abs(v).T)).sum(1, keepdims=True))
            e = (u + F) * ds + size * p * E + F * wide
            bound["dv"][ks, n] += (u + F) * (p.T @ np.abs(d))
            bound["dq"][qs, n] += e @ np.abs(k)
            dk = e.T @ np.abs(q)
            bound["dk"][ks, n] += dk[:, :dn]
            if h["k_rope"] is not None:
                bound["dk_rope"][ks] += dk[:, dn:]
    for name, r in ref.items():
        close(g[name], r, bound[name], name)


def pages(lens, page, spare=2, seed=0):
    """(page_table, number of pages): a random order of distinct pages, unused entries -1."""
    need = [-(-int(n) // page) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def check_decode(q, cache, table, lens, dc, scale, o, lse):
    run = lambda c: mla.decode(host(q), c, np.asarray(table), lens, dc, scale)
    c = np.nan_to_num(host(cache))       # what lies in rows that no token sees has no part in the result
    ref, ref_lse = run(c)
    u = U[o.dtype]
    mag = np.zeros(ref.shape)
    for b in range(q.shape[0]):          # sum_j P |row|
        L = max(0, min(int(lens[b]), table.shape[1] * c.shape[1]))
        at = np.asarray(table)[b][np.arange(L) // c.shape[1]]
        here = (at >= 0) & (at < c.shape[0])
        rows = np.where(here[:, None], c[np.where(here, at, 0), np.arange(L) % c.shape[1]], 0.0)
        for i in range(q.shape[1]):
            ok = here & (np.arange(L) < L - (q.shape[1] - 1) + i)
            if ok.any():
                p, _ = mla._softmax(host(q[b, i]) @ rows[ok].T * scale)
                mag[b, i] = p @ np.abs(rows[ok, :dc])
    close(o, ref, u * np.abs(ref) + (u + F) * mag, "o")
    if lse is not None:
        check_lse(lse, ref_lse)
