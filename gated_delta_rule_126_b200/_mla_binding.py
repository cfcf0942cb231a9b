"""ctypes binding of ``include/mla.h`` (argument marshalling only), as ``_binding`` is of ``kda.h``."""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import _binding
from ._binding import DTYPE_CODE, _check, _dims, _need, _offsets, _ptr, _shapes, _stream_handle

_declared = None


def _lib():
    global _declared
    lib = _binding.load()
    if _declared is not lib:
        c = ctypes
        vp, i32, i64, sz, f32 = c.c_void_p, c.c_int, c.c_int64, c.c_size_t, c.c_float
        lib.mla_append.restype = i32
        lib.mla_append.argtypes = [vp, i64, vp, i64, i32, vp, f32, vp, i32, vp, vp, i32, i64, vp, i32, vp, i32, i32,
                                   i32, i32, vp, i64, i64, i32, vp, i64, i64, vp, vp, vp]
        lib.mla_decode_workspace_size.restype = sz
        lib.mla_decode_workspace_size.argtypes = [i32] * 6
        lib.mla_decode.restype = i32
        lib.mla_decode.argtypes = [vp, i32, vp, i32, i32, vp, i32, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp, sz, vp]
        packed = [vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, i64, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32]
        lib.mla_prefill.restype = i32
        lib.mla_prefill.argtypes = packed + [vp, vp, vp]
        lib.mla_backward_workspace_size.restype = sz
        lib.mla_backward_workspace_size.argtypes = [i64, i64] + [i32] * 5
        lib.mla_backward.restype = i32
        lib.mla_backward.argtypes = packed + [vp] * 8 + [sz, vp]
        lib.mla_status.restype = i32
        lib.mla_status.argtypes = [vp]
        _declared = lib
    return lib


@contextlib.contextmanager
def _on(stream, dev):
    """The device and stream a call runs on: what it allocates belongs to that stream."""
    with torch.cuda.device(dev):
        if stream is None:
            yield torch.cuda.current_stream()
        else:
            with torch.cuda.stream(stream):
                yield stream


def _rows(rows, used, *shape, dtype, device):
    """An output of which a call writes the first ``used`` rows; the rest are zero."""
    t = torch.empty(rows, *shape, dtype=dtype, device=device)
    if used < rows:
        t[used:].zero_()
    return t


def _strided(t, name, dtype, device):
    """A CUDA tensor whose last dimension is contiguous; the others may have any non-negative stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _written(t, name):
    """An output's rows must be apart from one another: every stride covers what lies inside it."""
    inside = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda p: p[1]):
        if size > 1 and stride < inside:
            raise ValueError(f"{name}'s rows overlap (strides {t.stride()})")
        if size > 1:
            inside = stride * (size - 1) + inside
    return t


def _type(t, name):
    if t.dtype not in DTYPE_CODE:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return t.dtype


def mla_append(c, k_rope, cache, page_table, past_lens, cu_seqlens, norm_weight=None, eps=1e-6, inv_freq=None,
               interleaved=False, q_rope=None, packed=False, out=None, stream=None):
    """Norm, rotation and the write into the paged cache (see ``mla_append`` in mla.h).

    c [T,d_latent], k_rope [T,d_rope] or None (d_rope = 0), q_rope [T,H,d_rope] or None:
    float32 or bfloat16, contiguous in the last dimension (slices of a projection do).
    cache [num_pages,page_size,d_latent+d_rope] is updated in place; page_table
    [N,max_pages], past_lens [N], cu_seqlens [N+1] int32 on the device; norm_weight
    [d_latent] and inv_freq [d_rope/2] float32 or None (no norm, no rotation).

    Returns a dict: "cache"; "q_rope" when q_rope is given; "c" and "k_rope", the packed
    rows as they were cached, when ``packed``.  ``out`` may supply "q_rope" (the input
    itself rotates in place), "c" and "k_rope".
    """
    lib = _lib()
    T, dc = _dims(c, "c", 2)
    dr = 0 if k_rope is None else _dims(k_rope, "k_rope", 2)[1]
    pages, page, _ = _dims(cache, "cache", 3)
    N, width = _dims(page_table, "page_table", 2)
    H = 0 if q_rope is None else _dims(q_rope, "q_rope", 3)[1]
    given = dict(out or {})
    for name in given:
        if name not in ("q_rope", "c", "k_rope") or (name == "q_rope" and q_rope is None) or (
                name != "q_rope" and not packed) or (name == "k_rope" and not dr):
            raise ValueError(f"out[{name!r}] is not an output of this call")
    _shapes(k_rope=(k_rope, (T, dr)), cache=(cache, (pages, page, dc + dr)), past_lens=(past_lens, (N,)),
            cu_seqlens=(cu_seqlens, (N + 1,)), norm_weight=(norm_weight, (dc,)), inv_freq=(inv_freq, (dr // 2,)),
            q_rope=(q_rope, (T, H, dr)))
    for name, shape in (("q_rope", (T, H, dr)), ("c", (T, dc)), ("k_rope", (T, dr))):
        _shapes(**{f"out[{name!r}]": (given.get(name), shape)})
    dev, dt = c.device, _type(c, "c")
    _strided(c, "c", dt, None)
    if dr:
        _strided(k_rope, "k_rope", dt, dev)
    _need(cache, "cache", dt, dev)
    for name, t in (("page_table", page_table), ("past_lens", past_lens), ("cu_seqlens", cu_seqlens)):
        _need(t, name, torch.int32, dev)
    for name, t in (("norm_weight", norm_weight), ("inv_freq", inv_freq)):
        if t is not None:
            _need(t, name, torch.float32, dev)
    if q_rope is not None:
        _strided(q_rope, "q_rope", dt, dev)
    if "q_rope" in given:
        _strided(given["q_rope"], "out['q_rope']", dt, dev)
        _written(given["q_rope"], "out['q_rope']")
    for name in ("c", "k_rope"):
        if name in given:
            _need(given[name], f"out[{name!r}]", dt, dev)
    st = lambda t, i: 0 if t is None else t.stride(i)
    with _on(stream, dev) as use:
        res = {"cache": cache}
        if q_rope is not None:
            res["q_rope"] = given["q_rope"] if "q_rope" in given else torch.empty(T, H, dr, dtype=dt, device=dev)
        if packed:
            res["c"] = given["c"] if "c" in given else torch.empty(T, dc, dtype=dt, device=dev)
            if dr:
                res["k_rope"] = given["k_rope"] if "k_rope" in given else torch.empty(T, dr, dtype=dt, device=dev)
        qo = res.get("q_rope")
        status = lib.mla_append(_ptr(c), st(c, 0), _ptr(k_rope), st(k_rope, 0), DTYPE_CODE[dt], _ptr(norm_weight),
                                float(eps), _ptr(inv_freq), int(bool(interleaved)), _ptr(cu_seqlens),
                                _ptr(past_lens), N, T, _ptr(page_table), width, _ptr(cache), pages, page, dc, dr,
                                _ptr(q_rope), st(q_rope, 0), st(q_rope, 1), H, _ptr(qo), st(qo, 0), st(qo, 1),
                                _ptr(res.get("c")), _ptr(res.get("k_rope")), _stream_handle(use))
    _check(status, "mla_append")
    return res


def mla_decode_workspace_size(B, n, H, d_latent, d_rope, dtype=torch.bfloat16):
    return int(_lib().mla_decode_workspace_size(int(B), int(n), int(H), int(d_latent), int(d_rope), DTYPE_CODE[dtype]))


def mla_decode(q, cache, page_table, seq_lens, d_latent, scale, o=None, lse=None, want_lse=False, workspace=None,
               stream=None):
    """Absorbed latent attention over the paged cache (see ``mla_decode`` in mla.h).

    q [B,n,H,d_latent+d_rope], cache [num_pages,page_size,d_latent+d_rope] (float32 or
    bfloat16), page_table [B,max_pages] and seq_lens [B] int32 on the device; seq_lens
    counts the n new tokens.  scale is 1 / sqrt of the expanded head's size (it cannot be
    told from the absorbed shapes).  Returns ``(o [B,n,H,d_latent], lse [B,n,H] or None)``.
    """
    lib = _lib()
    B, n, H, W = _dims(q, "q", 4)
    pages, page, _ = _dims(cache, "cache", 3)
    width = _dims(page_table, "page_table", 2)[1]
    dc = int(d_latent)
    if not 1 <= dc <= W:
        raise ValueError(f"d_latent must lie in 1..{W}, got {dc}")
    _shapes(cache=(cache, (pages, page, W)), page_table=(page_table, (B, width)), seq_lens=(seq_lens, (B,)),
            o=(o, (B, n, H, dc)), lse=(lse, (B, n, H)))
    dev, dt = q.device, _type(q, "q")
    _need(q, "q", dt)
    _need(cache, "cache", dt, dev)
    _need(page_table, "page_table", torch.int32, dev)
    _need(seq_lens, "seq_lens", torch.int32, dev)
    for name, t, want in (("o", o, dt), ("lse", lse, torch.float32), ("workspace", workspace, None)):
        if t is not None:
            _need(t, name, want, dev)
    with _on(stream, dev) as use:
        if o is None:
            o = torch.empty(B, n, H, dc, dtype=dt, device=dev)
        if lse is None and want_lse:
            lse = torch.empty(B, n, H, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(max(mla_decode_workspace_size(B, n, H, dc, W - dc, dt), 256), dtype=torch.uint8,
                                    device=dev)
        st = lib.mla_decode(_ptr(q), DTYPE_CODE[dt], _ptr(cache), pages, page, _ptr(page_table), width,
                            _ptr(seq_lens), B, n, H, dc, W - dc, float(scale), _ptr(o), _ptr(lse), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream_handle(use))
    _check(st, "mla_decode")
    return o, lse


def _packed(q, k, v, cu_q, cu_k, k_rope, scale, cu_q_host, cu_k_host, o, lse, dO=None):
    """Checks shared by mla_prefill and mla_backward; returns sizes and the library's leading arguments."""
    Tq, H, d = _dims(q, "q", 3)
    Tk, _, dn = _dims(k, "k", 3)
    dv = _dims(v, "v", 3)[2]
    dr = 0 if k_rope is None else _dims(k_rope, "k_rope", 2)[1]
    _shapes(q=(q, (Tq, H, dn + dr)), k=(k, (Tk, H, dn)), v=(v, (Tk, H, dv)), k_rope=(k_rope, (Tk, dr)),
            o=(o, (Tq, H, dv)), lse=(lse, (Tq, H)), dO=(dO, (Tq, H, dv)))
    N, cq = _offsets(cu_q, cu_q_host, Tq)
    M, ck = _offsets(cu_k, cu_k_host, Tk)
    if N != M:
        raise ValueError(f"cu_q holds {N} sequences, cu_k {M}")
    dev, dt = q.device, _type(q, "q")
    _strided(q, "q", dt, None)
    _strided(k, "k", dt, dev)
    _strided(v, "v", dt, dev)
    if dr:
        _strided(k_rope, "k_rope", dt, dev)
    _need(cu_q, "cu_q", torch.int32, dev)
    _need(cu_k, "cu_k", torch.int32, dev)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    lead = [_ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0), k.stride(1), _ptr(k_rope),
            k_rope.stride(0) if dr else 0, _ptr(v), v.stride(0), v.stride(1), DTYPE_CODE[dt], _ptr(cu_q),
            ctypes.c_void_p(cq.data_ptr()), _ptr(cu_k), ctypes.c_void_p(ck.data_ptr()), N, H, dn, dr, dv, scale]
    return (Tq, Tk, H, dn, dr, dv, dev, dt, cq, ck), lead


def mla_prefill(q, k, v, cu_q, cu_k, k_rope=None, scale=None, causal=True, cu_q_host=None, cu_k_host=None, o=None,
                lse=None, want_lse=False, stream=None):
    """Expanded latent attention over packed sequences (see ``mla_prefill`` in mla.h).

    q [Tq,H,d_nope+d_rope], k [Tk,H,d_nope], v [Tk,H,d_v], k_rope [Tk,d_rope] shared by the
    heads or None (d_rope = 0): float32 or bfloat16, contiguous in the last dimension.
    cu_q, cu_k [N+1] int32 on the device and their host copies as in ``kda_prefill``.
    scale defaults to 1 / sqrt(d_nope + d_rope).  Returns ``(o [Tq,H,d_v], lse [Tq,H] or None)``;
    rows that belong to no sequence are zero, or left as they were in a given o or lse.
    """
    lib = _lib()
    (Tq, Tk, H, dn, dr, dv, dev, dt, cq, ck), lead = _packed(q, k, v, cu_q, cu_k, k_rope, scale, cu_q_host, cu_k_host,
                                                             o, lse)
    for name, t, want in (("o", o, dt), ("lse", lse, torch.float32)):
        if t is not None:
            _need(t, name, want, dev)
    with _on(stream, dev) as use:
        if o is None:
            o = _rows(Tq, int(cq[-1]), H, dv, dtype=dt, device=dev)
        if lse is None and want_lse:
            lse = _rows(Tq, int(cq[-1]), H, dtype=torch.float32, device=dev)
        st = lib.mla_prefill(*lead, int(bool(causal)), _ptr(o), _ptr(lse), _stream_handle(use))
    _check(st, "mla_prefill")
    return o, lse


def mla_backward_workspace_size(total_q, total_k, H, d_nope, d_rope, d_v, dtype=torch.bfloat16):
    return int(_lib().mla_backward_workspace_size(int(total_q), int(total_k), int(H), int(d_nope), int(d_rope),
                                                  int(d_v), DTYPE_CODE[dtype]))


def mla_backward(q, k, v, cu_q, cu_k, o, lse, dO, k_rope=None, scale=None, causal=True, cu_q_host=None,
                 cu_k_host=None, workspace=None, stream=None):
    """Gradients of ``mla_prefill`` (see ``mla_backward`` in mla.h).

    Inputs as there, its outputs o [Tq,H,d_v] and lse [Tq,H], and dO [Tq,H,d_v].  Returns a
    dict of tensors in the inputs' dtype: dq, dk, dv and dk_rope (None without k_rope; summed
    over the heads).  Rows that belong to no sequence come back zero.
    """
    lib = _lib()
    (Tq, Tk, H, dn, dr, dv, dev, dt, cq, ck), lead = _packed(q, k, v, cu_q, cu_k, k_rope, scale, cu_q_host, cu_k_host,
                                                             o, lse, dO)
    _need(o, "o", dt, dev)
    _need(lse, "lse", torch.float32, dev)
    _need(dO, "dO", dt, dev)
    tq, tk = int(cq[-1]), int(ck[-1])

    if workspace is not None:
        _need(workspace, "workspace", None, dev)
    like = dict(dtype=dt, device=dev)
    with _on(stream, dev) as use:
        out = dict(dq=_rows(Tq, tq, H, dn + dr, **like), dk=_rows(Tk, tk, H, dn, **like), dv=_rows(Tk, tk, H, dv, **like),
                   dk_rope=_rows(Tk, tk, dr, **like) if dr else None)
        if workspace is None:
            workspace = torch.empty(max(mla_backward_workspace_size(tq, tk, H, dn, dr, dv, dt), 256),
                                    dtype=torch.uint8, device=dev)
        st = lib.mla_backward(*lead, int(bool(causal)), _ptr(o), _ptr(lse), _ptr(dO), _ptr(out["dq"]),
                              _ptr(out["dk"]), _ptr(out["dk_rope"]), _ptr(out["dv"]), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream_handle(use))
    _check(st, "mla_backward")
    return out


def mla_status(stream=None):
    """Waits for the stream; the status flagged by the mla_* kernels run so far on the current device (0 = fine)."""
    return int(_lib().mla_status(_stream_handle(stream)))
