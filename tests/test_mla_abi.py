"""The latent-attention entry points export what mla.h declares and refuse bad arguments on
the host (no GPU: every check returns before a CUDA call), and the binding checks shapes."""
import ctypes
import os
import re

import pytest
import torch

from gated_delta_rule_126_b200 import _binding, _mla_binding, build
from gated_delta_rule_126_b200 import mla_append, mla_backward, mla_decode, mla_prefill

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
BF = torch.bfloat16
FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _mla_binding._lib()


def test_exports(lib):
    text = open(os.path.join(ROOT, "include", "mla.h")).read()
    declared = set(re.findall(r"KDA_API\s+[\w\s\*]+?\b(mla_\w+)\s*\(", text))
    assert declared == {"mla_append", "mla_decode", "mla_decode_workspace_size", "mla_prefill", "mla_backward",
                        "mla_backward_workspace_size", "mla_status"}
    out = os.popen(f"nm -D --defined-only {_binding.LIB_PATH}").read()
    assert {ln.split()[-1] for ln in out.splitlines() if " T " in ln and "mla" in ln} == declared


def _append(lib, **kw):
    g = lambda n, d: kw.get(n, d)
    return lib.mla_append(g("c", FAKE), g("cs", 576), g("kr", FAKE), 576, g("dt", 1), g("w", FAKE), g("eps", 1e-6), None,
                          0, g("cu", FAKE), g("past", FAKE), g("N", 2), g("T", 4), g("table", FAKE), g("mp", 3),
                          g("cache", FAKE), g("pages", 8), g("page", 16), g("dc", 512), g("dr", 64), g("q", FAKE),
                          g("qs", 64), 64, g("H", 4), g("qo", FAKE), 64, 64, None, None, None)


def test_append_refusals(lib):
    for bad in (dict(N=-1), dict(T=-1), dict(mp=-1), dict(pages=-1), dict(page=0), dict(dc=0), dict(dr=-2), dict(dt=2),
                dict(eps=-1.0), dict(eps=float("nan")), dict(H=0), dict(qo=None), dict(dr=0), dict(cs=-1), dict(qs=-1),
                dict(c=None), dict(kr=None), dict(cu=None), dict(past=None), dict(table=None), dict(cache=None),
                dict(c=ODD), dict(cache=ODD), dict(qo=ODD)):
        assert _append(lib, **bad) == INVALID, bad
    for bad in (dict(dc=513), dict(dr=66), dict(dr=63), dict(H=65536), dict(T=1 << 31)):
        assert _append(lib, **bad) == UNSUPPORTED, bad
    assert _append(lib, N=0) == 0 and _append(lib, T=0) == 0


def _decode(lib, **kw):
    g = lambda n, d: kw.get(n, d)
    ws = lib.mla_decode_workspace_size(2, 1, 4, 512, 64, 1)
    return lib.mla_decode(g("q", FAKE), g("dt", 1), g("cache", FAKE), g("pages", 8), g("page", 16), g("table", FAKE),
                          g("mp", 3), g("lens", FAKE), g("B", 2), g("n", 1), g("H", 4), g("dc", 512), g("dr", 64),
                          g("scale", 0.1), g("o", FAKE), None, g("ws", FAKE), g("size", ws), None)


def test_decode_refusals(lib):
    size = lib.mla_decode_workspace_size
    assert size(2, 1, 4, 512, 64, 1) > 0 and size(2, 1, 4, 513, 64, 1) == 0 and size(-1, 1, 4, 512, 64, 1) == 0
    assert size(2, 0, 4, 512, 64, 1) > 0 and size(0, 0, 1, 1, 0, 0) > 0          # no tokens is a size like another
    assert size(1, 1, 0, 512, 64, 1) == 0 and size(1, 2, 40000, 512, 64, 1) == 0
    for bad in (dict(dt=5), dict(B=-1), dict(n=-1), dict(H=0), dict(dc=0), dict(dr=-1), dict(page=0), dict(pages=-1),
                dict(mp=-1), dict(scale=float("inf")), dict(q=None), dict(o=None), dict(lens=None), dict(table=None),
                dict(cache=None), dict(q=ODD), dict(o=ctypes.c_void_p((1 << 20) + 8)), dict(cache=ODD)):
        assert _decode(lib, **bad) == INVALID, bad
    for bad in (dict(dc=520), dict(dr=65), dict(B=65537), dict(n=65537)):
        assert _decode(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(size=256), dict(ws=ctypes.c_void_p((1 << 20) + 64))):
        assert _decode(lib, **bad) == WORKSPACE, bad
    assert _decode(lib, B=0) == 0 and _decode(lib, n=0) == 0


def _prefill(lib, backward=False, cq=(0, 4), ck=(0, 6), N=1, **kw):
    g = lambda n, d: kw.get(n, d)
    arr = lambda c: None if c is None else (ctypes.c_int32 * len(c))(*c)
    lead = [g("q", FAKE), g("qs", 384), 192, g("k", FAKE), 512, g("ks", 256), g("kr", FAKE), 64, g("v", FAKE), 512, 256,
            g("dt", 1), g("cqd", FAKE), arr(cq), g("ckd", FAKE), arr(ck), N, g("H", 2), g("dn", 128), g("dr", 64),
            g("dv", 128), g("scale", 0.1), 1]
    if not backward:
        return lib.mla_prefill(*lead, g("o", FAKE), None, None)
    ws = lib.mla_backward_workspace_size(4, 6, 2, 128, 64, 128, 1)
    return lib.mla_backward(*lead, g("o", FAKE), g("lse", FAKE), g("dO", FAKE), g("dq", FAKE), g("dk", FAKE),
                            g("dkr", FAKE), g("dvo", FAKE), g("ws", FAKE), g("size", ws), None)


@pytest.mark.parametrize("backward", [False, True])
def test_prefill_and_backward_refusals(lib, backward):
    f = lambda **kw: _prefill(lib, backward, **kw)
    for bad in (dict(N=-1), dict(dt=9), dict(H=0), dict(dn=0), dict(dr=-1), dict(dv=0), dict(scale=float("nan")),
                dict(cq=(1, 4)), dict(ck=(0, -1)), dict(cq=(0, 4, 3), ck=(0, 6, 6), N=2), dict(cq=None), dict(cqd=None),
                dict(ckd=None), dict(q=None), dict(k=None), dict(v=None), dict(kr=None), dict(qs=-1), dict(ks=-8),
                dict(q=ODD), dict(kr=ODD), dict(o=None), dict(o=ODD)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(dn=129), dict(dr=65), dict(dv=129), dict(H=65536)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(cq=(0,), ck=(0,), N=0) == 0
    if backward:
        for bad in (dict(lse=None), dict(dO=None), dict(dq=None), dict(dk=None), dict(dkr=None), dict(dvo=None),
                    dict(dO=ODD), dict(dk=ODD)):
            assert f(**bad) == INVALID, bad
        for bad in (dict(ws=None), dict(size=255), dict(ws=ctypes.c_void_p((1 << 20) + 16))):
            assert f(**bad) == WORKSPACE, bad
        size = lib.mla_backward_workspace_size
        assert size(4, 6, 2, 129, 64, 128, 1) == 0 and size(-1, 6, 2, 128, 64, 128, 1) == 0
        assert size(1 << 40, 6, 2, 128, 64, 128, 1) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU failure mode")
def test_valid_calls_without_gpu_report_cuda_error(lib):
    assert _append(lib) == 4 and _decode(lib) == 4
    assert _prefill(lib) == 4 and _prefill(lib, True) == 4
    assert _prefill(lib, dt=0) == 4 and _prefill(lib, True, dt=0) == 4 and _decode(lib, dt=0, size=1 << 30) == 4


def z(*s, dtype=BF):
    return torch.zeros(*s, dtype=dtype)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_binding_checks(lib):
    args = dict(c=z(5, 16), k_rope=z(5, 4), cache=z(3, 8, 20), page_table=i32([0, 1], [2, 0]), past_lens=i32(0, 3),
                cu_seqlens=i32(0, 2, 5))
    with pytest.raises(ValueError, match="CUDA"):
        mla_append(**args)
    for name, bad in [("k_rope", z(4, 4)), ("cache", z(3, 8, 16)), ("past_lens", i32(0)), ("cu_seqlens", i32(0, 5)),
                      ("norm_weight", z(4)), ("inv_freq", z(4)), ("q_rope", z(5, 2, 6))]:
        with pytest.raises(ValueError, match="shape"):
            mla_append(**{**args, name: bad})
    with pytest.raises(ValueError, match="not an output"):
        mla_append(**args, out={"c": z(5, 16)})
    with pytest.raises(ValueError, match="not an output"):
        mla_append(**args, out={"q": z(5, 16)})
    dec = dict(q=z(2, 1, 3, 20), cache=z(3, 8, 20), page_table=i32([0, 1], [2, 0]), seq_lens=i32(4, 9), d_latent=16,
               scale=0.1)
    with pytest.raises(ValueError, match="CUDA"):
        mla_decode(**dec)
    for name, bad in [("cache", z(3, 8, 24)), ("page_table", i32([0, 1])), ("seq_lens", i32(1)), ("o", z(2, 1, 3, 20)),
                      ("lse", z(2, 1, 4))]:
        with pytest.raises(ValueError, match="shape"):
            mla_decode(**{**dec, name: bad})
    with pytest.raises(ValueError, match="d_latent"):
        mla_decode(**{**dec, "d_latent": 21})
    pre = dict(q=z(6, 2, 12), k=z(7, 2, 8), v=z(7, 2, 8), cu_q=i32(0, 6), cu_k=i32(0, 7), k_rope=z(7, 4))
    with pytest.raises(ValueError, match="CUDA"):
        mla_prefill(**pre)
    for name, bad in [("q", z(6, 2, 8)), ("k", z(7, 1, 8)), ("v", z(6, 2, 8)), ("k_rope", z(6, 4)), ("o", z(6, 2, 9))]:
        with pytest.raises(ValueError, match="shape"):
            mla_prefill(**{**pre, name: bad})
    with pytest.raises(ValueError, match="tokens"):
        mla_prefill(**{**pre, "cu_k": i32(0, 8)})
    with pytest.raises(ValueError, match="sequences"):
        mla_prefill(**{**pre, "cu_k": i32(0, 3, 7)})
    with pytest.raises(ValueError, match="shape"):
        mla_backward(**pre, o=z(6, 2, 8), lse=z(6, 3), dO=z(6, 2, 8))


def test_overlapping_output_rows_are_refused():
    with pytest.raises(ValueError, match="overlap"):
        _mla_binding._written(torch.zeros(1, 4).expand(3, 4), "x")
    _mla_binding._written(torch.zeros(5, 3, 10)[..., 4:], "x")
    _mla_binding._written(torch.zeros(3, 5, 4).transpose(0, 1), "x")


def test_binding_refuses_another_devices_stream():
    class Stream:  # as much of a torch.cuda.Stream as the check sees
        device_index, cuda_stream = 1, 0

    with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cuda:0"):
        _mla_binding._on(Stream(), 0)
