"""The latent-attention operators against the 64-bit oracle (needs a GPU)."""
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_126_b200 import (mla_append, mla_backward, mla_decode, mla_decode_workspace_size, mla_prefill,
                                       mla_status)
from oracle import mla
from tests.mla_check import (U, check_backward, check_decode, check_lse, check_prefill, close, host, i32, offsets,
                             packed, pages)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(autouse=True)
def no_kernel_flagged_an_error():
    yield
    assert mla_status() == 0


def rnd(*s, dtype=F32, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*s, generator=gen, device="cuda").to(dtype)


# ------------------------------------------------------------------------------ append
APPEND = [  # lens, past, dc, dr, H, page
    ([1], [0], 512, 64, 32, 64),
    ([1, 1, 1], [0, 63, 1000], 512, 64, 7, 64),
    ([5, 0, 70, 1], [3, 9, 60, 0], 256, 32, 4, 16),
    ([3, 2], [1, 0], 100, 6, 3, 1),
    ([9], [2], 8, 0, 0, 4),
    ([0, 4, 0], [5, 5, 5], 192, 16, 1, 3),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", APPEND)
def test_append(case, interleaved, dtype):
    lens, past, dc, dr, H, page = case
    T, cu = sum(lens), offsets(lens)
    table, n = pages([p + m for p, m in zip(past, lens)], page)
    x = rnd(T + 3, dc + dr, dtype=dtype, seed=1)                    # three rows behind the last sequence
    q = rnd(T + 3, max(H, 1), 40 + dr, dtype=dtype, seed=2)[..., 40:] if H else None
    cache = rnd(n, page, dc + dr, dtype=dtype, seed=3)
    w, f = 1 + 0.1 * rnd(dc, seed=4), torch.tensor(10000.0 ** (-np.arange(0, dr, 2) / max(dr, 1)), device="cuda").float()
    before = host(cache)
    kr = x[:, dc:] if dr else None
    out = {"c": torch.full((T + 3, dc), 7.0, device="cuda", dtype=dtype)}
    got = mla_append(x[:, :dc], kr, cache, i32(table), i32(past), i32(cu), norm_weight=w, eps=1e-5,
                     inv_freq=f if dr else None, interleaved=interleaved, q_rope=q, packed=True, out=out)
    assert got["cache"] is cache
    ref = mla.append(host(x[:, :dc]), None if kr is None else host(kr), before, table, past, cu, host(w), 1e-5,
                     host(f) if dr else None, interleaved, None if q is None else host(q))
    u = U[dtype]
    # float32 steps: the norm's sum (512 terms) and three roundings, sin and cos 2 ulp, angle reduced to 2^-25 of a turn
    tol = lambda r, m: u * np.abs(r) + 1e-6 * m
    close(cache, ref[0], tol(ref[0], 8 + np.abs(ref[0])), "cache")
    assert (got["c"][T:] == 7.0).all()                              # rows behind the last sequence are left alone
    close(got["c"][:T], ref[1][:T], tol(ref[1][:T], 8.0), "c")
    if dr:
        close(got["k_rope"][:T], ref[2][:T], tol(ref[2][:T], 8.0), "k_rope")
    if H:
        close(got["q_rope"][:T], ref[3][:T], tol(ref[3][:T], 8.0), "q_rope")


def test_append_far_positions_in_place_and_plain():
    """Positions near 10^9 (page table of one far page), queries rotated in place, no norm."""
    dc, dr, H, page = 64, 64, 2, 1 << 28
    f = torch.tensor(10000.0 ** (-np.arange(0, dr, 2) / dr), device="cuda").float()
    c, kr, q = rnd(3, dc), rnd(3, dr, seed=1), rnd(3, H, dr, seed=2)
    past = [999_999_937, 1_048_576]
    q0 = host(q)
    cache = torch.zeros(1, 4, dc + dr, device="cuda")               # the table leads nowhere: only q and k_rope are written
    got = mla_append(c, kr, cache, i32([[-1] * 4] * 2), i32(past), i32([0, 2, 3]), inv_freq=f, q_rope=q, packed=True,
                     out={"q_rope": q})
    pos = [past[0], past[0] + 1, past[1]]
    assert (cache == 0).all() and got["q_rope"] is q
    close(got["c"], host(c), 0.0, "c")
    close(got["k_rope"], mla.rotate(host(kr), pos, host(f), False), 2e-6, "k_rope")   # |x| up to 4: 4 (2^-24 3 + 2^-25 2 pi)
    close(q, mla.rotate(q0, pos, host(f), False), 2e-6, "q")


def test_append_bad_places_are_skipped():
    table = np.array([[0, 9, -1], [1, 2, -3]])
    cache = torch.zeros(3, 2, 8, device="cuda")
    c = rnd(9, 8)
    mla_append(c, None, cache, i32(table), i32([0, -1]), i32([0, 7, 9]))
    x = host(cache)
    np.testing.assert_array_equal(x[0], host(c[:2]))                # positions 2..6: pages 9, -1 and behind the table
    np.testing.assert_array_equal(x[1, 0], host(c[8]))              # position -1 is skipped, position 0 written
    assert (x[1, 1] == 0).all() and (x[2] == 0).all()


# ------------------------------------------------------------------------------ decode
DECODE = [  # lens, n, H, dc, dr, page
    ([1], 1, 1, 512, 64, 64),
    ([1023], 1, 32, 512, 64, 64),
    ([64, 65, 63, 0, 1, 129], 1, 32, 512, 64, 64),
    ([700, 3, 0, 1, 2, 4097], 4, 32, 512, 64, 32),
    ([513, 100], 3, 5, 512, 0, 16),
    ([90, 31, 2000], 2, 64, 128, 64, 128),
    ([257] * 9, 1, 128, 256, 64, 1),
    ([50, 333], 2, 7, 384, 64, 24),
    ([77, 20], 1, 3, 100, 20, 16),
    ([40], 5, 2, 64, 0, 8),
    ([130], 9, 16, 512, 32, 64),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", DECODE)
def test_decode(case, dtype):
    lens, n, H, dc, dr, page = case
    table, num = pages(lens, page)
    cache = rnd(num, page, dc + dr, dtype=dtype, seed=5)
    q = rnd(len(lens), n, H, dc + dr, dtype=dtype, seed=6)
    mask = torch.zeros(num, page, dtype=torch.bool, device="cuda")   # rows that belong to a sequence
    for b, L in enumerate(lens):
        for j in range(0, L, page):
            mask[table[b, j // page], :min(page, L - j)] = True
    cache[~mask] = NAN                                               # what no token sees may hold anything
    scale = 1 / math.sqrt(128 + dr)
    o, lse = mla_decode(q, cache, i32(table), i32(lens), dc, scale, want_lse=True)
    check_decode(q, cache, table, lens, dc, scale, o, lse)
    again, _ = mla_decode(q, cache, i32(table), i32(lens), dc, scale)
    assert torch.equal(o, again)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_bad_pages_and_lengths(dtype):
    """Pages outside the pool are left out, lengths behind the table's width are cut, negative ones are empty."""
    table = np.array([[0, 99, 2], [-1, -5, 77], [1, 0, 2], [1, 1, 1]])
    lens = [96, 96, 5000, -3]
    cache, q = rnd(3, 32, 576, dtype=dtype), rnd(4, 2, 8, 576, dtype=dtype, seed=1)
    o, lse = mla_decode(q, cache, i32(table), i32(lens), 512, 0.1, want_lse=True)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all() and (o[3] == 0).all()
    check_decode(q, cache, table, lens, 512, 0.1, o, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_sharp_scores_and_shared_pages(dtype):
    """Scores of some hundreds (one key takes all) and a prefix page shared by two sequences."""
    table = np.array([[3, 1], [3, 2]])
    cache, q = rnd(4, 64, 576, dtype=dtype), rnd(2, 1, 16, 576, dtype=dtype, seed=1)
    o, lse = mla_decode(8 * q, cache, i32(table), i32([100, 128]), 512, 1.0, want_lse=True)
    ref, ref_lse = mla.decode(host(8 * q), host(cache), table, [100, 128], 512, 1.0)
    # scores near 600, off by sqrt(576) 2^-23 of absolute sums near 3000: 9e-3, which P takes in full
    assert np.abs(host(lse) - ref_lse).max() <= 1e-2
    assert np.abs(host(o) - ref).max() <= 4 * (2e-2 + 2 * U[dtype])


# ------------------------------------------------------------------------------ prefill and backward
PACKED = [  # q_lens, k_lens, H, dn, dr, dv
    ([1], [1], 1, 128, 64, 128),
    ([128], [128], 2, 128, 64, 128),
    ([127, 129, 1, 0, 64], [127, 129, 1, 0, 64], 3, 128, 64, 128),
    ([300], [300], 2, 128, 0, 128),
    ([5, 200, 130], [500, 333, 130], 2, 128, 64, 128),
    ([140, 7, 0, 3], [20, 0, 9, 3], 2, 128, 64, 128),
    ([513, 255], [513, 700], 1, 128, 64, 128),
    ([65, 70], [65, 90], 3, 72, 24, 80),
    ([66], [66], 2, 33, 7, 65),
    ([10, 100], [10, 100], 2, 64, 0, 64),
    ([20], [30], 1, 1, 1, 1),
    ([150, 70], [150, 190], 34, 24, 8, 20),   # enough blocks for the larger tiles of the CUDA cores
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", PACKED)
def test_prefill_and_backward(case, causal, dtype):
    a, dO = packed(*case, dtype)
    o, lse = mla_prefill(**a, causal=causal, want_lse=True)
    check_prefill(a, o, lse, causal)
    g = mla_backward(**a, o=o, lse=lse, dO=dO, causal=causal)
    check_backward(a, dO, g, causal)
    plain, none = mla_prefill(**a, causal=causal)
    assert none is None and torch.equal(o, plain)
    again = mla_backward(**a, o=o, lse=lse, dO=dO, causal=causal)
    for name, t in g.items():
        assert t is None or torch.equal(t, again[name]), name


@pytest.mark.parametrize("dims", [(128, 64, 128), (64, 32, 64)])
@pytest.mark.parametrize("lens", [[2] * 60, [64] * 12, [300, 200, 33], [777]])
def test_gradients_lose_no_precision_where_keys_are_few(lens, dims):
    """dq and dk against what rounding the exact result makes.  Rounding dS and rounding the output are two independent
    roundings of the same kind, so the sum's error is sqrt(2) times one's: 1.5 asked (delta from the rounded output
    would give up to 2.7)."""
    a, dO = packed(lens, lens, 4, *dims, BF, seed=7)
    o, lse = mla_prefill(**a, want_lse=True)
    g = mla_backward(**a, o=o, lse=lse, dO=dO)
    ref = mla.backward(host(a["q"]), host(a["k"]), host(a["v"]), a["cu_q_host"], a["cu_k_host"], host(dO), k_rope=host(a["k_rope"]))
    for n in ("dq", "dk", "dv"):
        off = lambda x: np.linalg.norm(x - ref[n])
        assert off(host(g[n])) <= 1.5 * off(host(torch.tensor(ref[n]).to(BF))), n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_lens,k_lens,H,causal", [
    ([500], [500], 2, True),                        # 64-row tiles, clusters of eight blocks
    ([700, 33], [700, 40], 3, True),                # of four
    ([600, 33, 600], [600, 33, 500], 5, True),      # of two, queries that see nothing
    ([200] * 30, [200] * 30, 4, True),              # one block
    ([300], [300], 1, True),                        # 32-row tiles
    ([5], [1000], 1, False),                        # a long chain of keys, dk and dv of one short one
    ([1000], [3], 2, False),
    ([16] * 20, [16] * 20, 8, True)])
def test_clusters_share_chains(q_lens, k_lens, H, causal, dtype):
    """Blocks that share a tile's chain on the CUDA cores give the formula's sums, the same ones every time."""
    a, dO = packed(q_lens, k_lens, H, 40, 8, 48, dtype, seed=3)
    o, lse = mla_prefill(**a, causal=causal, want_lse=True)
    check_prefill(a, o, lse, causal=causal)
    g = mla_backward(**a, o=o, lse=lse, dO=dO, causal=causal)
    check_backward(a, dO, g, causal=causal)
    o2, lse2 = mla_prefill(**a, causal=causal, want_lse=True)
    g2 = mla_backward(**a, o=o, lse=lse, dO=dO, causal=causal)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_outside_the_sequences(dtype):
    """Rows behind the last sequence hold NaN: nothing of them is read into a sum, nothing written."""
    a, dO = packed([70, 130], [70, 200], 2, 128, 64, 128, dtype)
    wide = {n: torch.full((t.shape[0] + 40, *t.shape[1:]), NAN, dtype=dtype, device="cuda")
            for n, t in list(a.items()) + [("dO", dO)] if torch.is_tensor(t) and t.dtype == dtype}
    for n, t in wide.items():
        t[:-40] = dO if n == "dO" else a[n]
    big = dict(a, **{n: wide[n] for n in ("q", "k", "v", "k_rope")})
    o = torch.full((240, 2, 128), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((240, 2), 5.0, device="cuda")
    mla_prefill(**big, o=o, lse=lse)
    assert (o[200:] == 5).all() and (lse[200:] == 5).all()
    check_prefill(a, o[:200], lse[:200])
    g = mla_backward(**big, o=o, lse=lse, dO=wide["dO"])
    for n, rows in (("dq", 200), ("dk", 270), ("dv", 270), ("dk_rope", 270)):
        assert (g[n][rows:] == 0).all()
        g[n] = g[n][:rows]
    check_backward(a, dO, g)


def test_neighbours_do_not_leak():
    """A NaN in one packed sequence stays in it, in every tile that the sequences share."""
    a, dO = packed([100, 90, 40], [100, 90, 40], 2, 128, 64, 128, BF)
    for n in ("k", "v", "k_rope", "q"):
        a[n] = a[n].clone()
        a[n][100:190] = NAN
    dO[100:190] = NAN
    o, lse = mla_prefill(**a, want_lse=True)
    g = mla_backward(**a, o=o, lse=lse, dO=dO)
    for t in [o, lse] + [g[n] for n in ("dq", "dk", "dv", "dk_rope")]:
        keep = torch.cat((t[:100], t[190:]))
        assert torch.isfinite(keep).all()
    assert torch.isnan(o[100:190]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_alignment_and_scale(dtype):
    """Head-major and offset layouts give what the packed layout gives; another scale is taken."""
    a, dO = packed([150, 33], [150, 60], 3, 128, 64, 128, dtype)
    o, lse = mla_prefill(**a, scale=0.2, want_lse=True)
    check_prefill(a, o, lse, scale=0.2)
    g = mla_backward(**a, o=o, lse=lse, dO=dO, scale=0.2)
    check_backward(a, dO, g, scale=0.2)
    b = dict(a)
    for n in ("q", "k", "v"):
        b[n] = a[n].transpose(0, 1).contiguous().transpose(0, 1)            # [H, T, d] in memory
    wide = torch.zeros(a["k_rope"].shape[0], 72, dtype=dtype, device="cuda")
    wide[:, 8:] = a["k_rope"]
    b["k_rope"] = wide[:, 8:]
    o2, lse2 = mla_prefill(**b, scale=0.2, want_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    odd = dict(a)
    for n in ("q", "k", "v"):                                                # one element off any 16-byte boundary
        t = torch.zeros(a[n].numel() + 1, dtype=dtype, device="cuda")[1:].view(a[n].shape)
        odd[n] = t.copy_(a[n])
    o3, lse3 = mla_prefill(**odd, scale=0.2, want_lse=True)
    check_prefill(a, o3, lse3, scale=0.2)
    check_backward(a, dO, mla_backward(**odd, o=o3, lse=lse3, dO=dO, scale=0.2), scale=0.2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_scales_that_are_not_positive(scale, dtype):
    a, dO = packed([50, 140], [50, 200], 2, 128, 64, 128, dtype)
    o, lse = mla_prefill(**a, scale=scale, want_lse=True)
    check_prefill(a, o, lse, scale=scale)
    check_backward(a, dO, mla_backward(**a, o=o, lse=lse, dO=dO, scale=scale), scale=scale)
    table, n = pages([70, 200], 64)
    cache, q = rnd(n, 64, 576, dtype=dtype), rnd(2, 2, 8, 576, dtype=dtype, seed=1)
    o, lse = mla_decode(q, cache, i32(table), i32([70, 200]), 512, scale, want_lse=True)
    check_decode(q, cache, table, [70, 200], 512, scale, o, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_queries_or_no_keys(dtype):
    a, dO = packed([0, 0], [5, 130], 2, 128, 64, 128, dtype)
    o, lse = mla_prefill(**a, want_lse=True)
    assert o.shape == (0, 2, 128)
    g = mla_backward(**a, o=o, lse=lse, dO=dO)
    assert all((g[n] == 0).all() for n in ("dk", "dv", "dk_rope")) and g["dk"].shape == (135, 2, 128)
    a, dO = packed([3, 200], [0, 0], 2, 128, 64, 128, dtype)
    o, lse = mla_prefill(**a, want_lse=True)
    assert (o == 0).all() and torch.isneginf(lse).all()
    g = mla_backward(**a, o=o, lse=lse, dO=dO)
    assert (g["dq"] == 0).all() and g["dk"].shape == (0, 2, 128)
    a, dO = packed([0], [0], 1, 128, 64, 128, dtype)
    assert mla_prefill(**a)[0].shape == (0, 1, 128)
    cache, table = rnd(3, 16, 576, dtype=dtype), i32([[0, 1]] * 2)
    assert mla_decode(rnd(2, 0, 4, 576, dtype=dtype), cache, table, i32([3, 9]), 512, 0.1)[0].shape == (2, 0, 4, 512)
    mla_append(rnd(0, 512, dtype=dtype), rnd(0, 64, dtype=dtype), cache, table, i32([3, 9]), i32([0, 0, 0]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_heads_that_share_keys(dtype):
    """Keys and values broadcast over the heads (stride 0): the gradients come back per head."""
    a, dO = packed([60, 33], [60, 90], 1, 128, 64, 128, dtype)
    q, dO = rnd(93, 3, 192, dtype=dtype, seed=3), rnd(93, 3, 128, dtype=dtype, seed=4)
    shared = dict(a, q=q, k=a["k"].expand(-1, 3, -1), v=a["v"].expand(-1, 3, -1))
    o, lse = mla_prefill(**shared, want_lse=True)
    check_prefill(shared, o, lse)
    check_backward(shared, dO, mla_backward(**shared, o=o, lse=lse, dO=dO))


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with workspaces of its own, give what they give alone."""
    table, n = pages([3000, 2500], 64)
    cache, lens, table_d = rnd(n, 64, 576, dtype=BF), i32([3000, 2500]), i32(table)
    q = [rnd(2, 1, 32, 576, dtype=BF, seed=s) for s in (1, 2)]
    a, dO = packed([300, 200], [300, 200], 4, 128, 64, 128, BF)

    def work(x):
        d, _ = mla_decode(x, cache, table_d, lens, 512, 0.07)
        o, lse = mla_prefill(**a, want_lse=True)
        return [d, o, lse] + list(mla_backward(**a, o=o, lse=lse, dO=dO).values())

    want = [work(x) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = work(q[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(want[i], got[i]))


def test_many_short_sequences():
    """More tiles than the host lists, and more sequences than a block has threads."""
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 40, 700)]
    a, dO = packed(lens, lens, 2, 128, 64, 128, BF)
    o, lse = mla_prefill(**a, want_lse=True)
    check_prefill(a, o, lse)
    check_backward(a, dO, mla_backward(**a, o=o, lse=lse, dO=dO))
    table, n = pages(lens, 16)
    cache, q = rnd(n, 16, 192, dtype=BF), rnd(700, 1, 4, 192, dtype=BF, seed=1)
    o, lse = mla_decode(q, cache, i32(table), i32(lens), 128, 0.1, want_lse=True)
    check_decode(q, cache, table, lens, 128, 0.1, o, lse)


def test_gradient_against_differences():
    """dq, dk, dv and dk_rope of the f32 path along a random direction, against central differences in 64 bits."""
    a, dO = packed([40, 9], [40, 20], 2, 32, 16, 24, F32)
    o, lse = mla_prefill(**a, want_lse=True)
    g = mla_backward(**a, o=o, lse=lse, dO=dO)
    h = {n: host(a[n]) for n in ("q", "k", "v", "k_rope")}
    loss = lambda x: (mla.prefill(x["q"], x["k"], x["v"], a["cu_q_host"], a["cu_k_host"], k_rope=x["k_rope"])[0] * host(dO)).sum()
    rng = np.random.default_rng(3)
    for n in h:
        d = rng.standard_normal(h[n].shape)
        eps = 1e-5
        num = (loss(dict(h, **{n: h[n] + eps * d})) - loss(dict(h, **{n: h[n] - eps * d}))) / (2 * eps)
        size = np.abs(host(g["d" + n]) * d).sum()
        # float32 gradients: relative errors to 4e-5 of absolute sums; differences' own error is under 1e-8
        assert abs((host(g["d" + n]) * d).sum() - num) <= 4e-5 * size + 1e-6, n


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_layer_served(dtype):
    """Prompt (append, expand, prefill), then steps of 1 and 3 tokens (append, absorb, decode): each step's output
    is the expanded attention over all tokens so far."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s, sd=1.0: (sd * torch.randn(*s, generator=gen, device="cuda"))
    H, dn, dr, dv, dc, page = 4, 128, 64, 128, 512, 32
    wk, wv, w = r(H, dc, dn, sd=dc ** -0.5), r(H, dc, dv, sd=dc ** -0.5), 1 + 0.1 * r(dc)
    f = torch.tensor(10000.0 ** (-np.arange(0, dr, 2) / dr), device="cuda").float()
    prompts, steps, B = [90, 1, 37], [1, 3, 1], 3
    ends = [p + sum(steps) for p in prompts]
    table, n = pages(ends, page)
    table_d = i32(table)
    cache = torch.full((n, page, dc + dr), NAN, dtype=dtype, device="cuda")
    scale = (dn + dr) ** -0.5
    c_all, k_all = [[] for _ in range(B)], [[] for _ in range(B)]
    past = [0] * B
    for step, lens in enumerate([prompts] + [[s] * B for s in steps]):
        cu = offsets(lens)
        x, q = r(cu[-1], dc + dr).to(dtype), r(cu[-1], H, dn + dr).to(dtype)
        out = mla_append(x[:, :dc], x[:, dc:], cache, table_d, i32(past), i32(cu), norm_weight=w, inv_freq=f,
                         q_rope=q[..., dn:], packed=True, out={"q_rope": q[..., dn:]})
        for b in range(B):
            c_all[b].append(host(out["c"][cu[b]:cu[b + 1]]))
            k_all[b].append(host(out["k_rope"][cu[b]:cu[b + 1]]))
        past = [p + m for p, m in zip(past, lens)]
        # the reference: expanded attention in 64 bits over the rows as cached
        cat = [np.concatenate(v) for v in c_all], [np.concatenate(v) for v in k_all]
        c64 = np.concatenate(cat[0])
        k64, v64 = np.einsum("lc,hcd->lhd", c64, host(wk)), np.einsum("lc,hcd->lhd", c64, host(wv))
        ref, _ = mla.prefill(host(q), k64, v64, cu, offsets(past), k_rope=np.concatenate(cat[1]), scale=scale)
        if step == 0:
            k = torch.einsum("lc,hcd->lhd", out["c"].float(), wk).to(dtype)
            v = torch.einsum("lc,hcd->lhd", out["c"].float(), wv).to(dtype)
            o, _ = mla_prefill(q, k, v, i32(cu), i32(cu), k_rope=out["k_rope"], scale=scale)
        else:
            m = lens[0]
            qa = torch.cat((torch.einsum("thd,hcd->thc", q[..., :dn].float(), wk).to(dtype), q[..., dn:]), -1)
            ol, _ = mla_decode(qa.view(B, m, H, dc + dr), cache, table_d, i32(past), dc, scale)
            o = torch.einsum("thc,hcd->thd", ol.float().view(-1, H, dc), wv)
        # keys, values, absorbed queries and outputs are rounded (u each): scores are off by 2 u sqrt(192) |q||k| scale,
        # about 8 u, and so is P in relative terms; outputs of size 1 and below: 16 u over the largest
        assert np.abs(host(o) - ref).max() <= 16 * max(U[dtype], 2e-6) * max(1.0, np.abs(ref).max()), step


def test_streams_and_graphs():
    """Another stream than the current one, and a captured step replayed on new data and lengths."""
    table, n = pages([400, 400], 64)
    cache, q = rnd(n, 64, 576, dtype=BF), rnd(2, 1, 8, 576, dtype=BF, seed=1)
    lens, table_d = i32([100, 399]), i32(table)
    want, _ = mla_decode(q, cache, table_d, lens, 512, 0.07)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = mla_decode(q, cache, table_d, lens, 512, 0.07, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    a, dO = packed([130], [130], 2, 128, 64, 128, BF)
    o, lse = mla_prefill(**a, want_lse=True)
    g = mla_backward(**a, o=o, lse=lse, dO=dO)
    torch.cuda.synchronize()
    o2, lse2 = mla_prefill(**a, want_lse=True, stream=side)
    g2 = mla_backward(**a, o=o2, lse=lse2, dO=dO, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and all(torch.equal(g[x], g2[x]) for x in g)

    row, pos = rnd(2, 576, dtype=BF, seed=9), i32([100, 399])
    cu, ends = i32([0, 1, 2]), i32([101, 400])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla_append(row[:, :512], row[:, 512:], cache, table_d, pos, cu)
        og, _ = mla_decode(q, cache, table_d, ends, 512, 0.07)
        pg, pl = mla_prefill(**a, want_lse=True)
        gg = mla_backward(**a, o=pg, lse=pl, dO=dO)
    for k in range(2):
        row.copy_(rnd(2, 576, dtype=BF, seed=20 + k))
        pos.copy_(i32([7 + k, 300]))
        ends.copy_(i32([8 + k, 301]))
        graph.replay()
        torch.cuda.synchronize()
        check_decode(q, cache, table, [8 + k, 301], 512, 0.07, og, None)
        assert torch.equal(cache[int(table[0, 0]), 7 + k], row[0])
        assert torch.equal(pg, o) and all(torch.equal(g[x], gg[x]) for x in g)


def test_captured_on_the_cuda_cores():
    """Float32 calls, their clusters and their join, captured with one workspace for two decodes and replayed on new data."""
    a, dO = packed([300, 90], [300, 90], 2, 72, 24, 80, F32)
    lens = [700, 31]
    table, n = pages(lens, 16)
    cache, q = rnd(n, 16, 288, dtype=F32), rnd(2, 1, 12, 288, dtype=F32, seed=1)
    table_d, lens_d = i32(table), i32(lens)
    ws = torch.empty(mla_decode_workspace_size(2, 1, 12, 256, 32, F32), dtype=torch.uint8, device="cuda")
    mla_prefill(**a)
    mla_decode(q, cache, table_d, lens_d, 256, 0.07)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = mla_prefill(**a, want_lse=True)
        g = mla_backward(**a, o=o, lse=lse, dO=dO)
        first, _ = mla_decode(q, cache, table_d, lens_d, 256, 0.07, workspace=ws)
        second, _ = mla_decode(q, cache, table_d, lens_d, 256, 0.2, workspace=ws)
    for k in range(2):
        b, dO2 = packed([300, 90], [300, 90], 2, 72, 24, 80, F32, seed=30 + k)
        for name in ("q", "k", "v", "k_rope"):
            a[name].copy_(b[name])
        dO.copy_(dO2)
        q.copy_(rnd(2, 1, 12, 288, dtype=F32, seed=40 + k))
        graph.replay()
        torch.cuda.synchronize()
        check_prefill(a, o, lse)
        check_backward(a, dO, g)
        check_decode(q, cache, table, lens, 256, 0.07, first, None)
        check_decode(q, cache, table, lens, 256, 0.2, second, None)


def test_long_cache_offsets():
    """A pool of more than 2^31 elements: rows at its far end are found."""
    page, W, num = 64, 576, 60_000                                   # 2.2e9 elements, 4.4 GB
    cache = torch.empty(num, page, W, dtype=BF, device="cuda")
    table = np.array([[num - 1, num - 3, 5]])
    for p in table[0]:
        cache[int(p)] = rnd(page, W, dtype=BF, seed=int(p))
    c, cu, past = rnd(2, W, dtype=BF, seed=2), i32([0, 2]), i32([62])
    mla_append(c[:, :512], c[:, 512:], cache, i32(table), past, cu)
    assert torch.equal(cache[num - 1, 62], c[0]) and torch.equal(cache[num - 1, 63], c[1])
    q = rnd(1, 1, 32, W, dtype=BF, seed=3)
    o, _ = mla_decode(q, cache, i32(table), i32([150]), 512, 0.07)
    small = torch.stack([cache[int(p)] for p in table[0]])
    want, _ = mla_decode(q, small, i32([[0, 1, 2]]), i32([150]), 512, 0.07)
    assert torch.equal(o, want)
