"""The latent-attention oracle against closed forms, differences and an equivalence (CPU)."""
import numpy as np
import pytest

from oracle import mla

rng = np.random.default_rng(7)


def small(Tq, Tk, H=2, dn=5, dr=4, dv=3):
    r = lambda *s: rng.standard_normal(s)
    return r(Tq, H, dn + dr), r(Tk, H, dn), r(Tk, H, dv), r(Tk, dr)


def test_one_key_and_equal_keys():
    q, k, v, kr = small(1, 1)
    o, lse = mla.prefill(q, k, v, [0, 1], [0, 1], k_rope=kr, scale=0.5)
    np.testing.assert_allclose(o[0], v[0], atol=1e-15)
    np.testing.assert_allclose(lse[0], 0.5 * ((q[0, :, :5] * k[0]).sum(1) + q[0, :, 5:] @ kr[0]), atol=1e-14)
    q, k, v, kr = small(1, 6)
    o, lse = mla.prefill(q, 0 * k, v, [0, 1], [0, 6], k_rope=0 * kr)
    np.testing.assert_allclose(o[0], v.mean(0), atol=1e-15)      # equal scores: the mean
    np.testing.assert_allclose(lse, np.log(6.0))


def test_mask_and_empty_rows():
    q, k, v, kr = small(5, 3)                                     # more queries than keys: two see nothing
    o, lse = mla.prefill(q, k, v, [0, 5], [0, 3], k_rope=kr)
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all()
    np.testing.assert_allclose(o[2], v[0], atol=1e-15)
    o1, _ = mla.prefill(q[4:], k, v, [0, 1], [0, 3], k_rope=kr, causal=False)
    np.testing.assert_allclose(o[4], o1[0], atol=1e-15)


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_by_differences(causal):
    q, k, v, kr = small(4, 6)
    cq, ck, dO = [0, 3, 4], [0, 4, 6], rng.standard_normal((4, 2, 3))
    loss = lambda q, k, v, kr: (mla.prefill(q, k, v, cq, ck, k_rope=kr, causal=causal)[0] * dO).sum()
    g = mla.backward(q, k, v, cq, ck, dO, k_rope=kr, causal=causal)
    args = dict(dq=q, dk=k, dv=v, dk_rope=kr)
    for name, x in args.items():
        num, eps = np.zeros(x.shape), 1e-5
        for i in np.ndindex(*x.shape):
            at = x[i]
            x[i] = at + eps
            up = loss(q, k, v, kr)
            x[i] = at - eps
            num[i] = (up - loss(q, k, v, kr)) / (2 * eps)
            x[i] = at
        # central differences: error eps^2 f''' / 6 + rounding 2^-53 |f| / eps, both under 1e-9 here
        np.testing.assert_allclose(g[name], num, atol=1e-8, err_msg=name)


def test_absorbed_equals_expanded():
    """softmax(q_nope (c W_k)^T + q_rope kr^T) (c W_v) is the absorbed form with q_nope W_k^T, times W_v."""
    L, H, dc, dn, dr, dv, page = 11, 3, 6, 4, 2, 5, 4
    c, kr = rng.standard_normal((L, dc)), rng.standard_normal((L, dr))
    wk, wv = rng.standard_normal((H, dc, dn)), rng.standard_normal((H, dc, dv))
    q = rng.standard_normal((2, H, dn + dr))                      # the last two tokens
    k, v = np.einsum("lc,hcd->lhd", c, wk), np.einsum("lc,hcd->lhd", c, wv)
    o, lse = mla.prefill(q, k, v, [0, 2], [0, L], k_rope=kr, scale=0.3)
    table = np.array([[2, 0, 3]])
    cache, _, _, _ = mla.append(c, kr, rng.standard_normal((4, page, dc + dr)), table, [0], [0, L])
    qa = np.concatenate([np.einsum("thd,hcd->thc", q[..., :dn], wk), q[..., dn:]], -1)[None]
    ol, lse2 = mla.decode(qa, cache, table, [L], dc, 0.3)
    np.testing.assert_allclose(np.einsum("thc,hcd->thd", ol[0], wv), o, atol=1e-12)
    np.testing.assert_allclose(lse2[0], lse, atol=1e-12)


def test_append_by_hand():
    c, kr = np.array([[3.0, 4.0]]), np.array([[1.0, 0.0]])
    cache, c2, k2, q2 = mla.append(c, kr, np.zeros((2, 2, 4)), np.array([[1, 0]]), [2], [0, 1],
                                   norm_weight=np.array([1.0, 2.0]), eps=0.0, inv_freq=np.array([np.pi / 4]),
                                   q_rope=np.array([[[0.0, 2.0]]]))
    r = np.sqrt(12.5)
    np.testing.assert_allclose(c2[0], [3 / r, 8 / r])
    np.testing.assert_allclose(k2[0], [0, 1], atol=1e-15)         # position 2 times pi/4: a quarter turn
    np.testing.assert_allclose(q2[0, 0], [-2, 0], atol=1e-15)
    np.testing.assert_allclose(cache[0, 0], [3 / r, 8 / r, 0, 1], atol=1e-15)   # position 2: second page of the table
    assert (cache[1] == 0).all() and (cache[0, 1] == 0).all()


def test_rotation_pairs_and_relative_position():
    x, f = rng.standard_normal((1, 6)), np.array([0.3, 0.07, 1.1])
    half, inter = mla.rotate(x, [5], f, False), mla.rotate(x, [5], f, True)
    order = [0, 3, 1, 4, 2, 5]                                    # interleaved pairs of the half-split ones
    np.testing.assert_allclose(mla.rotate(x[:, order], [5], f, True), half[:, order], atol=1e-14)
    assert not np.allclose(half, inter)
    y = rng.standard_normal((1, 6))
    for inter in (False, True):
        a = mla.rotate(x, [9], f, inter) @ mla.rotate(y, [4], f, inter).T
        b = mla.rotate(x, [105], f, inter) @ mla.rotate(y, [100], f, inter).T
        np.testing.assert_allclose(a, b, atol=1e-12)


def test_bad_pages_and_short_sequences():
    q, cache = rng.standard_normal((3, 2, 2, 6)), rng.standard_normal((2, 4, 6))
    table = np.array([[0, 7], [-1, 1], [0, 1]])
    o, lse = mla.decode(q, cache, table, [8, 8, 1], 4, 1.0)
    ok, _ = mla.decode(q[:1], cache, np.array([[0]]), [4], 4, 1.0)
    np.testing.assert_allclose(o[0, 1], ok[0, 1])                 # page 7 is left out: the first four rows remain
    assert (o[2, 0] == 0).all() and np.isneginf(lse[2, 0]).all()  # one row, two tokens: the first sees none
    np.testing.assert_allclose(o[2, 1], np.broadcast_to(cache[0, 0, :4], (2, 4)))
