"""Pins of the attention, bias and dropout oracle (no GPU): the generator's published answers, closed forms,
equivariance, and every gradient against central differences."""
import numpy as np
import pytest

from oracle import attention as oa
from oracle import so3


def test_philox_known_answers():
    # answers published with the generator: counter and key all zero, all ones, and digits of pi
    cases = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
             ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
             ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
              (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for ctr, key, want in cases:
        assert tuple(int(w) for w in oa.philox4x32(np.asarray([ctr], np.uint64), key)[0]) == want


def test_keep_factors_rate_and_scale():
    f = oa.keep_factors(np.arange(200_000), 0.3, 1234567890123, 5, 2)
    kept = (f != 0).mean()
    assert abs(kept - 0.7) < 5 * np.sqrt(0.21 / 200_000)          # five standard deviations
    t = int(np.floor(0.3 * 65536 + 0.5))
    assert np.all((f == 0) | (f == 65536.0 / (65536 - t)))
    assert np.any(f != oa.keep_factors(np.arange(200_000), 0.3, 1234567890123, 6, 2))
    assert np.any(f != oa.keep_factors(np.arange(200_000), 0.3, 1234567890123, 5, 3))
    assert np.all(oa.keep_factors(np.arange(100), 0.0, 1, 1, 1) == 1)


def _case(seed, n_dst=5, n_src=7, E=30, lmax=1, C=6, H=3, D=4):
    rng = np.random.default_rng(seed)
    K = (lmax + 1) ** 2
    cut = np.sort(rng.integers(0, E + 1, n_dst - 1))
    row_ptr = np.concatenate([[0], cut, [E]])
    return dict(row_ptr=row_ptr, src=rng.integers(0, n_src, E), q=rng.standard_normal((n_dst, H, 2, D)),
                k=rng.standard_normal((n_src, H, 2, D)), v=rng.standard_normal((n_src, K, C)),
                lam=rng.uniform(0.1, 0.9, H), scale=D ** -0.5, bias=rng.standard_normal((E, 2 * H)),
                mask=(rng.random(E) > 0.2).astype(np.uint8),
                factors=oa.keep_factors(np.arange(E * H).reshape(E, H), 0.2, seed, 1, 0))


def test_forward_against_a_dense_formula():
    c = _case(3)
    out = oa.attention_forward(**c)
    n_dst, H = len(c["row_ptr"]) - 1, len(c["lam"])
    E, Ch = len(c["src"]), c["v"].shape[2] // H
    own = np.zeros((n_dst, E), bool)
    for d in range(n_dst):
        own[d, c["row_ptr"][d]:c["row_ptr"][d + 1]] = True
    own &= c["mask"][None] != 0
    for h in range(H):
        maps = []
        for s in range(2):
            z = c["scale"] * c["q"][:, h, s] @ c["k"][c["src"], h, s].T + c["bias"][None, :, 2 * h + s]
            p = np.where(own, np.exp(z), 0.0)
            maps.append(p / np.maximum(p.sum(1, keepdims=True), 1e-300))
        w = (maps[0] - c["lam"][h] * maps[1]) * c["factors"][None, :, h]
        want = np.einsum("de,ekc->dkc", w, c["v"][c["src"]][:, :, h * Ch:(h + 1) * Ch])
        np.testing.assert_allclose(out[:, :, h * Ch:(h + 1) * Ch], want, atol=1e-12)


def test_empty_and_masked_rows_are_zero():
    c = _case(4)
    c["mask"][:] = 0
    assert np.all(oa.attention_forward(**c) == 0)
    c = _case(4)
    c["bias"][:] = -np.inf
    c["v"][:], c["k"][:] = np.nan, np.nan
    assert np.all(oa.attention_forward(**c) == 0)


def test_rotation_equivariance():
    c = _case(5, lmax=2)
    rng = np.random.default_rng(8)
    qr, _ = np.linalg.qr(rng.standard_normal((3, 3)))
    R = qr * np.sign(np.linalg.det(qr))
    Dm = np.zeros((9, 9))
    for l in range(3):
        Dm[l * l:(l + 1) ** 2, l * l:(l + 1) ** 2] = so3.wigner_d(l, R)
    rot = dict(c, v=np.einsum("ab,nbc->nac", Dm, c["v"]))
    np.testing.assert_allclose(oa.attention_forward(**rot), np.einsum("ab,nbc->nac", Dm, oa.attention_forward(**c)),
                               atol=1e-12)


@pytest.mark.parametrize("share", ["channel", "degree", "row"])
def test_dropout_commutes_with_rotations_within_a_degree(share):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((11, 9, 5))
    f = oa.dropout_factors(11, 2, 5, share, 0.4, 99, 3, 1)
    Dm = np.zeros((9, 9))
    for l in range(3):
        Dm[l * l:(l + 1) ** 2, l * l:(l + 1) ** 2] = np.linalg.qr(rng.standard_normal((2 * l + 1, 2 * l + 1)))[0]
    np.testing.assert_allclose(f * np.einsum("ab,nbc->nac", Dm, x), np.einsum("ab,nbc->nac", Dm, f * x), atol=1e-13)


@pytest.mark.parametrize("seed", [11, 12])
def test_gradients_against_differences(seed):
    c = _case(seed, n_dst=4, n_src=5, E=20, lmax=1, C=4, H=2, D=3)
    G = np.random.default_rng(seed + 100).standard_normal((4, 4, 4))
    res, _ = oa.attention_bounds(**c, grad_out=G)
    for name, key in (("grad_q", "q"), ("grad_k", "k"), ("grad_v", "v"), ("grad_lam", "lam"), ("grad_bias", "bias")):
        flat = c[key].reshape(-1)
        fd = np.zeros(flat.size)
        for i in range(flat.size):
            keep, h = flat[i], 1e-5
            flat[i] = keep + h
            up = (oa.attention_forward(**c) * G).sum()
            flat[i] = keep - h
            fd[i] = (up - (oa.attention_forward(**c) * G).sum()) / (2 * h)
            flat[i] = keep
        # central differences: h^2 of the third derivative (order 1) and 1e-16 / h of rounding
        np.testing.assert_allclose(res[name].reshape(-1), fd, atol=2e-9, err_msg=name)


def test_bias_buckets_and_gradient():
    borders = np.asarray([1.0, 2.0, 4.0], np.float32)
    dist = np.asarray([0.0, 0.999, 1.0, 2.0, 3.9, 4.0, 100.0, np.nan], np.float32)
    assert oa.buckets(dist, borders).tolist() == [0, 0, 1, 2, 2, 3, 3, 0]
    rng = np.random.default_rng(1)
    t, G = rng.standard_normal((4, 3)), rng.standard_normal((8, 3))
    g = oa.bias_backward(dist, borders, G)
    assert np.isclose((g * t).sum(), (oa.bias_forward(dist, borders, t) * G).sum())  # the adjoint
