"""CPU: the decoder operators' oracle pinned by differences, closed forms and brute force."""
import numpy as np
import pytest
import torch

import oracle.decoder as dec
from camera_bev_view_amd import ops


def test_rms_norm_gradients_by_differences():
    rng = np.random.default_rng(1)
    h, w, gy, gh = rng.normal(size=(5, 7)), rng.normal(size=7), rng.normal(size=(5, 7)), rng.normal(size=(5, 7))
    ref = dec.rms_norm(h, w, 1e-3, gy, gh)
    loss = lambda a, b: (dec.rms_norm(a, b, 1e-3)["y"] * gy).sum() + (a * gh).sum()
    e = 1e-6
    for i in range(5):
        for c in range(7):
            d = np.zeros_like(h)
            d[i, c] = e
            assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * e) - ref["gx"][i, c]) < 1e-8
    for c in range(7):
        d = np.zeros(7)
        d[c] = e
        assert abs((loss(h, w + d) - loss(h, w - d)) / (2 * e) - ref["gw"][c]) < 1e-8


def test_rms_norm_closed_form():
    h = np.full((2, 4), 3.0)
    assert np.allclose(dec.rms_norm(h, None, 0.0)["y"], 1.0, atol=1e-15)
    assert np.allclose(dec.rms_norm(h, None, 16.0)["rstd"], 0.2, atol=1e-15)
    # a gradient along h changes its length alone, which the norm takes away
    assert np.allclose(dec.rms_norm(h, None, 0.0, h)["gx"], 0.0, atol=1e-15)


def test_e4m3_numbers_are_torchs():
    b = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(dec.numbers("e4m3"), b.astype(np.float64))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_codes_are_the_nearest_numbers(kind):
    rng = np.random.default_rng(2)
    n = dec.numbers(kind)
    some = n[np.isfinite(n) & (np.abs(n) <= dec.MOST[kind])]
    x = rng.normal(size=4000) * rng.choice([1.0, 30.0, 200.0], size=4000)
    got = n[dec.codes(x, np.float32(1), kind)]
    best = np.abs(some[None] - np.clip(x, -dec.MOST[kind], dec.MOST[kind])[:, None]).min(axis=1)
    np.testing.assert_array_equal(np.abs(got - np.clip(x, -dec.MOST[kind], dec.MOST[kind])), best)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_ties_go_to_the_even_number(kind):
    up = dec.numbers(kind)[:127]
    mid = (up[:-1] + up[1:]) / 2
    got = dec.codes(mid, np.float32(1), kind)
    want = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(126) + 1)
    np.testing.assert_array_equal(got, want)
    back = dec.numbers(kind)[dec.codes(-mid, np.float32(1), kind)]
    np.testing.assert_array_equal(back, -up[want])


def test_row_scales():
    x = np.zeros((5, 8), np.float32)
    x[1, 3] = -254.0
    x[2, 0] = 1e-45
    x[3, 7] = np.inf
    x[4, 1] = np.nan
    c, s = dec.row_codes(x, "int8")
    assert s[0] == s[2] == np.float32(2.0 ** -126) and s[1] == 2.0 and np.isnan(s[3]) and np.isnan(s[4])
    assert dec.numbers("int8")[c[1, 3]] == -127 and not c[[0, 2, 3, 4]].any()


def test_cache_round_trip_and_drops():
    rng = np.random.default_rng(3)
    cache = dec.Cache(4, 2, 20, "int8")
    table = np.array([[2, 9], [0, 1]])
    k, v = rng.normal(size=(2, 70, 2, 20)).astype(np.float32), rng.normal(size=(2, 70, 2, 20)).astype(np.float32)
    cache.write(k, v, table, [30, 62], [70, 5])
    rk, rv = cache.read(table, [30, 62], 70, [70, 5])
    # sequence 0 has 34 tokens on page 2, then a page that does not exist; sequence 1 has two tokens on page 0, three on 1
    assert np.abs(rk[0, :34] - k[0, :34]).max() <= np.abs(k).max() / 254 * 1.001 and not rk[0, 34:].any()
    assert np.abs(rv[1, :5] - v[1, :5]).max() <= np.abs(v).max() / 254 * 1.001 and not rv[1, 5:].any()
    assert (cache.k_scale[0, 0] != 0).sum() == 2 and (cache.k_scale[1, 0] != 0).sum() == 3
    assert not cache.k_scale[3].any()


def test_attention_closed_forms():
    rng = np.random.default_rng(4)
    cache = dec.Cache(3, 1, 16, "e4m3")
    table = np.array([[1, 0]])
    k, v = rng.normal(size=(1, 100, 1, 16)).astype(np.float32), rng.normal(size=(1, 100, 1, 16)).astype(np.float32)
    cache.write(k, v, table, [0])
    _, vals = cache.read(table, [0], 100)
    q = np.zeros((1, 3, 2, 16))
    # no scores: the mean of what a query sees
    res = dec.attention(q, cache, table, [97], "chain")
    for t in range(3):
        assert np.allclose(res["out"][0, t, 0], vals[0, :98 + t, 0].mean(axis=0), atol=1e-14)
    res = dec.attention(q, cache, table, [97], "none")
    assert np.allclose(res["out"][0, 2, 1], vals[0, :97, 0].mean(axis=0), atol=1e-14)
    bits = np.zeros((1, 3, 3), bool)
    bits[0, 2, [0, 2]] = True
    res = dec.attention(q, cache, table, [97], "tree", bits=bits)
    assert np.allclose(res["out"][0, 2, 0], vals[0, list(range(97)) + [97, 99], 0].mean(axis=0), atol=1e-14)
    assert not dec.attention(q, cache, table, [-1], "chain")["out"].any()


def test_tree_ancestors():
    a = ops.tree_ancestors([-1, 0, 0, 2, -1], device="cpu")
    assert a.shape == (1, 5, 1) and a[0, :, 0].tolist() == [0b1, 0b11, 0b101, 0b1101, 0b10000]
    chain = ops.tree_ancestors([list(range(-1, 129))] * 2, device="cpu")
    assert chain.shape == (2, 130, 3)
    assert chain[1, 129].tolist() == [-1, -1, 3] and chain[0, 63].tolist() == [-1, 0, 0]
    assert chain[0, 62].tolist() == [(1 << 63) - 1, 0, 0]
    for bad in ([0], [-1, 1], [-1, -2], [[-1], [-1, 0]]):
        with pytest.raises(ValueError):
            ops.tree_ancestors(bad, device="cpu")
    assert ops.tree_ancestors(torch.tensor([[-1, 0]]), device="cpu")[0, 1].tolist() == [3]
