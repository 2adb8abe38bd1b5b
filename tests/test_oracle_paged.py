"""Pins of the fp64 definitions of the paged 8-bit cache."""
import numpy as np
import torch

from oracle import paged as O


def test_e4m3_values_and_rounding():
    t = O.e4m3_table()
    torch_t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(t, nan=1e9), np.nan_to_num(torch_t, nan=1e9))
    x = np.concatenate([np.linspace(-460, 460, 4001), np.linspace(-0.05, 0.05, 4001)])
    want = torch.tensor(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.to_e4m3(x.astype(np.float32)), want)
    assert np.isnan(O.to_e4m3([np.inf, -np.inf, np.nan])).all()


def test_scale_is_the_least_power_of_two():
    for a in (1e-12, 0.1, 1.75, 448.0, 449.0, 449.1, 1e5, 1e20):
        s = O.scale_of(a)
        assert s == 2.0 ** 32 or a <= 449 * s
        assert s == 2.0 ** -32 or a > 449 * s / 2
    assert O.scale_of(0.0) == 2.0 ** -32


def test_rotation_keeps_distances_and_composes():
    rng = np.random.default_rng(1)
    x, y = rng.normal(size=(2, 4, 3, 16))
    f = 10.0 ** -np.arange(6)
    for inter in (False, True):
        a, b = (O.rotate(z, [np.array([5, 5, 9, 9])] * 2, f, [2, 4], inter) for z in (x, y))
        assert np.allclose((a * b).sum(-1), (x * y).sum(-1))
        assert np.array_equal(a[..., 12:], x[..., 12:])
        twice = O.rotate(O.rotate(x, [np.full(4, 3)], f, [6], inter), [np.full(4, 4)], f, [6], inter)
        assert np.allclose(twice, O.rotate(x, [np.full(4, 7)], f, [6], inter))


def test_attention_of_one_token_and_of_equal_keys():
    page, d = 16, 8
    cache = np.zeros((3, 1, page, d))
    v = np.arange(3 * page * d).reshape(3, 1, page, d).astype(float)
    one = np.ones((3, 1))
    o, lse = O.attention(np.ones((2, 2, d)), [0, 1, 2], [1, 20], np.array([[2, 0], [0, 1]]), cache, v, one, 2 * one)
    assert np.array_equal(o[0, 0], 2 * v[2, 0, 0]) and lse[0, 0] == 0.0
    seen = np.concatenate([v[0, 0], v[1, 0, :4]])
    assert np.allclose(o[1, 1], 2 * seen.mean(0)) and np.allclose(lse[1], np.log(20))
    o, lse = O.attention(np.ones((3, 1, d)), [0, 3], [1], np.array([[0]]), cache, v, one, one)
    assert not o[:2].any() and np.isneginf(lse[:2]).all() and np.array_equal(o[2, 0], v[0, 0, 0])


def test_append_grows_a_page_scale_and_rounds_the_older_bytes():
    cache, scale = np.zeros((2, 1, 16, 4)), np.full((2, 1), 64.0)
    O.append(np.full((3, 1, 4), 0.3), [0, 3], [3], np.array([[1]]), cache, scale)
    s = scale[1, 0]
    assert s == O.scale_of(0.3) and np.abs(cache[1, 0, :3] * s - 0.3).max() <= 0.3 * 2.0 ** -4
    O.append(np.full((1, 1, 4), 300.0), [0, 1], [4], np.array([[1]]), cache, scale)
    assert scale[1, 0] == 1.0 and np.array_equal(cache[1, 0, :3], np.full((3, 4), O.to_e4m3(O.to_e4m3(0.3 / s) * s)))
    assert np.array_equal(cache[1, 0, 3], np.full(4, O.to_e4m3(300.0))) and scale[0, 0] == 64.0
