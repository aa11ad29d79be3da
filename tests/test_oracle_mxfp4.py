"""Pins of the MXFP4 and routing oracles against something other than themselves."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import mxfp4, route


def test_code_values():
    assert mxfp4.VALUES.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]


def test_encode_borders_and_ties():
    # (value, magnitude expected): the midpoints go to the even code
    for v, want in [(.25, 0), (.75, 1), (1.25, 1), (1.75, 2), (2.5, 2), (3.5, 4), (5, 4),
                    (np.nextafter(.25, 1), .5), (np.nextafter(.75, 0), .5),
                    (np.nextafter(1.25, 2), 1.5), (np.nextafter(1.75, 0), 1.5),
                    (np.nextafter(2.5, 3), 3), (np.nextafter(3.5, 0), 3),
                    (np.nextafter(5, 6), 6), (6, 6), (100, 6)]:
        assert mxfp4.VALUES[mxfp4.encode_rne(np.array([v]))][0] == want, v
        assert mxfp4.VALUES[mxfp4.encode_rne(np.array([-v]))][0] == -want, v
    assert mxfp4.encode_rne(np.array([-0.0, -0.1])).tolist() == [8, 8]


def test_scale_is_the_smallest_that_does_not_saturate():
    rng = np.random.default_rng(0)
    for a in list(np.exp(rng.normal(0, 20, 200)).astype(np.float32)) + \
            [6.0, np.nextafter(np.float32(6), np.float32(7)), 3.0, 1e-45, 2.0 ** -126, 3.4e38]:
        e = int(mxfp4.scale_exponent(np.array([a]))[0])
        f = Fraction(float(a))
        assert 6 * Fraction(2) ** e >= f
        assert e == -127 or 6 * Fraction(2) ** (e - 1) < f
    assert mxfp4.scale_exponent(np.array([0.0]))[0] == -127


def test_quantize_special_groups():
    x = np.zeros((1, 128), np.float32)
    x[0, 32:64] = np.linspace(-3, 3, 32)
    x[0, 70] = np.inf
    x[0, 100] = np.nan
    codes, byte = mxfp4.quantize(x)
    assert byte.tolist() == [[0, 126, 255, 255]]
    assert not codes[0, 64:].any() and not codes[0, :32].any()
    v = mxfp4.values(codes, byte)
    assert np.isnan(v[0, 64:]).all() and np.isfinite(v[0, :64]).all()
    assert np.abs(v[0, 32:64] - x[0, 32:64]).max() <= 0.5  # half the widest code step


def test_scale_words_by_hand():
    byte = np.arange(130 * 5, dtype=np.int64).reshape(130, 5).astype(np.uint8)
    w = mxfp4.scale_words(byte).view(np.uint32)
    assert w.shape == (2, 2, 32, 4)
    # row 37 = 32 * 1 + 5, groups 0..3
    assert w[0, 0, 5, 1] == sum(int(byte[37, g]) << (8 * g) for g in range(4))
    assert w[1, 1, 1, 0] == byte[129, 4] and w[1, 1, 2, 0] == 0


def test_pack_round_trip():
    codes = np.random.default_rng(1).integers(0, 16, (3, 64)).astype(np.uint8)
    assert (mxfp4.unpack(mxfp4.pack(codes)) == codes).all()
    assert mxfp4.pack(np.array([[1, 2]], np.uint8))[0, 0] == 0x21


@pytest.mark.parametrize("normalize", [True, False])
def test_route_against_torch_and_differences(normalize):
    rng = np.random.default_rng(2)
    t, e, k = 9, 7, 3
    x = rng.normal(size=(t, e))
    x[2, 3:] = -np.inf          # three open experts
    x[4, 1:] = -np.inf          # one
    x[5] = -np.inf              # none
    mask = np.ones(t, bool)
    mask[7] = False
    dw, dl = rng.normal(size=(t, k)), 0.7
    idx, w, counts, loss, n, p = route.route(x, k, normalize, mask)
    assert n == 7 and (idx[5] == -1).all() and (idx[7] == -1).all()
    assert idx[4].tolist() == [0, -1, -1] and counts.sum() == 5 * 3 + 3 + 1

    def value(y):
        """sum(dw * weights) + dl * loss with the choices and counts held."""
        xt = torch.tensor(y, requires_grad=True)
        live = torch.tensor((idx[:, 0] >= 0))
        q = torch.where(live[:, None], torch.softmax(torch.where(live[:, None], xt, 0.), 1), 0.)
        sel = torch.tensor(np.maximum(idx, 0))
        ww = q.gather(1, sel) * torch.tensor(idx >= 0)
        if normalize:
            ww = ww / torch.where(live, ww.sum(1), 1.)[:, None]
        ls = e / (k * n * n) * (torch.tensor(counts, dtype=torch.float64) * q.sum(0)).sum()
        return (torch.tensor(dw) * ww).sum() + dl * ls, xt, ww, ls

    v, xt, ww, ls = value(x)
    assert np.allclose(ww.detach().numpy(), w, atol=1e-14)
    assert math.isclose(float(ls.detach()), loss, rel_tol=1e-13)
    got = route.route_backward(p, idx, w, counts, n, dw, dl, normalize)
    (auto,) = torch.autograd.grad(v, xt)
    live = np.isfinite(x)
    assert np.allclose(got[live], np.nan_to_num(auto.numpy())[live], atol=1e-12)
    assert not got[~live].any()
    h = 1e-5
    for i, j in [(0, int(idx[0, 0])), (0, 6), (2, 1), (4, 0), (8, int(idx[8, 2]))]:
        up, dn = x.copy(), x.copy()
        up[i, j] += h
        dn[i, j] -= h
        num = (float(value(up)[0].detach()) - float(value(dn)[0].detach())) / (2 * h)
        assert abs(num - got[i, j]) < 1e-8


def test_ties_go_to_the_lowest_expert():
    idx, *_ = route.route(np.array([[1.0, 2.0, 2.0, -0.0, 0.0, 2.0]]), 6)
    assert idx[0].tolist() == [1, 2, 5, 0, 3, 4]
