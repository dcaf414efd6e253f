"""Pins of the continuation oracle (rotary positions, e4m3 codes, cache append, cache attention) by closed
forms and invariants; runs on the CPU."""
import math

import numpy as np
import pytest

import oracle as O
from oracle import continuation as OC


def _p(**kw):
    p = dict(theta=10000.0, dims=(44, 42, 42), half=False, scaling="none", factors=(1.0, 1.0, 1.0),
             trained=(0.0, 0.0, 0.0), fast=32.0, slow=1.0, magnitude=1.0)
    p.update(kw)
    return p


def _layout():
    return O.Layout([O.Segment(O.SEG_VIDEO, 24, 2, 3, 4, -1, 1, 1, O.ORDER_RASTER),
                     O.Segment(O.SEG_AUDIO, 9, 0, 0, 0, 3, 21, 218, 0)])


@pytest.mark.parametrize("half", [False, True])
def test_rotary_is_a_rotation_and_the_transpose_undoes_it(half):
    x = np.random.default_rng(0).standard_normal((2, 30, 2, 128))
    p = _p(half=half, dims=(30, 20, 14))
    y = OC.rotary(x, p, _layout(), [0, 7])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(OC.rotary(y, p, _layout(), [0, 7], transpose=True), x)
    assert np.array_equal(y[..., 64:], x[..., 64:])  # behind the bands


def test_interleaved_plain_rotation_equals_the_layer_rope():
    x = np.random.default_rng(1).standard_normal((1, 33, 2, 128))
    assert np.allclose(OC.rotary(x, _p(), _layout(), [0]), O.rope(x[0], O.positions(_layout()))[None])


def test_scalings():
    base = [w for *_, w in OC.frequencies(_p(dims=(64, 0, 0)))]
    lin = [w for *_, w in OC.frequencies(_p(dims=(64, 0, 0), scaling="linear", factors=(4.0, 1, 1)))]
    assert np.allclose(lin, np.array(base) / 4)
    ntk = [w for *_, w in OC.frequencies(_p(dims=(64, 0, 0), scaling="ntk", factors=(4.0, 1, 1)))]
    assert math.isclose(ntk[0], base[0]) and math.isclose(ntk[-1], base[-1] / 4)
    parts = [w for *_, w in OC.frequencies(_p(dims=(64, 0, 0), scaling="parts", factors=(4.0, 1, 1), trained=(600.0, 1, 1)))]
    assert math.isclose(parts[0], base[0]) and math.isclose(parts[-1], base[-1] / 4)
    assert all(b / 4 <= w <= b for w, b in zip(parts, base))


def test_e4m3_values_and_rounding():
    t = OC.E4M3
    assert t[0x7e] == 448.0 and t[0x01] == 2.0 ** -9 and t[0x38] == 1.0 and math.isnan(t[0xff])
    codes = np.array([c for c in range(256) if not math.isnan(t[c])], np.uint8)
    assert np.array_equal(OC.to_e4m3(t[codes])[t[codes] != 0], codes[t[codes] != 0])
    assert t[OC.to_e4m3(np.array([17.0, 19.0, 1e9, 2.0 ** -10, 3 * 2.0 ** -10]))].tolist() == \
        [16.0, 20.0, 448.0, 0.0, 2 * 2.0 ** -9]  # ties to the even mantissa
    x = np.random.default_rng(2).uniform(-448, 448, 4000)
    assert np.all(np.abs(t[OC.to_e4m3(x)] - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10))


def test_fit_scale():
    assert OC.fit_scale(448.0) == 1.0 and OC.fit_scale(448.1) == 2.0 and OC.fit_scale(224.0) == 0.5
    assert OC.fit_scale(0.0) == 2.0 ** -60


def test_append_grows_the_scale_of_a_shared_page_only_when_needed():
    codes, scales = np.zeros((2, 1, 16, 4), np.uint8), np.zeros((2, 1))
    table = np.array([[1, 0]])
    x = np.full((1, 20, 1, 4), 1.0)
    OC.append(codes, scales, table, x[:, :5], [0], [5], None)
    before = scales[1, 0]
    OC.append(codes, scales, table, 300 * x[:, :3], [5], [3], None)
    assert before == 2.0 ** -8 and scales[1, 0] == 1.0
    assert np.all(OC.E4M3[codes[1, 0, :5]] == 1.0) and np.all(OC.E4M3[codes[1, 0, 5:8]] == 288.0)  # 256 + 32 k
    OC.append(codes, scales, table, x[:, :12], [8], [12], None)
    assert scales[1, 0] == 1.0 and scales[0, 0] == before and np.all(codes[1, 0, 8:] == 0x38)
    assert np.all(codes[0, 0, 4:] == 0)


def test_cache_attention_weights():
    rng = np.random.default_rng(3)
    kc = OC.to_e4m3(rng.standard_normal((3, 1, 16, 8)) * 50)
    vc = np.full((3, 1, 16, 8), 0x38, np.uint8)
    ks, vs = np.full((3, 1), 0.02), np.full((3, 1), 3.0)
    q = rng.standard_normal((1, 4, 2, 8))
    o, lse, S, _ = OC.cache_attn(q, kc, vc, ks, vs, np.array([[2, 0, 1]]), [37], [4], 1, 0.3)
    assert np.allclose(o, 3.0) and np.allclose(S, 3.0)
    K = (OC.E4M3[kc] * 0.02)[[2, 0, 1], 0].reshape(-1, 8)
    assert np.isclose(lse[0, 1, 2], np.log(np.exp(K[:36] @ q[0, 2, 1] * 0.3).sum()))
    o, lse, *_ = OC.cache_attn(q, kc, vc, ks, vs, np.array([[2, 0, 1]]), [2], [4], 1, 0.3)
    assert np.all(o[0, :2] == 0) and np.all(lse[0, :, :2] == -np.inf) and np.allclose(o[0, 2:], 3.0)
