"""Rotary parameters whose frequencies leave the range of a double are refused (their angles would be NaN); CPU only."""
import pytest

from joint_video_audio_rope_b200 import build as B

B.build()
from joint_video_audio_rope_b200 import mmdit as M  # noqa: E402

from test_continuation_abi import FAKE, _cache, _desc, _layout, _rc, _rot  # noqa: E402

BAD = [  # theta, dim_t, dim_h, scaling, factors
    (1e4, 4, 60, M.SCALE_NTK, (1e-200, 1.0, 1.0)),     # theta f^2 = 0: its powers are infinite
    (1e4, 32, 32, M.SCALE_LINEAR, (1.0, 1e-300, 1.0)),  # w / f = 10^300 and a position of 10^9
    (1e-308, 64, 64, M.SCALE_NONE, (1.0, 1.0, 1.0)),   # theta^(-62/64)
]


@pytest.mark.parametrize("theta,dt,dh,scaling,factors", BAD)
def test_frequencies_out_of_range_are_refused(theta, dt, dh, scaling, factors):
    for half in (M.PAIR_INTERLEAVED, M.PAIR_HALF):
        p = M.rotary_params(theta, dt, dh, pairing=half, scaling=scaling, factors=factors)
        assert _rot(params=p) == M.EINVAL
        assert _rc(M.cache_append, 6 * FAKE, 7 * FAKE, _desc(), _cache(), FAKE, layout=_layout(), rotation=p) == M.EINVAL


@pytest.mark.parametrize("scaling", [M.SCALE_NONE, M.SCALE_LINEAR, M.SCALE_NTK, M.SCALE_PARTS])
@pytest.mark.parametrize("factor", [1e-6, 0.5, 1.0, 4.0, 1e6])
@pytest.mark.parametrize("theta", [1e-3, 1.0, 1e4, 1e12])
def test_ordinary_parameters_are_taken(scaling, factor, theta):
    p = M.rotary_params(theta, 4, 60, 64, scaling=scaling, factors=(factor,) * 3, trained=(21.0, 30.0, 52.0))
    d = _desc(n_tokens=0)  # nothing to launch: accepted before a CUDA call
    M.rotary(FAKE, 2 * FAKE, d, d, None, None, None, None, _layout(0), p, stream=0)
