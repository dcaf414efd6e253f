"""Calls without tokens, as an empty torch tensor gives them: its address is NULL.  CPU only, nothing is launched."""
import pytest

from joint_video_audio_rope_b200 import build as B

B.build()
from joint_video_audio_rope_b200 import mmdit as M  # noqa: E402

from test_continuation_abi import FAKE, _cache, _desc, _layout, _rc  # noqa: E402

torch = pytest.importorskip("torch")


def test_an_empty_tensor_has_no_address():
    assert torch.empty((2, 0, 4, 128), dtype=torch.bfloat16).data_ptr() == 0


def test_calls_without_tokens():
    d, none = _desc(n_tokens=0), 0
    rot = M.rotary_params(1e4, 64)
    for n in (0, 40):
        M.rotary(none, none, d, d, none, none, d, d, _layout(n), rot, stream=0)
        M.rotary(none, none, d, d, None, None, None, None, _layout(n), rot, stream=0)
        M.rotary(None, None, None, None, none, none, d, d, _layout(n), rot, stream=0)
        M.cache_append(none, none, d, _cache(), FAKE, layout=_layout(n), rotation=rot, stream=0)
    M.cache_append(none, none, d, _cache(), FAKE, stream=0)
    assert M.cache_attn_workspace_size(d, _cache()) == 0
    M.cache_attn(none, none, d, d, _cache(), FAKE, 0.1, stream=0)


def test_their_other_arguments_are_checked():
    d, none = _desc(n_tokens=0), 0
    rot = M.rotary_params(1e4, 64)
    assert _rc(M.rotary, none, none, _desc(), d, None, None, None, None, _layout(), rot) == M.EINVAL  # 40 tokens
    assert _rc(M.rotary, none, none, d, d, None, None, None, None, _layout(), M.rotary_params(1e4, 130)) == M.EINVAL
    assert _rc(M.rotary, none, FAKE, d, d, None, None, None, None, _layout(), rot) == M.EINVAL
    assert _rc(M.cache_append, none, none, d, _cache(), None) == M.EINVAL
    assert _rc(M.cache_append, none, none, d, _cache(heads=8), FAKE) == M.EINVAL
    assert _rc(M.cache_attn, none, none, d, d, _cache(), None, 0.1) == M.EINVAL
    assert _rc(M.cache_attn, none, none, d, d, _cache(), FAKE, -0.1) == M.EINVAL
