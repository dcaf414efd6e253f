"""The host's plan of attention over the cache at sizes that no machine holds; CPU only (every check is made before a CUDA
call)."""
import pytest

from joint_video_audio_rope_b200 import build as B

B.build()
from joint_video_audio_rope_b200 import mmdit as M  # noqa: E402

from test_continuation_abi import FAKE, _cache, _rc  # noqa: E402


@pytest.mark.parametrize("dtype,rows,parts", [(M.BF16, 300, 16), (M.BF16, 1, 4), (M.F32, 1, 1)])
def test_long_histories_are_split_for_the_running_sums(dtype, rows, parts):
    """More items than any split for the GPU's sake would need: a bf16 range is 2^17 tokens at most, of each warp where the
    rows are few; fp32 calls need none."""
    tile = 256 if rows > 32 else 8
    for tokens, n in ((2 ** 21, parts), (2 ** 17, 1)):
        c = _cache(heads=8, batch=148, max_pages=tokens // 128, page_tokens=128)
        d = M.make_desc(148, rows, 8, 128, dtype)
        items = -(-rows // tile) * 8 * 148
        size = M.cache_attn_workspace_size(d, c)
        assert size == (items * n * tile * (128 + 2) * 4 if n > 1 else 0)


def test_calls_beyond_the_grid_are_refused():
    c = _cache(heads=1, batch=65535, max_pages=(2 ** 31 - 2 ** 21) // 128, page_tokens=128)
    d = M.make_desc(65535, 2000, 1, 128, M.BF16)
    assert M.cache_attn_workspace_size(d, c) == 0
    assert _rc(M.cache_attn, 6 * FAKE, 7 * FAKE, d, d, c, FAKE, 0.1) == M.EINVAL


@pytest.mark.parametrize("scale", [3e38, float("inf"), -1.0, float("nan"), 0.0])
def test_scales_that_overflow_are_refused(scale):
    d = M.make_desc(2, 40, 4, 128, M.BF16)
    assert _rc(M.cache_attn, 6 * FAKE, 7 * FAKE, d, d, _cache(), FAKE, scale, workspace=FAKE * 16, ws_bytes=1 << 40) == M.EINVAL
