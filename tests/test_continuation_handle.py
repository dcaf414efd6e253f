"""The cache handle of the binding; CPU only."""
import pytest

from joint_video_audio_rope_b200 import build as B

B.build()
from joint_video_audio_rope_b200 import mmdit as M  # noqa: E402

torch = pytest.importorskip("torch")


def _arrays(dtype=torch.uint8):
    k, v = (torch.zeros((3, 2, 16, 64), dtype=torch.uint8).view(dtype) for _ in range(2))
    return k, v, torch.zeros((3, 2)), torch.zeros((3, 2)), torch.zeros((1, 3), dtype=torch.int32)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn])
def test_codes_are_e4m3_or_raw_bytes(dtype):
    x = _arrays(dtype)
    c = M.make_cache(*x)
    assert (c.k, c.v, c.n_pages) == (x[0].data_ptr(), x[1].data_ptr(), 3)


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int8, torch.bool])
def test_other_types_of_eight_bits_are_refused(dtype):
    good, bad = _arrays(), _arrays(dtype)
    for pair in ((bad[0], bad[1]), (good[0], bad[1]), (bad[0], good[1])):
        with pytest.raises(ValueError):
            M.make_cache(*pair, *good[2:])


def test_a_handle_keeps_its_tensors_alive():
    """A temporary (a clone, a .contiguous()) handed to make_cache would otherwise be freed, and its memory used for
    something else, while the handle still holds the address."""
    import gc
    import weakref
    x = _arrays()
    refs = [weakref.ref(t) for t in x]
    c = M.make_cache(*x)
    del x
    gc.collect()
    assert all(r() is not None for r in refs)
    del c
    gc.collect()
    assert all(r() is None for r in refs)
