"""Refusals of the continuation calls; every check is made before a CUDA call, so this runs on the CPU."""
import pytest

from joint_video_audio_rope_b200 import build as B

B.build()
from joint_video_audio_rope_b200 import mmdit as M  # noqa: E402

FAKE = 0x10000  # 16-byte aligned, never dereferenced


def _desc(**kw):
    d = dict(batch=2, n_tokens=40, heads=4, head_dim=128, dtype=M.BF16)
    d.update(kw)
    return M.make_desc(**d)


def _layout(n=40):
    return M.make_layout([dict(kind=M.SEG_AUDIO, n_tokens=n, t_num=21, t_den=218)])


def _cache(**kw):
    d = dict(k=FAKE, v=2 * FAKE, k_scale=3 * FAKE, v_scale=4 * FAKE, n_pages=10, heads=4, page_tokens=16,
             head_dim=128, page_table=5 * FAKE, batch=2, max_pages=5)
    d.update(kw)
    return M.Cache(*[d[f] for f, _ in M.Cache._fields_])


def _rc(fn, *args, **kw):
    with pytest.raises(M.MmditError) as e:
        fn(*args, **kw, stream=0)
    return e.value.status


def _rot(q=FAKE, q_out=2 * FAKE, qd=None, qod=None, k=3 * FAKE, k_out=4 * FAKE, kd=None, kod=None, layout=None,
         params=None, **kw):
    return _rc(M.rotary, q, q_out, qd or _desc(), qod or _desc(), k, k_out, kd or _desc(), kod or _desc(),
               layout or _layout(), params or M.rotary_params(1e4, 44, 42, 42), **kw)


def test_rotary_refusals():
    assert _rc(M.rotary, None, None, None, None, None, None, None, None, _layout(), M.rotary_params(1e4, 128)) == M.EINVAL
    assert _rot(q_out=None) == M.EINVAL
    assert _rot(q=None) == M.EINVAL                        # an output without an input
    assert _rot(q=FAKE + 8) == M.EINVAL
    assert _rot(q_out=4 * FAKE) == M.EINVAL                # both outputs the same
    assert _rot(q_out=3 * FAKE) == M.EINVAL                # q_out over k
    assert _rot(q_out=FAKE, qod=_desc(stride_tok=1024, stride_batch=40 * 1024)) == M.EINVAL  # in place, other strides
    assert _rot(qd=_desc(head_dim=96), qod=_desc(head_dim=96)) == M.EUNSUPPORTED
    assert _rot(qd=_desc(dtype=5)) == M.EUNSUPPORTED
    assert _rot(qod=_desc(heads=8)) == M.EINVAL
    assert _rot(kd=_desc(n_tokens=41), kod=_desc(n_tokens=41)) == M.EINVAL
    assert _rot(kd=_desc(dtype=M.F32), kod=_desc(dtype=M.F32)) == M.EINVAL
    assert _rot(qd=_desc(stride_tok=500)) == M.EINVAL
    assert _rot(qd=_desc(stride_batch=512)) == M.EINVAL
    assert _rot(qd=_desc(batch=70000)) == M.EINVAL
    assert _rot(layout=_layout(39)) == M.EINVAL            # too short without first
    for bad in (dict(dim_t=43), dict(dim_t=130), dict(dim_t=0), dict(dim_t=-2, dim_h=66)):
        assert _rot(params=M.rotary_params(1e4, **bad)) == M.EINVAL
    for theta in (0.0, -1.0, float("nan"), float("inf")):
        assert _rot(params=M.rotary_params(theta, 128)) == M.EINVAL
    for bad in (dict(pairing=2), dict(scaling=4), dict(magnitude=0.0), dict(magnitude=float("nan")),
                dict(scaling=M.SCALE_LINEAR, factors=(0.0, 1, 1)), dict(scaling=M.SCALE_NTK, factors=(float("inf"), 1, 1)),
                dict(scaling=M.SCALE_PARTS, factors=(2.0, 1, 1)),
                dict(scaling=M.SCALE_PARTS, factors=(2.0, 1, 1), trained=(21.0, 1, 1), beta_fast=1.0, beta_slow=1.0)):
        assert _rot(params=M.rotary_params(1e4, 128, **bad)) == M.EINVAL
    f = M.raw("mmdit_rotary")
    d = _desc()
    assert f(FAKE, 2 * FAKE, d, d, None, None, None, None, _layout(), M.rotary_params(1e4, 128), None, 2, None) == M.EINVAL
    assert f(FAKE, 2 * FAKE, None, d, None, None, None, None, _layout(), M.rotary_params(1e4, 128), None, 0, None) == M.EINVAL


BAD_CACHES = [(dict(k=None), M.EINVAL), (dict(v_scale=None), M.EINVAL), (dict(k=FAKE + 4), M.EINVAL),
              (dict(k_scale=FAKE + 2), M.EINVAL), (dict(v=FAKE), M.EINVAL), (dict(n_pages=0), M.EINVAL),
              (dict(heads=0), M.EINVAL), (dict(page_tokens=24), M.EUNSUPPORTED), (dict(head_dim=96), M.EUNSUPPORTED),
              (dict(page_table=None), M.EINVAL), (dict(max_pages=0), M.EINVAL), (dict(max_pages=1 << 28), M.EINVAL),
              (dict(batch=0), M.EINVAL), (dict(batch=3), M.EINVAL), (dict(page_table=FAKE + 2), M.EINVAL)]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(change, status):
    c = _cache(**change)
    assert _rc(M.cache_append, 6 * FAKE, 7 * FAKE, _desc(), c, FAKE) == status
    assert _rc(M.cache_attn, 6 * FAKE, 7 * FAKE, _desc(), _desc(), c, FAKE, 0.1) == status
    assert M.cache_attn_workspace_size(_desc(), c) == 0


def test_append_refusals():
    f = lambda k=6 * FAKE, v=7 * FAKE, d=None, c=None, s=FAKE, **kw: _rc(M.cache_append, k, v, d or _desc(), c or _cache(), s, **kw)
    assert f(k=None) == M.EINVAL
    assert f(s=None) == M.EINVAL
    assert f(v=7 * FAKE + 8) == M.EINVAL
    assert f(d=_desc(heads=8)) == M.EINVAL
    assert f(d=_desc(head_dim=64)) == M.EINVAL
    assert f(d=_desc(dtype=9)) == M.EUNSUPPORTED
    assert f(layout=_layout()) == M.EINVAL                   # without a rotation
    assert f(rotation=M.rotary_params(1e4, 128)) == M.EINVAL  # without a layout
    assert f(layout=_layout(), rotation=M.rotary_params(1e4, 130)) == M.EINVAL


def test_attention_refusals_and_workspace():
    f = lambda q=6 * FAKE, o=7 * FAKE, d=None, od=None, c=None, kv=FAKE, scale=0.1, **kw: _rc(
        M.cache_attn, q, o, d or _desc(), od or d or _desc(), c or _cache(), kv, scale, **kw)
    assert f(q=None) == M.EINVAL
    assert f(kv=None) == M.EINVAL
    assert f(o=6 * FAKE) == M.EINVAL
    assert f(o=7 * FAKE + 8) == M.EINVAL
    assert f(scale=0.0) == M.EINVAL
    assert f(scale=float("nan")) == M.EINVAL
    assert f(causal_block=-1) == M.EINVAL
    assert f(d=_desc(heads=6)) == M.EINVAL                   # no multiple of the cache's heads
    assert f(od=_desc(n_tokens=41)) == M.EINVAL
    assert f(od=_desc(dtype=M.F32)) == M.EINVAL
    long = _cache(max_pages=4000)
    one = _desc(n_tokens=1)
    n = M.cache_attn_workspace_size(one, long)
    assert n > 0 and n % 256 == 0
    assert f(d=one, c=long) == M.EWORKSPACE
    assert f(d=one, c=long, workspace=FAKE, ws_bytes=n - 1) == M.EWORKSPACE
    assert f(d=one, c=long, workspace=FAKE + 16, ws_bytes=n) == M.EINVAL


def test_copy_refusals():
    f = lambda c, s, d: _rc(M.cache_copy_pages, c, s, d)
    c = _cache(page_table=None, batch=0, max_pages=0)
    assert f(c, [0], [10]) == M.EINVAL
    assert f(c, [-1], [1]) == M.EINVAL
    assert f(c, [0, 1], [2, 2]) == M.EINVAL      # written twice
    assert f(c, [0, 1], [1, 2]) == M.EINVAL      # read and written
    assert f(c, [3], [3]) == M.EINVAL
    assert f(_cache(k=None), [0], [1]) == M.EINVAL
    assert M.raw("mmdit_cache_copy_pages")(c, -1, None, None, None) == M.EINVAL
    assert M.raw("mmdit_cache_copy_pages")(c, 1, None, None, None) == M.EINVAL
    assert M.raw("mmdit_cache_copy_pages")(c, 0, None, None, None) == M.OK
    with pytest.raises(ValueError):
        M.cache_copy_pages(c, [1, 2], [3], stream=0)


def test_make_cache_checks_its_tensors():
    torch = pytest.importorskip("torch")
    k = torch.zeros((3, 2, 16, 64), dtype=torch.uint8)
    s = torch.zeros((3, 2))
    t = torch.zeros((1, 3), dtype=torch.int32)
    c = M.make_cache(k, k.clone(), s, s.clone(), t)
    assert (c.n_pages, c.heads, c.page_tokens, c.head_dim, c.batch, c.max_pages) == (3, 2, 16, 64, 1, 3)
    for bad in ((k[:2], k, s, s, t), (k.float(), k, s, s, t), (k, k, s.double(), s, t), (k, k, s, s, t.long()),
                (k.transpose(1, 2), k.transpose(1, 2), s, s, t)):
        with pytest.raises(ValueError):
            M.make_cache(*bad)


def test_tensors_elsewhere_and_arrays_of_another_shape_are_refused():
    torch = pytest.importorskip("torch")
    d, c = _desc(), _cache()
    i32 = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 40, 4, 128), dtype=torch.bfloat16)
    for call in (lambda: M.cache_append(x, 7 * FAKE, d, c, FAKE, stream=0),
                 lambda: M.cache_append(6 * FAKE, 7 * FAKE, d, c, i32, stream=0),
                 lambda: M.cache_append(6 * FAKE, 7 * FAKE, d, c, i32.long(), stream=0),
                 lambda: M.cache_append(6 * FAKE, 7 * FAKE, d, c, FAKE, count=i32[:1], stream=0),
                 lambda: M.cache_attn(6 * FAKE, 7 * FAKE, d, d, c, i32, 0.1, stream=0),
                 lambda: M.cache_attn(6 * FAKE, 7 * FAKE, d, d, c, FAKE, 0.1, lse=torch.zeros((2, 4, 39)), stream=0),
                 lambda: M.cache_attn(x, 7 * FAKE, d, d, c, FAKE, 0.1, stream=0),
                 lambda: M.rotary(x, FAKE, d, d, None, None, None, None, _layout(), M.rotary_params(1e4, 64), stream=0),
                 lambda: M.rotary(FAKE, 2 * FAKE, d, d, None, None, None, None, _layout(), M.rotary_params(1e4, 64),
                                  first=i32.repeat(2), stream=0)):
        with pytest.raises(ValueError):
            call()
    k = torch.zeros((3, 2, 16, 64), dtype=torch.uint8)
    host = M.make_cache(k, k.clone(), torch.zeros((3, 2)), torch.zeros((3, 2)))
    with pytest.raises(ValueError):
        M.cache_copy_pages(host, [0], [1], stream=0)
