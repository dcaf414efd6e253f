"""Rotary positions, the paged 8-bit cache and attention over it against the fp64 oracle.

Tolerances (u = half a step of the output type relative to the value: bf16 2^-8, f32 2^-24):
* rotary, |err| <= u |y| + 2^-21 M (|x1| + |x2|): the angle, at most 1 half turn, is rounded once (2^-25 pi), sincospi is
  good to 2 ulp (2^-23), the magnitude and the products round three more times (3 2^-24): 4.0e-7 < 2^-21 together.
* append without rotation: equal codes and scales (dividing by a power of two is exact).  With it, a value next to a
  rounding border may take either neighbour: half an e4m3 step, 2^-4 |y| or 2^-10 of the scale below 2^-6, plus the rotary's error.
* attention, |err| <= u |o| + w S with S = sum p |v| of the row and channel: the fp16 probabilities round by 2^-11 (fp32 calls:
  two parts, 2^-22), scores of D / 16 truncated fp32 steps err by at most D / 16 2^-22 A (A: their largest sum of |terms|) and
  2^-22 (|t|) <= 2^-22 A in the exponent, ex2 by 2^-22; numerator and denominator both carry them: factor 2; the running sums
  over n keys add n / 16 truncated steps, 2^-23 each.
  lse: ln 2 times the exponent's error, 2^-22 |lse|, and the sum's."""
import math

import numpy as np
import pytest

import oracle as O
from oracle import continuation as OC

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def M():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from joint_video_audio_rope_b200 import build
    build.build()
    from joint_video_audio_rope_b200 import mmdit
    return mmdit


DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _tensor(rng, shape, dtype, pad_tok=0, pad_batch=0, fill=None):
    """A [B, N, H, D] view with room between its tokens and batch items, and the storage around it."""
    b, n, h, d = shape
    st = h * d + pad_tok
    sb = st * n + pad_batch
    flat = torch.full((b * sb + 64,), 3.0, dtype=DT[dtype], device="cuda")
    view = flat.as_strided((b, n, h, d), (sb, st, d, 1))
    if fill is None:
        fill = rng.standard_normal(shape)
    view.copy_(torch.from_numpy(np.asarray(fill, np.float32)).to(DT[dtype]))
    return view, flat


# ------------------------------------------------------------------ rotary

def _segments(M):
    return [dict(kind=M.SEG_VIDEO, n_tokens=30, T=2, H=3, W=5, t0=-2),
            dict(kind=M.SEG_VIDEO, n_tokens=5 * 6 * 7, T=5, H=6, W=7, order=M.ORDER_BLOCK444),
            dict(kind=M.SEG_AUDIO, n_tokens=45, t0=1, t_num=21, t_den=218), dict(kind=M.SEG_TEXT, n_tokens=6)]


def _olayout(segs):
    return O.Layout([O.Segment(s["kind"], s["n_tokens"], s.get("T", 0), s.get("H", 0), s.get("W", 0), s.get("t0", 0),
                               s.get("t_num", 1), s.get("t_den", 1), s.get("order", 0)) for s in segs])


def _params(M, dims, half, scaling):
    kw = dict(factors=(4.0, 2.0, 1.5), trained=(21.0, 30.0, 52.0), magnitude=1.0 if scaling == "none" else 1.14)
    kinds = {"none": M.SCALE_NONE, "linear": M.SCALE_LINEAR, "ntk": M.SCALE_NTK, "parts": M.SCALE_PARTS}
    m = M.rotary_params(10000.0, *dims, pairing=M.PAIR_HALF if half else M.PAIR_INTERLEAVED, scaling=kinds[scaling],
                        beta_fast=4.0, beta_slow=0.25, **kw)
    return m, dict(theta=10000.0, dims=dims, half=half, scaling=scaling, fast=4.0, slow=0.25, **kw)


def _turn_bound(x, p, dtype, y):
    bound = HALF_STEP[dtype] * np.abs(y)
    for c1, c2, *_ in OC.frequencies(p):
        size = 2.0 ** -21 * p["magnitude"] * (np.abs(x[..., c1]) + np.abs(x[..., c2]))
        bound[..., c1] += size
        bound[..., c2] += size
    return bound


ROTARY = [  # dtype, D, B, N, Hq, Hk, dims, half, scaling, transpose, pads, window
    ("bf16", 128, 1, 291, 3, 3, (44, 42, 42), False, "none", False, (0, 0), False),
    ("bf16", 128, 2, 33, 6, 2, (44, 42, 42), True, "parts", False, (24, 8), True),
    ("bf16", 64, 3, 1, 5, 1, (32, 0, 0), True, "none", False, (0, 0), True),
    ("bf16", 64, 2, 17, 2, 2, (24, 20, 20), False, "ntk", True, (8, 16), True),
    ("f32", 64, 2, 50, 4, 2, (22, 20, 20), True, "linear", True, (4, 12), True),
    ("f32", 128, 1, 7, 9, 3, (2, 0, 126), True, "parts", False, (0, 0), True),
    ("f32", 128, 2, 130, 1, 1, (10, 6, 0), False, "parts", True, (0, 0), True),
    ("f32", 64, 1, 291, 2, 1, (64, 0, 0), False, "ntk", False, (0, 0), False),
    # enough tokens that a thread streams several heads past its angles
    ("bf16", 64, 8, 1100, 9, 4, (24, 20, 20), True, "none", False, (8, 0), True),
    ("f32", 64, 8, 600, 10, 3, (32, 16, 16), False, "parts", True, (0, 4), True),
]


@pytest.mark.parametrize("case", ROTARY)
def test_rotary(M, case):
    dtype, D, B, N, hq, hk, dims, half, scaling, transpose, (pt, pb), window = case
    rng = np.random.default_rng(5)
    segs = _segments(M)
    mp, p = _params(M, dims, half, scaling)
    first = np.resize([40, 0, 280] if window else [0], B).astype(np.int32)
    q, _ = _tensor(rng, (B, N, hq, D), dtype, pt, pb)
    k, _ = _tensor(rng, (B, N, hk, D), dtype, 2 * pt, pb)
    qo, qflat = _tensor(rng, (B, N, hq, D), dtype, pt + 16, 32, fill=np.zeros((B, N, hq, D)))
    kc = k.clone()
    M.rotary(q, qo, M.desc_of(q), M.desc_of(qo), k, k, M.desc_of(k), M.desc_of(k), M.make_layout(segs), mp,
             first=torch.from_numpy(first).cuda() if window else None, transpose=transpose)
    torch.cuda.synchronize()
    for x, y in ((q, qo), (kc, k)):
        hx = _f64(x)
        ref = OC.rotary(hx, p, _olayout(segs), first, transpose)
        err, bound = np.abs(_f64(y) - ref), _turn_bound(hx, p, dtype, ref)
        assert np.all(err <= bound), (float((err - bound).max()), np.argwhere(err > bound)[:3])
        n = sum(dims)
        assert torch.equal(x[..., n:], y[..., n:])  # the unturned channels keep their bits
    inside = torch.zeros_like(qflat, dtype=torch.bool)
    inside.as_strided(qo.shape, qo.stride()).fill_(True)
    assert bool((qflat[~inside] == 3.0).all())  # the room between rows is not written


@pytest.mark.parametrize("half", [False, True])
def test_rotary_of_far_positions(M, half):
    """Positions around 10^6 and 10^9: an fp32 angle would be off by up to 0.06 and 60 rad."""
    mp, p = _params(M, (40, 12, 12), half, "none")
    segs = [dict(kind=M.SEG_VIDEO, n_tokens=2 * 3 * 5, T=2, H=3, W=5, t0=10 ** 9),
            dict(kind=M.SEG_AUDIO, n_tokens=10 ** 7, t0=0, t_num=21, t_den=218)]
    lay = M.make_layout(segs)
    rng = np.random.default_rng(6)
    q, _ = _tensor(rng, (2, 20, 2, 64), "f32")
    o = torch.empty_like(q)
    first = np.array([10, 9 * 10 ** 6], np.int32)
    M.rotary(q, o, M.desc_of(q), M.desc_of(o), None, None, None, None, lay, mp, first=torch.from_numpy(first).cuda())
    near = [dict(kind=M.SEG_VIDEO, n_tokens=30, T=2, H=3, W=5, t0=10 ** 9)]
    ref = np.stack([OC.rotary(_f64(q)[:1], p, _olayout(near + [dict(kind=M.SEG_AUDIO, n_tokens=40, t_num=21, t_den=218)]), [10])[0]] +
                   [np.zeros((20, 2, 64))])
    x = _f64(q)[1]
    for n in range(20):
        t = (9 * 10 ** 6 + n - 30) * 21 / 218
        for c1, c2, axis, w in OC.frequencies(p):
            c, s = (math.cos(t * w), math.sin(t * w)) if axis == 0 else (1.0, 0.0)
            ref[1, n, :, c1], ref[1, n, :, c2] = (c * x[n, :, c1] - s * x[n, :, c2], s * x[n, :, c1] + c * x[n, :, c2])
    # the oracle's own fp64 angle is off by half a step of 10^9 rad: 6e-8, taken on top
    bound = _turn_bound(_f64(q), p, "f32", ref) + 1e-7 * np.abs(_f64(q)).max()
    assert np.all(np.abs(_f64(o) - ref) <= bound)


def test_rotary_keeps_what_it_does_not_turn_whatever_it_holds(M):
    mp, _ = _params(M, (16, 0, 0), True, "none")
    q = torch.randn((1, 8, 2, 64), device="cuda")
    q[..., 16:] = float("nan")
    q[0, 3, 1, 20] = float("inf")
    o = torch.empty_like(q)
    for half in (False, True):
        mp.pairing = M.PAIR_HALF if half else M.PAIR_INTERLEAVED
        M.rotary(q, o, M.desc_of(q), M.desc_of(o), None, None, None, None, M.make_layout([dict(kind=M.SEG_AUDIO, n_tokens=8)]), mp)
        assert torch.isfinite(o[..., :16]).all()
        assert torch.equal(q[..., 16:].view(torch.int32), o[..., 16:].view(torch.int32))


@pytest.mark.parametrize("half", [False, True])
def test_rotary_transpose_is_the_gradient(M, half):
    """<R x, g> changes by <x', R^T g> for any step x': differences of a linear map are exact up to rounding."""
    mp, p = _params(M, (22, 20, 20), half, "parts")
    rng = np.random.default_rng(7)
    lay = M.make_layout(_segments(M))
    x, _ = _tensor(rng, (2, 40, 3, 64), "f32")
    step, _ = _tensor(rng, (2, 40, 3, 64), "f32")
    g, _ = _tensor(rng, (2, 40, 3, 64), "f32")
    first = torch.tensor([3, 200], dtype=torch.int32, device="cuda")
    d = M.desc_of(x)

    def turn(t, transpose=False):
        o = torch.empty_like(t)
        M.rotary(t, o, M.desc_of(t), M.desc_of(o), None, None, None, None, lay, mp, first=first, transpose=transpose)
        return o
    dx = turn(g, True)
    ref = OC.rotary(_f64(g), p, _olayout(_segments(M)), [3, 200], True)
    assert np.all(np.abs(_f64(dx) - ref) <= _turn_bound(_f64(g), p, "f32", ref))
    change = ((turn(x + step).double() - turn(x).double()) * g.double()).sum()
    # every output value is off by at most 2^-20 (|x| + |step|), weighted by |g|
    room = 4 * 2.0 ** -20 * float(((x.abs() + step.abs()).double().sum(-1) * g.abs().double().amax(-1)).sum())
    assert abs(float(change) - float((step.double() * dx.double()).sum())) <= room
    assert d.head_dim == 64


# ------------------------------------------------------------------ cache

def _new_cache(M, rng, n_pages, heads, page, D, batch, per, live=None):
    """Random codes (NaN codes too) and scales, and a shuffled page table."""
    kc, vc = (rng.integers(0, 256, (n_pages, heads, page, D)).astype(np.uint8) for _ in range(2))
    ks, vs = (2.0 ** rng.integers(-9, -3, (n_pages, heads)) for _ in range(2))
    table = rng.permutation(n_pages)[: batch * per].reshape(batch, per).astype(np.int32)
    dev = [torch.from_numpy(a).cuda() for a in (kc, vc, ks.astype(np.float32), vs.astype(np.float32), table)]
    return [kc, vc, ks, vs, table], dev, M.make_cache(*dev)


APPEND = [  # dtype, D, page, B, N, H, start, count, rotation (None or half)
    ("bf16", 128, 16, 3, 1, 3, [0, 15, 47], None, None),
    ("bf16", 64, 16, 2, 40, 2, [3, 16], [40, 17], None),
    ("f32", 64, 32, 2, 70, 3, [31, 0], [70, 0], None),
    ("bf16", 128, 64, 2, 130, 2, [1, 63], [130, 66], None),
    ("f32", 128, 128, 2, 129, 2, [127, 5], [129, 1], None),
    ("bf16", 128, 64, 1, 130, 5, [37], None, False),
    ("bf16", 128, 16, 2, 33, 3, [9, 100], [33, 20], True),
    ("f32", 64, 64, 2, 100, 2, [60, 10], None, True),
    ("f32", 128, 32, 1, 40, 2, [5], None, False),
    ("f32", 128, 128, 1, 200, 2, [100], None, True),
    ("bf16", 64, 128, 2, 9, 2, [0, 120], None, False),
    # so many items that a CTA takes several heads of its page, one or two of them in shared memory
    ("f32", 128, 128, 80, 3, 4, [7 * i % 300 for i in range(80)], None, True),
    ("f32", 128, 128, 80, 3, 5, [11 * i % 300 for i in range(80)], None, False),
    ("bf16", 128, 64, 200, 2, 4, [3 * i % 130 for i in range(200)], [i % 3 for i in range(200)], True),
    ("bf16", 64, 64, 200, 70, 3, [i % 70 for i in range(200)], None, None),
    ("f32", 64, 16, 300, 2, 6, [i % 40 for i in range(300)], None, False),
]


@pytest.mark.parametrize("case", APPEND)
@pytest.mark.parametrize("size", [0.01, 30.0])  # older tokens' scales hold, or have to grow
def test_append(M, case, size):
    dtype, D, page, B, N, H, start, count, half = case
    rng = np.random.default_rng(11)
    per = -(-(max(start) + N) // page) + 1
    host, dev, cache = _new_cache(M, rng, B * per + 2, H, page, D, B, per)
    host[0][host[0] & 127 == 127] = 5  # older tokens are values
    host[1][host[1] & 127 == 127] = 5
    dev[0].copy_(torch.from_numpy(host[0]))
    dev[1].copy_(torch.from_numpy(host[1]))
    spread = np.exp2(rng.integers(-3, 4, (B, N, 1, 1)))
    k, _ = _tensor(rng, (B, N, H, D), dtype, 16, 8, fill=rng.standard_normal((B, N, H, D)) * size * spread)
    v, _ = _tensor(rng, (B, N, H, D), dtype, 16, 8, fill=rng.standard_normal((B, N, H, D)) * size * spread)
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    ct = None if count is None else torch.tensor(count, dtype=torch.int32, device="cuda")
    count = [N] * B if count is None else count
    hk, kw, p = _f64(k), {}, None
    if half is not None:
        dh = 2 * (D // 6)
        mp, p = _params(M, (D - 2 * dh - 2, dh, dh), half, "parts")
        kw = dict(layout=M.make_layout(_segments(M)), rotation=mp)
        hk = OC.rotary(hk, p, _olayout(_segments(M)), start)
    M.cache_append(k, v, M.desc_of(k), cache, st, count=ct, **kw)
    torch.cuda.synchronize()
    OC.append(host[0], host[2], host[4], hk, start, count, np.zeros((B, N, H), bool))
    OC.append(host[1], host[3], host[4], _f64(v), start, count, None)
    assert np.array_equal(dev[3].cpu().numpy(), host[3]) and np.array_equal(dev[1].cpu().numpy(), host[1])
    assert np.array_equal(dev[2].cpu().numpy(), host[2])
    got = dev[0].cpu().numpy()
    if half is None:
        assert np.array_equal(got, host[0])
        return
    turn = _turn_bound(_f64(k), p, "f32", hk)
    seen = np.ones(got.shape, bool)
    for b in range(B):
        for i in range(count[b]):
            j, s = divmod(start[b] + i, page)
            pid = host[4][b, j]
            seen[pid, :, s] = False
            sc = host[2][pid][:, None]
            err = np.abs(OC.E4M3[got[pid, :, s]] * sc - hk[b, i])
            assert np.all(err <= 2.0 ** -4 * np.abs(hk[b, i]) + 2.0 ** -10 * sc + turn[b, i])
    assert np.array_equal(got[seen], host[0][seen])
    assert (got != host[0]).mean() < 1e-3  # only values next to a border of the rounding


def test_append_outside_the_cache(M):
    """Negative starts, starts and counts behind the capacity, and bad page ids store nothing there."""
    rng = np.random.default_rng(12)
    host, dev, cache = _new_cache(M, rng, 12, 2, 16, 64, 3, 3)
    host[4][1, 1], host[4][2, 0] = 12, -1
    dev[4].copy_(torch.from_numpy(host[4]))
    k, _ = _tensor(rng, (3, 50, 2, 64), "bf16")
    v, _ = _tensor(rng, (3, 50, 2, 64), "bf16")
    for start in ([-5, 0, 2], [48, 2 ** 31 - 20, -(2 ** 31)], [47, 30, 16]):
        M.cache_append(k, v, M.desc_of(k), cache, torch.tensor(start, dtype=torch.int32, device="cuda"),
                       count=torch.tensor([60, 50, -3], dtype=torch.int32, device="cuda"))
        OC.append(host[0], host[2], host[4], _f64(k), start, [60, 50, -3], np.zeros((3, 50, 2), bool))
        OC.append(host[1], host[3], host[4], _f64(v), start, [60, 50, -3], None)
        for d, h in zip(dev[:4], host):
            assert np.array_equal(d.cpu().numpy(), h)
    assert M.device_status() == M.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("half", [None, False, True])
def test_append_of_infinities_and_nan(M, dtype, half):
    rng = np.random.default_rng(13)
    host, dev, cache = _new_cache(M, rng, 5, 3, 32, 64, 1, 3)
    x = [rng.standard_normal((1, 60, 3, 64)) for _ in range(2)]
    x[0][0, 7, 1, 5], x[0][0, 40, 0, 63], x[1][0, 41, 2, 0], x[1][0, 59, 0, 9] = np.nan, np.inf, -np.inf, np.nan
    (k, _), (v, _) = (_tensor(rng, (1, 60, 3, 64), dtype, fill=a) for a in x)
    bad = ~(np.isfinite(x[0]) & np.isfinite(x[1])).all(-1)
    kw, hk, p = {}, _f64(k), None
    if half is not None:
        mp, p = _params(M, (24, 20, 20), half, "none")
        kw = dict(layout=M.make_layout(_segments(M)), rotation=mp)
        hk = np.where(bad[..., None], np.nan, OC.rotary(np.nan_to_num(hk), p, _olayout(_segments(M)), [0]))
    M.cache_append(k, v, M.desc_of(k), cache, torch.zeros(1, dtype=torch.int32, device="cuda"), **kw)
    OC.append(host[1], host[3], host[4], _f64(v), [0], [60], None)
    assert np.array_equal(dev[1].cpu().numpy(), host[1]) and np.array_equal(dev[3].cpu().numpy(), host[3])
    got = dev[0].cpu().numpy()
    for i in range(60):
        pid, s = host[4][0, i // 32], i % 32
        assert np.array_equal((got[pid, :, s] & 127 == 127).all(-1), bad[0, i])
        assert not (got[pid, :, s] & 127 == 127)[~bad[0, i]].any()
    if half is None:
        OC.append(host[0], host[2], host[4], hk, [0], [60], bad)
        assert np.array_equal(got, host[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_infinities_to_several_heads_of_a_cta(M, dtype):
    """300 items of 5 heads: heads with and without an infinity or NaN follow one another in a CTA."""
    rng = np.random.default_rng(15)
    B, N, H = 300, 3, 5
    host, dev, cache = _new_cache(M, rng, B + 2, H, 64, 64, B, 1)
    x = [rng.standard_normal((B, N, H, 64)) for _ in range(2)]
    for i, bad in enumerate((np.nan, np.inf, -np.inf)):
        x[i % 2][i::7, i, i + 1, 5 * i] = bad
    (k, _), (v, _) = (_tensor(rng, (B, N, H, 64), dtype, fill=a) for a in x)
    bad = ~(np.isfinite(x[0]) & np.isfinite(x[1])).all(-1)
    M.cache_append(k, v, M.desc_of(k), cache, torch.zeros(B, dtype=torch.int32, device="cuda"))
    OC.append(host[0], host[2], host[4], _f64(k), [0] * B, [N] * B, bad)
    OC.append(host[1], host[3], host[4], _f64(v), [0] * B, [N] * B, None)
    for d, h in zip(dev[:4], host):
        assert np.array_equal(d.cpu().numpy(), h)


def test_append_token_by_token_equals_its_definition(M):
    """40 tokens of growing size, one call each: the page's scale grows on the way."""
    rng = np.random.default_rng(14)
    host, dev, cache = _new_cache(M, rng, 4, 2, 16, 128, 1, 3)
    x = rng.standard_normal((1, 40, 2, 128)) * np.exp2(np.arange(40) / 6)[None, :, None, None]
    k, _ = _tensor(rng, x.shape, "bf16", fill=x)
    v, _ = _tensor(rng, x.shape, "bf16", fill=x[:, ::-1])
    for i in range(40):
        M.cache_append(k[:, i:i + 1], v[:, i:i + 1], M.desc_of(k[:, i:i + 1]), cache,
                       torch.tensor([i], dtype=torch.int32, device="cuda"))
        OC.append(host[0], host[2], host[4], _f64(k[:, i:i + 1]), [i], [1], np.zeros((1, 1, 2), bool))
        OC.append(host[1], host[3], host[4], _f64(v[:, i:i + 1]), [i], [1], None)
    for d, h in zip(dev[:4], host):
        assert np.array_equal(d.cpu().numpy(), h)


# ------------------------------------------------------------------ attention

def _attend(M, q, dev, cache, kv, ql, causal, scale, o=None, lse=True, stream=None):
    o = torch.full_like(q, 7.0) if o is None else o
    e = torch.full((q.shape[0], q.shape[2], q.shape[1]), 7.0, device="cuda") if lse else None
    n = M.cache_attn_workspace_size(M.desc_of(q), cache)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")  # NaN
    M.cache_attn(q, o, M.desc_of(q), M.desc_of(o), cache, kv, scale, q_len=ql, causal_block=causal, lse=e, workspace=ws,
                 ws_bytes=n, stream=stream)
    return o, e


def _check_attention(dtype, D, kv, got, lse, ref, q_len):
    o, l, S, A = ref
    w = (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22) + 2 * ((D / 16 + 2) * 2.0 ** -22 * A + 2.0 ** -22) \
        + (kv / 16 + 8) * 2.0 ** -23
    for b in range(o.shape[0]):
        n = min(max(int(q_len[b]), 0), o.shape[1])
        err = np.abs(got[b, :n] - o[b, :n])
        bound = HALF_STEP[dtype] * np.abs(o[b, :n]) + w[b, :, :n].T[..., None] * S[b, :n]
        assert np.all(err <= bound), (b, float((err / np.maximum(bound, 1e-30)).max()), np.argwhere(~(err <= bound))[:4])
        assert np.all(got[b, n:] == 7.0)  # rows behind the item's last stay as they were
        if lse is not None:
            dead = l[b, :, :n] == -np.inf
            assert np.array_equal(lse[b, :, :n] == -np.inf, dead)
            d = np.abs(np.where(dead, 0, lse[b, :, :n]) - np.where(dead, 0, l[b, :, :n]))
            assert np.all(d <= w[b, :, :n] + 2.0 ** -22 * np.abs(np.where(dead, 0, l[b, :, :n])))
            assert np.all(lse[b, :, n:] == 7.0)


ATTN = [  # dtype, D, page, B, N, H, Hk, per, kv_len, q_len, causal
    ("bf16", 128, 16, 4, 1, 3, 3, 14, [218, 1, 0, 17], None, 1),
    ("bf16", 64, 32, 2, 1, 6, 2, 50, [1600, 33], None, 0),
    ("f32", 64, 16, 3, 11, 2, 2, 30, [450, 5, 11], [11, 11, 4], 1),
    ("f32", 128, 128, 2, 3, 4, 1, 6, [700, 129], [3, 0], 0),
    ("bf16", 128, 64, 1, 1, 8, 1, 40, [2560], None, 1),
    ("bf16", 128, 64, 2, 16, 2, 2, 12, [700, 64], [16, 9], 5),
    ("bf16", 128, 128, 2, 17, 3, 1, 5, [600, 128], [17, 17], 0),
    ("bf16", 64, 16, 2, 70, 4, 2, 20, [300, 40], [70, 70], 1),
    ("f32", 64, 64, 1, 40, 2, 1, 4, [200], None, 7),
    ("bf16", 128, 32, 3, 130, 2, 1, 20, [640, 130, 90], [130, 130, 130], 1),
    ("bf16", 128, 64, 2, 300, 2, 2, 12, [700, 333], [300, 5], 60),
    ("bf16", 64, 64, 1, 257, 1, 1, 9, [513], None, 0),
    ("bf16", 64, 128, 2, 90, 9, 3, 4, [512, 100], [90, 90], 1),
    ("bf16", 128, 16, 1, 200, 2, 2, 80, [1279], None, 0),
    ("bf16", 128, 128, 1, 66, 2, 2, 40, [5000], None, 0),
    ("bf16", 64, 64, 2, 9, 2, 2, 10, [600, 9], None, 1),
    ("bf16", 128, 64, 2, 27, 1, 1, 9, [576, 40], [27, 20], 1),
    ("f32", 64, 32, 1, 2, 4, 2, 30, [900], None, 0),
    ("f32", 128, 16, 2, 5, 2, 2, 20, [300, 7], [5, 2], 3),
    ("bf16", 64, 32, 200, 65, 2, 2, 90, [2880] + [40, 1, 129] * 66 + [2800], None, 1),  # more items than SMs: not split
]


@pytest.mark.parametrize("case", ATTN)
def test_attention(M, case):
    """Every slot behind kv_len holds NaN codes or old data, every page outside the table NaN scales."""
    dtype, D, page, B, N, H, Hk, per, kv, ql, causal = case
    rng = np.random.default_rng(21)
    host, dev, cache = _new_cache(M, rng, B * per + 2, Hk, page, D, B, per)
    kc, vc, ks, vs, table = host
    held = np.zeros(kc.shape[:3], bool)
    for b in range(B):
        for n in range(kv[b]):
            held[table[b, n // page], :, n % page] = True
    for c in (kc, vc):
        nan = c & 127 == 127
        c[nan & held[..., None]] = 0x21
    unused = np.setdiff1d(np.arange(B * per + 2), table)
    ks[unused] = np.nan
    ks *= 2.0 ** -3
    vs *= rng.uniform(0.5, 2.0, vs.shape)
    vs = vs.astype(np.float32).astype(np.float64)
    for d, h in zip(dev, (kc, vc, ks.astype(np.float32), vs.astype(np.float32))):
        d.copy_(torch.from_numpy(h))
    q, _ = _tensor(rng, (B, N, H, D), dtype, 16, 24)
    o, flat = _tensor(rng, (B, N, H, D), dtype, 8, 16, fill=np.full((B, N, H, D), 7.0))
    kt = torch.tensor(kv, dtype=torch.int32, device="cuda")
    qt = None if ql is None else torch.tensor(ql, dtype=torch.int32, device="cuda")
    ql = [N] * B if ql is None else ql
    scale = 1 / math.sqrt(D)
    got, lse = _attend(M, q, dev, cache, kt, qt, causal, scale, o=o)
    assert M.device_status() == M.OK
    ref = OC.cache_attn(_f64(q), kc, vc, ks, vs, table, kv, ql, causal, scale)
    _check_attention(dtype, D, max(kv), _f64(got), _f64(lse), ref, ql)
    inside = torch.zeros_like(flat, dtype=torch.bool)
    inside.as_strided(o.shape, o.stride()).fill_(True)
    assert bool((flat[~inside] == 3.0).all())
    again, _ = _attend(M, q, dev, cache, kt, qt, causal, scale, lse=False)
    assert torch.equal(again, got)  # no order depends on the run


@pytest.mark.parametrize("N", [1, 40, 150])
def test_attention_of_values_of_very_different_size(M, N):
    """V scales from 2^-40 to 2^30 in one item, zero scales, Q rows of all sizes, one key that takes all the weight."""
    rng = np.random.default_rng(22)
    host, dev, cache = _new_cache(M, rng, 20, 1, 16, 128, 1, 20)
    kc, vc, ks, vs, table = host
    kc[kc & 127 == 127], vc[vc & 127 == 127] = 3, 3
    vs[:] = np.exp2(rng.integers(-40, 31, vs.shape))
    vs[table[0, 3]], ks[table[0, 5]] = 0.0, 0.0
    for d, h in zip(dev, (kc, vc, ks.astype(np.float32), vs.astype(np.float32))):
        d.copy_(torch.from_numpy(h))
    x = rng.standard_normal((1, N, 1, 128)) * np.exp2(rng.integers(-20, 3, (1, N, 1, 1)))
    x[0, 0, 0, 1:] *= 2.0 ** -12  # one channel far above the others
    q, _ = _tensor(rng, x.shape, "bf16", fill=x)
    kt = torch.tensor([309], dtype=torch.int32, device="cuda")
    got, lse = _attend(M, q, dev, cache, kt, None, 0, 0.05)
    ref = OC.cache_attn(_f64(q), kc, vc, ks, vs, table, [309], [N], 0, 0.05)
    _check_attention("bf16", 128, 309, _f64(got), _f64(lse), ref, [N])


@pytest.mark.parametrize("N", [2, 70])
def test_a_lost_token_reaches_only_the_rows_that_see_it(M, N):
    """NaN in K or V of a token: appended, then attended to causally."""
    rng = np.random.default_rng(23)
    host, dev, cache = _new_cache(M, rng, 8, 2, 32, 64, 1, 8)
    k, _ = _tensor(rng, (1, 150, 2, 64), "bf16")
    v, _ = _tensor(rng, (1, 150, 2, 64), "bf16")
    k[0, 149, 0, 3] = float("nan")
    v[0, 149, 1, 60] = float("inf")
    M.cache_append(k, v, M.desc_of(k), cache, torch.zeros(1, dtype=torch.int32, device="cuda"))
    q, _ = _tensor(rng, (1, N, 2, 64), "bf16")
    q[0, 0, 1, 5] = float("inf")
    o, lse = _attend(M, q, dev, cache, torch.tensor([150], dtype=torch.int32, device="cuda"), None, 1, 0.125)
    assert torch.isfinite(o[0, 1:N - 1]).all() and torch.isfinite(lse[0, :, 1:N - 1]).all() and torch.isfinite(o[0, 0, 0]).all()
    assert torch.isnan(o[0, N - 1]).all() and torch.isnan(o[0, 0, 1]).all()


@pytest.mark.parametrize("N", [1, 100])
def test_attention_skips_pages_that_are_not_there(M, N):
    rng = np.random.default_rng(24)
    host, dev, cache = _new_cache(M, rng, 30, 2, 16, 64, 2, 12)
    kc, vc, ks, vs, table = host
    kc[kc & 127 == 127], vc[vc & 127 == 127] = 3, 3
    table[0, 4], table[0, 7], table[1, :] = -1, 30, 2 ** 31 - 1
    for d, h in zip(dev, (kc, vc, ks.astype(np.float32), vs.astype(np.float32), table)):
        d.copy_(torch.from_numpy(h))
    q, _ = _tensor(rng, (2, N, 2, 64), "bf16")
    got, lse = _attend(M, q, dev, cache, torch.tensor([180, 150], dtype=torch.int32, device="cuda"), None, 0, 0.02)
    ref = OC.cache_attn(_f64(q), kc, vc, ks, vs, table, [180, 150], [N, N], 0, 0.02)
    assert np.all(ref[1][1] == -np.inf)
    _check_attention("bf16", 64, 180, _f64(got), _f64(lse), ref, [N, N])
    # lengths outside the capacity are taken as the nearest one inside
    more, _ = _attend(M, q, dev, cache, torch.tensor([10 ** 6, -4], dtype=torch.int32, device="cuda"),
                      torch.tensor([N + 5, N], dtype=torch.int32, device="cuda"), 0, 0.02)
    most, _ = _attend(M, q, dev, cache, torch.tensor([192, 0], dtype=torch.int32, device="cuda"), None, 0, 0.02)
    assert torch.equal(more, most)


def test_cache_arrays_past_32_bits(M):
    """Pages whose codes start more than 2^32 bytes into the array: append, attention and copies there."""
    n_pages, H, page, D = 16500, 16, 128, 128
    kc, vc = (torch.empty((n_pages, H, page, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 32
    ks, vs = (torch.zeros((n_pages, H), device="cuda") for _ in range(2))
    ids = [n_pages - 1, 3, n_pages - 2]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    cache = M.make_cache(kc, vc, ks, vs, table)
    rng = np.random.default_rng(25)
    k, _ = _tensor(rng, (1, 300, H, D), "bf16")
    v, _ = _tensor(rng, (1, 300, H, D), "bf16")
    M.cache_append(k, v, M.desc_of(k), cache, torch.zeros(1, dtype=torch.int32, device="cuda"))
    M.cache_copy_pages(cache, [n_pages - 2], [n_pages - 4])
    table[0, 2] = n_pages - 4
    small = [t[ids[:2] + [n_pages - 4]].cpu().numpy() for t in (kc, vc, ks, vs)]
    host = [np.zeros((3, H, page, D), np.uint8), np.zeros((3, H, page, D), np.uint8), np.zeros((3, H)), np.zeros((3, H))]
    for c, s, x in ((0, 2, k), (1, 3, v)):
        OC.append(host[c], host[s], np.array([[0, 1, 2]]), _f64(x), [0], [300], np.zeros((1, 300, H), bool))
        assert np.array_equal(small[s], host[s])
        assert np.array_equal(small[c].transpose(0, 2, 1, 3).reshape(-1, H, D)[:300], host[c].transpose(0, 2, 1, 3).reshape(-1, H, D)[:300])
    for N in (1, 64):
        q, _ = _tensor(rng, (1, N, H, D), "bf16")
        got, lse = _attend(M, q, None, cache, torch.tensor([300], dtype=torch.int32, device="cuda"), None, 0, 0.09)
        ref = OC.cache_attn(_f64(q), host[0], host[1], host[2], host[3], np.array([[0, 1, 2]]), [300], [N], 0, 0.09)
        _check_attention("bf16", D, 300, _f64(got), _f64(lse), ref, [N])


# ------------------------------------------------------------------ page copies

@pytest.mark.parametrize("n", [1, 3, 1000])
def test_copy_pages(M, n):
    rng = np.random.default_rng(31)
    host, dev, _ = _new_cache(M, rng, 2 * n + 3, 3, 16, 64, 1, 1)
    cache = M.make_cache(*dev[:4])
    ids = rng.permutation(2 * n + 3)
    src, dst = ids[:n].tolist(), ids[n:2 * n].tolist()
    if n == 3:
        src = [src[0]] * 3  # a fork to three
    M.cache_copy_pages(cache, src, dst)
    for d, h in zip(dev[:4], host):
        h[dst] = h[src]
        assert np.array_equal(d.cpu().numpy(), h.astype(d.cpu().numpy().dtype))


# ------------------------------------------------------------------ together

def _generate(M, turns, graph=False, stream=None):
    """A 2-item sequence continued `turns` times by a 12-token frame: rotate Q, store K and V, attend by frames; at
    the end item 1 is forked into a third sequence that goes on by itself."""
    rng = np.random.default_rng(41)
    B, N, H, Hk, D, page, per = 2, 12, 4, 2, 128, 16, 8
    host, dev, _ = _new_cache(M, rng, 40, Hk, page, D, B, per)
    for d in dev[:2]:
        d.fill_(0x7f)
    cache = M.make_cache(*dev)
    segs = [dict(kind=M.SEG_VIDEO, n_tokens=12 * 9, T=9, H=3, W=4, t0=-1)]
    mp, p = _params(M, (44, 42, 42), False, "none")
    lay = M.make_layout(segs)
    held = torch.zeros(B, dtype=torch.int32, device="cuda")
    xs = [[_tensor(rng, (B, N, h, D), "bf16")[0] for h in (H, Hk, Hk)] for _ in range(turns)]
    q, k, v = (torch.empty_like(x) for x in xs[0])
    qr, o = torch.empty_like(q), torch.empty_like(q)
    n = M.cache_attn_workspace_size(M.desc_of(q), cache)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")

    def step():
        M.rotary(q, qr, M.desc_of(q), M.desc_of(qr), None, None, None, None, lay, mp, first=held)
        M.cache_append(k, v, M.desc_of(k), cache, held, layout=lay, rotation=mp)
        held.add_(N)
        M.cache_attn(qr, o, M.desc_of(qr), M.desc_of(o), cache, held, 0.088, causal_block=N, workspace=ws, ws_bytes=n)
    outs = []
    run = step
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    for x in xs:
        for t, s in zip((q, k, v), x):
            t.copy_(s)
        run()
        outs.append(o.clone())
    return xs, outs, dev, cache, lay, (mp, p), segs, held, (q, k, v)


def test_a_sequence_is_continued(M):
    xs, outs, dev, cache, lay, (mp, p), segs, held, _ = _generate(M, 5)
    page, per = 16, 8
    kc, vc = np.zeros(dev[0].shape, np.uint8), np.zeros(dev[0].shape, np.uint8)
    ks, vs = np.zeros(dev[2].shape), np.zeros(dev[2].shape)
    table = dev[4].cpu().numpy()
    for i, ((q, k, v), got) in enumerate(zip(xs, outs)):
        at = [12 * i] * 2
        # the attention reads Q as the rotary stored it, in bf16
        hq = OC.rotary(_f64(q), p, _olayout(segs), at)
        hq = _f64(torch.from_numpy(hq.astype(np.float32)).to(torch.bfloat16))
        OC.append(kc, ks, table, OC.rotary(_f64(k), p, _olayout(segs), at), at, [12] * 2, np.zeros((2, 12, 2), bool))
        OC.append(vc, vs, table, _f64(v), at, [12] * 2, None)
        ref = OC.cache_attn(hq, kc, vc, ks, vs, table, [12 * (i + 1)] * 2, [12] * 2, 12, 0.088)
        # a value of Q or K on a rounding border may fall to the other side: a step of bf16 or e4m3 in one channel
        # of 128 moves a score by 2^-3 |q k| scale <= 2^-3 * 12 * 0.088 = 0.13 at most, and its weight, one of 12 or more,
        # by that share: 2 * 0.13 / 12 of the values' size
        err = np.abs(_f64(got) - ref[0])
        assert np.all(err <= 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -10 + 2 * 0.13 / 12) * ref[2])
        assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(ref[0])
    # fork item 1 (60 tokens: three whole pages, 12 tokens of a fourth): it shares the whole pages
    free = [x for x in range(40) if x not in table]
    M.cache_copy_pages(cache, [int(table[1, 3])], [free[0]])
    fork = table.copy()
    fork[0] = table[1]
    fork[0, 3], fork[0, 4] = free[0], free[1]
    forked = M.make_cache(*dev[:4], torch.from_numpy(fork).cuda())
    rng = np.random.default_rng(42)
    q, k, v = (_tensor(rng, (2, 12, h, 128), "bf16")[0] for h in (4, 2, 2))
    k[0], v[0] = k[1], v[1]  # the same continuation twice: the fork and its parent agree
    q[0] = q[1]
    M.cache_append(k, v, M.desc_of(k), forked, held, layout=lay, rotation=mp)
    o, _ = _attend(M, q, dev, forked, held + 12, None, 12, 0.088)
    assert torch.equal(o[0], o[1])
    assert M.device_status() == M.OK


def test_a_captured_step_replays(M):
    a, b = _generate(M, 5)[1], _generate(M, 5, graph=True)[1]
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_run_on_the_stream_they_are_given(M):
    s = torch.cuda.Stream()
    a = _generate(M, 3)[1]
    with torch.cuda.stream(s):
        b = _generate(M, 3)[1]
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_calls_at_once_with_a_workspace_each(M):
    rng = np.random.default_rng(43)
    host, dev, cache = _new_cache(M, rng, 130, 4, 64, 128, 1, 120)
    for d, h in zip(dev, host[:2]):
        h[h & 127 == 127] = 3
        d.copy_(torch.from_numpy(h))
    q = [_tensor(rng, (1, n, 4, 128), "bf16")[0] for n in (1, 2, 90)]
    kv = torch.tensor([7600], dtype=torch.int32, device="cuda")
    alone = [_attend(M, x, dev, cache, kv, None, 0, 0.01)[0] for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(5):
        got = []
        for x, s in zip(q, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(_attend(M, x, dev, cache, kv, None, 0, 0.01)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, got))


@pytest.mark.parametrize("dtype,N", [("bf16", 3), ("f32", 20), ("bf16", 90)])
def test_split_calls_in_two_graphs(M, dtype, N):
    """Long histories are split into key ranges and merged by a second kernel: two captured calls with a workspace
    each, replayed together and in either order, give what the plain call gives, for each length of the history."""
    rng = np.random.default_rng(45)
    host, dev, cache = _new_cache(M, rng, 330, 2, 16, 64, 2, 150)
    for d, h in zip(dev, host[:2]):
        h[h & 127 == 127] = 3
        d.copy_(torch.from_numpy(h))
    kv = torch.tensor([2400, 1111], dtype=torch.int32, device="cuda")
    runs = []
    for i in range(2):
        q, _ = _tensor(rng, (2, N, 6, 64), dtype)
        o = torch.zeros_like(q)
        n = M.cache_attn_workspace_size(M.desc_of(q), cache)
        assert n > 0
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            M.cache_attn(q, o, M.desc_of(q), M.desc_of(o), cache, kv, 0.01, causal_block=1, workspace=ws, ws_bytes=n)
        runs.append((q, o, graph, ws))
    streams = [torch.cuda.Stream() for _ in runs]
    for lengths in ([2400, 1111], [N, 2400], [17, 0], [2399, 2400]):
        kv.copy_(torch.tensor(lengths, dtype=torch.int32))
        want = [_attend(M, q, dev, cache, kv, None, 1, 0.01)[0] for q, *_ in runs]
        torch.cuda.synchronize()
        for order in (0, 1):
            for r, s in list(zip(runs, streams))[::1 if order else -1]:
                with torch.cuda.stream(s):
                    r[2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(w, r[1]) for w, r in zip(want, runs))


def test_empty_calls(M):
    host, dev, cache = _new_cache(M, np.random.default_rng(44), 4, 2, 16, 64, 1, 2)
    q = torch.empty((1, 0, 2, 64), device="cuda")
    d = M.make_desc(1, 0, 2, 64, M.F32)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    some = torch.zeros(1024, device="cuda")
    M.rotary(some, some, d, d, None, None, None, None, M.make_layout([dict(kind=M.SEG_TEXT, n_tokens=0)]), M.rotary_params(1e4, 64))
    M.cache_append(some, some, d, cache, z)
    M.cache_attn(some, some[512:], d, d, cache, z, 0.1)
    M.cache_copy_pages(cache, [], [])
    for a, h in zip(dev[:4], host):
        assert np.array_equal(a.cpu().numpy(), h.astype(a.cpu().numpy().dtype))
    assert q.numel() == 0
