"""The continuation calls at the ends of the ranges that their contract allows, against the fp64 oracle.  Bounds: those of
test_gpu_continuation.py, where nothing else is derived beside the test."""
import math

import numpy as np
import pytest

from oracle import continuation as OC

from test_gpu_continuation import (HALF_STEP, M, _attend, _check_attention, _f64, _new_cache, _olayout, _params,  # noqa: F401
                                   _segments, _tensor)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

KINDS = [("bf16", 128, 1), ("bf16", 64, 12), ("bf16", 128, 100), ("bf16", 64, 300), ("f32", 64, 3), ("f32", 128, 20)]


def _led(M, rng, dtype, D, N, lead, kv=150):
    """An item of `kv` tokens in pages of 16 whose token 53 leads every row's scores by `lead` nats (to the rounding of
    Q): channel 0 of Q and of that key's K.  Other scores are within a nat of 0."""
    host, dev, cache = _new_cache(M, rng, 12, 1, 16, D, 1, 10)
    kc, vc, ks, vs, table = host
    vc[vc & 127 == 127] = 3
    kc[:] = OC.to_e4m3(rng.standard_normal(kc.shape) * 0.5)
    kc[..., 0] = 0
    ks[:] = 1.0
    page, slot = table[0, 53 // 16], 53 % 16
    kc[page, 0, slot] = 0
    kc[page, 0, slot, 0] = OC.to_e4m3(np.array(40.0))
    x = rng.standard_normal((1, N, 1, D)) * 0.5
    x[..., 0] = lead / (40.0 * 0.0625)
    q, _ = _tensor(rng, x.shape, dtype, fill=x)
    return host, dev, cache, q, (page, slot)


def _check_led(M, dtype, D, N, host, dev, cache, q, kv=150):
    for d, h in zip(dev, (host[0], host[1], host[2].astype(np.float32), host[3].astype(np.float32))):
        d.copy_(torch.from_numpy(h))
    got, lse = _attend(M, q, dev, cache, torch.tensor([kv], dtype=torch.int32, device="cuda"), None, 0, 0.0625)
    ref = OC.cache_attn(_f64(q), *host, [kv], [N], 0, 0.0625)
    _check_attention(dtype, D, kv, _f64(got), _f64(lse), ref, [N])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [20, -8, -20, -32, -40])
@pytest.mark.parametrize("lead", [0.0, 14.0])
def test_attention_beside_a_page_whose_v_scale_is_zero(M, kind, size, lead):
    """The page's values are zeros whatever its codes; it counts in the sum of weights and nowhere else."""
    dtype, D, N = kind
    host, dev, cache, q, (page, _) = _led(M, np.random.default_rng(51), dtype, D, N, lead)
    host[3][:] = 2.0 ** size
    host[3][page] = 0.0
    _check_led(M, dtype, D, N, host, dev, cache, q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("half", [False, True])
def test_append_of_keys_that_overflow_when_they_are_turned(M, dtype, half):
    """Finite K whose turned value is beyond fp32: the token's K there is lost, as if it had held an infinity."""
    rng = np.random.default_rng(55)
    host, dev, cache = _new_cache(M, rng, 5, 3, 32, 64, 1, 3)
    x = rng.standard_normal((1, 60, 3, 64))
    big = 3.2e38  # its pairs' length is 4.5e38: some position turns a value beyond 3.4e38
    for tok, h in ((7, 1), (40, 0), (41, 2)):
        x[0, tok, h, :24] = big
    (k, _), (v, _) = (_tensor(rng, x.shape, dtype, fill=a) for a in (x, rng.standard_normal(x.shape)))
    mp, p = _params(M, (24, 20, 20), half, "none")
    turned = OC.rotary(_f64(k), p, _olayout(_segments(M)), [0])
    bad = (np.abs(turned) > 3.5e38).any(-1)
    near = ((np.abs(turned) > 3.3e38).any(-1)) & ~bad
    assert not near.any() and bad.any()
    M.cache_append(k, v, M.desc_of(k), cache, torch.zeros(1, dtype=torch.int32, device="cuda"),
                   layout=M.make_layout(_segments(M)), rotation=mp)
    OC.append(host[1], host[3], host[4], _f64(v), [0], [60], None)
    assert np.array_equal(dev[1].cpu().numpy(), host[1]) and np.array_equal(dev[3].cpu().numpy(), host[3])
    got = dev[0].cpu().numpy()
    for i in range(60):
        nan = got[host[4][0, i // 32], :, i % 32] & 127 == 127
        assert np.array_equal(nan.all(-1), bad[0, i]) and not nan[~bad[0, i]].any()


@pytest.mark.parametrize("half", [False, True])
def test_rotary_products_are_all_that_rounds(M, half):
    """Cosine and sine are rounded to fp32 once, 2^-24 of themselves, as are the first product and the result: with
    |c|, |s| <= M, |err| <= 2^-24 |y| + 2^-24 M (|x1| + |x2|) + 2^-24 M |x2|."""
    mp, p = _params(M, (40, 44, 44), half, "parts")
    n = 20000
    lay = M.make_layout([dict(kind=M.SEG_VIDEO, n_tokens=n, T=20, H=25, W=40, t0=10 ** 6)])
    x = torch.randn((1, n, 1, 128), generator=torch.Generator(device="cuda").manual_seed(56), device="cuda")
    y = torch.empty_like(x)
    M.rotary(x, y, M.desc_of(x), M.desc_of(y), None, None, None, None, lay, mp)
    j = torch.arange(n, device="cuda")
    pos = torch.stack([10 ** 6 + j // 1000, j // 40 % 25, j % 40], 1).double()
    xd, yd = x[0, :, 0].double(), y[0, :, 0].double()
    for c1, c2, axis, w in OC.frequencies(p):
        a = pos[:, axis] * w
        c, s = torch.cos(a) * p["magnitude"], torch.sin(a) * p["magnitude"]
        r1, r2 = xd[:, c1] * c - xd[:, c2] * s, xd[:, c1] * s + xd[:, c2] * c
        room = 2.0 ** -24 * p["magnitude"] * (xd[:, c1].abs() + xd[:, c2].abs() + torch.maximum(xd[:, c1].abs(), xd[:, c2].abs()))
        room = room * (1 + 2.0 ** -12)  # the oracle's angle: 2^-53 of 10^6 turns
        assert bool(((yd[:, c1] - r1).abs() <= 2.0 ** -24 * r1.abs() + room).all())
        assert bool(((yd[:, c2] - r2).abs() <= 2.0 ** -24 * r2.abs() + room).all())


@pytest.mark.parametrize("kind", [k for k in KINDS if k[0] == "bf16"])
def test_attention_past_a_leading_token_without_values(M, kind):
    """The leading token's V codes are zeros, so the output is what the others add, exp(-lead) of the weight and less.
    A weight is rounded to fp16 by 2^-11 of itself or 2^-39 of the row's largest, 2^-37 in the kernel of many rows: at 19
    nats, 2^27.4, by 2^-11.6, at 17.5 nats, 2^25.2, by 2^-11.8."""
    dtype, D, N = kind
    host, dev, cache, q, (page, slot) = _led(M, np.random.default_rng(52), dtype, D, N, 19.0 if N <= 32 else 17.5)
    host[1][page, :, slot] = 0
    host[3][:] = 2.0 ** -6
    _check_led(M, dtype, D, N, host, dev, cache, q)


@pytest.mark.parametrize("D,N", [(64, 3), (64, 12), (128, 5), (128, 20)])
@pytest.mark.parametrize("lead", [12.0, 16.0, 20.0])
def test_fp32_attention_past_a_leading_token_without_values(M, D, N, lead):
    """The same in fp32, whose weights are two fp16 parts: each is whole to 2^-22 of itself down to 2^-29 (20 nats) of the
    row's largest.  The scores are exact but for their rounding: K holds powers of two or zeros, Q a few bits, so that one
    product of 12 to 20 nats and others of less than one are summed, each step truncated by 2^-23 of its sum: lead 2^-23 D / 16,
    and with the exponent's own rounding (lead + 6) 2^-23; each moves a weight by its size, numerator and denominator alike."""
    rng = np.random.default_rng(58)
    host, dev, cache, q, (page, slot) = _led(M, rng, "f32", D, N, lead)
    kc, vc, ks, vs, table = host
    kc[:] = OC.to_e4m3(np.exp2(rng.integers(-3, 1, kc.shape)) * rng.choice([-1.0, 0.0, 1.0], kc.shape))
    kc[..., 0] = 0
    kc[page, 0, slot] = 0
    kc[page, 0, slot, 0] = OC.to_e4m3(np.array(32.0))
    vc[page, :, slot] = 0
    vs[:] = 2.0 ** -6
    x = np.round(rng.standard_normal((1, N, 1, D)) * 8) / 32
    x[..., 0] = lead / 2  # times 32 times the scale, 2^-4
    q.copy_(torch.from_numpy(x.astype(np.float32)))
    for d, h in zip(dev, (kc, vc, ks.astype(np.float32), vs.astype(np.float32))):
        d.copy_(torch.from_numpy(h))
    got, _ = _attend(M, q, dev, cache, torch.tensor([150], dtype=torch.int32, device="cuda"), None, 0, 0.0625)
    o, _, S, _ = OC.cache_attn(_f64(q), *host, [150], [N], 0, 0.0625)
    w = 2.0 ** -22 + 2 * ((lead * D / 16 + 2 * (lead + 6)) * 2.0 ** -23) + (150 / 16 + 8) * 2.0 ** -23
    assert np.all(np.abs(_f64(got) - o) <= 2.0 ** -24 * np.abs(o) + w * S)


@pytest.mark.parametrize("dtype,rows", [("bf16", 200), ("bf16", 20), ("bf16", 1)])
def test_the_running_sums_of_very_long_histories(M, dtype, rows):
    """2^21 cached tokens, positive values, enough items that ranges are not split to fill the GPU.  A tensor core
    truncates each of its sums by up to 2^-23; a running sum takes in 2^17 tokens at most, 2^13 steps of 16: 2^-10."""
    B, D, page, kv = 300 if rows <= 32 else 148, 64, 128, 2 ** 21 - 5
    per = 2 ** 21 // page
    g = torch.Generator(device="cuda").manual_seed(53)
    k = (torch.randn((per, 1, page, D), generator=g, device="cuda")).to(torch.float8_e4m3fn)
    v = torch.randint(0x30, 0x38, (per, 1, page, D), generator=g, device="cuda", dtype=torch.uint8)  # 0.5 .. 0.94
    ks, vs = (torch.ones((per, 1), device="cuda") for _ in range(2))
    table = torch.arange(per, dtype=torch.int32, device="cuda").repeat(B, 1)
    cache = M.make_cache(k.view(torch.uint8), v, ks, vs, table)
    q = torch.randn((B, rows, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    o, lse = _attend(M, q, None, cache, torch.full((B,), kv, dtype=torch.int32, device="cuda"), None, 0, 0.125)
    for b in (0, B - 1):
        s = (q[b, :2, 0].double() @ k.reshape(-1, D)[:kv].double().T) * 0.125
        w = torch.softmax(s, -1)
        ref = sum(a @ x.double() for a, x in zip(w.split(2 ** 19, 1), v.view(torch.float8_e4m3fn).reshape(-1, D)[:kv].split(2 ** 19)))
        err = (o[b, :2, 0].double() - ref).abs()
        assert bool((err <= (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11 + 2.0 ** -13) * ref).all()), float((err / ref).max())
        assert float((lse[b, 0, :2].double() - torch.logsumexp(s, -1)).abs().max()) <= 2.0 ** -12


@pytest.mark.parametrize("kind", [("bf16", 64, 2), ("bf16", 64, 70), ("f32", 64, 2), ("f32", 64, 40), ("f32", 128, 2)])
@pytest.mark.parametrize("size", [25, 37])
def test_keys_and_values_beyond_the_small_scales(M, kind, size):
    """K and V of 10^25 and 10^37, which the append stores with scales of 2^76 and 2^116, under a Q that brings the
    scores back to ordinary ones."""
    dtype, D, N = kind
    rng = np.random.default_rng(54)
    host, dev, cache = _new_cache(M, rng, 8, 2, 32, D, 1, 6)
    k, _ = _tensor(rng, (1, 150, 2, D), dtype, fill=rng.standard_normal((1, 150, 2, D)) * 10.0 ** size)
    v, _ = _tensor(rng, (1, 150, 2, D), dtype, fill=rng.standard_normal((1, 150, 2, D)) * 10.0 ** size)
    M.cache_append(k, v, M.desc_of(k), cache, torch.zeros(1, dtype=torch.int32, device="cuda"))
    OC.append(host[0], host[2], host[4], _f64(k), [0], [150], np.zeros((1, 150, 2), bool))
    OC.append(host[1], host[3], host[4], _f64(v), [0], [150], None)
    for d, h in zip(dev[:4], host):
        assert np.array_equal(d.cpu().numpy(), h)
    x = rng.standard_normal((1, N, 2, D)) * 10.0 ** -size
    q, _ = _tensor(rng, x.shape, dtype, fill=x)
    got, lse = _attend(M, q, dev, cache, torch.tensor([150], dtype=torch.int32, device="cuda"), None, 0, 0.1)
    ref = OC.cache_attn(_f64(q), *host, [150], [N], 0, 0.1)
    _check_attention(dtype, D, 150, _f64(got), _f64(lse), ref, [N])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_calls_allocate_no_device_memory(M, dtype):
    """Nothing but the caller's arrays and workspace, in any form of the calls, once their kernels are loaded."""
    rng = np.random.default_rng(59)
    host, dev, cache = _new_cache(M, rng, 400, 2, 16, 64, 1, 300)
    q = [_tensor(rng, (1, n, 4, 64), dtype)[0] for n in (1, 12, 100)]
    k, _ = _tensor(rng, (1, 100, 2, 64), dtype)
    o = [torch.empty_like(x) for x in q]
    d = [M.desc_of(x) for x in q]
    size = max(M.cache_attn_workspace_size(x, cache) for x in d)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    held = torch.tensor([4700], dtype=torch.int32, device="cuda")
    start = torch.tensor([4600], dtype=torch.int32, device="cuda")
    lay, free = M.make_layout(_segments(M)), sorted(set(range(400)) - set(host[4].ravel().tolist()))
    kw = [dict()] + [dict(layout=lay, rotation=_params(M, (24, 20, 20), half, "none")[0]) for half in (False, True)]

    def everything():
        for x in kw:
            M.cache_append(k, k, M.desc_of(k), cache, start, **x)
        for x in kw[1:]:
            M.rotary(q[2], o[2], d[2], d[2], None, None, None, None, lay, x["rotation"])
        for x, y, z in zip(q, o, d):
            M.cache_attn(x, y, z, z, cache, held, 0.125, causal_block=1, workspace=ws, ws_bytes=size)
        M.cache_copy_pages(cache, [int(host[4][0, 0])], [free[0]])
    everything()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        everything()
    torch.cuda.synchronize()
    assert (torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]) == before


@pytest.mark.parametrize("case", [  # D, page, B, N, H, Hk, per, kv, q_len, causal
    (64, 32, 1, 300, 2, 2, 20, [600], None, 60), (128, 64, 2, 111, 6, 2, 9, [570, 111], [111, 40], 1),
    (128, 16, 1, 257, 1, 1, 20, [310], None, 0)])
def test_fp32_attention_of_many_rows(M, case):
    D, page, B, N, H, Hk, per, kv, ql, causal = case
    rng = np.random.default_rng(57)
    host, dev, cache = _new_cache(M, rng, B * per + 2, Hk, page, D, B, per)
    kc, vc, ks, vs, table = host
    kc[kc & 127 == 127], vc[vc & 127 == 127] = 3, 3
    vs[:] = np.exp2(rng.integers(-30, 10, vs.shape))
    ks *= 2.0 ** -3
    for d, h in zip(dev, (kc, vc, ks.astype(np.float32), vs.astype(np.float32))):
        d.copy_(torch.from_numpy(h))
    q, _ = _tensor(rng, (B, N, H, D), "f32", 4, 8)
    kt = torch.tensor(kv, dtype=torch.int32, device="cuda")
    qt = None if ql is None else torch.tensor(ql, dtype=torch.int32, device="cuda")
    got, lse = _attend(M, q, dev, cache, kt, qt, causal, 0.1)
    ql = [N] * B if ql is None else ql
    ref = OC.cache_attn(_f64(q), kc, vc, ks, vs, table, kv, ql, causal, 0.1)
    _check_attention("f32", D, max(kv), _f64(got), _f64(lse), ref, ql)


@pytest.mark.parametrize("D,N", [(64, 3), (64, 15), (128, 40)])
@pytest.mark.parametrize("size", [-60, -45, -8, 30])
@pytest.mark.parametrize("zeros", [False, True])
def test_fp32_sums_of_small_and_large_scales(M, D, N, size, zeros):
    """A row's reference holds log2 of V's scale and its sum the scale's inverse: of the lse, where the two meet, only
    the result may be rounded, and of an exponent only what the reference leaves of it.  With scores of almost 0: an
    exponent of up to 16 rounds by 2^-21 (times ln 2), ex2 by 2^-22, eight sums and products by 2^-24 each, the logarithm and
    its product by 2^-24 of the lse each."""
    for kv in (17, 28, 40, 75, 160):
        host, dev, cache, q, _ = _led(M, np.random.default_rng(60 + kv), "f32", D, N, 0.0, kv)
        q.mul_(2.0 ** -7)
        host[3][:] = 2.0 ** size
        if zeros:
            host[3][host[4][0, 1]] = 0.0
        _check_led(M, "f32", D, N, host, dev, cache, q, kv)
        _, lse = _attend(M, q, dev, cache, torch.tensor([kv], dtype=torch.int32, device="cuda"), None, 0, 0.0625)
        _, want, _, A = OC.cache_attn(_f64(q), *host, [kv], [N], 0, 0.0625)
        bound = 0.7 * 2.0 ** -21 + 2.0 ** -22 + 8 * 2.0 ** -24 + 2.0 ** -23 * np.abs(want) + (D / 16 + 2) * 2.0 ** -22 * A
        assert np.all(np.abs(_f64(lse) - want) <= bound), float((np.abs(_f64(lse) - want) / bound).max())
