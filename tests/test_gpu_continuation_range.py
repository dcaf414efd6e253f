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
