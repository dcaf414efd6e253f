"""Attention over the cache after a bounded wait ran out: while the device error word is set, attention kernels skip their
work, so no form of the call writes its outputs (a merge of key ranges that were never written would give garbage);
after the word is read, the same call computes as before."""
import numpy as np
import pytest

from test_gpu_continuation import M, _attend, _new_cache, _tensor  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture()
def clear_flag(M):  # noqa: F811
    yield
    M.device_status()  # whatever happened, leave the device error word clear


@pytest.mark.parametrize("dtype,N,per,split", [("bf16", 1, 8, False), ("bf16", 1, 120, True), ("bf16", 100, 8, False),
                                               ("bf16", 100, 120, True), ("f32", 20, 8, False), ("f32", 20, 120, True)])
def test_calls_after_a_timeout_leave_their_outputs(M, clear_flag, dtype, N, per, split):  # noqa: F811
    rng = np.random.default_rng(61)
    host, dev, cache = _new_cache(M, rng, per, 2, 16, 64, 1, per)
    for d, h in zip(dev, host[:2]):
        h[h & 127 == 127] = 3
        d.copy_(torch.from_numpy(h))
    q, _ = _tensor(rng, (1, N, 2, 64), dtype)
    assert (M.cache_attn_workspace_size(M.desc_of(q), cache) > 0) == split
    kv = torch.tensor([16 * per - 3], dtype=torch.int32, device="cuda")
    want, lse = _attend(M, q, dev, cache, kv, None, 0, 0.01)
    assert M.device_status() == M.OK
    waited = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.selftest_wait_timeout(50, waited)
    torch.cuda.synchronize()
    assert int(waited.item()) == 1
    got, none = _attend(M, q, dev, cache, kv, None, 0, 0.01)
    torch.cuda.synchronize()
    assert bool((got == 7.0).all()) and bool((none == 7.0).all())
    assert M.device_status() == M.ETIMEOUT
    got, again = _attend(M, q, dev, cache, kv, None, 0, 0.01)
    assert torch.equal(got, want) and torch.equal(again, lse)
    assert M.device_status() == M.OK
