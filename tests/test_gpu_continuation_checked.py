"""Page ids outside the cache are part of the continuation calls' contract (pages that are not there): the device-checked
build takes them as the regular one does, reports nothing and computes the same.  Each build runs in a child process of its
own; the ids are never used as addresses."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import sys
    import numpy as np, torch
    sys.path.insert(0, {root!r})
    from joint_video_audio_rope_b200 import mmdit as M
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    per, page, H, D = 70, 16, 2, 64
    k, v = (torch.zeros((150, H, page, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((150, H), device="cuda") for _ in range(2))
    table = torch.randperm(150, generator=g, device="cuda")[:2 * per].to(torch.int32).reshape(2, per)
    table[0, 3], table[0, 40], table[1, 7] = -1, 150, 2 ** 31 - 1
    c = M.make_cache(k, v, ks, vs, table)
    x, y = rand(2, 1100, H, D).bfloat16(), rand(2, 1100, H, D).bfloat16()
    start = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    held = start + 1100
    M.cache_append(x, y, M.desc_of(x), c, start)
    out = {{"k": k, "v": v, "ks": ks, "vs": vs}}
    for n in (1, 12, 100):
        q = rand(2, n, 4, D).bfloat16()
        o, lse = torch.full_like(q, 7.0), torch.full((2, 4, n), 7.0, device="cuda")
        d = M.desc_of(q)
        size = M.cache_attn_workspace_size(d, c)
        ws = torch.full((max(size, 1),), 255, dtype=torch.uint8, device="cuda")
        M.cache_attn(q, o, d, d, c, held, 0.125, lse=lse, workspace=ws, ws_bytes=size)
        torch.cuda.synchronize()
        out["o%d" % n], out["lse%d" % n] = o.float(), lse
        print("STATUS", M.device_status())
    np.savez({path!r}, **{{a: b.cpu().numpy() for a, b in out.items()}})
""")


def _run(lib, path):
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, path=path)], env=dict(os.environ, MMDIT_LIB=lib),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert [l for l in r.stdout.splitlines() if l.startswith("STATUS")] == ["STATUS 0"] * 3, r.stdout
    return dict(np.load(path))


def test_both_builds_take_ids_outside_the_cache(tmp_path):
    from joint_video_audio_rope_b200 import build
    a = _run(build.build(), str(tmp_path / "regular.npz"))
    b = _run(build.build(device_checks=True), str(tmp_path / "checked.npz"))
    assert a.keys() == b.keys()
    for name in a:
        assert np.array_equal(a[name], b[name]), name
        assert not (a[name] == 7.0).all() and np.isfinite(a[name]).all(), name
