"""The continuation path of the attention layer as measurable cases: rotary positions, appending K and V to
a paged 8-bit cache, attention over that cache, and copying its pages.

With ``own`` false, ``run`` computes each operator in plain torch operations; with ``own`` true it makes the calls of
``joint_video_audio_rope_b200.mmdit`` that a user makes.  ``exact`` gives the same outputs in 64 bits from the
definitions:

rotary
    Channels form bands [t | h | w] of dim_t, dim_h, dim_w channels; channels behind them pass unchanged.  Pair i of
    a band of d channels is (2i, 2i + 1) or (i, i + d/2), turned by position * w_i and scaled by ``magnitude``; the
    transposed rotation is the gradient.  w_i = theta^(-2i/d), or scaled for longer sequences ("parts"): g w + (1 - g) w / f
    with g = clamp((trained w / 2 pi - slow) / (fast - slow), 0, 1).
cache_append
    Tokens start[b].. of item b go to pages of e4m3 codes with one scale per (page, head): 2^ceil(log2(amax / 448)) of
    the values, never below the scale that older tokens of the page already
    have; their codes are rounded again when it grows, and slots without a token stay as they were.
cache_attn
    o = softmax(scale q k^T) v over the first kv_len[b] cached tokens; with causal_block = c, query token i of
    item b sits at kv_len[b] - q_len[b] + i and sees the keys of its own and of earlier blocks of c tokens.
cache_copy_pages
    Pages src[i] are copied onto pages dst[i]: codes and scales of K and V.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
MIN_EXP = -60  # smallest scale of a cache page: 2^-60


# ------------------------------------------------------------------ cases

def _rotary(name, batch, n, hq, hk, d, dtype, pairing, dims, scaling, factor, transpose, far, seq):
    return dict(name=name, op="rotary", batch=batch, n=n, hq=hq, hk=hk, d=d, dtype=dtype, pairing=pairing,
                dim_t=dims[0], dim_h=dims[1], dim_w=dims[2], scaling=scaling, factor=factor, transpose=transpose,
                far=far, seq=seq)


def _append(name, batch, n, heads, d, page, dtype, rope, start):
    return dict(name=name, op="append", batch=batch, n=n, heads=heads, d=d, page=page, dtype=dtype, rope=rope,
                start=start)


def _attn(name, batch, nq, heads, kv_heads, d, page, dtype, kv, causal_block, ragged):
    return dict(name=name, op="attn", batch=batch, nq=nq, heads=heads, kv_heads=kv_heads, d=d, page=page, dtype=dtype,
                kv=kv, causal_block=causal_block, ragged=ragged)


def _copy(name, pairs, pages, heads, d, page):
    return dict(name=name, op="copy", pairs=pairs, pages=pages, heads=heads, d=d, page=page)


def listed():
    return [
        # one audio token of eight sequences that are generated side by side, half of each head turned
        _rotary("rotary_audio_token", 8, 1, 24, 8, 128, "bf16", "half", (64, 0, 0), "parts", 4.0, False, 100000, "audio"),
        # the gradient of Q and K of a 480p layer: 21x30x52 video, 218 audio and 512 text tokens
        _rotary("rotary_480p_grad", 1, 33490, 24, 24, 128, "bf16", "interleaved", (44, 42, 42), "parts", 2.0, True, 0, "clip"),
        # K and V of that audio token into the caches of the eight sequences
        _append("append_audio_token", 8, 1, 24, 128, 16, "bf16", "none", 200),
        # the conditioning clip's K and V, cached once before its continuation is generated; K turned on the way
        _append("append_480p_clip", 1, 32760, 24, 128, 64, "bf16", "interleaved", 0),
        # five more frames of two small fp32 sequences that end inside a page
        _append("append_frames_f32", 2, 7800, 12, 64, 64, "f32", "half", 1571),
        # one audio token over the audio history
        _attn("attn_audio_token", 4, 1, 24, 24, 128, 16, "bf16", 218, 1, True),
        # one token over the history of a 720p clip, K and V heads shared by three query heads
        _attn("attn_token_720p", 1, 1, 24, 8, 128, 64, "bf16", 75600, 0, False),
        # the audio tokens of one latent frame, fp32, over a 480p history
        _attn("attn_audio_frame_f32", 2, 11, 12, 12, 64, 32, "f32", 32760, 1, True),
        # all 218 audio tokens of a clip over its 480p video history
        _attn("attn_audio_clip", 1, 218, 24, 24, 128, 128, "bf16", 32760, 0, False),
        # three new 480p frames over a history of 24 frames, a frame seeing itself and the earlier ones
        _attn("attn_frames_480p", 1, 4680, 24, 24, 128, 64, "bf16", 37440, 1560, False),
        # forking a sequence to eight continuations: its tail page, eight times
        _copy("copy_fork_tail", 8, 64, 24, 128, 16),
        # closing the holes that finished sequences left
        _copy("copy_compact", 400, 1000, 24, 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attn", "attn", "copy"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotary":
        n, batch = _log(rng, 1, 16000), rng.randint(1, 2)
        hk = rng.choice([1, 2, 4, 8])
        seq = rng.choice(["audio", "clip"])
        pairing = rng.choice(["interleaved", "half"])
        if seq == "audio":
            dims = (rng.choice([d // 4, d // 2, d]), 0, 0)
        else:
            dh = 2 * rng.randint(2, d // 6)
            dims = (d - 2 * dh - 2 * rng.randint(0, 3), dh, dh)
        c = _rotary("", batch, n, hk * rng.choice([1, 2, 3]), hk, d, dtype, pairing, dims,
                    rng.choice(["none", "parts"]), round(rng.uniform(1.5, 8.0), 2), rng.random() < 0.5,
                    rng.choice([0, 1000, 1000000]), seq)
    elif op == "append":
        n, batch = _log(rng, 1, 8000), rng.randint(1, 3)
        c = _append("", batch, n, rng.choice([2, 6, 12, 24]), d, page, dtype,
                    rng.choice(["none", "interleaved", "half"]), rng.randint(0, 3000))
    elif op == "attn":
        nq, kv_heads = _log(rng, 1, 2500), rng.choice([2, 4, 8])
        c = _attn("", rng.randint(1, 3), nq, kv_heads * rng.choice([1, 2, 3]), kv_heads, d, page,
                  "f32" if dtype == "f32" and nq <= 64 else "bf16", max(nq, _log(rng, 30, 30000)),
                  rng.choice([0, 1, 60, 1560]), rng.random() < 0.5)
    else:
        pairs = _log(rng, 1, 300)
        c = _copy("", pairs, 2 * pairs + rng.randint(3, 200), rng.choice([2, 8, 24]), d, page)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _segments(case):
    """The sequence that the case's tokens are a part of, as layout segments: (kind, tokens, T, H, W, t0, t_num, t_den)."""
    if case["op"] == "rotary" and case["seq"] == "audio":
        return [("audio", case["far"] + case["n"] + 300, 0, 0, 0, 0, 21, 218)]
    if case["op"] == "rotary":
        frames = case["n"] // 1560
        if frames == 0:
            return [("audio", case["n"], 0, 0, 0, case["far"], 21, 218)]
        rest = case["n"] - 1560 * frames
        audio = min(rest, 218)
        return [("video", 1560 * frames, frames, 30, 52, case["far"] - 1, 1, 1),
                ("audio", audio, 0, 0, 0, case["far"], 21, 218), ("text", rest - audio, 0, 0, 0, 0, 1, 1)]
    frames = -(-(case["start"] + case["n"] + 40) // 1560)
    return [("video", 1560 * frames, frames, 30, 52, -2, 1, 1)]


def _params(case):
    """theta, dims, pairing, scaling, factors, trained extents, fast, slow, magnitude of the case's rotation."""
    if case["op"] == "rotary":
        scaled = case["scaling"] == "parts"
        return dict(theta=10000.0, dims=(case["dim_t"], case["dim_h"], case["dim_w"]), pairing=case["pairing"], scaled=scaled,
                    factors=(case["factor"], 2.0, 2.0), trained=(21.0, 30.0, 52.0), fast=4.0, slow=0.25,
                    magnitude=0.1 * math.log(case["factor"]) + 1.0 if scaled else 1.0)
    dh = 2 * (case["d"] // 6)
    return dict(theta=10000.0, dims=(case["d"] - 2 * dh, dh, dh), pairing=case["rope"], scaled=False, factors=(1.0, 1.0, 1.0),
                trained=(0.0, 0.0, 0.0), fast=4.0, slow=0.25, magnitude=1.0)


def _cache(g, n_pages, heads, page, d):
    """A cache whose pages hold values of different sizes: e4m3 codes and the scales that they were rounded with."""
    codes, scales = [], []
    for _ in range(2):
        size = torch.exp2(torch.randint(-2, 3, (n_pages, heads, 1, 1), generator=g, device=DEV).float())
        x = torch.randn((n_pages, heads, page, d), generator=g, device=DEV)
        s = x.abs().amax((2, 3), keepdim=True) / E4M3_MAX
        codes.append((x / s).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn))
        scales.append((s * size / 2).reshape(n_pages, heads).contiguous())
        del x
    return dict(k=codes[0], v=codes[1], k_scale=scales[0], v_scale=scales[1])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    st = dict(case=dict(case))
    if case["op"] == "rotary":
        dt = _dtype(case)
        for name, h in (("q", case["hq"]), ("k", case["hk"])):
            st[name] = torch.randn((case["batch"], case["n"], h, case["d"]), generator=g, device=DEV).to(dt)
            st[name + "_out"] = torch.zeros_like(st[name])
        ahead = case["far"] if case["seq"] == "audio" else 0
        st["first"] = ahead + torch.randint(0, 300 if case["seq"] == "audio" else 1, (case["batch"],), generator=g, device=DEV,
                                            dtype=torch.int32)
    elif case["op"] == "append":
        b, n, page = case["batch"], case["n"], case["page"]
        st["start"] = case["start"] + torch.randint(0, 40 if case["start"] else 1, (b,), generator=g, device=DEV, dtype=torch.int32)
        per = -(-(case["start"] + 40 + n) // page)
        st["cache"] = _cache(g, b * per + 3, case["heads"], page, case["d"])
        for name in ("k_scale", "v_scale"):  # the scales that an append leaves
            st["cache"][name] = torch.exp2(torch.ceil(torch.log2(st["cache"][name])))
        st["table"] = torch.randperm(b * per + 3, generator=g, device=DEV)[: b * per].to(torch.int32).reshape(b, per)
        st["count"] = torch.randint(max(1, n - n // 8), n + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
        st["count"][0] = n
        size = torch.exp2(torch.randint(-2, 3, (b, n, 1, 1), generator=g, device=DEV).float())
        for name in ("k_new", "v_new"):
            st[name] = (torch.randn((b, n, case["heads"], case["d"]), generator=g, device=DEV) * size).to(_dtype(case))
    elif case["op"] == "attn":
        b, page, kv, nq = case["batch"], case["page"], case["kv"], case["nq"]
        per = -(-kv // page)
        st["cache"] = _cache(g, b * per + 3, case["kv_heads"], page, case["d"])
        st["table"] = torch.randperm(b * per + 3, generator=g, device=DEV)[: b * per].to(torch.int32).reshape(b, per)
        lo = kv // 3 if case["ragged"] else max(1, kv - 7)
        st["kv_len"] = torch.randint(lo, kv + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
        st["kv_len"][0] = kv
        lo = max(1, nq // 2) if case["ragged"] else nq
        st["q_len"] = torch.minimum(torch.randint(lo, nq + 1, (b,), generator=g, device=DEV, dtype=torch.int32), st["kv_len"])
        st["q_len"][0] = nq
        st["q"] = torch.randn((b, nq, case["heads"], case["d"]), generator=g, device=DEV).to(_dtype(case))
        st["o"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((b, case["heads"], nq), device=DEV)
    else:
        st["cache"] = _cache(g, case["pages"], case["heads"], case["page"], case["d"])
        cpu = torch.Generator()
        cpu.manual_seed(int(seed))
        ids = torch.randperm(case["pages"], generator=cpu)
        fork = case["pairs"] <= 8
        st["src"] = ids[:1].repeat(case["pairs"]).tolist() if fork else ids[: case["pairs"]].tolist()
        st["dst"] = ids[case["pairs"]: 2 * case["pairs"]].tolist()
    return st


# ------------------------------------------------------------------ plain forms

def _positions(segments, index):
    """(t, h, w) in 64 bits of the tokens with these indices in the sequence; behind its end: (0, 0, 0)."""
    i = index.to(torch.float64)
    pos = [torch.zeros_like(i) for _ in range(3)]
    at = 0
    for kind, n, T, H, W, t0, num, den in segments:
        inside = (index >= at) & (index < at + n)
        j = i - at
        if kind == "video":
            t = torch.floor(j / (H * W))
            r = j - t * (H * W)
            h = torch.floor(r / W)
            found = (t + t0, h, r - h * W)
        elif kind == "audio":
            found = (t0 + j * num / den, 0.0 * j, 0.0 * j)
        else:
            found = (0.0 * j, 0.0 * j, 0.0 * j)
        pos = [torch.where(inside, f, p) for f, p in zip(found, pos)]
        at += n
    return pos


def _pairs(p):
    """For each pair of turned channels: its first and second channel, axis and frequency."""
    first, second, axis, freq = [], [], [], []
    at = 0
    for a, dim in enumerate(p["dims"]):
        for i in range(dim // 2):
            w = p["theta"] ** (-2.0 * i / dim)
            if p["scaled"]:
                turns = p["trained"][a] * w / (2 * math.pi)
                g = min(1.0, max(0.0, (turns - p["slow"]) / (p["fast"] - p["slow"])))
                w = g * w + (1.0 - g) * w / p["factors"][a]
            first.append(at + (2 * i if p["pairing"] == "interleaved" else i))
            second.append(at + (2 * i + 1 if p["pairing"] == "interleaved" else i + dim // 2))
            axis.append(a)
            freq.append(w)
        at += dim
    return first, second, axis, freq


def _turn(x, segments, p, index, transpose):
    """x [B, N, H, d] in 32 bits, turned by the positions of the tokens `index` [B, N]."""
    first, second, axis, freq = _pairs(p)
    first, second, axis = (torch.tensor(v, device=x.device) for v in (first, second, axis))
    pos = torch.stack(_positions(segments, index), -1)
    angle = pos[..., axis] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    c = (torch.cos(angle) * p["magnitude"]).float()[:, :, None]
    s = (torch.sin(angle) * (-p["magnitude"] if transpose else p["magnitude"])).float()[:, :, None]
    a, b = x[..., first], x[..., second]
    y = x.clone()
    y[..., first] = a * c - b * s
    y[..., second] = a * s + b * c
    return y


def _fit(amax):
    """The power of two s with amax / s in (224, 448], and 2^-60 at least."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e, e - 1) - 8
    return torch.ldexp(torch.ones_like(amax), torch.clamp(e, min=MIN_EXP))


def _store(x, codes, scale, table, start, count, page):
    """Values x [B, N, H, d] of the tokens start[b].. into the pages of one half of the cache."""
    b, n, h = x.shape[:3]
    per = table.shape[1]
    token = torch.arange(n, device=x.device)[None, :]
    index = (start[:, None] + token).long()
    live = token < count[:, None]
    at = index // page
    last = start + count - 1
    pages = torch.arange(per, device=x.device)[None, :]
    touched = (pages >= (start // page)[:, None]) & (pages <= (last // page)[:, None]) & (count > 0)[:, None]
    item = torch.arange(b, device=x.device)[:, None].expand(b, n)
    rows = (item * per + at)[live]
    amax = torch.zeros((b * per, h), device=x.device)
    amax.scatter_reduce_(0, rows[:, None].expand(-1, h), x.abs().amax(-1)[live], "amax")
    s = _fit(amax)
    ids = table.reshape(-1).long()
    older = (pages == (start // page)[:, None]) & (start % page > 0)[:, None]
    before = scale[ids]
    s = torch.where(older.reshape(-1, 1), torch.maximum(s, before), s)
    grown = (older & touched).reshape(-1, 1) & (s > before)
    again = grown.any(1).nonzero().reshape(-1)
    slot = torch.arange(page, device=x.device)
    held = (slot[None, :] < (start % page)[:, None])[torch.div(again, per, rounding_mode="floor")].reshape(-1, 1, page, 1)
    old = codes[ids[again]].view(torch.uint8)
    small = (old.view(torch.float8_e4m3fn).float() * (before[again] / s[again])[:, :, None, None]).to(torch.float8_e4m3fn)
    codes.view(torch.uint8)[ids[again]] = torch.where(held, small.view(torch.uint8), old)
    keep = touched.reshape(-1)
    scale[ids[keep]] = s[keep]
    y = (x[live] / s[rows][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    codes.view(torch.uint8)[ids[rows], :, (index % page)[live]] = y.view(torch.uint8)


def _attend(q, cache, table, kv_len, q_len, causal_block, o, lse):
    b, nq, h, d = q.shape
    hk, page = cache["k"].shape[1], cache["k"].shape[2]
    n = table.shape[1] * page
    ids = table.long()
    key = torch.arange(n, device=q.device)
    live = key[None, :] < kv_len[:, None]
    k = (cache["k"][ids].float() * cache["k_scale"][ids][..., None, None]).transpose(1, 2).reshape(b, hk, n, d)
    v = (cache["v"][ids].float() * cache["v_scale"][ids][..., None, None]).transpose(1, 2).reshape(b, hk, n, d)
    v = torch.where(live[:, None, :, None], v, 0.0)
    rows = q.float().reshape(b, nq, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, h // hk * nq, d)
    s = torch.matmul(rows, k.transpose(2, 3)).reshape(b, hk, h // hk, nq, n)
    s *= 1.0 / math.sqrt(d)
    seen = live[:, None, :]
    if causal_block:
        at = (kv_len - q_len)[:, None] + torch.arange(nq, device=q.device)[None, :]
        end = (torch.div(at, causal_block, rounding_mode="floor") + 1) * causal_block
        seen = seen & (key[None, None, :] < end[:, :, None])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s -= torch.where(m == -math.inf, 0.0, m)
    s.exp_()
    l = s.sum(-1)
    y = torch.matmul(s.reshape(b, hk, h // hk * nq, n), v).reshape(b, hk, h // hk, nq, d)
    y = torch.where(l[..., None] > 0, y / l[..., None], 0.0)
    y = y.reshape(b, h, nq, d).transpose(1, 2)
    r = (m[..., 0] + torch.log(l)).reshape(b, h, nq)
    valid = torch.arange(nq, device=q.device)[None, :] < q_len[:, None]
    o.copy_(torch.where(valid[:, :, None, None], y.to(o.dtype), o))
    lse.copy_(torch.where(valid[:, None, :], r, lse))


def _plain(st):
    case = st["case"]
    if case["op"] == "rotary":
        token = torch.arange(case["n"], device=DEV)[None, :]
        index = st["first"][:, None].long() + token
        for name in ("q", "k"):
            y = _turn(st[name].float(), _segments(case), _params(case), index, case["transpose"])
            st[name + "_out"].copy_(y)
        return st["q_out"], st["k_out"]
    c = st["cache"]
    if case["op"] == "append":
        k = st["k_new"].float()
        if case["rope"] != "none":
            index = st["start"][:, None].long() + torch.arange(case["n"], device=DEV)[None, :]
            k = _turn(k, _segments(case), _params(case), index, False)
        _store(k, c["k"], c["k_scale"], st["table"], st["start"], st["count"], case["page"])
        _store(st["v_new"].float(), c["v"], c["v_scale"], st["table"], st["start"], st["count"], case["page"])
        return c["k"], c["v"], c["k_scale"], c["v_scale"]
    if case["op"] == "attn":
        _attend(st["q"], c, st["table"], st["kv_len"], st["q_len"], case["causal_block"], st["o"], st["lse"])
        return st["o"], st["lse"]
    src, dst = (torch.tensor(st[x], device=DEV) for x in ("src", "dst"))
    for half in (c["k"].view(torch.uint8), c["v"].view(torch.uint8), c["k_scale"], c["v_scale"]):
        half[dst] = half[src]
    return c["k"], c["v"], c["k_scale"], c["v_scale"]


# ------------------------------------------------------------------ the framework's calls

def _plan(st):
    """What a user's program keeps from call to call: descriptors, layout, cache handle, workspace."""
    from joint_video_audio_rope_b200 import mmdit as M
    case, plan = st["case"], {"M": M}
    if case["op"] in ("rotary", "append"):
        kinds = {"video": M.SEG_VIDEO, "audio": M.SEG_AUDIO, "text": M.SEG_TEXT}
        keys = ("n_tokens", "T", "H", "W", "t0", "t_num", "t_den")
        plan["layout"] = M.make_layout([dict(zip(keys, s[1:]), kind=kinds[s[0]]) for s in _segments(case)])
        p = _params(case)
        plan["rotation"] = M.rotary_params(
            p["theta"], *p["dims"], pairing=M.PAIR_HALF if p["pairing"] == "half" else M.PAIR_INTERLEAVED,
            scaling=M.SCALE_PARTS if p["scaled"] else M.SCALE_NONE, factors=p["factors"], trained=p["trained"],
            beta_fast=p["fast"], beta_slow=p["slow"], magnitude=p["magnitude"])
    if "cache" in st:
        c = st["cache"]
        plan["cache"] = M.make_cache(c["k"], c["v"], c["k_scale"], c["v_scale"], st.get("table"))
    for name in ("q", "k", "q_out", "k_out", "k_new", "o"):
        if name in st:
            plan[name] = M.desc_of(st[name])
    if case["op"] == "attn":
        n = M.cache_attn_workspace_size(plan["q"], plan["cache"])
        plan["workspace"] = (torch.empty(max(n, 1), dtype=torch.uint8, device=DEV), n)
    return plan


def _framework(st):
    case = st["case"]
    if "plan" not in st:
        st["plan"] = _plan(st)
    plan = st["plan"]
    M = plan["M"]
    if case["op"] == "rotary":
        M.rotary(st["q"], st["q_out"], plan["q"], plan["q_out"], st["k"], st["k_out"], plan["k"], plan["k_out"],
                 plan["layout"], plan["rotation"], first=st["first"], transpose=case["transpose"])
        return st["q_out"], st["k_out"]
    c = st["cache"]
    if case["op"] == "append":
        turn = case["rope"] != "none"
        M.cache_append(st["k_new"], st["v_new"], plan["k_new"], plan["cache"], st["start"], count=st["count"],
                       layout=plan["layout"] if turn else None, rotation=plan["rotation"] if turn else None)
    elif case["op"] == "attn":
        ws, n = plan["workspace"]
        M.cache_attn(st["q"], st["o"], plan["q"], plan["o"], plan["cache"], st["kv_len"], 1.0 / math.sqrt(case["d"]),
                     q_len=st["q_len"], causal_block=case["causal_block"], lse=st["lse"], workspace=ws, ws_bytes=n)
        return st["o"], st["lse"]
    else:
        M.cache_copy_pages(plan["cache"], st["src"], st["dst"])
    return c["k"], c["v"], c["k_scale"], c["v_scale"]


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ work

def work(case):
    e = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "rotary":
        values = case["batch"] * case["n"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 2 * values * e, "flops": 3 * values}
    if case["op"] == "append":
        values = 2 * case["batch"] * case["n"] * case["heads"] * case["d"]
        scales = 2 * case["batch"] * case["heads"] * -(-case["n"] // case["page"])
        return {"bytes": values * (e + 1) + 4 * scales, "flops": (3 if case["rope"] == "none" else 5) * values}
    if case["op"] == "attn":
        b, nq, kv, cb = case["batch"], case["nq"], case["kv"], case["causal_block"]
        share = 2 / 3 if case["ragged"] else 1.0  # mean length of the further items
        items = 1 + (b - 1) * share
        held = 2 * items * kv * case["kv_heads"] * (case["d"] + 4 / case["page"])
        seen = kv
        if cb:  # the mean over the queries of the keys that one sees
            at = range(kv - nq, kv)
            seen = sum(min(kv, (p // cb + 1) * cb) for p in at) / nq
        queries = nq * (1 + (b - 1) * (0.75 if case["ragged"] else 1.0))
        return {"bytes": held + 2 * queries * case["heads"] * case["d"] * e + 4 * queries * case["heads"],
                "flops": 4 * queries * seen * (items / b) * case["heads"] * case["d"]}
    values = 2 * case["heads"] * case["page"] * case["d"] + 8 * case["heads"]
    return {"bytes": (2 if case["pairs"] > 8 else 1) * case["pairs"] * values, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_turn(x, case, index, transpose):
    """x [N, H, d] in 64 bits, by complex multiplication."""
    p = _params(case)
    y = x.clone()
    where = torch.zeros((index.shape[0], 3), dtype=torch.float64, device=x.device)
    begin = 0
    for kind, n, T, H, W, t0, num, den in _segments(case):
        j = index - begin
        here = (j >= 0) & (j < n)
        if kind == "video":
            found = torch.stack([t0 + j // (H * W), j // W % H, j % W], 1).double()
        elif kind == "audio":
            found = torch.stack([t0 + (j * num).double() / den, 0.0 * j, 0.0 * j], 1)
        else:
            found = torch.zeros_like(where)
        where[here] = found[here]
        begin += n
    begin = 0
    for a, dim in enumerate(p["dims"]):
        if dim == 0:
            continue
        i = torch.arange(dim // 2, device=x.device, dtype=torch.float64)
        w = torch.exp(-2.0 * i / dim * math.log(p["theta"]))
        if p["scaled"]:
            g = ((p["trained"][a] * w / (2.0 * math.pi) - p["slow"]) / (p["fast"] - p["slow"])).clamp(0.0, 1.0)
            w = w * (g + (1.0 - g) / p["factors"][a])
        band = x[..., begin:begin + dim]
        half = p["pairing"] == "half"
        re, im = (band[..., : dim // 2], band[..., dim // 2:]) if half else (band[..., 0::2], band[..., 1::2])
        turn = torch.polar(torch.full_like(w, p["magnitude"]).expand(index.shape[0], -1).contiguous(), where[:, a:a + 1] * w)
        z = torch.complex(re.contiguous(), im.contiguous()) * (turn.conj() if transpose else turn)[:, None, :]
        if half:
            y[..., begin:begin + dim // 2], y[..., begin + dim // 2:begin + dim] = z.real, z.imag
        else:
            y[..., begin:begin + dim:2], y[..., begin + 1:begin + dim:2] = z.real, z.imag
        begin += dim
    return y


def _exact_e4m3(x):
    """Values in 64 bits to the nearest e4m3 value, ties to the even one."""
    a = x.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        out = []
        for name in ("q", "k"):
            y = torch.empty(st[name].shape, dtype=torch.float64, device=DEV)
            for b in range(case["batch"]):
                index = int(st["first"][b]) + torch.arange(case["n"], device=DEV)
                y[b] = _exact_turn(st[name][b].double(), case, index, case["transpose"])
            out.append(y)
        return tuple(out)
    c = st["cache"]
    if case["op"] == "append":
        out = []
        for half in ("k", "v"):
            codes, scales = c[half].to(torch.float64), c[half + "_scale"].double()
            for b in range(case["batch"]):
                start, count, page = int(st["start"][b]), int(st["count"][b]), case["page"]
                x = st[half + "_new"][b, :count].double()
                if half == "k" and case["rope"] != "none":
                    x = _exact_turn(x, case, start + torch.arange(count, device=DEV), False)
                for j in range(start // page, (start + count - 1) // page + 1):
                    at, lo, hi = int(st["table"][b, j]), max(start, j * page), min(start + count, (j + 1) * page)
                    part = x[lo - start:hi - start].transpose(0, 1)
                    s = torch.exp2(torch.ceil(torch.log2((part.abs().amax((1, 2)) / E4M3_MAX).clamp(min=2.0 ** MIN_EXP))))
                    if lo > j * page:
                        s = torch.maximum(s, scales[at])
                        ratio = (scales[at] / s)[:, None, None]
                        old = codes[at, :, : lo - j * page]
                        codes[at, :, : lo - j * page] = torch.where(ratio < 1, _exact_e4m3(old * ratio), old)
                    codes[at, :, lo - j * page:hi - j * page] = _exact_e4m3(part / s[:, None, None])
                    scales[at] = s
            out.append((codes, scales))
        return out[0][0], out[1][0], out[0][1], out[1][1]
    if case["op"] == "attn":
        o, lse = st["o"].double(), st["lse"].double()
        group = case["heads"] // case["kv_heads"]
        for b in range(case["batch"]):
            n, nq = int(st["kv_len"][b]), int(st["q_len"][b])
            ids = st["table"][b].long()
            key = torch.arange(n, device=DEV)
            end = torch.full((nq,), n, device=DEV)
            if case["causal_block"]:
                cb = case["causal_block"]
                end = ((n - nq + torch.arange(nq, device=DEV)) // cb + 1) * cb
            for h in range(case["heads"]):
                kh = h // group
                k, v = ((c[x][ids, kh].double() * c[x + "_scale"][ids, kh].double()[:, None, None]).reshape(-1, case["d"])[:n]
                        for x in ("k", "v"))
                s = (st["q"][b, :nq, h].double() @ k.T) / math.sqrt(case["d"])
                s = torch.where(key[None, :] < end[:, None], s, -math.inf)
                lse[b, h, :nq] = torch.logsumexp(s, 1)
                o[b, :nq, h] = torch.exp(s - lse[b, h, :nq, None]) @ v
        return o, lse
    out = [c["k"].to(torch.float64), c["v"].to(torch.float64), c["k_scale"].double(), c["v_scale"].double()]
    for s, t in zip(st["src"], st["dst"]):
        for x in out:
            x[t] = x[s]
    return tuple(out)
