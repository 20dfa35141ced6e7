"""Workloads of the 4-bit paged cache and of rotary positions with several axes.

``run`` computes an operator in plain torch (``own`` false) or through the package's calls
(``own`` true).  A case is one operator at one size:

* ``axes``    rotates q- or k-shaped rows whose tokens have a position on each of several axes;
* ``append4`` rotates the new tokens of a ragged batch, writes them to 4-bit pages and reads the touched pages'
  tokens back as bf16 (the values that the codes stand for);
* ``attend4`` attends from the last tokens of each sequence to its 4-bit pages.

A 4-bit value is code * group scale * page scale: codes of 1 sign, 2 exponent and 1 mantissa bit (0, 1/2, 1, 3/2, 2,
3, 4, 6), one e4m3 scale per 16 neighbouring elements of a token's head, one power of two per page and kv head.

Sequence lengths come from the case alone (``_lengths``), values from the seed.
"""
import math

import torch

own = False

_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_TOP = 6.0 * 448.0  # largest code times largest group scale
_MIN_EXP = -64


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one step's keys after an image in the prompt: latency only
        _axes("axes_step", tokens=8, heads=40, d=128, rot=128, interleaved=False, order="sections", own_freqs=False, pairs="16,24,24", scaling="none"),
        # the queries of a prompt that holds a video (time, height, width), axes taken in turns
        _axes("axes_video_cycled", tokens=8192, heads=32, d=128, rot=128, interleaved=False, order="cycled", own_freqs=False, pairs="24,20,20", scaling="none"),
        # patches of images, height and width with frequencies of their own, odd token count
        _axes("axes_image_own", tokens=20011, heads=16, d=64, rot=64, interleaved=True, order="sections", own_freqs=True, pairs="16,16", scaling="linear"),
        # one decode step of a batch: one token a sequence, most into pages that hold earlier ones, queries rotated along
        _append("append4_step", batch=64, q_lo=1, q_hi=1, kv_lo=1000, kv_hi=32768, hq=32, hkv=8, d=128, page=64, scaling="none", pairs=""),
        # prompts of uneven lengths with images in them, one of them a continuation
        _append("append4_prompt_axes", batch=5, q_lo=301, q_hi=4097, kv_lo=4100, kv_hi=9001, hq=32, hkv=8, d=128, page=64, scaling="bands", pairs="24,20,20"),
        # one short sequence, one token: latency only
        _attend("decode4_single_short", batch=1, q_lo=1, q_hi=1, kv_lo=129, kv_hi=129, hq=8, hkv=2, d=64, page=16, window=0, sinks=0),
        # the 32K decode batch, all of it resident
        _attend("decode4_batch_32k", batch=8, q_lo=1, q_hi=1, kv_lo=32768, kv_hi=32768, hq=32, hkv=8, d=128, page=64, window=0, sinks=0),
        # one 512K sequence: all parallelism from the length
        _attend("decode4_one_512k", batch=1, q_lo=1, q_hi=1, kv_lo=524288, kv_hi=524288, hq=40, hkv=8, d=128, page=64, window=0, sinks=0),
        # a ragged batch of layers with a window and sinks
        _attend("decode4_window_sinks", batch=61, q_lo=1, q_hi=1, kv_lo=3, kv_hi=40000, hq=32, hkv=8, d=128, page=32, window=4096, sinks=4),
        # several tokens a sequence (drafts to verify) over medium contexts
        _attend("verify4_ragged", batch=16, q_lo=2, q_hi=7, kv_lo=500, kv_hi=16000, hq=24, hkv=8, d=64, page=16, window=0, sinks=0),
        # a chunk of a long prompt
        _attend("chunk4_32k", batch=1, q_lo=2048, q_hi=2048, kv_lo=32768, kv_hi=32768, hq=32, hkv=8, d=128, page=64, window=0, sinks=0),
        # uneven prompts with a window and sinks
        _attend("prompt4_ragged_window", batch=6, q_lo=65, q_hi=3001, kv_lo=2000, kv_hi=7003, hq=40, hkv=8, d=128, page=32, window=1024, sinks=16),
    ]


def _axes(name, **kw):
    return {"name": name, "op": "axes", **kw}


def _append(name, **kw):
    return {"name": name, "op": "append4", "order": "cycled", "own_freqs": False, "interleaved": False, **kw}


def _attend(name, **kw):
    return {"name": name, "op": "attend4", **kw}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, pairs, axes):
    """`pairs` as `axes` whole numbers above zero."""
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))


def draw(rng):
    op = rng.choice(["axes", "append4", "attend4", "attend4", "attend4"])
    d = rng.choice([64, 128, 128])
    scaling = rng.choice(["none", "linear", "bands"])
    kind = {"order": rng.choice(["sections", "cycled"]), "own_freqs": rng.random() < 0.3, "interleaved": rng.random() < 0.5, "scaling": scaling}
    if op == "axes":
        rot = rng.choice([d, d, d // 2, d - 16])
        return {"op": op, "tokens": _log(rng, 1, 8000), "heads": rng.randint(1, 40), "d": d, "rot": rot,
                "pairs": _split(rng, rot // 2, rng.randint(2, 4)), **kind}
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append4":
        batch = _log(rng, 1, 64)
        hi = 1 if rng.random() < 0.4 else max(1, _log(rng, 1, 8000 // batch))
        kv_hi = hi + _log(rng, 1, 8000)
        return {"op": op, "batch": batch, "q_lo": rng.randint(1, hi), "q_hi": hi, "kv_lo": max(hi, kv_hi // 3), "kv_hi": kv_hi,
                "hq": hq, "hkv": hkv, "d": d, "page": page, "pairs": _split(rng, d // 2, rng.randint(2, 4)) if rng.random() < 0.5 else "", **kind}
    kind = rng.choice(["decode", "decode", "verify", "prompt", "prompt"])
    if kind == "prompt":
        batch = rng.randint(1, 4)
        hi = _log(rng, 30, 3000 // batch)
        kv_hi = hi + (0 if rng.random() < 0.4 else _log(rng, 1, 6000))
    else:
        batch = _log(rng, 1, 64)
        hi = 1 if kind == "decode" else rng.randint(2, 16)
        kv_hi = hi + _log(rng, 1, 1500000 // batch // hkv)
    windowed = rng.random() < 0.4
    return {"op": op, "batch": batch, "q_lo": max(1, hi // 2), "q_hi": hi, "kv_lo": max(hi, kv_hi // 4), "kv_hi": kv_hi, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "window": _log(rng, 1, 5000) if windowed else 0,
            "sinks": rng.choice([0, 1, 4, 33]) if windowed else 0}


def _spread(lo, hi, n, at):
    """n whole numbers over [lo, hi], uneven, the same for the same arguments; the largest is hi."""
    v = [lo + int((hi - lo) * ((at + i * 0.6180339887) % 1.0)) for i in range(n)]
    v[n // 2] = hi
    return v


def _lengths(case):
    n = _spread(case["q_lo"], case["q_hi"], case["batch"], 0.31)
    kv = [max(a, b) for a, b in zip(n, _spread(case["kv_lo"], case["kv_hi"], case["batch"], 0.77))]
    return n, kv


def _back(case):
    """Tokens to read back of each sequence: from the first slot of the first page that its new tokens touch."""
    n, kv = _lengths(case)
    return [b - (b - a) // case["page"] * case["page"] for a, b in zip(n, kv)]


def _scaling_args(name):
    return {"none": {}, "linear": {"factor": 4.0}, "bands": {"factor": 8.0, "low_freq": 1.0, "high_freq": 4.0, "original_max": 8192}}[name]


def _pairs(case):
    return [int(x) for x in case["pairs"].split(",")] if case["pairs"] else []


# ------------------------------------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _grid(axes, first, n):
    """Positions of n tokens on each axis: a grid whose last two axes are 24 and 36 wide, from `first` on."""
    i = torch.arange(n, device="cuda")
    last, mid = i % 36, i // 36 % 24
    rest = i // (36 * 24)
    return torch.stack([last + 3 * rest] if axes == 1 else [rest * (a + 1) for a in range(axes - 2)] + [mid, last]) + first


def _filled(gen, n_pages, hkv, page, d):
    """4-bit pages as appends of normal values leave them: codes, group scales, page scales."""
    codes = torch.empty(n_pages, hkv, page, d // 2, dtype=torch.uint8, device="cuda")
    groups = torch.empty(n_pages, hkv, page, d // 16, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.exp2(torch.randint(-9, -7, (n_pages, hkv), generator=gen, device="cuda").float())
    step = max(1, (1 << 26) // (hkv * page * d))
    for a in range(0, n_pages, step):
        x = _randn(gen, min(step, n_pages - a), hkv, page, d // 16, 16) / scales[a:a + step, :, None, None, None]
        g = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        groups[a:a + step] = g
        c = _codes(x / g.float().clamp(min=2.0 ** -9)[..., None]).flatten(-2)
        codes[a:a + step] = c[..., 0::2] | c[..., 1::2] << 4
    return codes, groups, scales


def _paged_state(case, gen):
    n, kv = _lengths(case)
    page, hkv, d, batch = case["page"], case["hkv"], case["d"], case["batch"]
    rows = [(x + page - 1) // page for x in kv]
    width, used = max(rows), sum(rows)
    n_pages = used + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda")[:used].to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor(rows, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < at[:, None]] = order
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    s = {"case": case, "table": table, "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
         "lens": torch.tensor(kv, dtype=torch.int32, device="cuda"), "total": starts[-1], "max_q": max(n), "max_kv": max(kv)}
    for key in ("k", "v"):
        s[key + "_pages"], s[key + "_groups"], s[key + "_scales"] = _filled(gen, n_pages, hkv, page, d)
    if own:
        from host_offloaded_kv_gb300 import clo
        s["cache"] = clo.PagedCache(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["k_groups"], s["v_groups"])
    return s


def _plan(case):
    from host_offloaded_kv_gb300 import clo
    axes = {"axis_pairs": _pairs(case), "axis_order": case["order"], "axis_own_freqs": case["own_freqs"]} if case["pairs"] else {}
    return clo.clo_rope_plan_init(rot_dim=case.get("rot", case["d"]), interleaved=case["interleaved"], theta=500000.0,
                                  scaling=case["scaling"], **_scaling_args(case["scaling"]), **axes)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    if case["op"] == "axes":
        x = _randn(gen, case["tokens"], case["heads"], case["d"]).to(torch.bfloat16)
        first = torch.randint(0, 30000, (1,), generator=gen, device="cuda")
        s = {"case": case, "x": x, "pos": _grid(len(_pairs(case)), first, case["tokens"]).contiguous()}
    else:
        s = _paged_state(case, gen)
        # scores with a spread of about 2: a few tokens carry most of a row's weight
        s["q"] = (_randn(gen, s["total"], case["hq"], case["d"]) * 2.0).to(torch.bfloat16)
        if case["op"] == "append4":
            s["k"] = _randn(gen, s["total"], case["hkv"], case["d"]).to(torch.bfloat16)
            s["v"] = (_randn(gen, s["total"], case["hkv"], case["d"]) * 2.0).to(torch.bfloat16)
            back = _back(case)
            s["back_starts"] = torch.tensor([sum(back[:i]) for i in range(len(back) + 1)], dtype=torch.int32, device="cuda")
            s["back_total"] = sum(back)
            # a prompt with images: positions on every axis; without axes the rows' places in the cache
            s["pos"] = _grid(len(_pairs(case)), 100, s["total"]).contiguous() if case["pairs"] else None
    if own and case["op"] != "attend4":
        s["plan"] = _plan(case)
    return s


# ------------------------------------------------------------------------------------------- operators
def run(s):
    case = s["case"]
    if case["op"] == "axes":
        return _own_axes(s) if own else _plain_axes(s)
    if case["op"] == "append4":
        return _own_append(s) if own else _plain_append(s)
    return _own_attend(s) if own else _plain_attend(s)


def _own_axes(s):
    from host_offloaded_kv_gb300 import clo
    return clo.clo_rope(s["plan"], s["x"], s["pos"])


def _own_append(s):
    c = s["cache"]
    q = c.append(s["k"], s["v"], s["starts"], s["lens"], s["table"], rope=s["plan"], positions=s["pos"], q=s["q"], max_q=s["max_q"])
    k, v = c.read(s["back_starts"], s["lens"], s["table"], s["back_total"])
    return {"q": q, "k": k, "v": v, "ks": s["k_scales"], "vs": s["v_scales"]}


def _own_attend(s):
    case = s["case"]
    return s["cache"].attention(s["q"], s["starts"], s["lens"], s["table"], max_q=s["max_q"], window=case["window"], sinks=case["sinks"])


def _scaled(f, scaling):
    a = _scaling_args(scaling)
    if scaling == "linear":
        return f / a["factor"]
    if scaling == "bands":
        turns = a["original_max"] * f / (2 * math.pi)
        keep = ((turns - a["low_freq"]) / (a["high_freq"] - a["low_freq"])).clamp(0, 1)
        return f * keep + f / a["factor"] * (1 - keep)
    return f


def _axis_of_pairs(case, rot):
    """Axis of each pair, and its place among the axis' pairs."""
    left, axis, at = _pairs(case) or [rot // 2], [], []
    if case["order"] == "sections":
        axis = [a for a, n in enumerate(left) for _ in range(n)]
    else:
        want, taken = list(left), 0
        while len(axis) < rot // 2:
            if want[taken % len(want)] > 0:
                want[taken % len(want)] -= 1
                axis.append(taken % len(want))
            taken += 1
    seen = [0] * len(left)
    for a in axis:
        at.append(seen[a])
        seen[a] += 1
    return axis, at, left


def _frequencies(case, rot):
    """(radians per position of each pair, in 64 bits, its axis)."""
    axis, at, count = _axis_of_pairs(case, rot)
    if case["own_freqs"] and case["pairs"]:
        power = [i / count[a] for i, a in zip(at, axis)]
    else:
        power = [2.0 * i / rot for i in range(rot // 2)]
    f = 500000.0 ** -torch.tensor(power, dtype=torch.float64, device="cuda")
    return _scaled(f, case["scaling"]), torch.tensor(axis, device="cuda")


def _rotate(x, pos, rot, case):
    """Rows of x's type rotated by pos [axes][tokens]; angles in 64 bits."""
    f, axis = _frequencies(case, rot)
    angle = pos.to(torch.float64)[axis].T * f
    c, s = torch.cos(angle).to(x.dtype)[:, None, :], torch.sin(angle).to(x.dtype)[:, None, :]
    head, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        out = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        out = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((out, rest), dim=-1)


def _plain_axes(s):
    return _rotate(s["x"].float(), s["pos"], s["case"]["rot"], s["case"]).to(torch.bfloat16)


def _token_places(starts, lens, table, total, page):
    """(position, page id, slot) of each token of a ragged batch whose tokens are the sequences' last ones."""
    n = (starts[1:] - starts[:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=total)
    pos = lens.long()[seq] - n[seq] + (torch.arange(total, device="cuda") - starts.long()[seq])
    return pos, table[seq, pos // page].long(), pos % page


def _codes(y):
    """Codes (uint8: sign, then the level's index) of the nearest levels, ties to the even index."""
    a = y.abs()
    i = (a > 0.25).to(torch.uint8)
    for k, edge in enumerate((0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        i += (a >= edge) if k % 2 == 0 else (a > edge)
    return i | (y < 0).to(torch.uint8) << 3


def _round_e4m3(x):
    """fp64 values (0 .. 448) to the nearest e4m3 ones, ties to even."""
    step = torch.exp2((torch.frexp(x)[1] - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def _values(codes, groups, scales):
    """fp32 values [..., d] of codes [..., d / 2] under group scales [..., d / 16] and page scales [...]."""
    level = torch.tensor(_LEVELS + tuple(-x for x in _LEVELS), device="cuda")
    x = torch.stack((level[(codes & 15).long()], level[(codes >> 4).long()]), dim=-1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * (groups.float() * scales[..., None])[..., None]).flatten(-2)


def _plain_append(s):
    case = s["case"]
    page = case["page"]
    places, pid, slot = _token_places(s["starts"], s["lens"], s["table"], s["total"], page)
    pos = places.expand(max(1, len(_pairs(case))), -1) if s["pos"] is None else s["pos"]
    q = _rotate(s["q"].float(), pos, case["d"], case).to(torch.bfloat16)
    first = torch.full((s["k_pages"].shape[0],), page, dtype=torch.int64, device="cuda").scatter_reduce(0, pid, slot, "amin")
    # values next to a border between two codes: in 64 bits
    for key, x in (("k", _rotate(s["k"].double(), pos, case["d"], case)), ("v", s["v"].double())):
        pages, groups, scales = s[key + "_pages"], s[key + "_groups"], s[key + "_scales"]
        amax = x.abs().amax(-1)
        top = torch.zeros_like(scales, dtype=torch.float64).scatter_reduce(0, pid[:, None].expand_as(amax), amax, "amax")
        mant, ex = torch.frexp(top)
        need = torch.exp2((ex - 12 + (mant > _TOP / 4096)).clamp(min=_MIN_EXP).float())
        need = torch.where(top > 0, need, torch.full_like(need, 2.0 ** _MIN_EXP))
        new = torch.where((first > 0)[:, None], torch.maximum(scales, need), need)
        touched = (first < page)[:, None]
        # tokens already in a touched page: their group scales under the new page scale
        old = (groups.float() * (scales / new)[:, :, None, None]).to(torch.float8_e4m3fn)
        keep = torch.arange(page, device="cuda")[None, :] < first[:, None]
        sel = (touched & keep)[:, None, :, None]
        groups.view(torch.uint8).copy_(torch.where(sel, old.view(torch.uint8), groups.view(torch.uint8)))
        scales.copy_(torch.where(touched, new, scales))
        x = (x / scales[pid].double()[..., None]).unflatten(-1, (-1, 16))
        g = _round_e4m3(x.abs().amax(-1) / 6.0)
        c = _codes(torch.where(g[..., None] > 0, x / g[..., None], torch.zeros_like(x))).flatten(-2)
        groups.view(torch.uint8)[pid, :, slot] = g.float().to(torch.float8_e4m3fn).view(torch.uint8)
        pages[pid, :, slot] = c[..., 0::2] | c[..., 1::2] << 4
    _, pid, slot = _token_places(s["back_starts"], s["lens"], s["table"], s["back_total"], page)
    read = lambda key: _taken(s, key, pid, slot, s[key + "_scales"][pid]).to(torch.bfloat16)  # noqa: E731
    return {"q": q, "k": read("k"), "v": read("v"), "ks": s["k_scales"], "vs": s["v_scales"]}


def _taken(s, key, pid, slot, scales):
    return _values(s[key + "_pages"][pid, :, slot], s[key + "_groups"].view(torch.uint8)[pid, :, slot].view(torch.float8_e4m3fn), scales)


def _plain_attend(s):
    case = s["case"]
    page, hkv, d, batch = case["page"], case["hkv"], case["d"], case["batch"]
    g, length, rows = case["hq"] // hkv, s["max_kv"], s["max_q"]
    j = torch.arange(length, device="cuda")
    pid = s["table"].long()[:, j // page].clamp(min=0)
    take = lambda key: _taken(s, key, pid, j % page, s[key + "_scales"][pid]).permute(0, 2, 1, 3)  # [batch, hkv, length, d]  # noqa: E731
    n = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(rows, device="cuda")
    at = (s["starts"][:-1].long()[:, None] + i).clamp(max=s["total"] - 1)
    q = s["q"].float()[at].view(batch, rows, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, g * rows, d)
    p = (s["lens"].long() - n)[:, None] + i
    see = (j <= p[..., None]) & (j < s["lens"].long()[:, None, None])
    if case["window"]:
        see &= (j > p[..., None] - case["window"]) | (j < case["sinks"])
    see = see[:, None, None].expand(batch, hkv, g, rows, length).reshape(batch, hkv, g * rows, length)
    sc = torch.matmul(q, take("k").transpose(-1, -2)).mul_(d ** -0.5).masked_fill_(~see, -math.inf)
    m = sc.amax(-1, keepdim=True)
    w = sc.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, take("v")) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(batch, hkv, g, rows, d).permute(0, 3, 1, 2, 4).reshape(batch, rows, hkv * g, d).to(torch.bfloat16)
    return o[(i < n[:, None])]


# ------------------------------------------------------------------------------------------- work
def work(case):
    d = case["d"]
    if case["op"] == "axes":
        e = case["tokens"] * case["heads"] * d
        return {"bytes": 4 * e + 8 * case["tokens"] * len(_pairs(case)), "flops": 3 * e}
    n, kv = _lengths(case)
    page, hkv, hq = case["page"], case["hkv"], case["hq"]
    row = d // 2 + d // 16  # bytes of a token's codes and group scales, of one kv head, K or V
    if case["op"] == "append4":
        t, back = sum(n), sum(_back(case))
        scales = 16 * hkv * sum((b - 1) // page - (b - a) // page + 1 for a, b in zip(n, kv))
        return {"bytes": 4 * t * hq * d + 2 * t * hkv * (2 * d + row) + 2 * back * hkv * (2 * d + row) + scales + 8 * t * len(_pairs(case)),
                "flops": 3 * t * (hq + hkv) * d}
    w, sinks = case["window"], case["sinks"]
    seen = pairs = 0
    for a, b in zip(n, kv):
        first = b - a  # position of the first query
        lo = max(0, first - w + 1) if w else 0
        seen += b - lo + min(lo, sinks if w else 0)
        for p in range(first, b):
            low = max(0, p - w + 1) if w else 0
            pairs += p + 1 - low + min(low, sinks if w else 0)
    return {"bytes": 4 * sum(n) * hq * d + 2 * seen * hkv * row + 8 * hkv * (seen // page + len(n)), "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "axes":
        return _exact_rotation(s["x"], s["pos"], case["rot"], case)
    n, kv = _lengths(case)
    if case["op"] == "append4":
        return _exact_append(s, case, n, kv)
    if work(case)["flops"] > 4e12:
        return None
    return _exact_attend(s, case, n, kv)


def _exact_rotation(x, pos, rot, case):
    """Pair by pair: complex multiplication by the unit number of its axis' position."""
    pairs, y = _pairs(case) or [rot // 2], x.double().clone()
    left, used, turn = list(pairs), [0] * len(pairs), 0
    for i in range(rot // 2):
        if case["order"] == "sections":
            a = next(k for k, m in enumerate(left) if m)
        else:
            while not left[turn % len(pairs)]:
                turn += 1
            a = turn % len(pairs)
            turn += 1
        left[a] -= 1
        e = used[a] / pairs[a] if case["own_freqs"] and case["pairs"] else i / (rot / 2)
        used[a] += 1
        f = float(_scaled(torch.tensor(500000.0 ** -e, dtype=torch.float64), case["scaling"]))
        z = torch.polar(torch.ones(pos.shape[1], dtype=torch.float64, device="cuda"), pos[a].double() * f)
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        t = torch.complex(x[..., lo].double(), x[..., hi].double()) * z[:, None]
        y[..., lo], y[..., hi] = t.real, t.imag
    return y


def _nearest(x, levels):
    """The nearest of ascending `levels` to each of x >= 0 (fp64), ties to the one of even index; at most the largest."""
    up = torch.searchsorted(levels, x.contiguous()).clamp(1, levels.numel() - 1)
    lo, hi = levels[up - 1], levels[up]
    high = (x - lo > hi - x) | ((x - lo == hi - x) & (up % 2 == 0))
    return torch.where(high, hi, lo)


def _exact_append(s, case, n, kv):
    page, d = case["page"], case["d"]
    place = torch.cat([torch.arange(b - a, b, device="cuda") for a, b in zip(n, kv)])
    pos = torch.stack([place] * max(1, len(_pairs(case)))) if s["pos"] is None else s["pos"]
    out = {"q": _exact_rotation(s["q"], pos, d, case), "k": [], "v": []}
    new = {"k": _exact_rotation(s["k"], pos, d, case), "v": s["v"].double()}
    scales = {"k": s["k_scales"].double().clone(), "v": s["v_scales"].double().clone()}
    level = torch.tensor(_LEVELS, dtype=torch.float64, device="cuda")
    e4m3 = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    table, t0 = s["table"].tolist(), 0
    for b, (a, total) in enumerate(zip(n, kv)):
        for key in ("k", "v"):
            fresh = new[key][t0:t0 + a]
            begin = (total - a) // page * page
            ids = table[b][begin // page:(total + page - 1) // page]
            lead = total - a - begin  # tokens of the first touched page that were there
            for k, i in enumerate(ids):
                lo, hi = max(k * page, lead), min((k + 1) * page, total - begin)
                put = fresh[lo - lead:hi - lead]
                part, ex = torch.frexp(put.abs().amax(-1).amax(0) / _TOP)  # part in [1/2, 1): the power of two at or above it
                need = torch.exp2((ex - (part == 0.5).to(ex.dtype)).double()).clamp(min=2.0 ** _MIN_EXP)
                old = scales[key][i].clone()
                now = torch.maximum(old, need) if lo > k * page else need
                scales[key][i] = now
                if lo > k * page:  # earlier tokens: their group scales shrink as the page's grows
                    c = s[key + "_pages"][i, :, :lo - k * page].int()
                    c = torch.stack((c & 15, c >> 4), dim=-1).flatten(-2)
                    sign = 1.0 - (c >> 3).double() * 2
                    was = s[key + "_groups"][i, :, :lo - k * page].double() * (old / now)[:, None, None]
                    g = _nearest(was, e4m3) * now[:, None, None]
                    out[key].append(((level[(c & 7).long()] * sign).unflatten(-1, (-1, 16)) * g[..., None]).flatten(-2).transpose(0, 1))
                x = (put / now[:, None]).unflatten(-1, (-1, 16))
                g = _nearest(x.abs().amax(-1) / 6.0, e4m3)[..., None]
                y = _nearest((x.abs() / g).nan_to_num(0.0, 0.0), level) * x.sign() * g * now[:, None, None]
                out[key].append(y.flatten(-2))
        t0 += a
    out["k"], out["v"] = torch.cat(out["k"]), torch.cat(out["v"])
    return {**out, "ks": scales["k"], "vs": scales["v"]}


def _exact_attend(s, case, n, kv):
    page, hkv, d, g = case["page"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    out, table, t0 = torch.zeros(s["total"], case["hq"], d, dtype=torch.float64, device="cuda"), s["table"].long(), 0
    level = torch.tensor(_LEVELS, dtype=torch.float64, device="cuda")
    for b, (a, total) in enumerate(zip(n, kv)):
        ids = table[b, :(total + page - 1) // page]
        p = torch.arange(total - a, total, device="cuda").repeat_interleave(g)[:, None]
        for h in range(hkv):
            held = []
            for key in ("k", "v"):
                c = s[key + "_pages"][:, h][ids].reshape(-1, d // 2)[:total].int()
                x = torch.empty(total, d, dtype=torch.float64, device="cuda")
                for odd in (0, 1):
                    part = c >> 4 if odd else c & 15
                    x[:, odd::2] = level[(part & 7).long()] * (1 - 2 * (part >> 3)).double()
                scale = s[key + "_groups"].view(torch.uint8)[:, h][ids].view(torch.float8_e4m3fn).double() * s[key + "_scales"][ids, h].double()[:, None, None]
                held.append(x * scale.reshape(-1, d // 16)[:total].repeat_interleave(16, dim=1))
            k, v = held
            rows = s["q"][t0:t0 + a, h * g:(h + 1) * g].double().reshape(a * g, d)
            for r in range(0, a * g, 4096):
                pr = p[r:r + 4096]
                j = torch.arange(total, device="cuda")[None, :]
                hide = j > pr
                if case["window"]:
                    hide |= (j <= pr - case["window"]) & (j >= case["sinks"])
                sc = (rows[r:r + 4096] @ k.T / math.sqrt(d)).masked_fill(hide, -math.inf)
                o = torch.softmax(sc, -1) @ v
                at = torch.arange(r, min(r + 4096, a * g), device="cuda")
                out[t0 + at // g, h * g + at % g] = o
        t0 += a
    return out
