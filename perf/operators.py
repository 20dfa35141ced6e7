"""Workloads of the paged-cache operators: rotary positions, paged append and read-back, paged attention.

``run`` computes an operator in plain torch (``own`` false) or through the package's calls
(``own`` true).  A case is one operator at one size:

* ``rope``   rotates q- or k-shaped rows by their positions;
* ``append`` rotates and writes the new tokens of a ragged batch to their pages, then reads the
  touched pages' tokens back as bf16 (with 8-bit pages the read-back is the values that the codes stand for);
* ``attend`` attends from the last tokens of each sequence to its pages.

Sequence lengths come from the case alone (``_lengths``), values from the seed.
"""
import math

import torch

own = False

_E4M3_MAX = 448.0
_MIN_EXP = -64


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a prompt's queries before clo_decode_step's layout: 32 heads of 128, half layout
        _rope("rope_prompt_half", tokens=8192, heads=32, d=128, rot=128, interleaved=False, scaling="none", pos_hi=32768),
        # one step's keys of a long-context model: interleaved, half of each head, far positions
        _rope("rope_step_inter_part", tokens=8, heads=40, d=128, rot=64, interleaved=True, scaling="yarn", pos_hi=524288),
        # one decode step of a batch: one token a sequence into bf16 pages, queries rotated along
        _append("append_step_bf16", batch=64, q_lo=1, q_hi=1, kv_lo=1000, kv_hi=32768, hq=32, hkv=8, d=128, page=64, bits=16, scaling="none"),
        # prompts of uneven lengths into 8-bit pages, one of them a continuation
        _append("append_prompt_e4m3", batch=5, q_lo=301, q_hi=4097, kv_lo=4100, kv_hi=9001, hq=32, hkv=8, d=128, page=64, bits=8, scaling="bands"),
        # one short sequence, one token: latency only
        _attend("decode_single_short", batch=1, q_lo=1, q_hi=1, kv_lo=129, kv_hi=129, hq=8, hkv=2, d=64, page=16, bits=16, window=0, sinks=0),
        # the 32K decode batch, all of it resident
        _attend("decode_batch_32k", batch=8, q_lo=1, q_hi=1, kv_lo=32768, kv_hi=32768, hq=32, hkv=8, d=128, page=64, bits=16, window=0, sinks=0),
        # one 512K sequence in 8 bits: all parallelism from the length
        _attend("decode_one_512k_e4m3", batch=1, q_lo=1, q_hi=1, kv_lo=524288, kv_hi=524288, hq=40, hkv=8, d=128, page=64, bits=8, window=0, sinks=0),
        # a ragged batch of layers with a window and sinks, 8-bit pages
        _attend("decode_window_sinks_e4m3", batch=61, q_lo=1, q_hi=1, kv_lo=3, kv_hi=40000, hq=32, hkv=8, d=128, page=32, bits=8, window=4096, sinks=4),
        # several tokens a sequence (drafts to verify) over medium contexts
        _attend("verify_ragged", batch=16, q_lo=2, q_hi=7, kv_lo=500, kv_hi=16000, hq=24, hkv=8, d=64, page=16, bits=16, window=0, sinks=0),
        # a whole prompt
        _attend("prompt_8k", batch=1, q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, hq=32, hkv=8, d=128, page=64, bits=16, window=0, sinks=0),
        # a chunk of a long prompt over 8-bit pages
        _attend("chunk_e4m3_32k", batch=1, q_lo=2048, q_hi=2048, kv_lo=32768, kv_hi=32768, hq=32, hkv=8, d=128, page=64, bits=8, window=0, sinks=0),
        # uneven prompts with a window and sinks
        _attend("prompt_ragged_window", batch=6, q_lo=65, q_hi=3001, kv_lo=2000, kv_hi=7003, hq=40, hkv=8, d=128, page=32, bits=16, window=1024, sinks=16),
    ]


def _rope(name, **kw):
    return {"name": name, "op": "rope", **kw}


def _append(name, **kw):
    return {"name": name, "op": "append", "interleaved": False, **kw}


def _attend(name, **kw):
    return {"name": name, "op": "attend", **kw}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    scaling = rng.choice(["none", "linear", "bands", "yarn"])
    if op == "rope":
        rot = rng.choice([d, d, d // 2, d - 16])
        return {"op": op, "tokens": _log(rng, 1, 8000), "heads": rng.randint(1, 40), "d": d, "rot": rot,
                "interleaved": rng.random() < 0.5, "scaling": scaling, "pos_hi": _log(rng, 100, 1000000)}
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    page, bits = rng.choice([16, 32, 64, 128]), rng.choice([8, 16])
    if op == "append":
        batch = _log(rng, 1, 64)
        hi = 1 if rng.random() < 0.4 else max(1, _log(rng, 1, 8000 // batch))
        kv_hi = hi + _log(rng, 1, 8000)
        return {"op": op, "batch": batch, "q_lo": rng.randint(1, hi), "q_hi": hi, "kv_lo": max(hi, kv_hi // 3), "kv_hi": kv_hi,
                "hq": hq, "hkv": hkv, "d": d, "page": page, "bits": bits, "interleaved": rng.random() < 0.5, "scaling": scaling}
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
            "hkv": hkv, "d": d, "page": page, "bits": bits, "window": _log(rng, 1, 5000) if windowed else 0,
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


def _scaling_args(name):
    return {"none": {}, "linear": {"factor": 4.0}, "bands": {"factor": 8.0, "low_freq": 1.0, "high_freq": 4.0, "original_max": 8192},
            "yarn": {"factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original_max": 32768}}[name]


# ------------------------------------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


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
        if case["bits"] == 16:
            s[key + "_pages"] = _randn(gen, n_pages, hkv, page, d).to(torch.bfloat16)
            s[key + "_scales"] = None
        else:
            # pages as earlier appends left them: codes up to the format's largest value, power-of-two scales around 1/64
            exp = torch.randint(-8, -4, (n_pages, hkv), generator=gen, device="cuda")
            x = _randn(gen, n_pages, hkv, page, d) * 90.0
            s[key + "_pages"] = x.clamp_(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
            s[key + "_scales"] = torch.exp2(exp.to(torch.float32))
            del x
    if own:
        from host_offloaded_kv_gb300 import clo
        s["cache"] = clo.PagedCache(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    return s


def _plan(case):
    from host_offloaded_kv_gb300 import clo
    return clo.clo_rope_plan_init(rot_dim=case.get("rot", case["d"]), interleaved=case["interleaved"], theta=500000.0,
                                  scaling=case["scaling"], **_scaling_args(case["scaling"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    if case["op"] == "rope":
        x = _randn(gen, case["tokens"], case["heads"], case["d"]).to(torch.bfloat16)
        pos = torch.randint(0, case["pos_hi"], (case["tokens"],), generator=gen, device="cuda")
        s = {"case": case, "x": x, "pos": pos}
    else:
        s = _paged_state(case, gen)
        # scores with a spread of about 2: a few tokens carry most of a row's weight
        s["q"] = (_randn(gen, s["total"], case["hq"], case["d"]) * 2.0).to(torch.bfloat16)
        if case["op"] == "append":
            s["k"] = _randn(gen, s["total"], case["hkv"], case["d"]).to(torch.bfloat16)
            s["v"] = (_randn(gen, s["total"], case["hkv"], case["d"]) * 2.0).to(torch.bfloat16)
            # read-back: each sequence from the first slot of the first page that its new tokens touch
            n, kv = _lengths(case)
            back = [b - (b - a) // case["page"] * case["page"] for a, b in zip(n, kv)]
            s["back_starts"] = torch.tensor([sum(back[:i]) for i in range(len(back) + 1)], dtype=torch.int32, device="cuda")
            s["back_total"] = sum(back)
    if own and case["op"] != "attend":
        s["plan"] = _plan(case)
    return s


# ------------------------------------------------------------------------------------------- operators
def run(s):
    case = s["case"]
    if case["op"] == "rope":
        return _own_rope(s) if own else _plain_rope(s["x"], s["pos"], case)
    if case["op"] == "append":
        return _own_append(s) if own else _plain_append(s)
    return _own_attend(s) if own else _plain_attend(s)


def _own_rope(s):
    from host_offloaded_kv_gb300 import clo
    return clo.clo_rope(s["plan"], s["x"], s["pos"])


def _own_append(s):
    c = s["cache"]
    q = c.append(s["k"], s["v"], s["starts"], s["lens"], s["table"], rope=s["plan"], q=s["q"], max_q=s["max_q"])
    k, v = c.read(s["back_starts"], s["lens"], s["table"], s["back_total"])
    return {"q": q, "k": k, "v": v} if s["k_scales"] is None else {"q": q, "k": k, "v": v, "ks": s["k_scales"], "vs": s["v_scales"]}


def _own_attend(s):
    case = s["case"]
    return s["cache"].attention(s["q"], s["starts"], s["lens"], s["table"], max_q=s["max_q"], window=case["window"], sinks=case["sinks"])


def _frequencies(rot, scaling):
    """(radians per position of each pair, magnitude), in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = 500000.0 ** (-2.0 * i / rot)
    a = _scaling_args(scaling)
    if scaling == "linear":
        return f / a["factor"], 1.0
    if scaling == "bands":
        turns = a["original_max"] * f / (2 * math.pi)
        keep = ((turns - a["low_freq"]) / (a["high_freq"] - a["low_freq"])).clamp(0, 1)
        return f * keep + f / a["factor"] * (1 - keep), 1.0
    if scaling == "yarn":
        lo = max(0, math.floor(rot * math.log(a["original_max"] / (a["beta_fast"] * 2 * math.pi)) / (2 * math.log(500000.0))))
        hi = min(rot - 1, math.ceil(rot * math.log(a["original_max"] / (a["beta_slow"] * 2 * math.pi)) / (2 * math.log(500000.0))))
        slow = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - slow) + f / a["factor"] * slow, 0.1 * math.log(a["factor"]) + 1.0
    return f, 1.0


def _rotate(x, pos, rot, interleaved, scaling):
    """fp32 rows rotated by their positions; angles in 64 bits."""
    f, mag = _frequencies(rot, scaling)
    angle = pos.to(torch.float64)[:, None] * f
    c, s = (torch.cos(angle) * mag).to(torch.float32)[:, None, :], (torch.sin(angle) * mag).to(torch.float32)[:, None, :]
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        out = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        out = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((out, rest), dim=-1)


def _plain_rope(x, pos, case):
    return _rotate(x.float(), pos, case["rot"], case["interleaved"], case["scaling"]).to(torch.bfloat16)


def _token_places(starts, lens, table, total, page):
    """(sequence, position, page id, slot) of each token of a ragged batch whose tokens are the sequences' last ones."""
    n = (starts[1:] - starts[:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=total)
    pos = lens.long()[seq] - n[seq] + (torch.arange(total, device="cuda") - starts.long()[seq])
    return seq, pos, table[seq, pos // page].long(), pos % page


def _plain_append(s):
    case = s["case"]
    page = case["page"]
    seq, pos, pid, slot = _token_places(s["starts"], s["lens"], s["table"], s["total"], page)
    rot = lambda x: _rotate(x.float(), pos, case["d"], case["interleaved"], case["scaling"])  # noqa: E731
    q = rot(s["q"]).to(torch.bfloat16)
    first = torch.full((s["k_pages"].shape[0],), page, dtype=torch.int64, device="cuda").scatter_reduce(0, pid, slot, "amin")
    for key, x in (("k", rot(s["k"])), ("v", s["v"].float())):
        pages, scales = s[key + "_pages"], s[key + "_scales"]
        if scales is None:
            pages[pid, :, slot] = x.to(torch.bfloat16)
            continue
        amax = x.abs().amax(-1)
        top = torch.zeros_like(scales).scatter_reduce(0, pid[:, None].expand_as(amax), amax, "amax")
        mant, ex = torch.frexp(top)
        need = torch.exp2((ex - 9 + (mant > 0.875)).clamp(min=_MIN_EXP).float())
        need = torch.where(top > 0, need, torch.full_like(need, 2.0 ** _MIN_EXP))
        new = torch.where((first > 0)[:, None], torch.maximum(scales, need), need)
        touched = (first < page)[:, None]
        # tokens already in a touched page: their values under the new scale
        old = (pages.float() * (scales / new)[:, :, None, None]).to(torch.float8_e4m3fn)
        keep = torch.arange(page, device="cuda")[None, :] < first[:, None]
        sel = (touched & keep)[:, None, :, None]
        pages.view(torch.uint8).copy_(torch.where(sel, old.view(torch.uint8), pages.view(torch.uint8)))
        scales.copy_(torch.where(touched, new, scales))
        pages.view(torch.uint8)[pid, :, slot] = (x / scales[pid][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    _, _, pid, slot = _token_places(s["back_starts"], s["lens"], s["table"], s["back_total"], page)
    read = lambda p, c: p.view(torch.uint8)[pid, :, slot].view(torch.float8_e4m3fn).float() * c[pid][:, :, None]  # noqa: E731
    if s["k_scales"] is None:
        return {"q": q, "k": s["k_pages"][pid, :, slot], "v": s["v_pages"][pid, :, slot]}
    return {"q": q, "k": read(s["k_pages"], s["k_scales"]).to(torch.bfloat16), "v": read(s["v_pages"], s["v_scales"]).to(torch.bfloat16),
            "ks": s["k_scales"], "vs": s["v_scales"]}


def _plain_attend(s):
    case = s["case"]
    page, hkv, d, batch = case["page"], case["hkv"], case["d"], case["batch"]
    g, length, rows = case["hq"] // hkv, s["max_kv"], s["max_q"]
    j = torch.arange(length, device="cuda")
    pid = s["table"].long()[:, j // page].clamp(min=0)
    take = lambda p, c: _gather(p, c, pid, j % page)  # [batch, hkv, length, d] fp32  # noqa: E731
    n = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(rows, device="cuda")
    at = (s["starts"][:-1].long()[:, None] + i).clamp(max=s["total"] - 1)
    q = s["q"].float()[at].view(batch, rows, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, g * rows, d)
    p = (s["lens"].long() - n)[:, None] + i
    see = (j <= p[..., None]) & (j < s["lens"].long()[:, None, None])
    if case["window"]:
        see &= (j > p[..., None] - case["window"]) | (j < case["sinks"])
    see = see[:, None, None].expand(batch, hkv, g, rows, length).reshape(batch, hkv, g * rows, length)
    sc = torch.matmul(q, take(s["k_pages"], s["k_scales"]).transpose(-1, -2)).mul_(d ** -0.5).masked_fill_(~see, -math.inf)
    m = sc.amax(-1, keepdim=True)
    w = sc.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, take(s["v_pages"], s["v_scales"])) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(batch, hkv, g, rows, d).permute(0, 3, 1, 2, 4).reshape(batch, rows, hkv * g, d).to(torch.bfloat16)
    return o[(i < n[:, None])]


def _gather(pages, scales, pid, slot):
    if scales is None:
        return pages[pid, :, slot].float().permute(0, 2, 1, 3)
    x = pages.view(torch.uint8)[pid, :, slot].view(torch.float8_e4m3fn).float()
    return x.mul_(scales[pid][..., None]).permute(0, 2, 1, 3)


# ------------------------------------------------------------------------------------------- work
def work(case):
    d = case["d"]
    if case["op"] == "rope":
        e = case["tokens"] * case["heads"] * d
        return {"bytes": 4 * e + 8 * case["tokens"], "flops": 3 * e}
    n, kv = _lengths(case)
    size, page, hkv, hq = case["bits"] // 8, case["page"], case["hkv"], case["hq"]
    if case["op"] == "append":
        t, back = sum(n), sum(b - (b - a) // page * page for a, b in zip(n, kv))
        scales = 0 if size == 2 else 16 * hkv * sum((b - 1) // page - (b - a) // page + 1 for a, b in zip(n, kv))
        return {"bytes": 4 * t * hq * d + t * hkv * d * 2 * (2 + size) + back * hkv * d * 2 * (2 + size) + scales,
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
    pages = 0 if size == 2 else 8 * hkv * (seen // page + len(n))
    return {"bytes": 4 * sum(n) * hq * d + seen * hkv * d * 2 * size + pages, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotation(s["x"], s["pos"], case["rot"], case)
    n, kv = _lengths(case)
    if case["op"] == "append":
        return _exact_append(s, case, n, kv)
    if work(case)["flops"] > 4e12:
        return None
    return _exact_attend(s, case, n, kv)


def _exact_rotation(x, pos, rot, case):
    f, mag = _frequencies(rot, case["scaling"])
    z = torch.polar(torch.full((pos.numel(), rot // 2), mag, dtype=torch.float64, device="cuda"), pos.double()[:, None] * f)
    y = x.double().clone()
    half = rot // 2
    re = y[..., 0:rot:2] if case["interleaved"] else y[..., :half]
    im = y[..., 1:rot:2] if case["interleaved"] else y[..., half:rot]
    t = torch.complex(re.contiguous(), im.contiguous()) * z[:, None, :]
    re.copy_(t.real)
    im.copy_(t.imag)
    return y


def _exact_e4m3(x):
    """The nearest value with 3 mantissa bits and a smallest step of 2^-9, ties to even (|x| <= 448)."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def _exact_append(s, case, n, kv):
    page, d = case["page"], case["d"]
    pos = torch.cat([torch.arange(b - a, b, device="cuda") for a, b in zip(n, kv)])
    out = {"q": _exact_rotation(s["q"], pos, d, case), "k": [], "v": []}
    new = {"k": _exact_rotation(s["k"], pos, d, case), "v": s["v"].double()}
    scales = {} if case["bits"] == 16 else {"k": s["k_scales"].double().clone(), "v": s["v_scales"].double().clone()}
    table, t0 = s["table"].tolist(), 0
    for b, (a, total) in enumerate(zip(n, kv)):
        for key in ("k", "v"):
            fresh = new[key][t0:t0 + a]
            begin = (total - a) // page * page
            ids = table[b][begin // page:(total + page - 1) // page]
            have = torch.cat([s[key + "_pages"][i].double().transpose(0, 1) for i in ids])[:total - begin]
            lead = total - a - begin  # tokens of the first touched page that were there
            if case["bits"] == 16:
                out[key].append(torch.cat((have[:lead], fresh)))
                continue
            for k, i in enumerate(ids):
                lo, hi = max(k * page, lead), min((k + 1) * page, total - begin)
                amax = fresh[lo - lead:hi - lead].abs().amax(-1).amax(0)
                part, ex = torch.frexp(amax / _E4M3_MAX)  # part in [1/2, 1): the power of two at or above it
                need = torch.exp2((ex - (part == 0.5).to(ex.dtype)).double()).clamp(min=2.0 ** _MIN_EXP)
                old = scales[key][i].clone()
                now = torch.maximum(old, need) if lo > k * page else need
                scales[key][i] = now
                had = _exact_e4m3(have[k * page:lo] * (old / now)[:, None]) * now[:, None]
                put = _exact_e4m3(fresh[lo - lead:hi - lead] / now[:, None]) * now[:, None]
                out[key].append(torch.cat((had, put)))
        t0 += a
    out["k"], out["v"] = torch.cat(out["k"]), torch.cat(out["v"])
    return {**out, "ks": scales["k"], "vs": scales["v"]} if scales else out


def _exact_attend(s, case, n, kv):
    page, hkv, d, g = case["page"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    out, table, t0 = torch.zeros(s["total"], case["hq"], d, dtype=torch.float64, device="cuda"), s["table"].long(), 0
    for b, (a, total) in enumerate(zip(n, kv)):
        ids = table[b, :(total + page - 1) // page]
        p = torch.arange(total - a, total, device="cuda").repeat_interleave(g)[:, None]
        for h in range(hkv):
            k, v = s["k_pages"][:, h][ids].double(), s["v_pages"][:, h][ids].double()
            if case["bits"] == 8:
                k, v = k * s["k_scales"][ids, h].double()[:, None, None], v * s["v_scales"][ids, h].double()[:, None, None]
            k, v = k.reshape(-1, d)[:total], v.reshape(-1, d)[:total]
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
