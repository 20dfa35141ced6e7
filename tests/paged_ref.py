"""Plain 64-bit forms of the paged-cache operators, for the tests: numpy/torch on the CPU, loops over
sequences, heads and rows, written from the formulas in include/clo.h."""
import math

import torch

E4M3_MAX, MIN_EXP = 448.0, -64


def frequencies(rot, theta=10000.0, scaling="none", factor=1.0, low_freq=1.0, high_freq=4.0, beta_fast=32.0, beta_slow=1.0,
                original_max=0, magnitude=0.0, interleaved=False):
    out = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            w = min(1.0, max(0.0, (original_max * f / (2 * math.pi) - low_freq) / (high_freq - low_freq)))
            f = w * f + (1 - w) * f / factor
        elif scaling == "yarn":
            c = lambda n: rot * math.log(original_max / (2 * math.pi * n)) / (2 * math.log(theta))  # noqa: E731
            lo, hi = max(0, math.floor(c(beta_fast))), min(rot - 1, math.ceil(c(beta_slow)))
            w = 1 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = w * f + (1 - w) * f / factor
        out.append(f)
    mag = magnitude or (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)
    return torch.tensor(out, dtype=torch.float64), mag


def rotate(x, pos, rot, interleaved=False, transpose=False, **scaling):
    """fp64 [n][h][d] rotated by pos [n]."""
    f, mag = frequencies(rot, **scaling)
    a = pos.double()[:, None] * f
    c, s = (torch.cos(a) * mag)[:, None], (torch.sin(a) * mag)[:, None]
    if transpose:
        s = -s
    y = x.double().clone()
    ia = torch.arange(rot // 2) * 2 if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    p, q = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia] = p * c - q * s
    y[..., ib] = q * c + p * s
    return y


def e4m3_values(t):
    return t.view(torch.float8_e4m3fn).to(torch.float32).double()


def round_e4m3(x):
    """Nearest e4m3 value (ties to even, saturating; NaN stays), in fp64."""
    y = x.clamp(-E4M3_MAX, E4M3_MAX)
    e = torch.frexp(y)[1].clamp(min=-5)
    step = torch.ldexp(torch.ones_like(y), e - 4)
    return torch.round(y / step) * step


def needed_scale(amax):
    if amax == 0:
        return 2.0 ** MIN_EXP
    m, e = math.frexp(amax)
    return 2.0 ** max(MIN_EXP, e - 9 + (1 if m > 0.875 else 0))


class Pages:
    """A paged cache on the CPU: K and V values in fp64 (8-bit pages: code values) and scales."""

    def __init__(self, k, v, ks=None, vs=None):
        self.val = [k, v]  # [n_pages][h][s][d] fp64
        self.scale = [ks, vs]  # [n_pages][h] fp64 or None
        self.bits = 16 if ks is None else 8

    def append(self, side, new, seqs, table):
        """new fp64 [total][h][d]; seqs: (first row, rows, kv_len) per sequence.  Returns per written value the
        unrounded one ([n_pages][h][s][d], NaN where nothing was written)."""
        val, scale = self.val[side], self.scale[side]
        n_pages, heads, size, d = val.shape
        raw = torch.full_like(val, float("nan"))
        for b, (first, n, kv) in enumerate(seqs):
            by_page = {}
            for i in range(n):
                pos = kv - n + i
                if 0 <= pos < table.shape[1] * size:
                    by_page.setdefault(pos // size, []).append((pos % size, first + i))
            for logical, rows in by_page.items():
                page = int(table[b, logical])
                if not 0 <= page < n_pages:
                    continue
                slots, at = [r[0] for r in rows], [r[1] for r in rows]
                x = new[at].transpose(0, 1)  # [h][rows][d]
                raw[page][:, slots] = x
                if self.bits == 16:
                    val[page][:, slots] = x
                    continue
                for h in range(heads):
                    fin = x[h][torch.isfinite(x[h])]
                    s = needed_scale(float(fin.abs().max()) if fin.numel() else 0.0)
                    if slots[0] > 0:
                        old = float(scale[page, h])
                        if old >= s:
                            s = old
                        elif old > 0:
                            val[page, h, :slots[0]] = round_e4m3(val[page, h, :slots[0]] * (old / s))
                    scale[page, h] = s
                    val[page, h, slots] = round_e4m3(x[h] / s)
        return raw

    def row(self, side, page, h, slot):
        v = self.val[side][page, h, slot]
        return v if self.bits == 16 else v * max(float(self.scale[side][page, h]), 1e-30)


def attention(pages, q, seqs, table, group, scale=None, window=0, sinks=0):
    """(out, sum p|v|, max sum|q||k| * scale) in fp64; q [total][hq][d]; rows of no sequence are NaN."""
    total, hq, d = q.shape
    scale = scale or 1 / math.sqrt(d)
    n_pages, _, size, _ = pages.val[0].shape
    out = torch.full((total, hq, d), float("nan"), dtype=torch.float64)
    spread, reach = torch.zeros_like(out), torch.zeros(total, hq, 1, dtype=torch.float64)
    for b, (first, n, kv) in enumerate(seqs):
        cap = min(max(kv, 0), table.shape[1] * size)
        there = [j for j in range(cap) if 0 <= int(table[b, j // size]) < n_pages]
        for h in range(hq // group):
            if there:
                ks = torch.stack([pages.row(0, int(table[b, j // size]), h, j % size) for j in there])
                vs = torch.stack([pages.row(1, int(table[b, j // size]), h, j % size) for j in there])
            js = torch.tensor(there, dtype=torch.int64)
            for i in range(n):
                p = kv - n + i
                see = js <= p
                if window:
                    see &= (js > p - window) | (js < sinks)
                for g in range(group):
                    o = torch.zeros(d, dtype=torch.float64)
                    if bool(see.any()):
                        k, v, x = ks[see], vs[see], q[first + i, h * group + g].double()
                        s = (k @ x) * scale
                        m = s.max()
                        w = torch.exp(s - (m if not torch.isinf(m) or m > 0 else torch.zeros_like(m)))
                        if float(w.sum()) != 0:
                            o = (w[:, None] * v).sum(0) / w.sum()
                            spread[first + i, h * group + g] = (w[:, None] * v.abs()).sum(0) / w.sum()
                            reach[first + i, h * group + g] = (k.abs() @ x.abs()).max() * scale
                    out[first + i, h * group + g] = o
    return out, spread, reach


def attention_bound(want, spread, reach, d, bits):
    """What the kernels may be off: each weight is rounded to bf16 (half step 2^-8) or fp16 (2^-11) before the product with
    V, each score carries the rounding of a d-term fp32 sum (and, 8-bit pages, of q to fp16 relative to its row's
    largest element, below the same), which scales a weight by at most twice that; out is rounded to bf16 once."""
    scores = 2 * (d + 8) * 2.0 ** -24 * reach
    return (2.0 ** (-8 if bits == 16 else -11) + scores + 2.0 ** -18) * spread + 2.0 ** -8 * want.abs() + 1e-30
