"""Plain 64-bit forms of the 4-bit pages, for the tests: on the CPU, from the formulas in include/clo.h."""
import math

import torch

import paged_ref as ref

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 0 .. 448, ascending


def nearest(x, levels):
    """Index of the nearest level to each |x| (fp64), ties to the even index, at most the last."""
    a = x.abs().contiguous()
    up = torch.searchsorted(levels, a).clamp(1, len(levels) - 1)
    lo, hi = levels[up - 1], levels[up]
    return torch.where((a - lo > hi - a) | ((a - lo == hi - a) & (up % 2 == 0)), up, up - 1)


def needed_scale(amax):
    """The smallest 2^e, e >= -64, with amax <= 2688 * 2^e."""
    e = -64
    if amax > 0:
        e = max(e, math.ceil(math.log2(amax / 2688.0)) - 1)
    while amax > 2688.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def encode(x, scale):
    """(values of the codes [.., d], group scales [.., d / 16]) of rows x [.., d] under a page's scale."""
    g = (x / scale).unflatten(-1, (-1, 16))
    top = torch.where(torch.isfinite(g), g.abs(), 0.0).amax(-1)
    s = E4M3[nearest(top / 6.0, E4M3)]
    s = torch.where(torch.isinf(g).any(-1), 448.0, s)
    y = torch.where(s[..., None] > 0, g / s[..., None], 0.0)
    fin = torch.where(torch.isfinite(y), y, torch.where(torch.isnan(y), 0.0, torch.sign(y) * 6.0))
    code = LEVELS[nearest(fin, LEVELS)] * torch.sign(fin)
    return code.flatten(-2), torch.where(torch.isnan(g).any(-1), float("nan"), s)


def values(code, group, scale):
    """fp64 values of codes [n][h][s][d], group scales [n][h][s][d / 16], page scales [n][h]."""
    s = scale.clamp(min=1e-30)[:, :, None, None] if scale.dim() == 2 else scale
    return (code.unflatten(-1, (-1, 16)) * (group * s)[..., None]).flatten(-2)


def bytes_of(code):
    """uint8 [.., d / 2] of code values [.., d]."""
    c = nearest(code, LEVELS).to(torch.uint8) | (torch.signbit(code).to(torch.uint8) << 3)
    return c[..., 0::2] | c[..., 1::2] << 4


def codes_of(pages):
    """Code values [.., d] of uint8 [.., d / 2]."""
    c = torch.stack((pages & 15, pages >> 4), dim=-1).flatten(-2).long()
    return LEVELS[c & 7] * (1.0 - 2.0 * (c >> 3).double())


class Pages4:
    """4-bit pages on the CPU: codes' values, group scales and page scales in fp64, for K and V."""

    def __init__(self, code, group, scale):
        self.code, self.group, self.scale = code, group, scale

    def append(self, side, new, seqs, table):
        """As clo_paged_append; new fp64 [total][h][d].  Returns which slots were written, bool [n_pages][s]."""
        code, group, scale = self.code[side], self.group[side], self.scale[side]
        n_pages, heads, size, _ = code.shape
        written = torch.zeros(n_pages, size, dtype=torch.bool)
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
                written[page, slots] = True
                for h in range(heads):
                    x = new[at, h]
                    fin = x[torch.isfinite(x)]
                    s = needed_scale(float(fin.abs().max()) if fin.numel() else 0.0)
                    if slots[0] > 0:
                        old = float(scale[page, h])
                        if old >= s:
                            s = old
                        elif old > 0:
                            was = group[page, h, :slots[0]] * (old / s)
                            group[page, h, :slots[0]] = torch.where(torch.isnan(was), was, E4M3[nearest(was.nan_to_num(0.0), E4M3)])
                    scale[page, h] = s
                    code[page, h, slots], group[page, h, slots] = encode(x, s)
        return written

    def plain(self):
        """The values as a cache of the plain reference."""
        return ref.Pages(*(values(self.code[i], self.group[i], self.scale[i]) for i in range(2)))


def of_cache(cache):
    """Pages4 of what a device cache holds."""
    get = lambda t: t.contiguous().view(torch.uint8).cpu().view(torch.float8_e4m3fn).double()  # noqa: E731
    return Pages4([codes_of(t.cpu()) for t in (cache.k_pages, cache.v_pages)], [get(t) for t in (cache.k_group_scales, cache.v_group_scales)],
                  [t.cpu().double() for t in (cache.k_scales, cache.v_scales)])
