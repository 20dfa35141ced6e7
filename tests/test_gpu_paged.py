"""Rotary positions and the paged cache on the GPU, against plain 64-bit forms (tests/paged_ref.py)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def clo():
    from host_offloaded_kv_gb300 import clo as m

    m.load_library()
    return m


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def bf16(x):
    return x.to(BF16)


def rope_bound(want, x, mag=1.0):
    """One rounding to bf16 (half step 2^-8) of a value that hardware sine and cosine (2^-21 each, and the
    angle to 2^-20) put at most 2^-19 of the row's elements off."""
    return 2.0 ** -8 * want.abs() + 2.0 ** -18 * mag * x.double().abs().amax(-1, keepdim=True) + 1e-38


def check(got, want, bound, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(torch.where(inf, got, 0.0), torch.where(inf, want, 0.0)), f"{what}: infinities in other places"
    off = torch.where(nan | inf, 0.0, (got - want).abs() / bound)
    assert float(off.max() if off.numel() else 0.0) <= 1.0, f"{what}: {float(off.max()):.3g} of the bound"


# --------------------------------------------------------------------------------------------- rope
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 112), (128, 20), (80, 40), (2, 2), (1024, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,h", [(1, 1), (5, 3), (37, 40)])
def test_rope(clo, d, rot, interleaved, n, h):
    x = bf16(rand(d + rot + n, n, h, d))
    pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(n))
    pos[0] = 0
    pos[-1] = -12345
    kw = dict(scaling="yarn", factor=8.0, original_max=8192)
    plan = clo.clo_rope_plan_init(rot_dim=rot, interleaved=interleaved, **kw)
    mag = 0.1 * math.log(8.0) + 1.0
    for transpose in (False, True):
        got = clo.clo_rope(plan, x.cuda(), pos.cuda(), transpose=transpose)
        want = ref.rotate(x, pos, rot, interleaved, transpose, **kw)
        check(got, want, rope_bound(want, x, mag), f"transpose={transpose}")
        assert torch.equal(got.cpu()[..., rot:], x[..., rot:])  # the rest is copied


def test_rope_far_positions(clo):
    # 2^40 positions: fp64 angles of the reference carry 2^40 * 2^-53 radians, within the bound's 2^-18
    n, d = 64, 128
    x = bf16(rand(3, n, 1, d))
    pos = torch.randint(1 << 20, 1 << 30, (n,), generator=torch.Generator().manual_seed(4))
    plan = clo.clo_rope_plan_init(rot_dim=d, theta=500000.0)
    want = ref.rotate(x, pos, d, theta=500000.0)
    check(clo.clo_rope(plan, x.cuda(), pos.cuda()), want, rope_bound(want, x))


@pytest.mark.parametrize("offset", [0, 1, 8])
def test_rope_strides_alignment_and_in_place(clo, offset):
    # heads inside a fused row, the base on 16 bytes or not; in place leaves the neighbours alone
    n, h, d = 9, 6, 64
    buf = bf16(rand(5, n, 1000))
    dev = buf.cuda()
    view = dev.as_strided((n, h, d), (1000, d, 1), offset)
    x = buf.as_strided((n, h, d), (1000, d, 1), offset).clone()
    pos = torch.arange(100, 100 + n)
    plan = clo.clo_rope_plan_init(rot_dim=32)
    want = ref.rotate(x, pos, 32)
    check(clo.clo_rope(plan, view, pos.cuda()), want, rope_bound(want, x))
    assert clo.clo_rope(plan, view, pos.cuda(), out=view) is view
    check(view, want, rope_bound(want, x), "in place")
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided((n, h, d), (1000, d, 1), offset).fill_(False)
    assert torch.equal(dev.cpu()[mask], buf[mask])
    # heads outermost in memory
    t = x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    check(clo.clo_rope(plan, t, pos.cuda()), want, rope_bound(want, x), "heads first")


def test_rope_gradient_is_the_transpose(clo):
    # <g, R x> = <R^T g, x>, and differences: R is linear, so (R(x + e) - R(x)) . g for one element e is that element of R^T g
    n, h, d = 2, 2, 64
    plan = clo.clo_rope_plan_init(rot_dim=48, interleaved=True)
    pos = torch.tensor([7, 1000])
    g = bf16(rand(8, n, h, d))
    grad = clo.clo_rope(plan, g.cuda(), pos.cuda(), transpose=True)
    want = ref.rotate(g, pos, 48, True, True)
    check(grad, want, rope_bound(want, g))
    for e in (0, 1, 30, 47, 50):
        x = torch.zeros(n, h, d, dtype=BF16)
        x[..., e] = 1.0
        y = clo.clo_rope(plan, x.cuda(), pos.cuda()).cpu().double()
        diff = (y * g.double()).sum(-1)
        # y carries a bf16 rounding per element (2^-8 of |y| <= 1, two elements), grad one
        bound = 2 * (2.0 ** -8 + 2.0 ** -18) * g.double().abs().amax(-1) + 2.0 ** -8 * diff.abs()
        check(grad[..., e], diff, 2 * bound, f"element {e}")


def test_rope_empty(clo):
    plan = clo.clo_rope_plan_init(rot_dim=64)
    for shape in ((0, 4, 64), (3, 0, 64)):
        x = torch.empty(shape, dtype=BF16, device="cuda")
        assert clo.clo_rope(plan, x, torch.zeros(shape[0], dtype=torch.int64, device="cuda")).shape == x.shape


def test_binding_refusals_on_device(clo):
    plan = clo.clo_rope_plan_init(rot_dim=64)
    x = torch.zeros(2, 2, 64, dtype=BF16, device="cuda")
    pos = torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in (x.half(), x[0], x.transpose(1, 2)):
        with pytest.raises(ValueError):
            clo.clo_rope(plan, bad, pos)
    with pytest.raises(ValueError, match="positions"):
        clo.clo_rope(plan, x, pos.int())
    with pytest.raises(ValueError, match="expanded"):
        clo.clo_rope(plan, x, pos, out=x[:1].expand(2, 2, 64))
    c = clo.PagedCache.create(2, 2, 16, 64)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="block_table"):
        c.attention(x, i32(0, 2), i32(2), table.long())
    with pytest.raises(ValueError, match="q_starts"):
        c.attention(x, i32(0, 2, 2), i32(2), table)
    with pytest.raises(ValueError, match="head_dim"):
        c.attention(torch.zeros(2, 2, 128, dtype=BF16, device="cuda"), i32(0, 2), i32(2), table)
    with pytest.raises(clo.CLOError, match="multiple of n_kv_heads"):
        c.attention(torch.zeros(2, 3, 64, dtype=BF16, device="cuda"), i32(0, 2), i32(2), table)
    with pytest.raises(ValueError, match="scales"):
        clo.PagedCache(c.k_pages, c.v_pages, torch.ones(2, 2, device="cuda"), torch.ones(2, 2, device="cuda"))
    with pytest.raises(ValueError, match="dtypes"):
        clo.PagedCache(c.k_pages.float(), c.v_pages.float())


# --------------------------------------------------------------------------------------------- caches
class Case:
    """A batch on the CPU and on the device: seqs are (rows, kv_len); pages are handed out in shuffled order."""

    def __init__(self, clo, seqs, hkv, d, page, bits, seed, extra=3, holes=(), by_token=False, magnitude=1.0, fill=True, width=None):
        self.clo, self.bits, self.page, self.hkv, self.d = clo, bits, page, hkv, d
        self.seqs, at = [], 0
        for n, kv in seqs:
            self.seqs.append((at, n, kv))
            at += n
        self.total = at
        need = [max(0, -(-kv // page)) for _, kv in seqs]
        width = max(need + [1]) if width is None else width
        n_pages = sum(need) + extra
        gen = torch.Generator().manual_seed(seed)
        order = torch.randperm(n_pages, generator=gen).tolist()
        self.table = torch.full((len(seqs), width), -1, dtype=torch.int32)
        for b, r in enumerate(need):
            for j in range(min(r, width)):
                self.table[b, j] = order.pop()
        for b, j, v in holes:
            self.table[b, j] = v
        shape = (n_pages, hkv, page, d)
        self.codes, vals, self.scales = [], [], []
        for side in range(2):
            x = rand(seed + 10 + side, *shape) * magnitude
            if not fill:
                x.fill_(float("nan"))
            if bits == 16:
                c = bf16(x)
                vals.append(c.double())
                self.scales.append(None)
            else:
                c = ref.round_e4m3(x * 60).to(torch.float8_e4m3fn)
                vals.append(ref.e4m3_values(c))
                e = torch.randint(-9, -3, (n_pages, hkv), generator=gen)
                self.scales.append(torch.exp2(e.float()))
            self.codes.append(c)
        self.pages = ref.Pages(*vals, *[s if s is None else s.double() for s in self.scales])
        self.by_token = by_token

    def pages_like(self, c):
        """The pages on the device: heads outside slots, or slots outside heads."""
        d = c.view(torch.uint8).cuda().view(c.dtype) if c.dtype != BF16 else c.cuda()
        return d.transpose(1, 2).contiguous().transpose(1, 2) if self.by_token else d

    def device(self):
        dev = [self.pages_like(c) for c in self.codes]
        sc = [None if s is None else s.cuda() for s in self.scales]
        self.cache = self.clo.PagedCache(*dev, *sc)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.starts = i32([s[0] for s in self.seqs] + [self.total])
        self.lens = i32([s[2] for s in self.seqs])
        self.tab = self.table.cuda()
        return self.cache

    @property
    def max_q(self):
        return max(s[1] for s in self.seqs)

    def attend(self, q, window=0, sinks=0, scale=0.0, **kw):
        return self.cache.attention(q.cuda(), self.starts, self.lens, self.tab, max_q=kw.pop("max_q", self.max_q), window=window,
                                    sinks=sinks, softmax_scale=scale, **kw)

    def compare(self, got, q, window=0, sinks=0, scale=None, what=""):
        want, spread, reach = ref.attention(self.pages, q, self.seqs, self.table, q.shape[1] // self.hkv, scale, window, sinks)
        check(got, want, ref.attention_bound(want, spread, reach, self.d, self.bits), what)


# --------------------------------------------------------------------------------------------- append and read
def device_values(cache):
    out = []
    for p, s in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales)):
        v = p.cpu().double() if s is None else ref.e4m3_values(p.contiguous().view(torch.uint8).cpu())
        out.append((v, None if s is None else s.cpu().double()))
    return out


BATCHES = {"one": [(1, 1)], "steps": [(1, 17), (1, 64), (1, 33), (1, 1)], "ragged": [(0, 5), (7, 7), (33, 70), (1, 129), (130, 200)],
           "long": [(300, 517)], "short_cache": [(5, 3), (4, 0), (2, 90)]}


@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("d,page,bits,by_token", [(64, 16, 16, False), (128, 64, 16, True), (128, 32, 8, False), (64, 128, 8, True), (128, 16, 8, False)])
@pytest.mark.parametrize("mode", ["plain", "rope", "rope_q"])
def test_append_and_read(clo, batch, d, page, bits, by_token, mode):
    hkv, hq = 3, 7
    c = Case(clo, BATCHES[batch], hkv, d, page, bits, seed=len(batch) + d + page, by_token=by_token, magnitude=0.05 if batch == "ragged" else 1.0)
    cache = c.device()
    k, v, q = bf16(rand(1, c.total, hkv, d) * 3), bf16(rand(2, c.total, hkv, d)), bf16(rand(3, c.total, hq, d))
    pos = torch.cat([torch.arange(kv - n, kv) for _, n, kv in c.seqs])
    given = None
    if mode == "rope_q":
        given = pos * 3 + 1000
    rot, inter = (d, False) if mode == "rope" else (d // 2, True)
    plan = None if mode == "plain" else clo.clo_rope_plan_init(rot_dim=rot, interleaved=inter)
    k64 = k.double() if plan is None else ref.rotate(k, pos if given is None else given, rot, inter)
    before = device_values(cache)
    got_q = cache.append(k.cuda(), v.cuda(), c.starts, c.lens, c.tab, rope=plan, positions=None if given is None else given.cuda(),
                         q=q.cuda() if mode == "rope_q" else None, max_q=c.max_q)
    raws = [c.pages.append(0, k64, c.seqs, c.table), c.pages.append(1, v.double(), c.seqs, c.table)]
    if mode == "rope_q":
        want = ref.rotate(q, given, rot, inter)
        check(got_q, want, rope_bound(want, q), "q")
    else:
        assert got_q is None
    for side, (val, scale) in enumerate(device_values(cache)):
        raw, new = raws[side], ~torch.isnan(raws[side])
        if bits == 16:
            assert torch.equal(val[~new], before[side][0][~new]), "slots of other tokens changed"
            check(val[new], raw[new], 2.0 ** -8 * raw[new].abs() + (0 if plan is None or side else 2.0 ** -18 * 20) + 1e-38)
            if side or plan is None:
                assert torch.equal(val[new], raw[new])
            continue
        assert torch.equal(scale, c.pages.scale[side]), "scales"
        assert torch.equal(val[~new], c.pages.val[side][~new]), "codes of earlier tokens"
        if side or plan is None:
            assert torch.equal(val[new], c.pages.val[side][new])
        else:  # half a step of the format (2^-4 of the value, 2^-10 at the least) around the unrounded value
            x = (raw / scale[:, :, None, None])[new]
            slack = (2.0 ** -18 * 20 / scale)[:, :, None, None].expand_as(raw)[new]
            check(val[new], x, 2.0 ** -4 * x.abs() + 2.0 ** -10 + slack)
    # read back what the pages now hold, whole sequences and the batch's rows
    back = [(sum(max(s[2], 0) for s in c.seqs[:b]), max(s[2], 0), s[2]) for b, s in enumerate(c.seqs)]
    total = sum(r[1] for r in back)
    starts = torch.tensor([r[0] for r in back] + [total], dtype=torch.int32, device="cuda")
    gk, gv = cache.read(starts, c.lens, c.tab, total)
    for side, got in enumerate((gk, gv)):
        val, scale = device_values(cache)[side]
        for b, (first, n, _) in enumerate(back):
            for j in range(n):
                page_id = int(c.table[b, j // page])
                want = val[page_id, :, j % page] * (1.0 if scale is None else scale[page_id][:, None])
                assert torch.equal(got[first + j].cpu().double(), want)


def test_append_twice_grows_the_scale_of_a_page(clo):
    # token by token with growing values: the page's scale follows, the earlier codes are rescaled, never written anew
    d, page = 64, 16
    c = Case(clo, [(1, page)], 1, d, page, 8, seed=4, fill=False)
    cache = c.device()
    for i in range(page):
        x = bf16(rand(100 + i, 1, 1, d) * 2.0 ** (i - 6))
        c.seqs = [(0, 1, i + 1)]
        cache.append(x.cuda(), x.cuda(), c.starts, torch.tensor([i + 1], dtype=torch.int32, device="cuda"), c.tab, max_q=1)
        for side in range(2):
            c.pages.append(side, x.double(), c.seqs, c.table)
    page_id = int(c.table[0, 0])
    for side, (val, scale) in enumerate(device_values(cache)):
        assert float(scale[page_id, 0]) == float(c.pages.scale[side][page_id, 0])
        assert torch.equal(val[page_id], c.pages.val[side][page_id])


@pytest.mark.parametrize("bits", [16, 8])
def test_append_of_what_is_not_finite(clo, bits):
    d, page = 128, 32
    c = Case(clo, [(3, 3), (2, 40)], 2, d, page, bits, seed=9)
    cache = c.device()
    x = rand(5, c.total, 2, d)
    x[0, 0, 3], x[1, 1, 7], x[3, 0, 0], x[4, 1, 127] = float("inf"), float("nan"), -float("inf"), float("nan")
    x[2] = 0.0
    x[2, :, 0] = 1e-30
    x = bf16(x)
    cache.append(x.cuda(), x.cuda(), c.starts, c.lens, c.tab, max_q=3)
    for side, (val, scale) in enumerate(device_values(cache)):
        raw = c.pages.append(side, x.double(), c.seqs, c.table)
        new = ~torch.isnan(raw) if bits == 16 else None
        if bits == 16:
            assert torch.equal(val[new], raw[new])
        else:
            assert torch.equal(scale, c.pages.scale[side])
            assert torch.equal(torch.nan_to_num(val, nan=1e9), torch.nan_to_num(c.pages.val[side], nan=1e9))


def test_append_skips_pages_that_are_not_there(clo):
    # holes, numbers past the last page, positions past the table: nothing is written, reads give zeros
    d, page, hkv = 64, 16, 2
    for bits in (16, 8):
        c = Case(clo, [(40, 40), (20, 50), (1, 33)], hkv, d, page, bits, seed=6, holes=[(0, 1, -1), (1, 2, 1 << 20), (2, 2, -7)], width=3)
        cache = c.device()
        before = device_values(cache)
        k = bf16(rand(7, c.total, hkv, d))
        cache.append(k.cuda(), k.cuda(), c.starts, c.lens, c.tab, max_q=40)
        raw = c.pages.append(0, k.double(), c.seqs, c.table)
        val = device_values(cache)[0][0]
        same = torch.isnan(raw)
        assert torch.equal(val[same], (before[0][0] if bits == 16 else c.pages.val[0])[same])
        gk, _ = cache.read(c.starts, c.lens, c.tab, c.total)
        for first, n, kv in c.seqs:
            for i in range(n):
                pos, b = kv - n + i, [s[0] for s in c.seqs].index(first)
                pid = int(c.table[b, pos // page]) if pos // page < 3 else -1
                if not 0 <= pid < val.shape[0]:
                    assert not gk[first + i].any()


# --------------------------------------------------------------------------------------------- attention
ATTEND = [
    # seqs, hkv, group, d, page, bits, window, sinks
    ([(1, 1)], 1, 1, 64, 16, 16, 0, 0),
    ([(1, 130)], 2, 4, 128, 64, 16, 0, 0),
    ([(1, 300), (1, 17), (1, 1), (1, 64)], 2, 5, 128, 32, 16, 0, 0),
    ([(1, 300), (1, 17), (1, 1), (1, 64)], 2, 8, 128, 16, 8, 0, 0),
    ([(1, 513), (1, 100)], 1, 16, 64, 128, 8, 0, 0),
    ([(1, 1000), (1, 40), (1, 3)], 2, 3, 64, 16, 16, 100, 4),
    ([(1, 1000), (1, 40), (1, 3)], 2, 7, 128, 64, 8, 33, 70),
    ([(1, 700)], 1, 2, 128, 16, 16, 1, 0),
    ([(3, 200), (1, 77), (0, 50), (5, 5)], 2, 3, 128, 32, 16, 0, 0),
    ([(4, 300), (2, 31)], 1, 4, 64, 64, 8, 20, 3),
    ([(40, 40)], 2, 4, 128, 64, 16, 0, 0),
    ([(70, 200), (1, 64), (0, 9), (33, 33)], 2, 4, 128, 32, 16, 0, 0),
    ([(70, 200), (1, 64), (33, 33)], 1, 8, 128, 64, 8, 0, 0),
    ([(129, 129), (17, 260)], 1, 3, 64, 16, 16, 50, 5),
    ([(129, 129), (17, 260)], 2, 2, 64, 128, 8, 128, 1),
    ([(150, 400)], 1, 16, 128, 16, 16, 0, 0),
    ([(257, 300)], 2, 1, 128, 128, 8, 64, 0),
    ([(6, 3), (20, 0), (3, 40)], 1, 4, 128, 16, 16, 0, 0),
    ([(30, 10), (2, 1)], 1, 2, 64, 32, 8, 4, 2),
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(clo, case):
    seqs, hkv, group, d, page, bits, window, sinks = ATTEND[case]
    c = Case(clo, seqs, hkv, d, page, bits, seed=20 + case, by_token=case % 2 == 1)
    c.device()
    q = bf16(rand(50 + case, c.total, hkv * group, d) * 2)
    got = c.attend(q, window, sinks)
    c.compare(got, q, window, sinks)
    # max_q is a bound, not the length: another bound gives the same rows
    got = c.attend(q, window, sinks, max_q=None)
    c.compare(got, q, window, sinks, what="max_q of the whole call")


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("rows", [1, 3, 60])
def test_attention_ignores_what_masked_tokens_hold(clo, bits, rows):
    # NaN and infinities where no row, or not every row, looks: slots past the length, tokens before the window,
    # pages that are not there, and the rows' own later tokens
    d, page, hkv, group, kv, window, sinks = 128, 16, 2, 4, 300, 90, 3
    c = Case(clo, [(rows, kv), (rows, rows)], hkv, d, page, bits, seed=31, holes=[(0, 16, -1)])
    bad = [float("nan"), float("inf"), -float("inf")] if bits == 16 else [float("nan")] * 3
    for side in range(2):
        codes = c.codes[side].double() if bits == 16 else ref.e4m3_values(c.codes[side])
        last = int(c.table[0, (kv - 1) // page])
        codes[last, :, (kv - 1) % page + 1:] = bad[0]
        for n, j in enumerate((sinks, sinks + 5, kv - rows - window, kv - rows - window - 1)):
            codes[int(c.table[0, j // page]), :, j % page] = bad[n % 3]
        second = int(c.table[1, (rows - 1) // page])
        codes[second, :, (rows - 1) % page + 1:] = bad[1]
        if rows > 1:  # visible to the last row alone
            for b, k in ((0, kv), (1, rows)):
                codes[int(c.table[b, (k - 1) // page]), 0, (k - 1) % page, 5] = bad[(side + 1) % 3]
        c.codes[side] = bf16(codes) if bits == 16 else codes.to(torch.float8_e4m3fn)
        c.pages.val[side] = c.codes[side].double() if bits == 16 else ref.e4m3_values(c.codes[side])
    c.device()
    q = bf16(rand(77, c.total, hkv * group, d))
    c.compare(c.attend(q, window, sinks), q, window, sinks)


@pytest.mark.parametrize("rows", [1, 40])
def test_attention_of_lowest_and_infinite_scores(clo, rows):
    d, page = 64, 16
    low = torch.finfo(BF16).min
    c = Case(clo, [(rows, 50), (rows, 45)], 1, d, page, 16, seed=12)
    # sequence 0: every key the type's lowest value (scores of about -3e38 or below fp32's range); sequence 1: -infinity scores
    for b, value in ((0, low), (1, -float("inf"))):
        for j in range(4):
            if int(c.table[b, j]) >= 0:
                c.codes[0][int(c.table[b, j])] = 0.0
                c.codes[0][int(c.table[b, j]), :, :, 0] = value
    c.codes[0][int(c.table[0, 0]), :, 3, 0] = 0.5
    c.pages.val[0] = c.codes[0].double()
    c.device()
    q = torch.zeros(c.total, 2, d, dtype=BF16)
    q[..., 0] = 1.0
    got = c.attend(q).cpu()
    assert not got[rows:].any()  # every score -infinity: zeros
    want = ref.attention(c.pages, q, c.seqs, c.table, 2)[0]
    near = want[:rows]
    first = 50 - rows
    keep = [i for i in range(rows) if first + i >= 3]  # rows that see token 3: all weight is on it
    check(got[keep], near[keep], 2.0 ** -7 * near[keep].abs() + 1e-6)


def test_attention_scale_strides_stream_and_untouched_rows(clo):
    d, page, hkv, group = 128, 32, 2, 4
    for seqs in ([(1, 90), (1, 33)], [(40, 90), (3, 33)]):
        c = Case(clo, seqs, hkv, d, page, 16, seed=14)
        c.device()
        q = bf16(rand(3, c.total + 2, hkv * group, d))
        # q inside a fused projection, out inside a wider row; two rows behind the last sequence
        fused = torch.zeros(c.total + 2, hkv * (group + 2) * d, dtype=BF16, device="cuda")
        fused[:, :hkv * group * d] = q.cuda().view(c.total + 2, -1)
        qv = fused.as_strided((c.total + 2, hkv * group, d), (fused.stride(0), d, 1))
        wide = torch.full((c.total + 2, hkv * group, d + 8), 7.0, dtype=BF16, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.cache.attention(qv, c.starts, c.lens, c.tab, out=wide[..., :d], max_q=c.max_q, softmax_scale=0.3)
        side.synchronize()
        c.compare(wide[:c.total, :, :d], q[:c.total], scale=0.3)
        assert bool((wide[c.total:] == 7.0).all()) and bool((wide[..., d:] == 7.0).all())


def dense_on_device(c, q, window=0, sinks=0):
    """Attention of a Case in fp64 on the device, a (sequence, kv head) at a time: for sizes beyond the loops of paged_ref."""
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    spread, reach = torch.zeros_like(out), torch.zeros(*q.shape[:2], 1, dtype=torch.float64, device="cuda")
    group, d = q.shape[1] // c.hkv, c.d
    vals = [v.cuda() if s is None else v.cuda() * s.double().cuda()[:, :, None, None] for v, s in zip(c.pages.val, c.scales)]
    qd = q.double().cuda()
    for b, (first, n, kv) in enumerate(c.seqs):
        if n == 0:
            continue
        ids = c.table[b, :-(-kv // c.page)].long().cuda()
        j = torch.arange(kv, device="cuda")
        p = torch.arange(kv - n, kv, device="cuda")[:, None]
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        for h in range(c.hkv):
            k, v = (x[ids, h].reshape(-1, d)[:kv] for x in vals)
            for g in range(group):
                x = qd[first:first + n, h * group + g]
                w = torch.softmax((x @ k.T / math.sqrt(d)).masked_fill(~see, -math.inf), -1)
                out[first:first + n, h * group + g] = w @ v
                spread[first:first + n, h * group + g] = w @ v.abs()
                reach[first:first + n, h * group + g] = ((x.abs() @ k.abs().T) * see).amax(-1, keepdim=True) / math.sqrt(d)
    return out.cpu(), spread.cpu(), reach.cpu()


# Sizes at which the units of rows are more than the SMs (several to a block), are cut between blocks, or are split over
# blocks and joined; lengths of everything from one token on.
LARGE = [
    # seqs, hkv, group, d, page, bits, window, sinks
    ([(n, n + 7 * n % 90) for n in range(33, 63)], 6, 3, 64, 32, 16, 0, 0),
    ([(n, n + 7 * n % 90) for n in range(33, 63)], 6, 3, 64, 32, 8, 0, 0),
    ([(n, n + 300) for n in range(100, 126)], 7, 2, 128, 64, 16, 0, 0),
    ([(n, n + 300) for n in range(100, 126)], 7, 2, 128, 64, 8, 0, 0),
    ([(700, 900), (1, 3000), (300, 300), (0, 50), (1500, 4000)], 4, 4, 128, 64, 16, 0, 0),
    ([(700, 900), (1, 3000), (300, 300), (0, 50), (1500, 4000)], 4, 4, 128, 64, 8, 0, 0),
    ([(700, 900), (64, 3000), (300, 300), (1500, 4000)], 4, 4, 64, 16, 8, 400, 20),
    ([(700, 900), (64, 3000), (300, 300), (1500, 4000)], 4, 4, 64, 16, 16, 400, 20),
    ([(20, 21000)], 8, 4, 128, 64, 16, 0, 0),
    ([(20, 21000)], 8, 4, 128, 64, 8, 0, 0),
    ([(30, 20000), (5, 700), (17, 9000)], 8, 4, 64, 128, 8, 0, 0),
    ([(30, 20000), (5, 700), (17, 9000)], 8, 4, 64, 128, 16, 0, 0),
    ([(200, 9000), (130, 130)], 8, 8, 128, 32, 8, 0, 0),
    ([(200, 9000), (130, 130)], 8, 8, 128, 32, 16, 3000, 100),
    ([(1, 40000)], 3, 5, 128, 64, 8, 0, 0),
    ([(1, 40000), (1, 20)], 2, 16, 128, 64, 16, 0, 0),
    ([(3, 30000), (2, 1)], 4, 4, 64, 16, 16, 0, 0),
    ([(1, 5 + 37 * i) for i in range(70)], 4, 4, 128, 32, 8, 0, 0),
    # more sequences than a warp looks over at once, most short, some without rows, one long
    ([(i % 7 and 1, 1 + 13 * i % 97) for i in range(150)] + [(1, 6000)] + [(2, 3 + 5 * i) for i in range(150)], 2, 2, 128, 16, 16, 0, 0),
    ([(i % 7 and 1, 1 + 13 * i % 97) for i in range(150)] + [(1, 12000)] + [(2, 3 + 5 * i) for i in range(150)], 2, 2, 128, 16, 8, 0, 0),
    # as many units as fill the GPU, ragged
    ([(1, 200 + 450 * i) for i in range(20)], 8, 2, 128, 64, 16, 0, 0),
    ([(1, 200 + 450 * i) for i in range(20)], 8, 1, 64, 64, 8, 2500, 7),
    # few units of many rows, long enough to be cut all the same
    ([(30, 2500), (25, 40), (0, 9)], 3, 3, 128, 64, 16, 0, 0),
    ([(30, 2500), (25, 40), (0, 9)], 3, 3, 128, 64, 8, 0, 0),
    ([(90, 3100)], 1, 4, 64, 16, 16, 0, 0),
]


@pytest.mark.parametrize("case", range(len(LARGE)))
def test_attention_at_sizes_that_share_the_gpu(clo, case):
    seqs, hkv, group, d, page, bits, window, sinks = LARGE[case]
    seqs = [(n, max(n, kv)) for n, kv in seqs]
    c = Case(clo, seqs, hkv, d, page, bits, seed=200 + case)
    c.device()
    q = bf16(rand(300 + case, c.total, hkv * group, d) * 2)
    want, spread, reach = dense_on_device(c, q, window, sinks)
    bound = ref.attention_bound(want, spread, reach, d, bits)
    check(c.attend(q, window, sinks), want, bound)
    # without a workspace (one that is too small is none), and again with one that holds garbage
    check(c.attend(q, window, sinks, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), want, bound, "no workspace")
    size = c.cache.attention_workspace(hkv * group, len(seqs), c.total, c.tab.shape[1], c.max_q, window, sinks)
    work = torch.full((size + 64,), 0xff, dtype=torch.uint8, device="cuda")
    first = c.attend(q, window, sinks, workspace=work)
    check(first, want, bound, "given workspace")
    assert bool((work[size:] == 0xff).all()), "written past the workspace"
    assert torch.equal(first, c.attend(q, window, sinks, workspace=work)), "two runs differ"


def test_calls_on_named_streams_at_once(clo):
    """Two streams that the caller names, work of both in flight, outputs and workspaces of the current stream's allocator, whose
    freed memory the current stream overwrites at once."""
    cases, want = [], []
    for seed, seqs in ((31, [(1, 20000), (1, 700)]), (32, [(40, 9000), (2, 30)])):
        c = Case(clo, seqs, 4, 128, 64, 16, seed=seed)
        c.device()
        q = bf16(rand(seed, c.total, 16, 128)).cuda()
        assert c.cache.attention_workspace(16, len(seqs), c.total, c.tab.shape[1], c.max_q) > 0
        cases.append((c, q, torch.cuda.Stream()))
        want.append(c.cache.attention(q, c.starts, c.lens, c.tab, max_q=c.max_q).cpu())
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (c, q, s) in enumerate(cases):
            got[i].append(c.cache.attention(q, c.starts, c.lens, c.tab, max_q=c.max_q, stream=s))
            c.cache.attention(q, c.starts, c.lens, c.tab, max_q=c.max_q, stream=s)  # dropped before it has run
            torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
            torch.full((c.total, 16, 128), 3.0, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o.cpu(), want[i])


def test_streams_by_handle(clo):
    # the default stream, its other name, the thread's own, one of torch's as a number and as an object
    c = Case(clo, [(1, 9000)], 2, 64, 32, 16, seed=41)
    c.device()
    q = bf16(rand(41, c.total, 8, 64)).cuda()
    plan = clo.clo_rope_plan_init(rot_dim=64)
    pos = torch.tensor([70000], dtype=torch.int64, device="cuda")
    want = c.attend(q).cpu(), clo.clo_rope(plan, q, pos).cpu()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (0, 1, 2, side.cuda_stream, side):
        got = (c.cache.attention(q, c.starts, c.lens, c.tab, max_q=c.max_q, stream=stream), clo.clo_rope(plan, q, pos, stream=stream))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g.cpu(), w)
    del got, g
    torch.cuda.synchronize()


def test_attention_offsets_past_32_bits(clo):
    # pages whose element offsets pass 2^32: few tokens, far apart
    d, page, hkv = 128, 128, 1
    n_pages = (1 << 32) // (page * d) + 70
    for bits in (16, 8):
        dt = BF16 if bits == 16 else torch.float8_e4m3fn
        k = torch.empty((n_pages, hkv, page, d), dtype=dt, device="cuda")
        v = torch.empty_like(k)
        sc = [torch.ones(n_pages, hkv, device="cuda") for _ in range(2)] if bits == 8 else [None, None]
        cache = clo.PagedCache(k, v, *sc)
        ids = [n_pages - 1, 3, n_pages - 64]
        table = torch.tensor([ids], dtype=torch.int32, device="cuda")
        n = 2 * page + 60
        x = bf16(rand(1, n, hkv, d)), bf16(rand(2, n, hkv, d))
        starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        cache.append(x[0].cuda(), x[1].cuda(), starts, lens, table)
        gk, gv = cache.read(starts, lens, table, n)
        if bits == 16:
            assert torch.equal(gk.cpu(), x[0]) and torch.equal(gv.cpu(), x[1])
        local = torch.tensor([[0, 1, 2]], dtype=torch.int32)
        vals = [torch.zeros(3, hkv, page, d, dtype=torch.float64) for _ in range(2)]
        for side, got in enumerate((gk, gv)):
            for j in range(n):
                vals[side][j // page, :, j % page] = got[j].cpu().double()
        pages = ref.Pages(*vals)
        for rows in (1, 64):
            q = bf16(rand(5, rows, 4, d))
            st = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
            got = cache.attention(q.cuda(), st, lens, table)
            want, spread, reach = ref.attention(pages, q, [(0, rows, n)], local, 4)
            check(got, want, ref.attention_bound(want, spread, reach, d, bits))
        del cache, k, v


# --------------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("bits", [16, 8])
def test_prompt_then_steps_with_a_graph(clo, bits):
    # a prompt, then single-token steps: append with rotation, attention, the step captured once and replayed;
    # a second graph over its own buffers runs between the replays
    hq, hkv, d, page, prompt, steps = 8, 2, 128, 16, 45, 6
    plan = clo.clo_rope_plan_init(rot_dim=d, theta=500000.0)
    lens0 = [prompt, prompt - 12]
    caches, tables = [], []
    for g in range(2):
        caches.append(clo.PagedCache.create(12, hkv, page, d, kv_bits=bits))
        tables.append(torch.randperm(12, generator=torch.Generator().manual_seed(g))[:8].view(2, 4).to(torch.int32).cuda())
    total = sum(lens0)
    starts = torch.tensor([0, lens0[0], total], dtype=torch.int32, device="cuda")
    refs = []
    for g in range(2):
        k, v, q = (bf16(rand(40 + 10 * g + i, total, h, d)) for i, h in enumerate((hkv, hkv, hq)))
        lens = torch.tensor(lens0, dtype=torch.int32, device="cuda")
        qr = caches[g].append(k.cuda(), v.cuda(), starts, lens, tables[g], rope=plan, q=q.cuda())
        out = caches[g].attention(qr, starts, lens, tables[g], max_q=prompt)
        val = device_values(caches[g])
        pages = ref.Pages(val[0][0], val[1][0], val[0][1], val[1][1])
        seqs = [(0, lens0[0], lens0[0]), (lens0[0], lens0[1], lens0[1])]
        want, spread, reach = ref.attention(pages, qr.cpu(), seqs, tables[g].cpu(), hq // hkv)
        check(out, want, ref.attention_bound(want, spread, reach, d, bits), "prompt")
        refs.append(lens)
    ones = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    bufs, graphs = [], []
    for g in range(2):
        kb, vb, qb = (torch.zeros(2, h, d, dtype=BF16, device="cuda") for h in (hkv, hkv, hq))
        qr, ob = torch.empty_like(qb), torch.empty_like(qb)

        def step(g=g, kb=kb, vb=vb, qb=qb, qr=qr, ob=ob):
            refs[g].add_(1)
            caches[g].append(kb, vb, ones, refs[g], tables[g], rope=plan, q=qb, q_out=qr, max_q=1)
            caches[g].attention(qr, ones, refs[g], tables[g], out=ob, max_q=1)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        bufs.append((kb, vb, qb, qr, ob))
        graphs.append(graph)
    for i in range(steps):
        for g in range(2):
            for n, t in enumerate(bufs[g][:3]):
                t.copy_(bf16(rand(1000 + 100 * g + 10 * i + n, *t.shape)).cuda())
        for g in range(2):
            graphs[g].replay()
        torch.cuda.synchronize()
        for g in range(2):
            now = refs[g].tolist()
            assert now == [x + i + 1 for x in lens0]
            kb, vb, qb, qr, ob = bufs[g]
            pos = torch.tensor([x - 1 for x in now])
            want = ref.rotate(qb.cpu(), pos, d, theta=500000.0)
            check(qr, want, rope_bound(want, qb.cpu()), "rotated q")
            val = device_values(caches[g])
            pages = ref.Pages(val[0][0], val[1][0], val[0][1], val[1][1])
            want, spread, reach = ref.attention(pages, qr.cpu(), [(0, 1, now[0]), (1, 1, now[1])], tables[g].cpu(), hq // hkv)
            check(ob, want, ref.attention_bound(want, spread, reach, d, bits), f"step {i}")
            # the new key is the rotated one
            gk, gv = caches[g].read(ones, refs[g], tables[g], 2)
            kw = ref.rotate(kb.cpu(), pos, d, theta=500000.0)
            bound = rope_bound(kw, kb.cpu()) if bits == 16 else 2.0 ** -4 * kw.abs() + 2.0 ** -8 * 2.0 ** -2 + 1e-4
            check(gk, kw, bound, "key")


def test_paged_sequence_moves_to_the_host_pool(clo):
    # a prompt in pages, read back and offloaded: a decode step that selects every token agrees with the paged attention
    from host_offloaded_kv_gb300.clo import CLOContext
    from host_offloaded_kv_gb300.synth import Synth

    hq, hkv, d, page, n = 8, 2, 64, 32, 100
    plan = clo.clo_rope_plan_init(rot_dim=d)
    cache = clo.PagedCache.create(6, hkv, page, d)
    table = torch.tensor([[4, 0, 5, 2]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    k, v = bf16(rand(1, n, hkv, d)).cuda(), bf16(rand(2, n, hkv, d)).cuda()
    cache.append(k, v, starts, lens, table, rope=plan)
    gk, gv = cache.read(starts, lens, table, n)
    lib = CLOContext(n_layers=1, batch=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, max_tokens=n,
                     hash_R=Synth(3).hash_matrices(1, hkv, d), topk=n, tau=np.full(hkv, 2.0, dtype=np.float32))
    try:
        torch.cuda.synchronize()
        lib.append_kv(0, 0, gk.view(torch.int16), gv.view(torch.int16))
        q = clo.clo_rope(plan, bf16(rand(3, 1, hq, d)).cuda(), torch.tensor([n - 1], device="cuda"))
        out = torch.empty((1, 1, hq, d), dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        lib.decode_step(q.view(torch.int16).view(1, 1, hq, d).contiguous(), out)
        lib.sync()
        one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        paged = cache.attention(q, one, lens, table)
        want = out.cpu().double().view(1, hq, d)
        # both are within 2^-8 of the weighted mean of |V| <= 4.5 and one bf16 rounding of each other
        check(paged, want, 2.0 ** -8 * want.abs() + 2 * 2.0 ** -8 * 4.5 * torch.ones_like(want))
    finally:
        lib.close()
