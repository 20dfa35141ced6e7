"""4-bit pages on the GPU, against plain 64-bit forms (tests/paged4_ref.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

import paged4_ref as ref4  # noqa: E402
import paged_ref as ref  # noqa: E402
from test_gpu_paged import ATTEND, BATCHES, BF16, LARGE, bf16, check, dense_on_device, rand, rope_bound  # noqa: E402

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def clo():
    from host_offloaded_kv_gb300 import clo as m

    m.load_library()
    return m


class Case:
    """A batch on the CPU and on the device: seqs are (rows, kv_len); pages are handed out in shuffled order."""

    def __init__(self, clo, seqs, hkv, d, page, seed, extra=3, holes=(), by_token=False, width=None):
        self.clo, self.page, self.hkv, self.d, self.by_token = clo, page, hkv, d, by_token
        self.bits = 8  # for the bound of attention: fp16 products
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
        code, group, scale = [], [], []
        for side in range(2):
            c = torch.randint(0, 256, (n_pages, hkv, page, d // 2), generator=gen, dtype=torch.uint8)
            code.append(ref4.codes_of(c) + 0.0)
            group.append(ref4.E4M3[torch.randint(40, 72, (n_pages, hkv, page, d // 16), generator=gen)])
            scale.append(torch.exp2(torch.randint(-3, 2, (n_pages, hkv), generator=gen).double()))
        self.pages4 = ref4.Pages4(code, group, scale)
        self.scales = [None, None]

    @property
    def pages(self):
        return self.pages4.plain()

    def device(self):
        p = self.pages4
        like = lambda t: t.cuda().transpose(1, 2).contiguous().transpose(1, 2) if self.by_token else t.cuda()  # noqa: E731
        e4m3 = lambda t: t.float().to(torch.float8_e4m3fn).view(torch.uint8).cuda().view(torch.float8_e4m3fn)  # noqa: E731
        self.cache = self.clo.PagedCache(*(like(ref4.bytes_of(c)) for c in p.code), *(s.float().cuda() for s in p.scale), *(e4m3(g) for g in p.group))
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.starts, self.lens, self.tab = i32([s[0] for s in self.seqs] + [self.total]), i32([s[2] for s in self.seqs]), self.table.cuda()
        return self.cache

    @property
    def max_q(self):
        return max(s[1] for s in self.seqs)

    def attend(self, q, window=0, sinks=0, scale=0.0, **kw):
        return self.cache.attention(q.cuda(), self.starts, self.lens, self.tab, max_q=kw.pop("max_q", self.max_q), window=window, sinks=sinks,
                                    softmax_scale=scale, **kw)

    def compare(self, got, q, window=0, sinks=0, scale=None, what=""):
        want, spread, reach = ref.attention(self.pages, q, self.seqs, self.table, q.shape[1] // self.hkv, scale, window, sinks)
        check(got, want, limit(self.pages4, self.seqs, want, spread, reach, self.d), what)


def limit(pages4, seqs, want, spread, reach, d):
    """What the kernels may be off: as for 8-bit pages (paged_ref.attention_bound), and what fp16 loses of small weights.  A row's largest weight (times
    its page's scale) is held as 2^7 or more, one below 2^-14 is rounded by up to 2^-25, so each of the row's tokens adds at most
    2^-32 of the largest page scale times its code and group scale; the sum of the weights is one at least."""
    tokens = max(kv for _, _, kv in seqs)
    most = max(float((torch.isfinite(g) * g.nan_to_num(0.0)).max()) for g in pages4.group[1:]) * 6.0 * float(pages4.scale[1].max())
    return ref.attention_bound(want, spread, reach, d, 8) + 2.0 ** -32 * tokens * most


def same(cache, want, written=None):
    """The device cache holds exactly these values, group scales and page scales."""
    got = ref4.of_cache(cache)
    for side in range(2):
        assert torch.equal(got.scale[side], want.scale[side]), f"page scales of side {side}"
        assert torch.equal(got.group[side].nan_to_num(nan=-1.0), want.group[side].nan_to_num(nan=-1.0)), f"group scales of side {side}"
        gone = torch.isnan(want.group[side]).repeat_interleave(16, dim=-1)  # codes of a NaN group mean nothing
        assert torch.equal(torch.where(gone, 0.0, got.code[side]), torch.where(gone, 0.0, want.code[side])), f"codes of side {side}"


# --------------------------------------------------------------------------------------------- append and read
@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("d,page,by_token", [(64, 16, False), (128, 64, True), (128, 32, False), (64, 128, True), (128, 16, False), (128, 128, False)])
@pytest.mark.parametrize("mode", ["plain", "half", "part", "odd", "axes"])
def test_append_and_read(clo, batch, d, page, by_token, mode):
    # every code, group scale and page scale is that of the exactly rotated keys; q comes along
    hkv, hq = 3, 7
    c = Case(clo, BATCHES[batch], hkv, d, page, seed=len(batch) + d + page, by_token=by_token)
    cache = c.device()
    k, v, q = bf16(rand(1, c.total, hkv, d) * (0.01 if batch == "ragged" else 30)), bf16(rand(2, c.total, hkv, d)), bf16(rand(3, c.total, hq, d))
    pos = torch.cat([torch.arange(kv - n, kv) for _, n, kv in c.seqs])
    given = pos * 3 + 1000 if mode in ("part", "odd") else None
    rot, inter = {"half": (d, False), "part": (d // 2, True), "odd": (48, False), "axes": (d, False), "plain": (0, False)}[mode]
    pairs = (d // 2 - 20, 11, 9)
    plan = None if mode == "plain" else clo.clo_rope_plan_init(rot_dim=rot, interleaved=inter, **(dict(axis_pairs=pairs, axis_order="cycled") if mode == "axes" else {}))
    if mode == "axes":
        from test_rope_axes import rotate

        given = torch.stack([pos * 0 + 77, pos // 5, pos % 5])
        turned = lambda x: rotate(x, given, rot, pairs, "cycled")  # noqa: E731
    else:
        turned = lambda x: x.double() if plan is None else ref.rotate(x, pos if given is None else given, rot, inter)  # noqa: E731
    got_q = cache.append(k.cuda(), v.cuda(), c.starts, c.lens, c.tab, rope=plan, positions=None if given is None else given.cuda(),
                         q=None if plan is None else q.cuda(), max_q=c.max_q)
    c.pages4.append(0, turned(k), c.seqs, c.table)
    c.pages4.append(1, v.double(), c.seqs, c.table)
    if plan is not None:
        want = turned(q)
        check(got_q, want, rope_bound(want, q), "q")
    same(cache, c.pages4)
    # read back what the pages now hold: whole sequences
    back = [(sum(max(s[2], 0) for s in c.seqs[:b]), max(s[2], 0)) for b, s in enumerate(c.seqs)]
    total = sum(r[1] for r in back)
    starts = torch.tensor([r[0] for r in back] + [total], dtype=torch.int32, device="cuda")
    for side, got in enumerate(cache.read(starts, c.lens, c.tab, total)):
        want = torch.zeros(total, hkv, d, dtype=torch.float64)
        for b, (first, n) in enumerate(back):
            j = torch.arange(n)
            want[first:first + n] = c.pages.val[side][c.table[b, j // page].long(), :, j % page]
        assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("positions", [(0, 200), (1 << 19, (1 << 19) + 4000), (-4000, 4000)])
def test_codes_are_those_of_the_exact_rotation(clo, positions, interleaved):
    # 6 million keys: about as many lie within fp32's error of a border between two codes as would show in a comparison
    d, hkv, page, n = 128, 8, 64, 6016
    k = bf16(rand(11, n, hkv, d))
    pos = torch.randint(*positions, (n,), generator=torch.Generator().manual_seed(12))
    cache = clo.PagedCache.create(n // page, hkv, page, d, kv_bits=4, group=16)
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = clo.clo_rope_plan_init(rot_dim=d, theta=500000.0, interleaved=interleaved)
    cache.append(k.cuda(), k.cuda(), i32(0, n), i32(n), table, rope=plan, positions=pos.cuda())
    x = ref.rotate(k, pos, d, interleaved, theta=500000.0)
    got = ref4.of_cache(cache)
    for side, rows in ((0, x), (1, k.double())):
        rows = rows.view(-1, page, hkv, d).transpose(1, 2)
        need = torch.tensor([[ref4.needed_scale(float(m)) for m in r] for r in rows.abs().amax((-1, -2))], dtype=torch.float64)
        assert torch.equal(got.scale[side], need)
        code, group = ref4.encode(rows, need[:, :, None, None])
        assert torch.equal(got.group[side], group)
        assert torch.equal(got.code[side], code)


def test_append_token_by_token_grows_the_scale_of_a_page(clo):
    # growing values: the page's scale follows, the earlier tokens' group scales shrink, their codes stay
    d, page = 64, 16
    c = Case(clo, [(1, page)], 2, d, page, seed=4)
    cache = c.device()
    for i in range(page):
        x = bf16(rand(100 + i, 1, 2, d) * 2.0 ** (3 * i - 6))
        c.seqs = [(0, 1, i + 1)]
        cache.append(x.cuda(), x.cuda(), c.starts, torch.tensor([i + 1], dtype=torch.int32, device="cuda"), c.tab, max_q=1)
        for side in range(2):
            c.pages4.append(side, x.double(), c.seqs, c.table)
    same(cache, c.pages4)


def test_append_of_values_at_the_formats_ends(clo):
    # infinities, NaN, zeros, groups far below the page's largest value, the smallest and largest bf16 numbers, borders between codes
    d, page = 128, 32
    c = Case(clo, [(9, 9), (2, 40), (1, 70), (32, 32)], 2, d, page, seed=9)
    cache = c.device()
    x = rand(5, c.total, 2, d)
    x[0, 0, 3], x[1, 1, 7], x[9, 0, 0], x[10, 1, 127], x[11] = INF, NAN, -INF, NAN, 0.0
    x[2] = 0.0
    x[2, :, 0] = 1e-30
    x[3, 0, 16:32] *= 1e-5
    x[4, 0, :16], x[4, 0, 16:32], x[4, 1] = INF, NAN, -INF
    x[12:22] *= 2.0 ** 126
    x[22:] *= 2.0 ** -130
    # halfway between codes for a group scale of one over the page's: 6 is the group's largest
    x[5, 0, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0])
    x[6, 1, :16] = x[5, 0, :16] * 1.125
    x = bf16(x)
    cache.append(x.cuda(), x.cuda(), c.starts, c.lens, c.tab, max_q=32)
    for side in range(2):
        c.pages4.append(side, x.double(), c.seqs, c.table)
    same(cache, c.pages4)
    # a NaN or infinite page scale that was there is replaced by the needed one
    cache.k_scales.fill_(NAN)
    one = bf16(rand(6, 1, 2, d)).cuda()
    cache.append(one, one, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([10], dtype=torch.int32, device="cuda"), c.tab[:1])
    got = float(cache.k_scales[int(c.table[0, 0]), 0])
    assert got == ref4.needed_scale(float(one[0, 0].double().abs().max()))


def test_append_skips_pages_that_are_not_there(clo):
    d, page, hkv = 64, 16, 2
    c = Case(clo, [(40, 40), (20, 50), (1, 33)], hkv, d, page, seed=6, holes=[(0, 1, -1), (1, 2, 1 << 20), (2, 2, -7)], width=3)
    cache = c.device()
    k = bf16(rand(7, c.total, hkv, d))
    cache.append(k.cuda(), k.cuda(), c.starts, c.lens, c.tab, max_q=40)
    written = [c.pages4.append(side, k.double(), c.seqs, c.table) for side in range(2)][0]
    same(cache, c.pages4)
    gk, _ = cache.read(c.starts, c.lens, c.tab, c.total)
    for b, (first, n, kv) in enumerate(c.seqs):
        for i in range(n):
            pos = kv - n + i
            pid = int(c.table[b, pos // page]) if pos // page < 3 else -1
            there = 0 <= pid < written.shape[0]
            want = c.pages.val[0][pid, :, pos % page] if there else torch.zeros(hkv, d, dtype=torch.float64)
            assert torch.equal(gk[first + i].cpu().double(), want)


# --------------------------------------------------------------------------------------------- attention
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(clo, case):
    seqs, hkv, group, d, page, _, window, sinks = ATTEND[case]
    c = Case(clo, seqs, hkv, d, page, seed=20 + case, by_token=case % 2 == 1)
    c.device()
    q = bf16(rand(50 + case, c.total, hkv * group, d))
    c.compare(c.attend(q, window, sinks), q, window, sinks)
    c.compare(c.attend(q, window, sinks, max_q=None), q, window, sinks, what="max_q of the whole call")


@pytest.mark.parametrize("case", [i for i, x in enumerate(LARGE) if x[5] == 8])
def test_attention_at_sizes_that_share_the_gpu(clo, case):
    seqs, hkv, group, d, page, _, window, sinks = LARGE[case]
    c = Case(clo, seqs, hkv, d, page, seed=300 + case)
    c.device()
    q = bf16(rand(301 + case, c.total, hkv * group, d))
    want, spread, reach = dense_on_device(c, q, window, sinks)
    bound = limit(c.pages4, c.seqs, want, spread, reach, d)
    got = c.attend(q, window, sinks)
    check(got, want, bound)
    check(c.attend(q, window, sinks, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), want, bound, "no workspace")
    assert torch.equal(c.attend(q, window, sinks), got)  # the order of sums is fixed


@pytest.mark.parametrize("rows", [1, 3, 60])
def test_attention_ignores_what_masked_tokens_hold(clo, rows):
    # group scales of NaN where no row, or not every row, looks: slots past the length, before the window, the rows' own later tokens
    d, page, hkv, group, kv, window, sinks = 128, 16, 2, 4, 300, 90, 3
    c = Case(clo, [(rows, kv), (rows, rows)], hkv, d, page, seed=31, holes=[(0, 16, -1)])
    for side in range(2):
        g = c.pages4.group[side]
        g[int(c.table[0, (kv - 1) // page]), :, (kv - 1) % page + 1:] = NAN
        for j in (sinks, sinks + 5, kv - rows - window, kv - rows - window - 1):
            g[int(c.table[0, j // page]), :, j % page] = NAN
        g[int(c.table[1, (rows - 1) // page]), :, (rows - 1) % page + 1:] = NAN
        if rows > 1:  # visible to the last row alone
            for b, k in ((0, kv), (1, rows)):
                g[int(c.table[b, (k - 1) // page]), 0, (k - 1) % page, 5] = NAN
    c.device()
    q = bf16(rand(77, c.total, hkv * group, d))
    c.compare(c.attend(q, window, sinks), q, window, sinks)


@pytest.mark.parametrize("seqs,hkv,group,d,page,window,sinks,marks", [
    ([(1300, 1300)], 2, 4, 128, 64, 0, 0, [(0, 0, 0, 2), (0, 1, 300, 0), (0, 1, 1000, 7)]),
    ([(900, 1500), (20, 20)], 2, 4, 64, 32, 300, 5, [(0, 0, 2, 1), (0, 0, 6, 2), (0, 1, 700, 3), (1, 1, 19, 0)]),
    ([(40, 9000)], 2, 2, 128, 64, 0, 0, [(0, 0, 100, 7), (0, 1, 8970, 4)]),
    ([(200, 6000)], 2, 3, 64, 16, 0, 0, [(0, 0, 0, 3), (0, 1, 5900, 0)]),
    ([(3, 30000)], 2, 3, 128, 16, 0, 0, [(0, 0, 29999, 3), (0, 1, 29998, 0)])])
def test_rows_are_nan_where_they_see_a_group_of_nan(clo, seqs, hkv, group, d, page, window, sinks, marks):
    c = Case(clo, seqs, hkv, d, page, seed=80)
    clean = [g.clone() for g in c.pages4.group]
    for b, h, j, g in marks:
        p = int(c.table[b, j // page])
        clean[1][p, h, j % page, g] = 0.0
        c.pages4.group[1][p, h, j % page, g] = NAN
    c.device()
    q = bf16(rand(81, c.total, hkv * group, d))
    c.pages4.group = clean
    want, spread, reach = dense_on_device(c, q, window, sinks)
    bound = limit(c.pages4, c.seqs, want, spread, reach, d)
    for b, h, j, g in marks:
        first, n, kv = c.seqs[b]
        pos = torch.arange(kv - n, kv)
        see = (pos >= j) & ((pos - window < j) | (j < sinks) if window else True)
        want[first:first + n, h * group:(h + 1) * group, 16 * g:16 * g + 16] += torch.where(see, NAN, 0.0)[:, None, None]
    check(c.attend(q, window, sinks), want, bound)
    check(c.attend(q, window, sinks, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), want, bound, "no workspace")


@pytest.mark.parametrize("seqs", [[(1, 60000), (1, 25000)], [(200, 3000)]])
@pytest.mark.parametrize("power", [1e-30, 2.0 ** -64, 2.0 ** 100])
def test_page_scales_at_the_ends_of_their_range(clo, seqs, power):
    # V's scales: weights that are nearly equal over many tokens, divided by such scales; K's stay small enough that q.K is
    c = Case(clo, seqs, 2, 64, 128, seed=130)
    c.pages4.scale[1] = (c.pages4.scale[1] * power).clamp(min=1e-30).float().double()
    c.device()
    q = bf16(rand(131, c.total, 8, 64) * 1e-3)
    want, spread, reach = dense_on_device(c, q)
    unit = float(want.abs().max())  # (the bound's floor of 1e-30 is about values near one)
    bound = limit(c.pages4, c.seqs, want, spread, reach, 64) / unit
    for work in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):
        check(c.attend(q, workspace=work).double() / unit, want / unit, bound)


def test_group_scales_at_the_ends_of_their_range(clo):
    # 448 and 2^-9 beside each other in a row, and zero: values are exact in the products
    for rows in (1, 50):
        c = Case(clo, [(rows, 200)], 2, 128, 32, seed=140)
        for side in range(2):
            pick = torch.randint(0, 3, c.pages4.group[side].shape, generator=torch.Generator().manual_seed(side))
            c.pages4.group[side] = torch.tensor([448.0, 2.0 ** -9, 0.0], dtype=torch.float64)[pick]
            c.pages4.scale[side].fill_(2.0 ** -9)
        c.device()
        q = bf16(rand(141, rows, 8, 128) * 0.1)
        c.compare(c.attend(q), q)


def test_empty_calls_and_unwritten_rows(clo):
    c = Case(clo, [(2, 40), (0, 9), (3, 50)], 2, 64, 16, seed=150)
    cache = c.device()
    q = bf16(rand(151, c.total + 2, 4, 64)).cuda()
    out = torch.full_like(q, 7.0)
    cache.attention(q, c.starts, c.lens, c.tab, out=out, max_q=3)
    c.compare(out[:c.total], q[:c.total].cpu())
    assert bool((out[c.total:] == 7.0).all())  # rows behind the last sequence are left as they were
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert cache.attention(q[:0], none, none[:0], c.tab[:0]).shape == (0, 4, 64)
    k, v = cache.read(none, none[:0], c.tab[:0], 0)
    assert k.shape == v.shape == (0, 2, 64)
    before = ref4.of_cache(cache)
    cache.append(k, v, none, none[:0], c.tab[:0])
    cache.append(k, v, c.starts * 0, c.lens, c.tab)
    same(cache, before)
    # rows beyond max_q are left out by every call
    x = bf16(rand(152, c.total, 2, 64)).cuda()
    cache.append(x, x, c.starts, c.lens, c.tab, max_q=1)
    first = [(c.seqs[0][0], 1, 39), (0, 0, 9), (c.seqs[2][0], 1, 48)]
    for side in range(2):
        c.pages4.append(side, x.cpu().double(), first, c.table)
    same(cache, c.pages4)


def test_offsets_past_32_bits(clo):
    # codes beyond 2^32 bytes, group scales beyond 2^32 bytes: few tokens, far apart
    d, page, hkv = 128, 128, 4
    n_pages = (1 << 32) // (page * hkv * d // 16) + 70
    cache = clo.PagedCache.create(n_pages, hkv, page, d, kv_bits=4, group=16)
    assert cache.k_group_scales.numel() > 1 << 32 and cache.k_pages.numel() > 1 << 34
    table = torch.tensor([[n_pages - 1, 3, n_pages - 64]], dtype=torch.int32, device="cuda")
    n = 2 * page + 60
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x = [bf16(rand(i, n, hkv, d)) for i in (1, 2)]
    cache.append(x[0].cuda(), x[1].cuda(), i32(0, n), i32(n), table)
    c = Case(clo, [(n, n)], hkv, d, page, seed=1, extra=0)
    for side, got in enumerate(cache.read(i32(0, n), i32(n), table, n)):
        c.pages4.append(side, x[side].double(), c.seqs, c.table)
        ids = c.table[0].long()[torch.arange(n) // page]
        assert torch.equal(got.cpu().double(), c.pages.val[side][ids, :, torch.arange(n) % page])
    for rows in (1, 64):
        q = bf16(rand(5, rows, 8, d))
        got = cache.attention(q.cuda(), i32(0, rows), i32(n), table)
        want, spread, reach = ref.attention(c.pages, q, [(0, rows, n)], c.table, 2)
        check(got, want, limit(c.pages4, c.seqs, want, spread, reach, d))


# --------------------------------------------------------------------------------------------- together
def test_prompt_then_steps_with_a_graph(clo):
    # a prompt with an image, then single-token steps: append with rotation by three axes, attention, the step captured once and replayed; a
    # second graph over its own buffers runs on another stream at the same time
    hq, hkv, d, page, prompt, steps = 8, 2, 128, 16, 45, 5
    pairs = (24, 20, 20)
    plan = clo.clo_rope_plan_init(rot_dim=d, theta=500000.0, axis_pairs=pairs, axis_order="cycled")
    lens0 = [prompt, prompt - 12]
    total = sum(lens0)
    starts = torch.tensor([0, lens0[0], total], dtype=torch.int32, device="cuda")
    ones = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lens, caches, tables, bufs, graphs, streams = [], [], [], [], [], []
    for g in range(2):
        cache = clo.PagedCache.create(12, hkv, page, d, kv_bits=4, group=16)
        table = torch.randperm(12, generator=torch.Generator().manual_seed(g))[:8].view(2, 4).to(torch.int32).cuda()
        k, v, q = (bf16(rand(40 + 10 * g + i, total, h, d)) for i, h in enumerate((hkv, hkv, hq)))
        at = torch.randint(0, 60, (3, total), generator=torch.Generator().manual_seed(g)).cuda()
        n = torch.tensor(lens0, dtype=torch.int32, device="cuda")
        qr = cache.append(k.cuda(), v.cuda(), starts, n, table, rope=plan, positions=at, q=q.cuda())
        out = cache.attention(qr, starts, n, table, max_q=prompt)
        seqs = [(0, lens0[0], lens0[0]), (lens0[0], lens0[1], lens0[1])]
        held = ref4.of_cache(cache)
        want, spread, reach = ref.attention(held.plain(), qr.cpu(), seqs, table.cpu(), hq // hkv)
        check(out, want, limit(held, seqs, want, spread, reach, d), "prompt")
        kb, vb, qb = (torch.zeros(2, h, d, dtype=BF16, device="cuda") for h in (hkv, hkv, hq))
        pb, qo, ob = torch.zeros(3, 2, dtype=torch.int64, device="cuda"), torch.empty_like(qb), torch.empty_like(qb)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            n.add_(1)
            cache.append(kb, vb, ones, n, table, rope=plan, positions=pb, q=qb, q_out=qo, max_q=1)
            cache.attention(qo, ones, n, table, out=ob, max_q=1)
        for x, y in ((lens, n), (caches, cache), (tables, table), (bufs, (kb, vb, qb, pb, qo, ob)), (graphs, graph), (streams, torch.cuda.Stream())):
            x.append(y)
    for i in range(steps):
        for g in range(2):
            for n, t in enumerate(bufs[g][:3]):
                t.copy_(bf16(rand(1000 + 100 * g + 10 * i + n, *t.shape)).cuda())
            bufs[g][3].fill_(50 + i)
        torch.cuda.synchronize()
        before = [ref4.of_cache(c) for c in caches]
        for g in range(2):
            with torch.cuda.stream(streams[g]):
                graphs[g].replay()
        torch.cuda.synchronize()
        for g in range(2):
            kb, vb, qb, pb, qo, ob = (t.cpu() for t in bufs[g])
            now = lens[g].tolist()
            assert now == [x + i + 1 for x in lens0]
            seqs = [(0, 1, now[0]), (1, 1, now[1])]
            before[g].append(0, ref.rotate(kb, torch.tensor([50 + i] * 2), d, theta=500000.0), seqs, tables[g].cpu())
            before[g].append(1, vb.double(), seqs, tables[g].cpu())
            same(caches[g], before[g])
            want = ref.rotate(qb, torch.tensor([50 + i] * 2), d, theta=500000.0)
            check(qo, want, rope_bound(want, qb), "rotated q")
            want, spread, reach = ref.attention(before[g].plain(), qo, seqs, tables[g].cpu(), hq // hkv)
            check(ob, want, limit(before[g], seqs, want, spread, reach, d), f"step {i}")


def test_sequence_moves_to_the_host_pool(clo):
    # a prompt in 4-bit pages, read back and offloaded: a decode step that selects every token agrees with the paged attention
    from host_offloaded_kv_gb300.clo import CLOContext
    from host_offloaded_kv_gb300.synth import Synth  # noqa: F401

    hq, hkv, d, n = 8, 2, 128, 200
    import numpy as np

    c = Case(clo, [(1, n)], hkv, d, 64, seed=170)
    cache = c.device()
    one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    k, v = cache.read(one, c.lens, c.tab, n)
    q = bf16(rand(171, 1, hq, d)).cuda()
    want = c.attend(q.cpu())
    R = np.random.default_rng(0).standard_normal((128, d)).astype(np.float32)
    R16 = torch.from_numpy(R).to(BF16).view(torch.int16).numpy().view(np.uint16)
    ctx = CLOContext(n_layers=1, batch=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, max_tokens=n + 8, hash_R=R16, topk=n, tau=np.full((1, hkv), 2.0, np.float32),
                     persist_mask=np.zeros((1, hkv), np.uint8), warmup_steps=0)
    try:
        ctx.append_kv(0, 0, k.view(torch.int16), v.view(torch.int16), src_is_device=True)
        out = torch.empty(1, 1, hq, d, dtype=torch.float32, device="cuda")
        ctx.decode_step(q.view(1, 1, hq, d).view(torch.int16), out, io_on_device=True)
        ctx.sync()
    finally:
        ctx.close()
    # two roundings to bf16 of the output and of the weights (2^-8 each), as sums over values of size `spread`
    _, spread, _ = ref.attention(c.pages, q.cpu(), c.seqs, c.table, hq // hkv)
    off = (out.view(1, hq, d).cpu().double() - want.cpu().double()).abs()
    assert bool((off <= 4 * 2.0 ** -8 * spread + 1e-6).all())


# --------------------------------------------------------------------------------------------- binding
def test_binding_refusals(clo):
    pages = [torch.zeros(2, 2, 16, 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(2, 2, device="cuda") for _ in range(2)]
    groups = [torch.zeros(2, 2, 16, 4, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    make = clo.PagedCache
    make(*pages, *scales, *groups)
    for bad, text in (((*pages,), "scales"), ((*pages, *scales), "group_scales"), ((*pages, *scales, groups[0], None), "group_scales"),
                      ((*pages, *scales, groups[0], groups[1][..., :3]), "v_group_scales"), ((*pages, *scales, groups[0].float(), groups[1]), "k_group_scales"),
                      ((*pages, *scales, groups[0].transpose(0, 1), groups[1]), "k_group_scales"), ((*pages, scales[0].double(), scales[1], *groups), "k_scales"),
                      ((*pages, *scales, groups[0].cpu(), groups[1]), "k_group_scales"), ((pages[0], pages[1][..., :16], *scales, *groups), "shapes"),
                      ((pages[0].view(torch.float8_e4m3fn), pages[1].view(torch.float8_e4m3fn), *scales, *groups), "group_scales")):
        with pytest.raises(ValueError, match=text):
            make(*bad)
    with pytest.raises(clo.CLOError, match="head_dim"):
        wide = make(*(torch.zeros(2, 2, 16, 48, dtype=torch.uint8, device="cuda") for _ in range(2)), *scales,
                    *(torch.zeros(2, 2, 16, 6, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)))
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        wide.attention(torch.zeros(1, 2, 96, dtype=BF16, device="cuda"), i32(0, 1), i32(1), i32(0)[None])


def test_what_an_append_writes_gets_a_new_version(clo):
    c = Case(clo, [(5, 5)], 2, 64, 16, seed=160)
    cache = c.device()
    x = bf16(rand(161, 5, 2, 64)).cuda()
    pages = [cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales, cache.k_group_scales, cache.v_group_scales]
    old = [t._version for t in pages]
    cache.append(x, x, c.starts, c.lens, c.tab)
    now = [t._version for t in pages]
    assert all(a > b for a, b in zip(now, old))
    cache.read(c.starts, c.lens, c.tab, 5), cache.attention(x, c.starts, c.lens, c.tab)
    assert [t._version for t in pages] == now
    with pytest.raises(ValueError, match="gradient"):
        cache.attention(x.clone().requires_grad_(), c.starts, c.lens, c.tab)


# --------------------------------------------------------------------------------------------- rows at which one kernel gives way to another
ROWS = [
    # seqs, hkv, group, d, page, window, sinks: 17 to 24 rows per kv head of 64 and of 128, 25, and both sides of 8 and 16
    ([(6, 500), (1, 40), (3, 7), (0, 20)], 2, 4, 64, 16, 0, 0),
    ([(7, 900), (5, 64), (7, 7)], 1, 3, 64, 64, 100, 5),
    ([(3, 333), (2, 2)], 2, 8, 64, 128, 0, 0),
    ([(24, 700), (17, 20), (1, 1)], 2, 1, 64, 32, 0, 0),
    ([(25, 700), (17, 20), (1, 1)], 2, 1, 64, 32, 64, 3),
    ([(6, 500), (1, 40), (3, 7), (0, 20)], 2, 4, 128, 16, 0, 0),
    ([(8, 300), (1, 9)], 2, 1, 128, 64, 0, 0),
    ([(9, 300), (1, 9)], 2, 1, 64, 64, 0, 0),
    ([(16, 300), (1, 9)], 1, 1, 128, 32, 0, 0),
    # long enough to be cut between blocks
    ([(6, 20000), (4, 900), (2, 3)], 2, 4, 64, 64, 0, 0),
    ([(7, 3 + 150 * i) for i in range(40)], 4, 3, 64, 16, 0, 0),
]


@pytest.mark.parametrize("case", range(len(ROWS)))
def test_attention_at_every_width_of_rows(clo, case):
    seqs, hkv, group, d, page, window, sinks = ROWS[case]
    c = Case(clo, [(min(n, kv), kv) for n, kv in seqs], hkv, d, page, seed=400 + case)
    c.device()
    q = bf16(rand(401 + case, c.total, hkv * group, d))
    want, spread, reach = dense_on_device(c, q, window, sinks)
    bound = limit(c.pages4, c.seqs, want, spread, reach, d)
    first = c.attend(q, window, sinks)
    check(first, want, bound)
    check(c.attend(q, window, sinks, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), want, bound, "no workspace")
    work = torch.full((c.cache.attention_workspace(hkv * group, len(seqs), c.total, c.table.shape[1], max_q=c.max_q, window=window, sinks=sinks),), 0xff,
                      dtype=torch.uint8, device="cuda")
    assert torch.equal(c.attend(q, window, sinks, workspace=work), first)  # whatever the workspace held


def test_queries_that_are_not_finite_spoil_their_own_rows(clo):
    for rows in (1, 5, 40):
        c = Case(clo, [(rows, 150), (rows, 90)], 2, 64, 32, seed=420 + rows)
        c.device()
        q = bf16(rand(421, c.total, 4, 64))
        clean = c.attend(q)
        q[0, 1, 3], q[rows, 2, 60] = NAN, INF
        got = c.attend(q)
        same_rows = torch.ones(c.total, 4, dtype=torch.bool)
        same_rows[0, 1] = same_rows[rows, 2] = False
        assert torch.isnan(got[0, 1]).all()
        assert torch.equal(got.cpu()[same_rows], clean.cpu()[same_rows])


def test_strided_rows_in_a_wider_buffer(clo):
    # q, out, k, v and the read-back inside wider buffers; what lies between them is left as it was
    d, hkv, group, page = 64, 2, 3, 16
    c = Case(clo, [(5, 37), (1, 20)], hkv, d, page, seed=430)
    cache = c.device()
    wide = lambda h, fill: torch.full((c.total + 1, h + 2, d + 8), fill, dtype=BF16, device="cuda")  # noqa: E731
    q, out = wide(hkv * group, 0.5), wide(hkv * group, 7.0)
    src = bf16(rand(431, c.total, hkv * group, d))
    q[:c.total, 1:-1, 8:] = src.cuda()
    cache.attention(q[:c.total, 1:-1, 8:], c.starts, c.lens, c.tab, out=out[:c.total, 1:-1, 8:], max_q=5)
    c.compare(out[:c.total, 1:-1, 8:], src)
    keep = torch.ones(out.shape, dtype=torch.bool)
    keep[:c.total, 1:-1, 8:] = False
    assert bool((out.cpu()[keep] == 7.0).all())
    k, v = wide(hkv, 0.25), wide(hkv, 0.25)
    x = bf16(rand(432, c.total, hkv, d))
    k[:c.total, 1:-1, 8:] = x.cuda()
    v[:c.total, 1:-1, 8:] = x.cuda() * 2
    cache.append(k[:c.total, 1:-1, 8:], v[:c.total, 1:-1, 8:], c.starts, c.lens, c.tab, max_q=5)
    for side in range(2):
        c.pages4.append(side, x.double() * (1 + side), c.seqs, c.table)
    same(cache, c.pages4)
    ko, vo = wide(hkv, 3.0), wide(hkv, 3.0)
    cache.read(c.starts, c.lens, c.tab, c.total, k_out=ko[:c.total, 1:-1, 8:], v_out=vo[:c.total, 1:-1, 8:])
    a, b = cache.read(c.starts, c.lens, c.tab, c.total)
    keep = torch.ones(ko.shape, dtype=torch.bool)
    keep[:c.total, 1:-1, 8:] = False
    for o, want in ((ko, a), (vo, b)):
        assert torch.equal(o[:c.total, 1:-1, 8:], want) and bool((o.cpu()[keep] == 3.0).all())


def test_thousands_of_sequences(clo):
    # single tokens and pairs of 2000 sequences under the C names, some without rows, some without tokens
    d, page, hkv, group = 64, 16, 1, 2
    seqs = [((i % 3), 0 if i % 50 == 0 else (i % 3) + i % 30) for i in range(2000)]
    seqs = [(min(n, kv), kv) for n, kv in seqs]
    c = Case(clo, seqs, hkv, d, page, seed=440)
    cache = c.device()
    x = bf16(rand(441, c.total, hkv, d))
    clo.clo_paged_append(cache, x.cuda(), x.cuda(), c.starts, c.lens, c.tab, max_q=2)
    for side in range(2):
        c.pages4.append(side, x.double(), c.seqs, c.table)
    same(cache, c.pages4)
    k, _ = clo.clo_paged_read(cache, c.starts, c.lens, c.tab, c.total, max_q=2)
    q = bf16(rand(442, c.total, hkv * group, d))
    want, spread, reach = ref.attention(c.pages, q, c.seqs, c.table, group)
    check(clo.clo_paged_attention(cache, q.cuda(), c.starts, c.lens, c.tab, max_q=2), want, limit(c.pages4, c.seqs, want, spread, reach, d))
    vals = c.pages.val[0]
    want = torch.stack([vals[int(c.table[b, (kv - n + i) // page]), :, (kv - n + i) % page] for b, (_, n, kv) in enumerate(c.seqs) for i in range(n)])
    assert torch.equal(k.cpu().double(), want)
