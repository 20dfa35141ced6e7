"""4-bit pages on the GPU where ranges and borders end."""
import math

import pytest

torch = pytest.importorskip("torch")

import paged4_ref as ref4  # noqa: E402
from test_gpu_paged import BF16, rand  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def clo():
    from host_offloaded_kv_gb300 import clo as m

    m.load_library()
    return m


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def e4m3(t):
    return t.float().to(torch.float8_e4m3fn).cuda()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rows,tokens", [(1, 60000), (1, 300), (200, 3000)])
def test_outputs_near_the_end_of_bf16(clo, bits, rows, tokens):
    # every V is 1.5 * 2^e, so every output is: finite whether units are cut and joined or stay whole.  Weights are rounded to fp16 for the
    # product and not for the sum (2^-11), sums to fp32 (below 2^-14 for so many equal terms), the output to bf16 (2^-8)
    hkv, group, d, page = 2, 4, 64, 64
    n = -(-tokens // page)
    for e in (120, 124, 126):
        if bits == 8:
            pages = [torch.zeros(n, hkv, page, d), torch.full((n, hkv, page, d), 1.5)]
            cache = clo.PagedCache(*(p.to(torch.float8_e4m3fn).cuda() for p in pages), torch.ones(n, hkv).cuda(), torch.full((n, hkv), 2.0 ** e).cuda())
        else:
            codes = [ref4.bytes_of(torch.full((n, hkv, page, d), x, dtype=torch.float64)).cuda() for x in (0.0, 6.0)]
            cache = clo.PagedCache(*codes, torch.ones(n, hkv).cuda(), torch.full((n, hkv), 2.0 ** (e - 2)).cuda(), *(e4m3(torch.ones(n, hkv, page, d // 16)) for _ in range(2)))
        q = rand(1, rows, hkv * group, d).to(BF16).cuda()
        for work in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):
            got = cache.attention(q, i32([0, rows]), i32([tokens]), torch.arange(n, dtype=torch.int32, device="cuda")[None], max_q=rows, workspace=work).double()
            off = float((got / (1.5 * 2.0 ** e) - 1).abs().max())
            assert off <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14, (e, work is None, off)


@pytest.mark.parametrize("d", [64, 128])
def test_read_back_of_large_scales(clo, d):
    # group scale times page scale lies past fp32's range, code times both does not
    hkv, page = 3, 16
    gen = torch.Generator().manual_seed(d)
    code = torch.tensor([0.0, 0.5, -0.5, -0.0], dtype=torch.float64)[torch.randint(0, 4, (2, hkv, page, d), generator=gen)]
    group = torch.full((2, hkv, page, d // 16), 448.0, dtype=torch.float64)
    scale = torch.full((2, hkv), 1.0, dtype=torch.float64) * 2.0 ** 120
    cache = clo.PagedCache(*(ref4.bytes_of(code).cuda() for _ in range(2)), *(scale.float().cuda() for _ in range(2)), *(e4m3(group) for _ in range(2)))
    k, v = cache.read(i32([0, 2 * page]), i32([2 * page]), i32([[1, 0]]), 2 * page)
    want = ref4.values(code, group, scale)[[1, 0]].transpose(1, 2).reshape(2 * page, hkv, d)
    assert torch.isfinite(want).all() and float(want.abs().max()) < 2.0 ** 128
    for got in (k, v):
        assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("page", [16, 128])
def test_page_scales_are_those_of_the_exact_rotation(clo, page, interleaved):
    # The largest key of a page lies within 2^-24 of 2688 * 2^e: the factor on the rotated elements is chosen to put it there.  Pair 0 turns by
    # one radian per position; a page of 128 is shared out to several warps, and the key stands in its last row.
    trials, d, hkv = 300, 64, 1
    gen = torch.Generator().manual_seed(page + interleaved)
    cache = clo.PagedCache.create(trials, hkv, page, d, kv_bits=4, group=16)
    want = torch.zeros(trials, dtype=torch.float64)
    a, b = (0, 1) if interleaved else (0, 32)
    done = 0
    while done < trials:
        p, q = (float(x) for x in torch.randn(2, generator=gen).to(BF16))
        pos = int(torch.randint(0, 2000, (1,), generator=gen))
        s, c = math.sin(pos), math.cos(pos)
        x, y = abs(p * c - q * s), abs(q * c + p * s)
        if x < 0.1 or x < 1.1 * y:
            continue
        e = math.ceil(math.log2(x / 2688.0))
        magnitude = float(torch.tensor(2688.0 * 2.0 ** e / x, dtype=torch.float32))
        off = magnitude * x / (2688.0 * 2.0 ** e) - 1.0
        if abs(off) < 1e-12:  # what 64 bits do not decide
            continue
        rows = torch.zeros(page, hkv, d, dtype=BF16)
        rows[-1, 0, a], rows[-1, 0, b] = p, q
        plan = clo.clo_rope_plan_init(rot_dim=d, interleaved=interleaved, magnitude=magnitude)
        where = torch.full((page,), pos, dtype=torch.int64).cuda()
        cache.append(rows.cuda(), torch.zeros_like(rows).cuda(), i32([0, page]), i32([page]), i32([[done]]), rope=plan, positions=where)
        want[done] = 2.0 ** (e + (off > 0))
        done += 1
    got = cache.k_scales[:, 0].cpu().double()
    assert torch.equal(got, want), f"{int((got != want).sum())} of {trials} scales"


@pytest.mark.parametrize("page", [16, 64])
def test_codes_at_borders_are_those_of_the_exact_rotation(clo, page):
    # A key within 2^-24 of the border between two codes, by the choice of the factor as above.  Pair 1 does not turn (its frequency is nearly zero):
    # its first element is the group's largest and takes the page's scale and the group's far from their own borders.
    trials, d, rot = 400, 64, 16
    gen = torch.Generator().manual_seed(page)
    cache = clo.PagedCache.create(trials, 1, page, d, kv_bits=4, group=16)
    want, got_at = torch.zeros(trials, dtype=torch.float64), []
    done = 0
    while done < trials:
        p, q = (float(x) for x in torch.randn(2, generator=gen).to(BF16))
        pos = int(torch.randint(0, 2000, (1,), generator=gen))
        x, y = p * math.cos(pos) - q * math.sin(pos), q * math.cos(pos) + p * math.sin(pos)
        border = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)[done % 7]
        # group scale 1 and page scale 2^e: the key at border * 2^e, the largest element at about 6 * 2^e, the other one of the pair below it
        if abs(x) < 0.01 or abs(y) * border >= 5.9 * abs(x):
            continue
        e = math.floor(math.log2(abs(x) / border)) + 1
        magnitude = float(torch.tensor(border * 2.0 ** e / abs(x), dtype=torch.float32))
        off = magnitude * abs(x) / (border * 2.0 ** e) - 1.0
        if abs(off) < 1e-12:
            continue
        row = torch.zeros(1, 1, d, dtype=BF16)
        row[0, 0, 0], row[0, 0, 8], row[0, 0, 1] = p, q, float(torch.tensor(6.0 * 2.0 ** e / magnitude).to(BF16))
        row[0, 0, 32] = 2000.0 * 2.0 ** e  # not rotated: the page's largest, which makes its scale 2^e
        plan = clo.clo_rope_plan_init(rot_dim=rot, theta=1e300, magnitude=magnitude)
        cache.append(row.cuda(), torch.zeros_like(row).cuda(), i32([0, 1]), i32([1]), i32([[done]]), rope=plan, positions=torch.tensor([pos]).cuda())
        lo = max(v for v in ref4.LEVELS.tolist() if v < border)
        hi = min(v for v in ref4.LEVELS.tolist() if v > border)
        want[done] = math.copysign(hi if off > 0 else lo, x) * 2.0 ** e
        got_at.append(2.0 ** e)
        done += 1
    now = ref4.of_cache(cache)
    scale = torch.tensor(got_at, dtype=torch.float64)
    assert torch.equal(now.scale[0][:, 0], scale) and torch.equal(now.group[0][:, 0, 0, 0], torch.ones(trials, dtype=torch.float64))
    assert torch.equal(now.code[0][:, 0, 0, 0] * scale, want)
