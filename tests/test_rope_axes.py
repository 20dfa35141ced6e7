"""Rotary positions with several axes: plans and refusals on the CPU, kernels on the GPU against 64-bit forms."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import paged_ref as ref  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def clo():
    import __graft_entry__ as ge

    ge.build()
    from host_offloaded_kv_gb300 import clo as m

    m.load_library()
    return m


def axes_of(pairs, order):
    """Axis of each pair, as the header states it."""
    if order == "sections":
        return [a for a, n in enumerate(pairs) for _ in range(n)]
    left, out = list(pairs), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def frequencies(rot, pairs, order, own, **scaling):
    axis = axes_of(pairs, order)
    if not own:
        f, mag = ref.frequencies(rot, **scaling)
        return f, mag, axis
    series = [ref.frequencies(2 * n, **scaling) for n in pairs]
    used, f = [0] * len(pairs), []
    for a in axis:
        f.append(series[a][0][used[a]])
        used[a] += 1
    return torch.stack(f), series[0][1], axis


def rotate(x, pos, rot, pairs, order, own=False, interleaved=False, transpose=False, **scaling):
    """fp64 [n][h][d] rotated by pos [axes][n]."""
    f, mag, axis = frequencies(rot, pairs, order, own, **scaling)
    a = pos.double()[axis].T * f
    c, s = (torch.cos(a) * mag)[:, None], (torch.sin(a) * mag)[:, None] * (-1 if transpose else 1)
    y = x.double().clone()
    ia = torch.arange(rot // 2) * 2 if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    p, q = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia] = p * c - q * s
    y[..., ib] = q * c + p * s
    return y


def bound(want, x, mag=1.0):
    # one rounding to bf16 (half step 2^-8 of the value), sines and cosines off by 7.5e-8 and three fp32 roundings: below 2^-18 of the row
    return 2.0 ** -8 * want.abs() + 2.0 ** -18 * mag * x.double().abs().amax(-1, keepdim=True) + 1e-38


def check(got, want, limit, what=""):
    off = ((got.detach().cpu().double() - want).abs() / limit).max() if want.numel() else 0.0
    assert float(off) <= 1.0, f"{what}: {float(off):.3g} of the bound"


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).to(BF16)


PLANS = [(128, (16, 24, 24), "sections", False), (128, (24, 20, 20), "cycled", False), (64, (16, 16), "sections", True), (128, (1, 62, 1), "cycled", True),
         (96, (10, 3, 5, 30), "cycled", False), (48, (23, 1), "sections", False), (20, (4, 3, 3), "cycled", True), (64, (32,), "sections", True)]
SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="bands", factor=8.0, original_max=8192),
            dict(scaling="yarn", factor=16.0, original_max=32768)]


# ------------------------------------------------------------------------------------------------ CPU
@pytest.mark.parametrize("rot,pairs,order,own", PLANS)
@pytest.mark.parametrize("scaling", SCALINGS)
def test_plan_holds_each_pairs_axis_and_frequency(clo, rot, pairs, order, own, scaling):
    plan = clo.clo_rope_plan_init(rot_dim=rot, theta=500000.0, axis_pairs=pairs, axis_order=order, axis_own_freqs=own, **scaling)
    f, mag, axis = frequencies(rot, pairs, order, own, theta=500000.0, **scaling)
    assert plan.n_axes == len(pairs) and list(plan.axis)[:rot // 2] == axis
    got = torch.tensor([t * 2.0 ** -64 * 2 * math.pi for t in plan.turn][:rot // 2], dtype=torch.float64)
    # a power in fp64 (a few steps of 2^-53) and a fraction rounded to 2^-63 turns
    assert float(((got - f).abs() / (f * 2.0 ** -48 + 2.0 ** -60)).max()) <= 1.0
    assert abs(plan.magnitude - mag) <= 2.0 ** -23 * mag


def test_cycled_axes_skip_those_that_are_used_up(clo):
    plan = clo.clo_rope_plan_init(rot_dim=16, axis_pairs=(4, 1, 3), axis_order="cycled")
    assert list(plan.axis)[:8] == [0, 1, 2, 0, 2, 0, 2, 0]


def test_one_axis_is_the_plan_without(clo):
    a, b = clo.clo_rope_plan_init(rot_dim=64), clo.clo_rope_plan_init(rot_dim=64, axis_pairs=(32,), axis_order="cycled", axis_own_freqs=True)
    assert bytes(a) == bytes(b)


def test_plan_refusals(clo):
    bad = [dict(axis_pairs=(16, 15)), dict(axis_pairs=(32, 0)), dict(axis_pairs=(33, -1)), dict(n_axes=5), dict(n_axes=-1), dict(n_axes=2),
           dict(axis_pairs=(16, 16), axis_order=2), dict(axis_pairs=(2 ** 31 - 1, 2 ** 31 - 1, 34, 2))]
    for kw in bad:
        with pytest.raises(clo.CLOError, match="clo_rope_plan_init"):
            clo.clo_rope_plan_init(rot_dim=64, **kw)
    for kw, text in ((dict(axis_pairs=(8,) * 5), "axes"), (dict(axis_pairs=()), "axes"), (dict(axis_order="mixed"), "axis_order"),
                     (dict(axis_pairs=(16, 16), n_axes=3), "n_axes")):
        with pytest.raises(ValueError, match=text):
            clo.clo_rope_plan_init(rot_dim=64, **kw)
    # a plan that names an axis beyond its own is none of clo_rope_plan_init's, and refused before anything is read
    plan = clo.clo_rope_plan_init(rot_dim=64, axis_pairs=(16, 16))
    rows = clo.clo_rows(0x10000, 512, 64)
    for field in ("axis", "n_axes"):
        p = clo.clo_rope_plan.from_buffer_copy(bytes(plan))
        if field == "axis":
            p.axis[31] = 2
        else:
            p.n_axes = 5
        rc = clo.load_library().clo_rope(ctypes.byref(p), ctypes.byref(rows), ctypes.byref(rows), 0x30000, 4, 8, 64, 0, None)
        assert rc == clo.CLO_ERR_INVALID and "clo_rope_plan_init" in clo.clo_last_error()


# ------------------------------------------------------------------------------------------------ GPU
@pytest.mark.gpu
@pytest.mark.parametrize("rot,pairs,order,own", PLANS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,h,d", [(1, 1, 128), (37, 5, 128), (1300, 9, 128), (257, 40, 64), (6, 3, 130)])
def test_rotation(clo, rot, pairs, order, own, interleaved, n, h, d):
    if rot > d:
        pytest.skip("more rotated elements than the head has")
    x = rand(rot + n, n, h, d)
    pos = torch.randint(-50000, 1 << 20, (len(pairs), n), generator=torch.Generator().manual_seed(n))
    kw = SCALINGS[(n + rot) % 4]
    mag = ref.frequencies(rot, **kw)[1]
    plan = clo.clo_rope_plan_init(rot_dim=rot, interleaved=interleaved, axis_pairs=pairs, axis_order=order, axis_own_freqs=own, **kw)
    where = pos.cuda() if len(pairs) > 1 else pos[0].cuda()
    for transpose in (False, True):
        got = clo.clo_rope(plan, x.cuda(), where, transpose=transpose)
        want = rotate(x, pos, rot, pairs, order, own, interleaved, transpose, **kw)
        check(got, want, bound(want, x, mag), f"transpose={transpose}")
        assert torch.equal(got.cpu()[..., rot:], x[..., rot:])


@pytest.mark.gpu
def test_equal_positions_on_every_axis_are_one_axis(clo):
    # text tokens: the same bits as the plan of one axis; in place, heads inside a fused row, another stream
    n, h, d = 700, 12, 128
    buf = rand(1, n, 2000).cuda()
    one = clo.clo_rope_plan_init(rot_dim=d)
    three = clo.clo_rope_plan_init(rot_dim=d, axis_pairs=(24, 20, 20), axis_order="cycled")
    pos = torch.arange(5, 5 + n).cuda()
    want = clo.clo_rope(one, buf.as_strided((n, h, d), (2000, d, 1), 16), pos)
    view = buf.clone().as_strided((n, h, d), (2000, d, 1), 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert clo.clo_rope(three, view, pos.expand(3, n).contiguous(), out=view, stream=s) is view
    s.synchronize()
    assert torch.equal(view, want)


@pytest.mark.gpu
def test_gradient_is_the_transpose(clo):
    # R is linear: (R x) . g for the unit vector of element e is element e of R^T g
    n, h, d, rot = 2, 2, 64, 48
    pairs = (9, 8, 7)
    plan = clo.clo_rope_plan_init(rot_dim=rot, axis_pairs=pairs, axis_order="cycled")
    pos = torch.tensor([[7, 1000], [3, 20], [0, 400]])
    g = rand(8, n, h, d)
    grad = clo.clo_rope(plan, g.cuda(), pos.cuda(), transpose=True)
    for e in (0, 1, 30, 47, 50):
        x = torch.zeros(n, h, d, dtype=BF16)
        x[..., e] = 1.0
        y = clo.clo_rope(plan, x.cuda(), pos.cuda()).cpu().double()
        diff = (y * g.double()).sum(-1)
        # y carries a bf16 rounding per element (2^-8 of |y| <= 1, two elements), grad one
        limit = 2 * (2.0 ** -8 + 2.0 ** -18) * g.double().abs().amax(-1) + 2.0 ** -8 * diff.abs()
        check(grad[..., e], diff, 2 * limit, f"element {e}")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("pairs,order,interleaved", [((16, 24, 24), "sections", False), ((24, 20, 20), "cycled", True)])
def test_append_rotates_by_several_axes(clo, bits, pairs, order, interleaved):
    # keys and queries of two sequences, the second a single token; without positions every axis has the row's place in the cache
    d, hkv, hq, page = 128, 2, 6, 32
    starts, lens = torch.tensor([0, 75, 76], dtype=torch.int32), torch.tensor([75, 40], dtype=torch.int32)
    table = torch.tensor([[3, 0, 2], [1, 4, -1]], dtype=torch.int32).cuda()
    k, v, q = rand(1, 76, hkv, d), rand(2, 76, hkv, d), rand(3, 76, hq, d)
    plan = clo.clo_rope_plan_init(rot_dim=d, interleaved=interleaved, axis_pairs=pairs, axis_order=order)
    own = torch.cat([torch.arange(75), torch.tensor([39])]).expand(3, 76)
    for pos in (torch.randint(0, 5000, (3, 76), generator=torch.Generator().manual_seed(4)), None):
        c = clo.PagedCache.create(5, hkv, page, d, kv_bits=bits)
        if bits == 8:
            c.k_pages.view(torch.uint8).zero_(), c.v_pages.view(torch.uint8).zero_()
        got = c.append(k.cuda(), v.cuda(), starts.cuda(), lens.cuda(), table, rope=plan, positions=None if pos is None else pos.cuda(), q=q.cuda(), max_q=75)
        back, _ = c.read(starts.cuda(), lens.cuda(), table, 76, max_q=75)
        at = own if pos is None else pos
        want = rotate(q, at, d, pairs, order, interleaved=interleaved)
        check(got, want, bound(want, q))
        want = rotate(k, at, d, pairs, order, interleaved=interleaved)
        # 8-bit codes: half a step of e4m3, 2^-4 of the value or 2^-10 (half the smallest step, 2^-9) of the page's scale, which is at
        # most the 1 that a new cache's pages have: the single token's page keeps it, as the slots before it are taken to hold tokens
        more = 0 if bits == 16 else 2.0 ** -4 * want.abs() + 2.0 ** -10
        check(back, want, bound(want, k) + more)


@pytest.mark.gpu
def test_positions_of_other_shapes_are_refused(clo):
    plan = clo.clo_rope_plan_init(rot_dim=64, axis_pairs=(16, 16))
    x = torch.zeros(6, 2, 64, dtype=BF16, device="cuda")
    for shape in ((6,), (12,), (6, 2), (3, 6), (2, 5), (1, 2, 6)):
        with pytest.raises(ValueError, match="positions"):
            clo.clo_rope(plan, x, torch.zeros(shape, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="positions"):
        clo.clo_rope(plan, x, torch.zeros(6, 2, dtype=torch.int64, device="cuda").T)
    with pytest.raises(ValueError, match="positions"):
        clo.clo_rope(plan, x, torch.zeros(2, 6, dtype=torch.int32, device="cuda"))
    one = clo.clo_rope_plan_init(rot_dim=64)
    with pytest.raises(ValueError, match="positions"):
        clo.clo_rope(one, x, torch.zeros(2, 6, dtype=torch.int64, device="cuda"))
    empty = clo.clo_rope(plan, x[:0], torch.zeros(2, 0, dtype=torch.int64, device="cuda"))
    assert empty.shape == (0, 2, 64)
