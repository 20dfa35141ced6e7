"""Rotary positions where a warp takes four rounds of heads (long calls of many heads), and several warps a token, the last partly filled."""
import pytest

torch = pytest.importorskip("torch")

from test_rope_axes import SCALINGS, bound, check, rand, rotate  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def clo():
    from host_offloaded_kv_gb300 import clo as m

    m.load_library()
    return m


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes,order", [(1, "sections"), (3, "sections"), (4, "cycled")])
@pytest.mark.parametrize("n,h,d,rot", [(1300, 21, 64, 64), (1300, 37, 128, 128), (1216, 17, 64, 48), (1217, 33, 64, 32), (1215, 37, 128, 96), (1300, 9, 128, 16), (1216, 65, 128, 112)])
def test_rotation(clo, n, h, d, rot, axes, order, interleaved):
    x = rand(n + h, n, h, d)
    pairs = (rot // 2,) if axes == 1 else tuple(rot // 2 // axes + (i < rot // 2 % axes) for i in range(axes))
    pos = torch.randint(-50000, 1 << 20, (axes, n), generator=torch.Generator().manual_seed(h))
    kw = SCALINGS[(h + axes) % 4]
    plan = clo.clo_rope_plan_init(rot_dim=rot, interleaved=interleaved, axis_pairs=pairs, axis_order=order, **kw)
    where = (pos if axes > 1 else pos[0]).cuda()
    for transpose in (False, True):
        want = rotate(x, pos, rot, pairs, order, False, interleaved, transpose, **kw)
        got = clo.clo_rope(plan, x.cuda(), where, transpose=transpose)
        check(got, want, bound(want, x, plan.magnitude), f"transpose={transpose}")
        assert torch.equal(got.cpu()[..., rot:], x[..., rot:])
        # in place, heads inside a wider row: the same bits, and nothing beside the heads is written
        buf = torch.full((n, h * d + 48), 7.0, dtype=torch.bfloat16, device="cuda")
        view = buf.as_strided((n, h, d), (h * d + 48, d, 1), 16)
        view.copy_(x)
        assert clo.clo_rope(plan, view, where, out=view, transpose=transpose) is view
        assert torch.equal(view, got)
        assert (buf[:, :16] == 7.0).all() and (buf[:, 16 + h * d:] == 7.0).all()
