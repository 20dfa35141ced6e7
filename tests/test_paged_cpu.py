"""Rotary plans and the refusals of the paged-cache calls (no GPU: nothing is launched)."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import paged_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def clo():
    import __graft_entry__ as ge

    ge.build()
    from host_offloaded_kv_gb300 import clo as m

    m.load_library()
    return m


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="bands", factor=8.0, original_max=8192),
            dict(scaling="yarn", factor=16.0, original_max=4096), dict(scaling="yarn", factor=1.0, original_max=100),
            dict(scaling="yarn", factor=4.0, original_max=4096, magnitude=0.75)]


@pytest.mark.parametrize("rot", [2, 20, 64, 128])
@pytest.mark.parametrize("theta", [10000.0, 500000.0])
@pytest.mark.parametrize("kw", SCALINGS)
def test_plan_holds_the_frequencies_as_turns(clo, rot, theta, kw):
    plan = clo.clo_rope_plan_init(rot_dim=rot, theta=theta, **kw)
    f, mag = ref.frequencies(rot, theta=theta, **kw)
    assert plan.rot_dim == rot and plan.interleaved == 0 and plan.ready == 1
    assert abs(plan.magnitude - mag) <= 2.0 ** -24 * mag
    for i in range(rot // 2):
        # a few fp64 roundings of the frequency, and the last bits of the 64-bit fraction
        assert abs(plan.turn[i] / 2.0 ** 64 - float(f[i]) / (2 * math.pi)) <= 8 * 2.0 ** -53 * float(f[i]) + 2.0 ** -61


@pytest.mark.parametrize("kw,text", [(dict(rot_dim=0), "rot_dim"), (dict(rot_dim=7), "rot_dim"), (dict(rot_dim=130), "rot_dim"),
                                     (dict(rot_dim=64, theta=1.0), "theta"), (dict(rot_dim=64, theta=float("nan")), "theta"),
                                     (dict(rot_dim=64, scaling=9), "scaling"), (dict(rot_dim=64, factor=0.5), "factor"),
                                     (dict(rot_dim=64, magnitude=-1.0), "magnitude"),
                                     (dict(rot_dim=64, scaling="bands", factor=2.0), "original_max"),
                                     (dict(rot_dim=64, scaling="bands", original_max=10, low_freq=4.0, high_freq=4.0), "low_freq"),
                                     (dict(rot_dim=64, scaling="yarn", original_max=10, beta_slow=0.0), "beta")])
def test_plan_refuses(clo, kw, text):
    with pytest.raises(clo.CLOError) as e:
        clo.clo_rope_plan_init(**kw)
    assert e.value.status == clo.CLO_ERR_INVALID and text in str(e.value)


def test_plan_refuses_unknown_names(clo):
    with pytest.raises(ValueError, match="unknown scaling"):
        clo.clo_rope_plan_init(rot_dim=64, scaling="other")
    with pytest.raises(TypeError, match="no field"):
        clo.clo_rope_plan_init(rot_dim=64, base=3)


def _rows(clo, ptr=0x10000, token=1024, head=128):
    return clo.clo_rows(ptr, token, head)


def _rope(clo, plan=None, x=None, y=None, pos=0x30000, n=4, h=8, d=128):
    plan = plan or clo.clo_rope_plan_init(rot_dim=128)
    x, y = x or _rows(clo), y or _rows(clo, 0x20000)
    return clo.load_library().clo_rope(ctypes.byref(plan), ctypes.byref(x), ctypes.byref(y), pos, n, h, d, 0, None)


def test_rope_refusals(clo):
    bad = [dict(d=127), dict(d=2048), dict(n=-1), dict(h=-1), dict(d=64), dict(x=clo.clo_rows(None, 8, 8)), dict(pos=None),
           dict(pos=0x30004), dict(y=_rows(clo, 0x20001)), dict(y=_rows(clo, 0x10000, token=2048)), dict(plan=clo.clo_rope_plan())]
    for kw in bad:
        assert _rope(clo, **kw) == clo.CLO_ERR_INVALID, kw
        assert clo.clo_last_error().startswith("clo_rope"), kw
    assert clo.load_library().clo_rope(None, None, None, None, 1, 1, 64, 0, None) == clo.CLO_ERR_INVALID
    assert _rope(clo, n=0, x=clo.clo_rows(None, 0, 0)) == clo.CLO_OK  # no rows: nothing is read


def _cache(clo, **kw):
    c = dict(k_pages=0x100000, v_pages=0x200000, k_scales=None, v_scales=None, n_pages=4, k_stride_page=16384, k_stride_head=8192,
             k_stride_token=128, v_stride_page=16384, v_stride_head=8192, v_stride_token=128, n_kv_heads=2, head_dim=128,
             page_size=64, kv_bits=16)
    c.update(kw)
    return clo.clo_paged_cache(**c)


def _batch(clo, **kw):
    b = dict(q_starts=0x1000, kv_lens=0x2000, block_table=0x3000, table_stride=4, max_pages=4, batch=2, total_q=2, max_q=1)
    b.update(kw)
    return clo.clo_paged_batch(**b)


CACHE_FAULTS = [dict(k_pages=None), dict(v_pages=0x200008), dict(head_dim=96), dict(kv_bits=4), dict(page_size=48), dict(n_kv_heads=0),
                dict(n_pages=0), dict(n_pages=1 << 31), dict(k_stride_page=0), dict(v_stride_token=130), dict(k_stride_head=-8192),
                dict(k_stride_page=1 << 40), dict(kv_bits=8), dict(kv_bits=8, k_scales=0x4000, v_scales=0x5002),
                dict(kv_bits=8, k_scales=0x4000, v_scales=0x5000, k_stride_token=72)]
BATCH_FAULTS = [dict(q_starts=None), dict(kv_lens=0x2002), dict(block_table=None), dict(batch=-1), dict(batch=65536), dict(total_q=-1),
                dict(total_q=(1 << 30) + 1), dict(max_q=-1), dict(max_pages=-1), dict(max_pages=1 << 24)]


@pytest.mark.parametrize("call", ["append", "read", "attention"])
def test_paged_calls_refuse(clo, call):
    lib = clo.load_library()
    plan = clo.clo_rope_plan_init(rot_dim=128)

    def run(c=None, b=None, k=None, v=None, plan=plan, q=None, q_out=None, hq=4, scale=0.0, window=0, sinks=0, pos=None, work=None):
        c, b = ctypes.byref(c or _cache(clo)), ctypes.byref(b or _batch(clo))
        k, v = ctypes.byref(k or _rows(clo)), ctypes.byref(v or _rows(clo, 0x20000))
        opt = lambda r: None if r is None else ctypes.byref(r)  # noqa: E731
        if call == "append":
            return lib.clo_paged_append(c, b, opt(plan), pos, k, v, opt(q), opt(q_out), hq, None)
        if call == "read":
            return lib.clo_paged_read(c, b, k, v, None)
        return lib.clo_paged_attention(c, b, k, v, hq, scale, window, sinks, work, 0, None)

    bad = [dict(c=_cache(clo, **kw)) for kw in CACHE_FAULTS] + [dict(b=_batch(clo, **kw)) for kw in BATCH_FAULTS]
    bad += [dict(k=_rows(clo, 0x10008)), dict(v=_rows(clo, 0x20000, token=1028)), dict(k=_rows(clo, None)), dict(v=_rows(clo, 0x20000, head=100))]
    if call == "append":
        short = clo.clo_rope_plan_init(rot_dim=24)
        wide = clo.clo_rope_plan_init(rot_dim=128)
        r = _rows(clo, 0x40000)
        bad += [dict(plan=short), dict(plan=wide, c=_cache(clo, head_dim=64)), dict(plan=clo.clo_rope_plan()), dict(q=r), dict(q_out=r),
                dict(q=r, q_out=r, hq=0), dict(q=r, q_out=r, plan=None), dict(q=r, q_out=_rows(clo, 0x40000, token=2048)),
                dict(q=r, q_out=_rows(clo, 0x50002)), dict(pos=0x30004)]
    if call == "attention":
        bad += [dict(hq=0), dict(hq=3), dict(hq=34), dict(scale=float("nan")), dict(scale=-1.0), dict(window=-1), dict(sinks=-1),
                dict(v=_rows(clo)), dict(work=0x4008)]
    for kw in bad:
        assert run(**kw) == clo.CLO_ERR_INVALID, kw
        assert clo.clo_last_error().startswith("clo_paged_" + call), kw
    for b in (dict(batch=0, q_starts=None, kv_lens=None, block_table=None), dict(total_q=0), dict(max_q=0)):
        assert run(b=_batch(clo, **b)) == clo.CLO_OK  # nothing to do, nothing launched


def test_attention_workspace_sizes(clo):
    lib = clo.load_library()

    def size(hq=32, window=0, sinks=0, **b):
        out = ctypes.c_int64(-1)
        batch = _batch(clo, **dict(dict(batch=1, total_q=1, max_q=1, max_pages=4096, table_stride=4096), **b))
        rc = lib.clo_paged_attention_workspace(ctypes.byref(_cache(clo)), ctypes.byref(batch), hq, window, sinks, ctypes.byref(out))
        assert rc == clo.CLO_OK
        return out.value

    for long in (dict(), dict(batch=600, total_q=600), dict(total_q=300, max_q=300), dict(total_q=300, max_q=9)):
        assert size(**long) > 0 and size(**long) % 16 == 0
        # sequences that the table or a window keeps short need none
        assert size(**dict(long, max_pages=1)) == 0
        assert size(window=16, **dict(long, batch=1)) == 0
    # the size goes by the sizes, not by the lengths that the call meets
    assert size(max_pages=4096) == size(max_pages=1 << 20)
    assert size(batch=0) == size(total_q=0) == size(max_q=0) == 0
    batch, out = _batch(clo), ctypes.c_int64(-1)
    for args in ((0, 0, 0), (3, 0, 0), (4, -1, 0), (4, 0, -1)):
        rc = lib.clo_paged_attention_workspace(ctypes.byref(_cache(clo)), ctypes.byref(batch), *args, ctypes.byref(out))
        assert rc == clo.CLO_ERR_INVALID and clo.clo_last_error().startswith("clo_paged_attention_workspace"), args
    assert lib.clo_paged_attention_workspace(ctypes.byref(_cache(clo)), ctypes.byref(batch), 4, 0, 0, None) == clo.CLO_ERR_INVALID


def test_binding_refuses_host_tensors(clo):
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    plan = clo.clo_rope_plan_init(rot_dim=64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        clo.clo_rope(plan, x, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        clo.PagedCache(torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="kv_bits"):
        clo.PagedCache.create(1, 1, 16, 64, kv_bits=4)


def test_struct_layouts_match_header(clo):
    names = ["clo_rope_config", "clo_rope_plan", "clo_rows", "clo_paged_cache", "clo_paged_batch"]
    body = "".join(f'printf("%zu ", sizeof({n}));' for n in names)
    tmp = os.path.join(ROOT, "host_offloaded_kv_gb300", "_lib", "paged_layout_probe.c")
    with open(tmp, "w") as f:
        f.write('#include <stdio.h>\n#include "clo.h"\nint main(){' + body + "}\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), tmp, "-o", tmp[:-2]], check=True)
    sizes = [int(x) for x in subprocess.run([tmp[:-2]], capture_output=True, text=True).stdout.split()]
    assert sizes == [ctypes.sizeof(getattr(clo, n)) for n in names]


def test_reference_rounding_is_the_formats():
    codes = torch.arange(256, dtype=torch.uint8)
    vals = ref.e4m3_values(codes)
    fin = torch.sort(vals[torch.isfinite(vals)].unique())[0]
    assert torch.equal(ref.round_e4m3(fin), fin)
    x = torch.randn(4096, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * torch.exp2(torch.arange(4096) % 20 - 11.0)
    x = x.clamp(-448, 448)
    near = (fin[None, :] - x[:, None]).abs().min(1)[0]
    assert torch.equal((ref.round_e4m3(x) - x).abs(), near)


def test_a_lost_copy_is_never_hidden(tmp_path):
    # rows of a unit whose wait gave up are NaN, also where V would have them computed again; parts carry that to the join
    from host_offloaded_kv_gb300 import _build

    src = tmp_path / "row_end.cu"
    src.write_text('''#include <cstdio>
#include "clo_paged_attend.cuh"
using namespace clo;
int main() {
  for (int i = 0; i < 4; ++i) {
    const RowEnd e = row_end(i & 2, i & 1);
    const float mark = part_mark(e);
    printf("%d %d %d ", (int)(e == RowEnd::nan), (int)(e == RowEnd::again), (int)(row_end(mark == kPartLost, mark == kPartSpoilt) == e));
  }
}
''')
    exe = str(tmp_path / "row_end")
    csrc = os.path.join(ROOT, "host_offloaded_kv_gb300", "csrc")
    subprocess.run([_build._nvcc(), "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", csrc, "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert got == "0 0 1  0 1 1  1 0 1  1 0 1".split()
    # every place that computes rows again asks row_end first
    for name in ("clo_paged_few.cuh", "clo_paged_prompt.cu"):
        text = open(os.path.join(csrc, name)).read()
        calls = [m for m in range(len(text)) if text.startswith("attend_row<", m)]
        assert len(calls) >= 2
        for at in calls:
            assert "row_end(" in text[at - 1500:at], f"{name}: a row is computed again unasked"


def test_plans_and_configs_are_what_they_say(clo):
    cfg = clo.clo_rope_config_default()
    cfg.rot_dim = 64
    plan = clo.clo_rope_plan_init(cfg)
    assert plan.rot_dim == 64
    with pytest.raises(TypeError, match="exclude"):  # one of them would be ignored
        clo.clo_rope_plan_init(cfg, rot_dim=32)
    with pytest.raises(TypeError, match="clo_rope_config"):
        clo.clo_rope_plan_init(plan)
    x, pos = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    for bad in (cfg, None, 64):  # a config is shorter than the plan that the call reads
        with pytest.raises(TypeError, match="clo_rope_plan"):
            clo.clo_rope(bad, x, pos)
