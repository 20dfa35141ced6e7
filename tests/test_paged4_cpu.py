"""4-bit pages without a GPU: refusals of the C calls and of the binding, the reference's rounding."""
import ctypes
import os
import random
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

import paged4_ref as ref4  # noqa: E402
import test_paged_cpu as base  # noqa: E402
import test_prompt_schedule_cpu as barriers  # noqa: E402


@pytest.fixture(scope="module")
def clo():
    import __graft_entry__ as ge

    ge.build()
    from host_offloaded_kv_gb300 import clo as m

    m.load_library()
    return m


GOOD = dict(kv_bits=4, k_scales=0x4000, v_scales=0x5000, k_group_scales=0x6000, v_group_scales=0x7000)
FAULTS = [dict(k_scales=None), dict(v_scales=None), dict(v_scales=0x5002), dict(k_group_scales=None), dict(v_group_scales=None),
          dict(k_group_scales=0x6008), dict(v_group_scales=0x7004), dict(k_stride_token=48), dict(v_stride_head=8208), dict(k_stride_page=1 << 41),
          dict(v_pages=0x200008), dict(head_dim=96), dict(kv_bits=2), dict(kv_bits=6)]


@pytest.mark.parametrize("call", ["append", "read", "attention", "workspace"])
def test_calls_refuse(clo, call):
    lib = clo.load_library()

    def run(batch=None, **kw):
        c, b = base._cache(clo, **{**GOOD, **kw}), base._batch(clo, **(batch or {}))
        k, v = base._rows(clo), base._rows(clo, 0x20000)
        at = [ctypes.byref(x) for x in (c, b, k, v)]
        if call == "append":
            return lib.clo_paged_append(at[0], at[1], None, None, at[2], at[3], None, None, 0, None)
        if call == "read":
            return lib.clo_paged_read(*at, None)
        if call == "workspace":
            return lib.clo_paged_attention_workspace(at[0], at[1], 4, 0, 0, ctypes.byref(ctypes.c_int64()))
        return lib.clo_paged_attention(*at, 4, 0.0, 0, 0, None, 0, None)

    for kw in FAULTS:
        assert run(**kw) == clo.CLO_ERR_INVALID, kw
        assert clo.clo_last_error().startswith("clo_paged_"), kw
    for b in (dict(batch=0, q_starts=None, kv_lens=None, block_table=None), dict(total_q=0), dict(max_q=0)):
        assert run(batch=b) == clo.CLO_OK  # nothing to do, nothing launched


def test_workspace_goes_by_the_sizes(clo):
    lib = clo.load_library()

    def size(max_pages, total=1, max_q=1, window=0):
        out = ctypes.c_int64(-1)
        b = base._batch(clo, batch=1, total_q=total, max_q=max_q, max_pages=max_pages, table_stride=max_pages)
        c = base._cache(clo, **GOOD)
        assert lib.clo_paged_attention_workspace(ctypes.byref(c), ctypes.byref(b), 32, window, 0, ctypes.byref(out)) == clo.CLO_OK
        return out.value

    for total in (1, 300):
        assert size(4096, total, total) > 0 and size(4096, total, total) % 16 == 0
        assert size(1, total, total) == 0 and size(4096, total, total, window=16) == 0


@pytest.mark.parametrize("kw", [dict(kv_bits=4), dict(kv_bits=4, group=32), dict(kv_bits=4, group=0), dict(kv_bits=8, group=16), dict(group=16), dict(kv_bits=2, group=16)])
def test_a_cache_of_4_bits_states_its_group(clo, kw):
    with pytest.raises(ValueError, match="kv_bits"):
        clo.PagedCache.create(1, 1, 16, 64, **kw)


def test_host_tensors_are_refused(clo):
    pages = [torch.zeros(1, 1, 16, 32, dtype=torch.uint8) for _ in range(2)]
    with pytest.raises(ValueError, match="CUDA tensor"):
        clo.PagedCache(*pages, torch.ones(1, 1), torch.ones(1, 1), *(torch.zeros(1, 1, 16, 4, dtype=torch.float8_e4m3fn) for _ in range(2)))


def test_reference_rounding():
    # every value of the formats is its own nearest; borders go to the even index; large values to the last
    for levels in (ref4.LEVELS, ref4.E4M3):
        assert torch.equal(ref4.nearest(levels, levels), torch.arange(len(levels)))
        mid = (levels[1:] + levels[:-1]) / 2
        got = ref4.nearest(mid, levels)
        assert (got % 2 == 0).all() and ((got == torch.arange(len(mid))) | (got == torch.arange(1, len(mid) + 1))).all()
        assert int(ref4.nearest(levels[-1:] * 2, levels)) == len(levels) - 1
    assert torch.equal(ref4.codes_of(ref4.bytes_of(ref4.LEVELS)), ref4.LEVELS)
    assert torch.equal(ref4.codes_of(ref4.bytes_of(-ref4.LEVELS)), -ref4.LEVELS)
    for a, e in ((0.0, -64), (2688.0, 0), (2688.0001, 1), (1.0, -11), (2.0 ** -100, -64), (5.25, -9)):
        assert ref4.needed_scale(a) == 2.0 ** e


def test_pairs_are_rotated_in_integers_to_2_to_the_minus_48(tmp_path):
    # against 64-bit-mantissa arithmetic: angles of every size, exponents 50 apart, zeros, magnitudes; rounded to the odd neighbour
    from host_offloaded_kv_gb300 import _build

    src = tmp_path / "exact.cu"
    src.write_text(r'''
#include <cstdio>
#include <random>
#include "clo_rotate_exact.cuh"
using namespace clo;
static float of(uint16_t x) { const uint32_t b = (uint32_t)x << 16; float f; memcpy(&f, &b, 4); return f; }
int main() {
  std::mt19937_64 g(1);
  const long double turn = 6.283185307179586476925286766559005768L / 18446744073709551616.0L;
  long bad = 0, even = 0;
  for (int i = 0; i < 1000000; ++i) {
    uint64_t a = g();
    if (i % 5 == 0) a >>= g() % 60;
    if (i % 7 == 0) a = (a & 3) << 62;
    uint16_t p = (g() & 0x807f) | (100 + g() % 50) << 7, q = (g() & 0x807f) | (100 + g() % 50) << 7;
    if (i % 11 == 0) p = 0;
    if (i % 13 == 0) q &= 0x8000;
    const float m = i % 3 == 0 ? 1.f : 1.f + (g() % 1000) / 777.f;
    float x[2];
    rotate_exact(p, q, a, m, &x[0], &x[1]);
    const long double s = sinl((int64_t)a * turn), c = cosl((int64_t)a * turn), P = of(p), Q = of(q);
    const long double want[2] = {(P * c - Q * s) * m, (Q * c + P * s) * m}, slack = ldexpl(fmaxl(fabsl(P), fabsl(Q)) * m, -48);
    for (int k = 0; k < 2; ++k) {
      bad += !(want[k] >= nextafterf(x[k], -INFINITY) - slack && want[k] <= nextafterf(x[k], INFINITY) + slack);
      uint32_t b;
      memcpy(&b, &x[k], 4);
      even += !(b & 1) && fabsl(want[k] - x[k]) > slack;
    }
  }
  printf("%ld %ld\n", bad, even);
}
''')
    exe = str(src)[:-3]
    subprocess.run([_build._nvcc(), "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(base.ROOT, "host_offloaded_kv_gb300", "csrc"),
                    str(src), "-o", exe], check=True)
    assert subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split() == ["0", "0"]


SHAPES = [(d, 4, tiles) for d in (64, 128) for tiles in (1, 2)]


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    # the prompt kernel's rings for 4-bit pages, from its source
    body = "".join(f'printf("%d %d %d %d\\n", Cfg<{d}, 4, {t}>::kSlots, Cfg<{d}, 4, {t}>::kRawSide, Cfg<{d}, 4, {t}>::kMeta, Cfg<{d}, 4, {t}>::kBytes);'
                   for d, _, t in SHAPES)
    text = open(barriers.SOURCE).read()
    parts = re.findall(r"^constexpr int k(?:Tok|Rows) = \d+;", text, re.M)
    parts += re.findall(r"^template <int D, int BITS, int TILES>\nstruct Cfg \{.*?^\};", text, re.M | re.S)
    src = tmp_path_factory.mktemp("cfg4") / "cfg.cpp"
    src.write_text("#include <cstdint>\n#include <cstdio>\n" + "\n".join(parts) + "\nint main() {" + body + "}\n")
    subprocess.run(["g++", "-std=c++17", str(src), "-o", str(src)[:-4]], check=True)
    rows = subprocess.run([str(src)[:-4]], capture_output=True, text=True, check=True).stdout.split("\n")
    return {shape: tuple(map(int, row.split())) for shape, row in zip(SHAPES, rows)}


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "d%d_bits%d_tiles%d" % s)
def test_prompt_kernels_barriers_keep_in_step(sizes, shape):
    *rings, memory = sizes[shape]
    assert 2 * rings[1] <= 12 and memory + 4096 <= 227 * 1024  # barriers of the rings, shared memory beside the static part
    for seed in range(10):
        rng = random.Random(seed)
        barriers.Block(barriers.some_units(rng), shape, tuple(rings), rng).run()
