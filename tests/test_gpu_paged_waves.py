"""Decode attention whose units stay whole: the waves of blocks that a call takes."""
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_third_block_where_it_saves_a_wave(tmp_path):
    text = open(os.path.join(ROOT, "host_offloaded_kv_gb300", "csrc", "clo_paged_few.cuh")).read()
    rule = re.search(r"^constexpr bool third_block_pays\(.*$", text, re.M).group(0)
    src = tmp_path / "rule.cpp"
    src.write_text("#include <cstdint>\n#include <cstdio>\nconstexpr int kSms = 152;\n" + rule + '\nint main() { for (int u = 1; u <= 4000; ++u) printf("%d ", third_block_pays(u)); }\n')
    subprocess.run(["g++", "-std=c++17", str(src), "-o", str(src)[:-4]], check=True)
    got = subprocess.run([str(src)[:-4]], capture_output=True, text=True, check=True).stdout.split()
    waves = lambda units, per_sm: -(-units // (152 * per_sm))  # noqa: E731
    assert [x == "1" for x in got] == [waves(u, 3) < waves(u, 2) for u in range(1, 4001)]
    assert [got[u - 1] for u in (304, 305, 456, 457, 608, 609)] == ["0", "1", "1", "0", "0", "1"]


@pytest.mark.gpu
@pytest.mark.parametrize("bits,d", [(16, 128), (16, 64), (8, 128), (8, 64), (4, 128), (4, 64)])
@pytest.mark.parametrize("rows", [1, 3])
def test_a_sequence_is_the_same_in_batches_of_every_size(bits, d, rows):
    # 8, 160, 360, 512 and 1024 units: one block to an SM up to several waves of two or three; the sequence's bits depend on none of them
    from host_offloaded_kv_gb300 import clo

    hkv, group, page, most = 8, 4, 16, 128
    gen = torch.Generator(device="cuda").manual_seed(rows)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    lens = torch.randint(rows, 250, (most,), generator=torch.Generator().manual_seed(d), dtype=torch.int32)
    table = torch.arange(most * 16, dtype=torch.int32, device="cuda").view(most, 16)
    cache = clo.PagedCache.create(most * 16, hkv, page, d, kv_bits=bits, **({"group": 16} if bits == 4 else {}))
    total = int(lens.sum())
    starts = torch.zeros(most + 1, dtype=torch.int32)
    starts[1:] = lens.cumsum(0)
    cache.append(randn(total, hkv, d).bfloat16(), randn(total, hkv, d).bfloat16(), starts.cuda(), lens.cuda(), table)
    q = randn(most * rows, hkv * group, d).bfloat16()
    outs = {}
    for n in (1, 20, 45, 64, 128):
        at = torch.arange(n + 1, dtype=torch.int32, device="cuda") * rows
        outs[n] = cache.attention(q[:n * rows], at, lens[:n].cuda(), table[:n], max_q=rows)
    for n, out in outs.items():
        assert torch.equal(out, outs[most][:n * rows]), n
