"""What the calls over pages read of their callers' structs (no GPU)."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
import ctypes, mmap, sys
sys.path.insert(0, sys.argv[1])
from host_offloaded_kv_gb300 import clo
lib, libc = clo.load_library(), ctypes.CDLL(None, use_errno=True)
# a cache whose last two fields lie in memory that cannot be read
size, page = ctypes.sizeof(clo.clo_paged_cache) - 16, mmap.PAGESIZE
assert clo.clo_paged_cache.k_group_scales.offset == size
area = mmap.mmap(-1, 2 * page)
base = ctypes.addressof(ctypes.c_char.from_buffer(area))
libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
assert libc.mprotect(base + page, page, 0) == 0
full = clo.clo_paged_cache(k_pages=0x100000, v_pages=0x200000, k_scales=0x4000, v_scales=0x5000, n_pages=4, k_stride_page=16384, k_stride_head=8192,
                           k_stride_token=128, v_stride_page=16384, v_stride_head=8192, v_stride_token=128, n_kv_heads=2, head_dim=128, page_size=64,
                           kv_bits=int(sys.argv[2]))
at = base + page - size
ctypes.memmove(at, ctypes.addressof(full), size)
b = clo.clo_paged_batch(q_starts=0x1000, kv_lens=0x2000, block_table=0x3000, table_stride=4, max_pages=4, batch=2, total_q=0, max_q=1)
rows = ctypes.byref(clo.clo_rows(0x10000, 1024, 128))
cache, batch, out = ctypes.c_void_p(at), ctypes.byref(b), ctypes.c_int64()
print(lib.clo_paged_append(cache, batch, None, None, rows, rows, None, None, 0, None), lib.clo_paged_read(cache, batch, rows, rows, None),
      lib.clo_paged_attention_workspace(cache, batch, 4, 0, 0, ctypes.byref(out)), lib.clo_paged_attention(cache, batch, rows, rows, 4, 0.0, 0, 0, None, 0, None))
"""


@pytest.mark.parametrize("bits", [16, 8])
def test_group_scales_are_read_for_4_bit_pages_only(bits):
    # a caller that was compiled before the fields were there
    import __graft_entry__ as ge

    ge.build()
    r = subprocess.run([sys.executable, "-c", PROBE, ROOT, str(bits)], capture_output=True, text=True)
    assert (r.returncode, r.stdout.split()) == (0, ["0"] * 4), r.stderr
