"""Edges of the calls over HBM pages on the GPU: what padded batches, other streams, odd bounds and extreme values meet."""
import pytest

torch = pytest.importorskip("torch")

import paged_ref as ref  # noqa: E402
from test_gpu_paged import Case, bf16, check, dense_on_device, rand  # noqa: E402

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def clo():
    from host_offloaded_kv_gb300 import clo as m

    m.load_library()
    return m


def dense(c, q, window=0, sinks=0):
    """dense_on_device, with zeros for sequences that hold no token."""
    seqs = c.seqs
    c.seqs = [(first, n if kv > 0 else 0, kv) for first, n, kv in seqs]
    try:
        return dense_on_device(c, q, window, sinks)
    finally:
        c.seqs = seqs


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("rows,d", [(6, 128), (30, 64)])
def test_units_without_tokens_between_others_in_one_block(clo, bits, rows, d):
    # 24 or 120 rows per kv head, more units than blocks, so that a block goes from units with tokens to padded ones and on
    seqs = []
    for i in range(110):
        seqs += [(rows, rows + 40 + 37 * i % 600), (rows, 0)] + ([(rows, 0)] if i % 3 == 0 else [])
    c = Case(clo, seqs, 3, d, 64, bits, seed=61, width=11)
    c.device()
    q = bf16(rand(62, c.total, 12, d) * 2)
    want, spread, reach = dense(c, q)
    bound = ref.attention_bound(want, spread, reach, d, bits)
    first = c.attend(q)
    check(first, want, bound)
    none = torch.empty(16, dtype=torch.uint8, device="cuda")
    whole = c.attend(q, workspace=none)
    check(whole, want, bound, "no workspace")
    for _ in range(40):
        assert torch.equal(c.attend(q), first) and torch.equal(c.attend(q, workspace=none), whole)
