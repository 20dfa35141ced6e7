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


# --------------------------------------------------------------------------------------------- streams
def stream_of_memory(address):
    """The stream that torch's allocator took this memory for."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]


def test_new_memory_belongs_to_the_named_stream(clo):
    # what the current stream has just freed may still be written there: a call on another stream must not get it
    n, h, d = 4096, 8, 128
    plan = clo.clo_rope_plan_init(rot_dim=d)
    x = bf16(rand(71, n, h, d)).cuda()
    pos = torch.arange(n, device="cuda")
    c = Case(clo, [(1, 20000)], 2, 64, 64, 16, seed=72)
    c.device()
    q = bf16(rand(73, 1, 8, 64)).cuda()
    want = clo.clo_rope(plan, x, pos).cpu(), c.attend(q).cpu()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        old = torch.empty_like(x)
        freed = old.data_ptr()
        del old
        got = clo.clo_rope(plan, x, pos, stream=stream)
        assert got.data_ptr() != freed and stream_of_memory(got.data_ptr()) == side.cuda_stream
        k, v = c.cache.read(c.starts, c.lens, c.tab, 1, stream=stream)
        assert stream_of_memory(k.data_ptr()) == stream_of_memory(v.data_ptr()) == side.cuda_stream
        out = c.attend(q, stream=stream)
        assert stream_of_memory(out.data_ptr()) == side.cuda_stream
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), want[0]) and torch.equal(out.cpu(), want[1])
        del got, k, v, out
    torch.cuda.synchronize()
    # the default stream by either name, from another current stream
    with torch.cuda.stream(side):
        for stream in (0, 1, torch.cuda.default_stream()):
            assert stream_of_memory(clo.clo_rope(plan, x, pos, stream=stream).data_ptr()) == 0
        assert stream_of_memory(clo.clo_rope(plan, x, pos).data_ptr()) == side.cuda_stream
    torch.cuda.synchronize()


def test_workspace_belongs_to_the_named_stream(clo):
    c = Case(clo, [(1, 30000)], 2, 64, 64, 16, seed=74)
    c.device()
    q = bf16(rand(75, 1, 8, 64)).cuda()
    want = c.attend(q)
    size = c.cache.attention_workspace(8, 1, 1, c.tab.shape[1], 1)
    assert size > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = lambda: sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == side.cuda_stream)  # noqa: E731
    out, before = torch.empty_like(want), held()
    c.attend(q, out=out, stream=side)
    torch.cuda.synchronize()
    assert held() >= before + size
    assert torch.equal(out, want)
