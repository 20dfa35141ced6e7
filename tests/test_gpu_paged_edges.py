"""Edges of the calls over HBM pages on the GPU: what padded batches, other streams, odd bounds and extreme values meet."""
import math

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


# --------------------------------------------------------------------------------------------- V that is not finite
def put_v(c, marks):
    """V of (sequence, kv head, token, element) set to a value, on the CPU side of a Case (before device())."""
    for b, h, j, e, value in marks:
        page = int(c.table[b, j // c.page])
        for t in (c.codes[1], c.pages.val[1]):
            if t.dtype is torch.float8_e4m3fn:
                t.view(torch.uint8)[page, h, j % c.page, e] = 0x7f
            else:
                t[page, h, j % c.page, e] = value


def with_marks(c, q, marks, window=0, sinks=0):
    """(want, bound): the fp64 attention with V zero at the marks, then each mark's value where a row sees it."""
    vals = c.pages.val[1].clone()
    for b, h, j, e, _ in marks:
        c.pages.val[1][int(c.table[b, j // c.page]), h, j % c.page, e] = 0.0
    want, spread, reach = dense(c, q, window, sinks)
    c.pages.val[1] = vals
    group = q.shape[1] // c.hkv
    add = torch.zeros_like(want)
    for b, h, j, e, value in marks:
        first, n, kv = c.seqs[b]
        pos = torch.arange(kv - n, kv)
        see = (pos >= j) & ((pos - window < j) | (j < sinks) if window else True)
        add[first:first + n, h * group:(h + 1) * group, e] += torch.where(see, value, 0.0)[:, None]
    return want + add, ref.attention_bound(want, spread, reach, c.d, c.bits)


NAN, INF = float("nan"), float("inf")
SPOILT = [
    # seqs, hkv, group, d, page, window, sinks, marks (8-bit pages: all NaN)
    ([(1300, 1300)], 2, 4, 128, 64, 0, 0, [(0, 0, 0, 5, NAN), (0, 1, 300, 9, INF), (0, 1, 1000, 9, -INF), (0, 1, 1001, 70, -INF)]),
    ([(1300, 1300)], 2, 4, 64, 16, 0, 0, [(0, 0, 1299, 63, NAN), (0, 1, 640, 0, NAN), (0, 1, 641, 0, INF)]),
    ([(900, 1500), (20, 20)], 2, 4, 128, 32, 300, 5, [(0, 0, 2, 1, NAN), (0, 0, 6, 2, NAN), (0, 1, 700, 3, INF), (1, 1, 19, 4, NAN)]),
    # one row tile, units cut between blocks and joined
    ([(40, 9000)], 2, 2, 128, 64, 0, 0, [(0, 0, 100, 7, NAN), (0, 1, 8999, 8, INF), (0, 1, 8970, 9, NAN)]),
    ([(40, 9000)], 2, 2, 64, 128, 2000, 3, [(0, 0, 6990, 7, NAN), (0, 0, 1, 8, INF), (0, 1, 4, 9, NAN)]),
    # two row tiles, joined
    ([(200, 6000)], 2, 3, 128, 16, 0, 0, [(0, 0, 0, 127, NAN), (0, 1, 5900, 3, NAN)]),
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("case", range(len(SPOILT)))
def test_rows_are_not_finite_where_they_see_it(clo, case, bits):
    seqs, hkv, group, d, page, window, sinks, marks = SPOILT[case]
    if bits == 8:
        marks = [(b, h, j, e, NAN) for b, h, j, e, _ in marks]
    c = Case(clo, seqs, hkv, d, page, bits, seed=80 + case)
    put_v(c, marks)
    c.device()
    q = bf16(rand(81 + case, c.total, hkv * group, d))
    want, bound = with_marks(c, q, marks, window, sinks)
    check(c.attend(q, window, sinks), want, bound)
    check(c.attend(q, window, sinks, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), want, bound, "no workspace")


@pytest.mark.parametrize("rows,kv", [(300, 300), (40, 5000)])
def test_large_values_and_infinities_of_no_weight(clo, rows, kv):
    # values whose weighted sum passes fp32's range before it is divided by the weights' sum, and an infinity of a weight below fp32's
    # normal range (2^-134 of the row's largest), whose product with it is an infinity all the same
    d = 128
    c = Case(clo, [(rows, kv)], 1, d, 64, 16, seed=91)
    for t in (c.codes[0], c.pages.val[0]):
        t[..., 0] = 0.0
    put_v(c, [(0, 0, j, 3, 2.0 ** 119) for j in range(kv)] + [(0, 0, 5, 4, INF)])
    page = int(c.table[0, 0])
    for t in (c.codes[0], c.pages.val[0]):
        t[page, 0, 5] = 0.0
        t[page, 0, 5, 0] = -64.0
        t[page, 0, 6:7, 0] = 64.0
    c.device()
    q = bf16(rand(92, rows, 2, d) * 0.01)
    q[..., 0] = bf16(torch.tensor(134 * math.log(2) / 128 * math.sqrt(d)))
    got = c.attend(q)[..., :5].cpu().double()
    pos = torch.arange(kv - rows, kv)
    late = pos >= 6
    # channel 3: the weighted mean of equal values; weights are rounded to bf16 above and not below the line
    assert ((got[late][..., 3] / 2.0 ** 119 - 1).abs() <= 2 * 2.0 ** -8).all()
    assert (got[late][..., 4] == INF).all()


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("value", [NAN, INF])
def test_one_value_that_is_not_finite_does_not_stall_a_prompt(clo, bits, value):
    if bits == 8 and value == INF:
        pytest.skip("8-bit pages hold no infinity")
    times = []
    for marks in ([], [(0, 0, 0, 5, value)]):
        c = Case(clo, [(8192, 8192)], 2, 128, 64, bits, seed=95)
        put_v(c, marks)
        c.device()
        q = bf16(rand(96, 8192, 8, 128)).cuda()
        out = c.attend(q)
        assert bool(torch.isfinite(out).all()) == (not marks)
        runs = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            c.attend(q, out=out)
            b.record()
            b.synchronize()
            runs.append(a.elapsed_time(b))
        times.append(min(runs))
    print(f"{times[0] * 1e3:.0f} us, with it {times[1] * 1e3:.0f} us")
    assert times[1] < 20 * times[0]  # row by row it would be hundreds of times


# --------------------------------------------------------------------------------------------- padded decode batches
def best_time(call, n=5):
    runs = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        runs.append(a.elapsed_time(b))
    return min(runs)


@pytest.mark.parametrize("bits", [16, 8])
def test_sequences_without_rows_cost_no_work(clo, bits):
    # inactive slots of a decode batch in front of an active one, whole units (no workspace): each read the active one's pages
    none = torch.empty(16, dtype=torch.uint8, device="cuda")
    times, q = [], bf16(rand(101, 1, 8, 128)).cuda()
    for slots in (0, 600):
        c = Case(clo, [(0, 0)] * slots + [(1, 20000)], 2, 128, 64, bits, seed=100)
        c.device()
        got = c.attend(q, workspace=none)
        want, spread, reach = dense(c, q.cpu())
        check(got, want, ref.attention_bound(want, spread, reach, 128, bits))
        times.append(best_time(lambda: c.attend(q, workspace=none)))
    print(f"{times[0] * 1e3:.0f} us, with 600 inactive slots {times[1] * 1e3:.0f} us")
    assert times[1] < 2 * times[0]  # 601 times the bytes otherwise


@pytest.mark.parametrize("d,bits", [(128, 16), (64, 8)])
def test_decode_batches_of_any_pattern_of_rows(clo, d, bits):
    # sequences without rows first, last and between, with and without tokens, beside longer ones; whole units and shares
    for seed in range(6):
        pick = torch.randint(0, 4, (40,), generator=torch.Generator().manual_seed(seed)).tolist()
        seqs = [[(0, 0), (0, 70), (1, 300 + 97 * i), (2, 1 + 5 * i)][k] for i, k in enumerate(pick)]
        if not any(n for n, _ in seqs):
            continue
        seqs = [(n, max(n, kv)) for n, kv in seqs]
        c = Case(clo, seqs, 2, d, 32, bits, seed=seed)
        c.device()
        q = bf16(rand(110 + seed, c.total, 6, d))
        want, spread, reach = dense(c, q)
        bound = ref.attention_bound(want, spread, reach, d, bits)
        check(c.attend(q), want, bound)
        check(c.attend(q, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), want, bound, "no workspace")


# --------------------------------------------------------------------------------------------- rows beyond max_q
@pytest.mark.parametrize("bits", [16, 8])
def test_rows_beyond_max_q_are_left_out_by_every_call(clo, bits):
    # of sequences with 9, 2 and 6 rows, the first 4 rows at most; keys, queries, read-back and attention agree on it
    d, hkv, hq, most = 64, 2, 4, 4
    seqs = [(9, 40), (2, 2), (6, 6)]
    c = Case(clo, seqs, hkv, d, 16, bits, seed=120)
    cache = c.device()
    before = [p.clone() for p in (cache.k_pages, cache.v_pages)]
    plan = clo.clo_rope_plan_init(rot_dim=d)
    k, q = bf16(rand(121, c.total, hkv, d)).cuda(), bf16(rand(122, c.total, hq, d)).cuda()
    mark = lambda h: torch.full((c.total, h, d), 7.0, dtype=BF16, device="cuda")  # noqa: E731
    q_out, k_out, v_out, out = mark(hq), mark(hkv), mark(hkv), mark(hq)
    cache.append(k, k, c.starts, c.lens, c.tab, rope=plan, q=q, q_out=q_out, max_q=most)
    cache.read(c.starts, c.lens, c.tab, c.total, k_out=k_out, v_out=v_out, max_q=most)
    cache.attention(q, c.starts, c.lens, c.tab, out=out, max_q=most)
    left = torch.cat([torch.arange(n) >= most for n, _ in seqs]).cuda()
    for t in (q_out, k_out, v_out, out):
        assert bool((t[left] == 7.0).all()) and not bool((t[~left] == 7.0).all(-1).any())
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in seqs])
    want = clo.clo_rope(plan, q, pos.cuda())
    assert torch.equal(q_out[~left], want[~left])
    for pages, old in zip((cache.k_pages, cache.v_pages), before):
        for first, n, kv in c.seqs:
            for i in range(most, n):
                j, b = kv - n + i, [s[0] for s in c.seqs].index(first)
                page = int(c.table[b, j // 16])
                assert torch.equal(pages.view(torch.uint8)[page, :, j % 16], old.view(torch.uint8)[page, :, j % 16])


# --------------------------------------------------------------------------------------------- scales at the ends of their range
@pytest.mark.parametrize("power", [1e-30, 2.0 ** -64, 3e33])
@pytest.mark.parametrize("seqs", [[(1, 60000), (1, 25000)], [(1, 30000), (2, 700)] + [(1, 24000)] * 38])
def test_decode_with_scales_at_the_ends_of_their_range(clo, seqs, power):
    # weights that are nearly equal over many tokens, divided by such scales, sum up to 1e34 times the tokens
    c = Case(clo, seqs, 2, 64, 128, 8, seed=130)
    c.scales[1] = (c.scales[1] * (64 if power > 1e-30 else 0) * power).clamp(min=1e-30)
    c.pages.scale[1] = c.scales[1].double()
    c.device()
    q = bf16(rand(131, c.total, 8, 64) * 1e-3)
    want, spread, reach = dense(c, q)
    assert float(want.abs().max()) < 3e38
    unit = float(want.abs().max())  # (the bound's floor of 1e-30 is about values near one)
    bound = ref.attention_bound(want / unit, spread / unit, reach, 64, 8)
    check(c.attend(q).double() / unit, want / unit, bound)
    check(c.attend(q, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")).double() / unit, want / unit, bound, "no workspace")


def test_prompt_with_scales_at_the_end_of_their_range(clo):
    # weights of up to 2^15 (the running maximum lags by up to 2^8) over scales of 1e-30: a whole unit's sum passes fp32's range
    rows, kv, d = 200, 20000, 64
    c = Case(clo, [(rows, kv)], 1, d, 64, 8, seed=133)
    c.scales[1] = torch.full_like(c.scales[1], 1e-30)
    c.scales[0] = torch.full_like(c.scales[0], 2.0 ** -8)
    for t in (c.codes[0], c.pages.val[0]):
        t.view(torch.uint8).zero_() if t.dtype is torch.float8_e4m3fn else t.zero_()
    for j in range(256, kv):
        page = int(c.table[0, j // 64])
        c.codes[0].view(torch.uint8)[page, 0, j % 64, 0] = 0x7e  # 448
        c.pages.val[0][page, 0, j % 64, 0] = 448.0
    c.pages.scale = [s.double() for s in c.scales]
    c.device()
    q = torch.zeros(rows, 2, d, dtype=BF16)
    q[..., 0] = bf16(torch.tensor(7.5 * math.log(2) * math.sqrt(d) / 1.75))
    want, spread, reach = dense(c, q)
    unit = float(want.abs().max())
    bound = ref.attention_bound(want / unit, spread / unit, reach, d, 8)
    for work in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):
        check(c.attend(q, workspace=work).double() / unit, want / unit, bound)


# --------------------------------------------------------------------------------------------- autograd
def test_rows_that_require_a_gradient_are_refused_while_it_is_recorded(clo):
    n, h, d = 5, 2, 64
    plan, pos = clo.clo_rope_plan_init(rot_dim=d), torch.arange(n, device="cuda")
    x = bf16(rand(141, n, h, d)).cuda()
    g = x.clone().requires_grad_()
    c = Case(clo, [(n, n)], h, d, 16, 16, seed=142)
    cache = c.device()
    at = (c.starts, c.lens, c.tab)
    calls = [lambda t: clo.clo_rope(plan, t, pos), lambda t: clo.clo_rope(plan, x, pos, out=t), lambda t: cache.append(t, x, *at),
             lambda t: cache.append(x, t, *at), lambda t: cache.append(x, x, *at, rope=plan, q=t),
             lambda t: cache.append(x, x, *at, rope=plan, q=x, q_out=t), lambda t: cache.read(*at, n, k_out=t),
             lambda t: cache.read(*at, n, v_out=t), lambda t: cache.attention(t, *at), lambda t: cache.attention(x, *at, out=t)]
    for call in calls:
        for t in (g, g * 2):  # a leaf, and what was computed from one
            with pytest.raises(ValueError, match="gradient"):
                call(t)
    with pytest.raises(ValueError, match="gradient"):
        clo.PagedCache(cache.k_pages.clone().requires_grad_(), cache.v_pages)
    want = clo.clo_rope(plan, x, pos)
    with torch.no_grad():
        for call in calls:
            call(g.clone())
        assert torch.equal(clo.clo_rope(plan, g, pos), want)
    with torch.inference_mode():
        y = clo.clo_rope(plan, g, pos)
        assert torch.equal(y, want)
        cache.append(y, y, *at, rope=plan, q=y, q_out=y)
        cache.attention(y, *at, out=torch.empty_like(y))
    assert torch.equal(clo.clo_rope(plan, g.detach(), pos), want)
    assert not want.requires_grad


@pytest.mark.parametrize("bits", [16, 8])
def test_what_a_call_writes_gets_a_new_version(clo, bits):
    n, h, d = 5, 2, 64
    plan, pos = clo.clo_rope_plan_init(rot_dim=d), torch.arange(n, device="cuda")
    x = bf16(rand(151, n, h, d)).cuda()
    c = Case(clo, [(n, n)], h, d, 16, bits, seed=152)
    cache = c.device()
    at = (c.starts, c.lens, c.tab)
    out = [torch.empty_like(x) for _ in range(5)]
    work = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    pages = [t for t in (cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales) if t is not None]
    read = [x, pos, *at]
    now = lambda ts: [t._version for t in ts]  # noqa: E731

    def raises(call, ts):
        old, kept = now(ts), now(read)
        call()
        assert all(a > b for a, b in zip(now(ts), old)) and now(read) == kept

    raises(lambda: clo.clo_rope(plan, x, pos, out=out[0]), [out[0]])
    raises(lambda: cache.append(x, x, *at, rope=plan, q=x, q_out=out[1]), pages + [out[1]])
    raises(lambda: cache.read(*at, n, k_out=out[2], v_out=out[3]), out[2:4])
    raises(lambda: cache.attention(x, *at, out=out[4], workspace=work), [out[4], work])
    old = now(pages)
    cache.read(*at, n), cache.attention(x, *at)
    with pytest.raises(ValueError):
        cache.append(x, x[:2], *at)
    assert now(pages) == old
    # autograd notices that what it saved was overwritten
    w = torch.ones_like(x, requires_grad=True)
    y = (w * out[0]).sum()
    clo.clo_rope(plan, x, pos, out=out[0])
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    with torch.inference_mode():  # tensors without a version
        clo.clo_rope(plan, x, pos, out=torch.empty_like(x))


# --------------------------------------------------------------------------------------------- threads
def test_other_threads_run_while_a_launch_waits(clo):
    # the launch queue is full behind 0.6 s of other work: a call waits for room, and a second thread goes on
    import threading
    import time

    x = bf16(rand(161, 1, 1, 64)).cuda()
    plan, pos, out = clo.clo_rope_plan_init(rot_dim=64), torch.zeros(1, dtype=torch.int64, device="cuda"), torch.empty_like(x)
    clo.clo_rope(plan, x, pos, out=out)
    torch.cuda.synchronize()
    longest, done = [0.0], threading.Event()

    def tick():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            longest[0], last = max(longest[0], now - last), now

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        t0 = time.perf_counter()
        torch.cuda._sleep(1_200_000_000)
        for _ in range(5000):
            clo.clo_rope(plan, x, pos, out=out)
        took = time.perf_counter() - t0
        torch.cuda.synchronize()
    finally:
        done.set()
        thread.join()
    assert took > 0.3, "the queue was not full"
    assert longest[0] < 0.2, f"the second thread stood still for {longest[0]:.2f} s"


def test_arguments_of_no_truth_or_kind_are_refused(clo):
    x = bf16(rand(171, 2, 2, 64)).cuda()
    plan, pos = clo.clo_rope_plan_init(rot_dim=64), torch.zeros(2, dtype=torch.int64, device="cuda")
    out = torch.zeros_like(x)
    with pytest.raises(RuntimeError, match="ambiguous"):  # the error of the truth value itself
        clo.clo_rope(plan, x, pos, out=out, transpose=torch.ones(2))
    torch.cuda.synchronize()
    assert not out.any()  # refused before the launch
    for bad in (dict(stream="side"), dict(stream=object()), dict(stream=1.5)):
        with pytest.raises((AttributeError, TypeError, ValueError)):
            clo.clo_rope(plan, x, pos, out=out, **bad)
    c = Case(clo, [(2, 2)], 2, 64, 16, 16, seed=172)
    cache = c.device()
    at = (c.starts, c.lens, c.tab)
    for bad in (dict(max_q=1.5), dict(max_q="1"), dict(window=None), dict(sinks=1 << 40), dict(softmax_scale="x"), dict(workspace=x)):
        with pytest.raises((TypeError, ValueError)):
            cache.attention(x, *at, **bad)


# --------------------------------------------------------------------------------------------- rotation at any position
def rotated_exactly(plan, x, pos):
    """fp64 rotation by the plan's own turns, position * turn modulo one turn in integers, and what fp32 may be off by: cosine and sine
    by 7.5e-8, and two roundings of a product and a sum (2^-24 each)."""
    import numpy as np

    half = plan.rot_dim // 2
    turn = np.array(plan.turn[:half], dtype=np.uint64)
    with np.errstate(over="ignore"):
        frac = pos.numpy().astype(np.uint64)[:, None] * turn
    angle = torch.from_numpy(frac.astype(np.float64)) * (2 * math.pi / 2.0 ** 64)
    c, s = (torch.cos(angle) * plan.magnitude)[:, None], (torch.sin(angle) * plan.magnitude)[:, None]
    y, off = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    ia = torch.arange(half) * 2 if plan.interleaved else torch.arange(half)
    ib = ia + 1 if plan.interleaved else ia + half
    p, q = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = p * c - q * s, q * c + p * s
    off[..., ia] = off[..., ib] = (7.5e-8 + 2 * 2.0 ** -24) * plan.magnitude * (p.abs() + q.abs())
    return y, off


def rounded_once(got, want, off):
    """got is want, off by at most `off`, rounded to bf16: within half a step of want, where off reaches the next value too."""
    got = got.cpu().double()
    e = torch.frexp(torch.maximum(got.abs(), want.abs()))[1]
    half_step = torch.ldexp(torch.ones_like(want), e - 9)  # 8 significant bits
    over = (got - want).abs() / (half_step + off)
    assert float(over.max()) <= 1.0, f"{float(over.max()):.6f} of the bound"


POSITIONS = [(0, 1 << 20), (1 << 31, 1 << 33), (1 << 33, 1 << 45), (1 << 45, (1 << 63) - 1), (-(1 << 62), 0)]


@pytest.mark.parametrize("lo,hi", POSITIONS)
@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (64, 64, True), (128, 48, True), (96, 96, False), (64, 20, False)])
def test_rope_rounds_once_at_any_position(clo, lo, hi, d, rot, interleaved):
    n, h = 2000, 4
    gen = torch.Generator().manual_seed(d + rot)
    pos = torch.randint(lo, hi, (n,), generator=gen)
    plan = clo.clo_rope_plan_init(rot_dim=rot, interleaved=interleaved, theta=500000.0, scaling="yarn", factor=16.0, original_max=32768)
    x = bf16(rand(181, n, h, d))
    rounded_once(clo.clo_rope(plan, x.cuda(), pos.cuda()), *rotated_exactly(plan, x, pos))


@pytest.mark.parametrize("lo,hi", POSITIONS)
def test_append_rounds_once_at_any_position(clo, lo, hi):
    n, hkv, hq, d = 700, 2, 4, 128
    pos = torch.randint(lo, hi, (n,), generator=torch.Generator().manual_seed(182))
    plan = clo.clo_rope_plan_init(rot_dim=d)
    c = Case(clo, [(n, n)], hkv, d, 64, 16, seed=183)
    cache = c.device()
    k, q = bf16(rand(184, n, hkv, d)), bf16(rand(185, n, hq, d))
    got = cache.append(k.cuda(), k.cuda(), c.starts, c.lens, c.tab, rope=plan, positions=pos.cuda(), q=q.cuda())
    rounded_once(got, *rotated_exactly(plan, q, pos))
    rounded_once(cache.read(c.starts, c.lens, c.tab, n)[0], *rotated_exactly(plan, k, pos))


# --------------------------------------------------------------------------------------------- many sequences, C names
@pytest.mark.parametrize("bits", [16, 8])
def test_thousands_of_sequences_under_the_c_names(clo, bits):
    # sequences with 0 to 2 rows, in every block of the lookups, through the functions that carry the C names
    pick = torch.randint(0, 3, (3000,), generator=torch.Generator().manual_seed(190)).tolist()
    seqs = [(n, n + 11 * i % 30) for i, n in enumerate(pick)]
    hkv, hq, d = 2, 4, 64
    c = Case(clo, seqs, hkv, d, 16, bits, seed=191, width=2)
    cache = c.device()
    plan = clo.clo_rope_plan_init(rot_dim=d)
    k, v, q = bf16(rand(192, c.total, hkv, d)), bf16(rand(193, c.total, hkv, d)), bf16(rand(194, c.total, hq, d))
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in seqs])
    at = (c.starts, c.lens, c.tab)
    qr = clo.clo_paged_append(cache, k.cuda(), v.cuda(), *at, rope=plan, q=q.cuda(), max_q=2)
    assert torch.equal(qr, clo.clo_rope(plan, q.cuda(), pos.cuda()))
    gk, gv = clo.clo_paged_read(cache, *at, c.total, max_q=2)
    kr = clo.clo_rope(plan, k.cuda(), pos.cuda())
    if bits == 16:
        assert torch.equal(gk, kr) and torch.equal(gv, v.cuda())
    else:  # a code's half step (2^-4 of the value, 2^-10 of the scale at the least) and kr's own rounding
        for got, x, side in ((gk, kr, 0), (gv, v.cuda(), 1)):
            scale = (cache.k_scales, cache.v_scales)[side]
            page = torch.cat([c.table[b, (torch.arange(kv - n, kv) // 16)].long() for b, (n, kv) in enumerate(seqs)]).cuda()
            bound = (2.0 ** -4 + 2.0 ** -7) * x.double().abs() + 2.0 ** -10 * scale[page].double()[:, :, None]
            check(got, x.double().cpu(), bound.cpu())
    # the pages as they are now, for the reference
    for side, (p, s) in enumerate(((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales))):
        c.pages.val[side] = p.cpu().double() if s is None else ref.e4m3_values(p.contiguous().view(torch.uint8).cpu())
        c.scales[side] = None if s is None else s.cpu()
    want, spread, reach = dense(c, qr.cpu())
    bound = ref.attention_bound(want, spread, reach, d, bits)
    check(clo.clo_paged_attention(cache, qr, *at, max_q=2), want, bound)
    size = clo.clo_paged_attention_workspace(cache, hq, len(seqs), c.total, c.tab.shape[1], 2)
    assert size == cache.attention_workspace(hq, len(seqs), c.total, c.tab.shape[1], 2)


def test_capture_on_a_named_stream(clo):
    # the capturing stream named in the call (outputs and workspace from the graph's memory), replayed with other inputs beside eager calls
    c = Case(clo, [(1, 9000), (1, 300)], 2, 128, 64, 8, seed=201)
    c.device()
    plan = clo.clo_rope_plan_init(rot_dim=128)
    q, pos = bf16(rand(202, 2, 8, 128)).cuda(), torch.tensor([8999, 299], device="cuda")
    assert c.cache.attention_workspace(8, 2, 2, c.tab.shape[1], 1) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = c.attend(clo.clo_rope(plan, q, pos, stream=side), stream=side)
    for i in range(3):
        q.copy_(bf16(rand(203 + i, 2, 8, 128)))
        eager = [c.attend(clo.clo_rope(plan, q, pos)) for _ in range(3)]
        graph.replay()
        eager += [c.attend(clo.clo_rope(plan, q, pos)) for _ in range(3)]
        torch.cuda.synchronize()
        for e in eager:
            assert torch.equal(out, e)


# --------------------------------------------------------------------------------------------- lengths past the table, expanded inputs
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("window,sinks", [(0, 0), (10, 4), (10, 0), (700, 100), (1 << 30, 1 << 30)])
@pytest.mark.parametrize("seqs", [[(3, 1000), (1, 33), (2, 40)], [(40, 1000), (20, 700), (33, 60)]])
def test_lengths_past_the_table(clo, seqs, window, sinks, bits):
    # the table holds 48 tokens of each sequence: rows behind them see what is there, or nothing
    c = Case(clo, seqs, 2, 64, 16, bits, seed=211, width=3)
    c.device()
    q = bf16(rand(212, c.total, 6, 64))
    c.compare(c.attend(q, window, sinks), q, window, sinks)


@pytest.mark.parametrize("bits", [16, 8])
def test_inputs_expanded_over_heads_and_tokens(clo, bits):
    hkv, hq, d = 2, 8, 128
    for seqs in ([(1, 90), (2, 33)], [(40, 90), (5, 33)]):
        c = Case(clo, seqs, hkv, d, 32, bits, seed=221)
        cache = c.device()
        plan = clo.clo_rope_plan_init(rot_dim=d)
        k1, q1 = bf16(rand(222, c.total, 1, d)).cuda(), bf16(rand(223, 1, hq, d)).cuda()
        k, q = k1.expand(c.total, hkv, d), q1.expand(c.total, hq, d)  # strides of zero
        pos = torch.cat([torch.arange(kv - n, kv) for n, kv in seqs]).cuda()
        assert torch.equal(clo.clo_rope(plan, q, pos), clo.clo_rope(plan, q.contiguous(), pos))
        qr = cache.append(k, k, c.starts, c.lens, c.tab, rope=plan, q=q, max_q=c.max_q)
        assert torch.equal(qr, clo.clo_rope(plan, q.contiguous(), pos))
        gk, gv = cache.read(c.starts, c.lens, c.tab, c.total)
        twin = Case(clo, seqs, hkv, d, 32, bits, seed=221)
        other = twin.device()
        other.append(k.contiguous(), k.contiguous(), c.starts, c.lens, c.tab, rope=plan, max_q=c.max_q)
        for a, b in zip((gk, gv), other.read(c.starts, c.lens, c.tab, c.total)):
            assert torch.equal(a, b)
        assert torch.equal(c.attend(q), c.attend(q.contiguous()))


@pytest.mark.parametrize("bits", [16, 8])
def test_empty_batches_tables_and_strided_read_back(clo, bits):
    d, hkv = 64, 2
    c = Case(clo, [(3, 20), (1, 7)], hkv, d, 16, bits, seed=231)
    cache = c.device()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = lambda n, h: bf16(rand(232, n, h, d)).cuda()  # noqa: E731
    plan = clo.clo_rope_plan_init(rot_dim=d)
    # no sequence; sequences without a row
    for starts, lens in ((i32(0), i32()), (i32(0, 0, 0), i32(5, 0))):
        table = torch.zeros(len(lens), 2, dtype=torch.int32, device="cuda")
        assert cache.append(rows(0, hkv), rows(0, hkv), starts, lens, table, rope=plan, q=rows(0, 4)).shape == (0, 4, d)
        assert cache.attention(rows(0, 4), starts, lens, table).shape == (0, 4, d)
        assert [t.shape for t in cache.read(starts, lens, table, 0)] == [(0, hkv, d)] * 2
    # a table without pages: nothing is written, read as zeros, attended to
    before = [t.clone() for t in cache._tensors if t is not None]
    for n in (1, 30):
        at = i32(0, n), i32(n), torch.zeros(1, 0, dtype=torch.int32, device="cuda")
        qr = cache.append(rows(n, hkv), rows(n, hkv), *at, rope=plan, q=rows(n, 4))
        assert torch.equal(qr, clo.clo_rope(plan, rows(n, 4), torch.arange(n, device="cuda")))
        assert not cache.attention(rows(n, 4), *at).any() and not any(t.any() for t in cache.read(*at, n))
    for a, b in zip(before, (t for t in cache._tensors if t is not None)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # into wider rows, heads outermost, the rest left alone
    want = cache.read(c.starts, c.lens, c.tab, c.total)
    wide = torch.full((c.total, hkv, d + 8), 7.0, dtype=BF16, device="cuda")
    outer = torch.full((hkv, c.total + 1, d), 7.0, dtype=BF16, device="cuda")
    cache.read(c.starts, c.lens, c.tab, c.total, k_out=wide[..., :d], v_out=outer.transpose(0, 1)[:c.total])
    assert torch.equal(wide[..., :d], want[0]) and bool((wide[..., d:] == 7.0).all())
    assert torch.equal(outer.transpose(0, 1)[:c.total], want[1]) and bool((outer[:, c.total] == 7.0).all())


@pytest.mark.parametrize("group", [2, 16])
def test_the_most_sequences_that_a_call_takes(clo, group):
    # 65,535 sequences of two tokens, both the call's: 4 rows per kv head, or 32 (the prompt kernel)
    batch, d, scale = 65535, 64, 0.2
    cache = clo.PagedCache.create(batch, 1, 16, d)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.randperm(batch, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda().view(batch, 1)
    starts, lens = torch.arange(0, 2 * batch + 1, 2, **i32), torch.full((batch,), 2, **i32)
    gen = torch.Generator(device="cuda").manual_seed(2)
    new = lambda h: torch.randn((2 * batch, h, d), generator=gen, device="cuda").to(BF16)  # noqa: E731
    k, v, q = new(1), new(1), new(group)
    times = [best_time(lambda: cache.append(k, v, starts, lens, table, max_q=2), 3)]
    gk, gv = cache.read(starts, lens, table, 2 * batch, max_q=2)
    assert torch.equal(gk, k) and torch.equal(gv, v)
    out = cache.attention(q, starts, lens, table, max_q=2, softmax_scale=scale)
    times.append(best_time(lambda: cache.attention(q, starts, lens, table, out=out, max_q=2, softmax_scale=scale), 3))
    print(f"append {times[0]:.2f} ms, attention {times[1]:.2f} ms")
    kd, vd, qd = (t.double().view(batch, 2, -1, d) for t in (k, v, q))
    sc = torch.einsum("bqhd,bkd->bqhk", qd, kd[:, :, 0]) * scale
    sc[:, 0, :, 1] = -math.inf
    w = torch.softmax(sc, -1)
    want, spread = torch.einsum("bqhk,bkd->bqhd", w, vd[:, :, 0]), torch.einsum("bqhk,bkd->bqhd", w, vd[:, :, 0].abs())
    reach = (torch.einsum("bqhd,bkd->bqhk", qd.abs(), kd[:, :, 0].abs()) * scale).amax(-1, keepdim=True)
    bound = ref.attention_bound(want, spread, reach, d, 16).view(2 * batch, group, d)
    check(out, want.view(2 * batch, group, d).cpu(), bound.cpu())
