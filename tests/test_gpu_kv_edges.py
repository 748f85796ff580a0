"""GPU tests of the cache calls at the ends of what they accept: scales and scores at
the limits, many chunks, sizes at which a launch or a workspace could not hold."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv_util as U  # noqa: E402
import test_gpu_kv as T  # noqa: E402
from lossless_rejection_sampling_spec_amd import binding  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = T.DEV


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    binding.lib()
    yield


@pytest.fixture(autouse=True)
def _seed():
    """Each test's values are its own, whichever tests run before it."""
    torch.manual_seed(11)


def repeated(cache, times):
    """The cache's first request `times` times over the same pages."""
    table = cache.page_table[:1].expand(times, -1).contiguous()
    return binding.KVCache(pages=cache.pages, page_table=table,
                           seq_lens=cache.seq_lens[:1].expand(times).contiguous(),
                           ref_counts=cache.ref_counts, page_size=cache.page_size,
                           kv_heads=cache.kv_heads, head_dim=cache.head_dim)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,heads", [(64, 4), (128, 4), (256, 2)])
@pytest.mark.parametrize("scale", [1e-38, 3e-39, 1e-44, 1e-30])
@pytest.mark.parametrize("batch,window", [(1, 200), (256, 700)])
def test_the_smallest_scales_with_a_window(dtype, d, heads, scale, batch, window):
    """Rows that see nothing of a wave's first tile, but of its later ones: the window of
    row 0 starts at the last position of a tile, those of the others behind it.  The
    result is the mean of the visible V."""
    rows = 6
    ctx = 639 + window - 1                             # row 0's first position: 639, 31 mod 32
    cache, K, V = T.make_attention(d, 16, 1, [rows], [ctx], d)
    q = torch.randn(rows, heads, d, device=DEV).to(T.DTYPES[dtype])
    cu = [rows * b for b in range(batch + 1)]
    out, st = binding.kv_attention(repeated(cache, batch), q.repeat(batch, 1, 1), T._i(cu),
                                   T._i([ctx] * batch), max_k=5, max_context=ctx + rows, scale=scale,
                                   window=window)
    assert st.cpu().tolist() == [0] * batch
    T.check_attention(out, q, K, V, [0, rows], [ctx], [rows], dtype, float(np.float32(scale)), window)
    assert (out.view(batch, -1) == out.view(batch, -1)[0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,heads", [(64, 1), (128, 20), (256, 2)])
@pytest.mark.parametrize("power", [10, 25, 31, 40, 90])
@pytest.mark.parametrize("batch", [1, 300])
def test_scores_far_beyond_the_exponents_of_fp32(dtype, d, heads, power, batch):
    """Queries of a single power of two: every score is exact, the largest ones are
    equal, and few of the others count beside them.  The result is the mean of V over the
    largest, and from 2^30 on that or NaN for the whole row."""
    rows, ctx = 3, 900
    cache, K, V = T.make_attention(d, 16, 1, [rows], [ctx], power)
    x = torch.zeros(rows, heads, d)
    for j in range(rows):
        for h in range(heads):
            x[j, h, (7 * j + 11 * h) % d] = (-1) ** h * 2.0 ** power
    q = x.to(T.DTYPES[dtype]).to(DEV)
    cu = [rows * b for b in range(batch + 1)]
    out, st = binding.kv_attention(repeated(cache, batch), q.repeat(batch, 1, 1), T._i(cu),
                                   T._i([ctx] * batch), max_k=2, max_context=ctx + rows, scale=1.0)
    assert st.cpu().tolist() == [0] * batch
    o = T._f64(out)
    for j in range(rows):
        for h in range(heads):
            s = (-1) ** h * K[0][:ctx + j + 1, 0, (7 * j + 11 * h) % d] * 2.0 ** power
            w = np.exp(s - s.max())
            want = w @ V[0][:ctx + j + 1, 0] / w.sum()
            mass = w @ np.abs(V[0][:ctx + j + 1, 0]) / w.sum()
            # the scores are exact: a step of s - m times log2 e, of exp2, of each sum
            # and of the result, and half a bf16 step of each weight of bf16 rows
            gap = np.minimum(s.max() - s, 200.0)
            rel = (T.HALF["bf16"] if dtype == "bf16" else 0) + 2.0 ** -20 + 2 * ctx * 2.0 ** -24
            tol = (mass * rel + (w * gap * 4 * 2.0 ** -24) @ np.abs(V[0][:ctx + j + 1, 0]) / w.sum()
                   + T.HALF[dtype] * np.abs(want))
            if np.abs(s).max() * 1.4427 >= 2.0 ** 30 and np.isnan(o[j, h]).all():
                assert np.isnan(o[-rows + j, h]).all()
                continue
            for b in {0, batch - 1}:
                assert np.all(np.abs(o[b * rows + j, h] - want) <= tol), (j, h, b)


def test_reserve_of_a_full_batch_over_very_many_layers():
    """1,024 requests and 20,000 layers: a workgroup for each request and layer would be
    more than a launch can have.  The shared tail is copied in every layer."""
    layers, page, batch = 20000, 16, 1024
    cache = binding.KVCache.create(layers=layers, num_pages=6, page_size=page, kv_heads=1, head_dim=64,
                                   requests=batch, max_context=64, device=DEV)
    cache.pages.random_(0, 256)
    rows = [0] * batch
    rows[0] = 20
    ctx, st = binding.kv_reserve(cache, T._i(T._cu(rows)))
    assert st.cpu().tolist() == [0] + [3] * (batch - 1)
    st = binding.kv_fork(cache, T._i([0]), T._i([batch - 1]))
    assert st.cpu().tolist() == [0]
    before = cache.pages.clone()
    rows[0], rows[-1] = 0, 1
    ctx, st = binding.kv_reserve(cache, T._i(T._cu(rows)))
    assert st.cpu().tolist() == [3] * (batch - 1) + [0] and int(ctx[-1]) == 20
    assert cache.page_table.cpu()[[0, -1], :2].tolist() == [[0, 1], [0, 2]]
    assert cache.ref_counts.cpu().tolist() == [2, 1, 1, 0, 0, 0]
    assert torch.equal(cache.pages[:, 2], before[:, 1])
    for p in (0, 1, 3, 4, 5):
        assert torch.equal(cache.pages[:, p], before[:, p])


def test_a_cache_of_more_requests_than_the_calls_take_is_refused():
    def make(**kw):
        return binding.KVCache.create(**{**dict(layers=1, num_pages=4, page_size=16, kv_heads=1,
                                                head_dim=64, requests=2, max_context=16, device=DEV),
                                         **kw})
    cache = make(requests=1024)
    assert binding.kv_compact(cache).cpu().tolist() == [0]
    assert binding.kv_fork(cache, T._i([0]), T._i([1023])).cpu().tolist() == [0]
    for kw in (dict(requests=1025), dict(layers=65536, num_pages=1)):
        with pytest.raises(ValueError, match="at most 1024 requests"):
            make(**kw)
    # a step in which no request has rows: the page calls take it, the others are not made
    cu = T._i([0, 0, 0])
    ctx, st = binding.kv_reserve(cache, cu)
    assert st.cpu().tolist() == [3, 3] and ctx.cpu().tolist() == [-1, -1]
    assert binding.kv_release(cache, T._i([0, 0]), ctx).cpu().tolist() == [0, 0]
    none = torch.empty(0, 1, 64, device=DEV)
    with pytest.raises(ValueError):
        binding.kv_append(cache, none, none, none, cu, ctx)
    with pytest.raises(ValueError):
        binding.kv_attention(cache, none, cu, ctx, max_k=0, max_context=16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_gives_the_same_bytes_whatever_the_call(dtype, d):
    """The rows of two requests in one call, in a call of each, and one by one."""
    rows, ctx, heads, kv = [9, 14], [5, 20], 6, 2
    x = torch.randn(sum(rows), heads + 2 * kv, d, device=DEV).to(T.DTYPES[dtype])
    w = 1 + 0.1 * torch.randn(2, d, device=DEV)
    cs = torch.from_numpy(T._rotation(64, d)).to(DEV)

    def make():
        cache = binding.KVCache.create(layers=1, num_pages=8, page_size=16, kv_heads=kv, head_dim=d,
                                       requests=2, max_context=64, device=DEV)
        cache.page_table.copy_(torch.arange(8, device=DEV).view(2, 4))
        return cache

    def append(cache, x, cu, ctx):
        q, st = binding.kv_append(cache, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:],
                                  T._i(cu), T._i(ctx), q_weight=w[0], k_weight=w[1], cos_sin=cs)
        assert all(s in (0, 3) for s in st.cpu().tolist())
        return q

    whole = make()
    q = append(whole, x, [0, 9, 23], ctx)
    apart = make()
    q2 = torch.cat([append(apart, x[:9], [0, 9, 9], ctx), append(apart, x[9:], [0, 0, 14], ctx)])
    single = make()
    q3 = torch.cat([append(single, x[i:i + 1], [0, 1, 1] if i < 9 else [0, 0, 1],
                           [5 + i, 0] if i < 9 else [0, 11 + i]) for i in range(23)])
    for other, oq in ((apart, q2), (single, q3)):
        assert torch.equal(whole.pages, other.pages) and torch.equal(q, oq)


def long_cache(d, page, kv, n, seed):
    """One sequence of n positions of random codes: (cache, K, V)."""
    rng, pages = np.random.default_rng(seed), -(-n // page)
    units = rng.integers(0, 256, (1, pages, kv, page * (d + d // 16)), np.uint8)
    units[..., page * d:] = rng.integers(122, 128, units[..., page * d:].shape, np.uint8)
    ids = rng.permutation(pages)
    K, V = (np.empty((pages * page, kv, d)) for _ in range(2))
    for i, p in enumerate(ids):
        for h in range(kv):
            K[i * page:(i + 1) * page, h], V[i * page:(i + 1) * page, h] = U.read_unit(units[0, p, h], page, d)
    return T._cache(units, ids.reshape(1, -1), [n], np.ones(pages), page, kv, d), K[:n], V[:n]


@pytest.mark.parametrize("dtype,d,heads,kv,batch", [("bf16", 128, 32, 4, 1024), ("bf16", 64, 32, 4, 1024),
                                                    ("bf16", 256, 16, 2, 1024), ("f32", 64, 16, 2, 1024),
                                                    ("bf16", 128, 4, 4, 1024), ("f32", 128, 4, 4, 1024)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50000, 40)])
def test_contexts_of_more_tiles_than_chunks_hold(dtype, d, heads, kv, batch, window, sinks):
    """A batch so large that a request has few chunks: long ones take chunks of hundreds
    of tiles, whose page ids are read 64 at a time.  One long request loses a page far
    inside a chunk; a bound of 2^20 positions changes the chunks again."""
    cache, K, V = long_cache(d, 64, kv, 70003, d)
    cache = repeated(cache, batch)
    rng = np.random.default_rng(heads)
    rows = [int(x) for x in rng.integers(1, 4, batch)]
    ctx = [int(x) for x in rng.integers(0, 500, batch)]
    some = {0: 70000, 1: 16384, 2: 16383, 5: 16352, 77: 33000, 1000: 65535, batch - 1: 2048}
    for b, c in some.items():
        ctx[b], rows[b] = c, 2
    rows[0] = 3
    cache.page_table[77, 300] = 1 << 25
    cu = T._cu(rows)
    q = torch.randn(int(cu[-1]), heads, d, device=DEV).to(T.DTYPES[dtype])
    want = [0] * batch
    want[77] = 8
    for bound in (70003, 1 << 20):
        out, st = binding.kv_attention(cache, q, T._i(cu), T._i(ctx), max_k=6, max_context=bound,
                                       window=window, sinks=sinks)
        assert st.cpu().tolist() == want
        o = T._f64(out)
        assert np.isnan(o[cu[77]:cu[78]]).all()
        for b in sorted(set(some) - {77}) + [3, 500]:
            n = ctx[b] + rows[b]
            for h in (0, kv - 1):                      # the last query head of a KV head
                at = (h + 1) * (heads // kv) - 1
                T.check_attention(out[cu[b]:cu[b + 1], at:at + 1], q[cu[b]:cu[b + 1], at:at + 1],
                                  [K[:n, h:h + 1]], [V[:n, h:h + 1]], [0, rows[b]], [ctx[b]], [rows[b]],
                                  dtype, d ** -0.5, window, sinks)


def test_a_page_table_whose_rows_are_part_of_longer_ones_is_refused():
    """The calls would use the entries behind a row, which are not the cache's."""
    wide = torch.full((2, 8), -1, dtype=torch.int32, device=DEV)
    pages = torch.zeros(1, 12, binding.kv_page_bytes(1, 64, 16), dtype=torch.uint8, device=DEV)

    def make(table):
        return binding.KVCache(pages=pages, page_table=table, seq_lens=T._i([0] * len(table)),
                               ref_counts=T._i([0] * 12), page_size=16, kv_heads=1, head_dim=64)

    for table in (wide[:, :4], wide[:, ::2], wide.t()[:2], wide[:1].expand(2, -1)):
        with pytest.raises(ValueError, match="page_table"):
            make(table)
    # a single row has no stride of its own
    for table in (wide[:1], wide[:1, :4], wide[0].as_strided((1, 4), (0, 1))):
        cache = make(table)
        ctx, st = binding.kv_reserve(cache, T._i([0, 16 * table.shape[1] + 1]))
        assert st.cpu().tolist() == [7]
        ctx, st = binding.kv_reserve(cache, T._i([0, 16 * table.shape[1]]))
        assert st.cpu().tolist() == [0]
        assert table.cpu().tolist() == [list(range(table.shape[1]))]
        assert wide.cpu()[0, table.shape[1]:].tolist() == [-1] * (8 - table.shape[1])
        wide.fill_(-1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("batch,heads,n", [(1, 3, 40007), (1, 1, 20000), (130, 2, 50001), (33, 5, 70000)])
def test_contexts_of_many_chunks_are_joined(dtype, d, batch, heads, n):
    """79 and 157 chunks of one user and 35 of a request in a small batch (a workgroup per
    row joins them, 64 at a time), 25 of some requests of a larger one (16 threads per
    row, 16 at a time)."""
    cache, K, V = long_cache(d, 16, 1, n, heads)
    cache = repeated(cache, batch)
    rng = np.random.default_rng(d)
    rows = [int(x) for x in rng.integers(1, 4, batch)]
    ctx = [int(x) for x in rng.integers(0, 3000, batch)]
    rows[0], ctx[0] = 3, n - 3
    some = {0}
    if batch > 1:
        some |= {7, 20, batch - 1}
        ctx[7], ctx[20] = 16 * 2048 + 5, 17 * 2048 - rows[20]
    cu = T._cu(rows)
    q = torch.randn(int(cu[-1]), heads, d, device=DEV).to(T.DTYPES[dtype])
    out, st = binding.kv_attention(cache, q, T._i(cu), T._i(ctx), max_k=2, max_context=n)
    assert st.cpu().tolist() == [0] * batch
    for b in some:
        m = ctx[b] + rows[b]
        T.check_attention(out[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], [K[:m]], [V[:m]], [0, rows[b]], [ctx[b]],
                          [rows[b]], dtype, d ** -0.5)


def test_sizes_past_32_bits_are_refused():
    """Their low 32 bits would be sizes that the call takes."""
    cache, q, cu, ctx, kw = T._small()
    binding.kv_attention(cache, q, cu, ctx, **kw)
    for change in (dict(window=(1 << 32) + 16), dict(window=20, sinks=1 << 32), dict(max_k=(1 << 32) + 4),
                   dict(max_context=(1 << 32) + 705), dict(max_context=(1 << 30) + 1)):
        with pytest.raises(ValueError):
            binding.kv_attention(cache, q, cu, ctx, **{**kw, **change})


def test_a_call_does_not_wait_for_a_thread_on_another_stream():
    """One thread in the middle of a call's launches; another's call on its own stream goes
    through, one on the same stream waits."""
    import threading
    cache, q, cu, ctx, kw = T._small()
    want, _ = binding.kv_attention(cache, q, cu, ctx, **kw)
    torch.cuda.synchronize()
    done = [threading.Event(), threading.Event()]
    outs = []

    def call(i, stream):
        with torch.cuda.stream(stream):
            outs.append(binding.kv_attention(cache, q, cu, ctx, **kw)[0])
        done[i].set()

    here = torch.cuda.current_stream()
    threads = [threading.Thread(target=call, args=a) for a in ((0, torch.cuda.Stream()), (1, here))]
    with binding._on(cache.device):
        for t in threads:
            t.start()
        assert done[0].wait(30) and not done[1].is_set()
    assert done[1].wait(30)
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(outs) == 2 and all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("batch,heads,window", [(1, 3, 0), (24, 3, 0), (24, 3, 37), (300, 10, 0)])
def test_what_lies_behind_the_last_position_changes_no_bit(dtype, d, batch, heads, window):
    """Stale bytes behind a request's last position, and pages it does not hold, as scales
    of NaN, as large values and as small ones: the same bits.  (Rows that fill up a tile of
    16 must not see them either: they share the moments at which maxima are raised.)"""
    rng = np.random.default_rng(d + batch)
    rows = [int(x) for x in rng.integers(1, 6, batch)]
    ctx = [int(x) for x in rng.integers(0, 400, batch)]
    page, n = 16, [c + r for c, r in zip(ctx, rows)]
    cache, K, V = T.make_attention(d, page, 1, [rows[0]] * 3, [700] * 3, batch)
    table = cache.page_table[0]
    pages = cache.pages.cpu().numpy().reshape(1, -1, 1, page * (d + d // 16))
    ids = table.cpu().numpy()
    cu = T._cu(rows)
    q = torch.randn(int(cu[-1]), heads, d, device=DEV).to(T.DTYPES[dtype]) * 2
    ks, vs = U.places(page, d)[2:]
    outs = []
    for fill in (255, 252, 140, 1):
        out = []
        for b in range(min(batch, 24)):            # a call of each request's own stale bytes
            host = np.full_like(pages, fill)
            held = -(-n[b] // page)
            host[0, ids[:held]] = pages[0, ids[:held]]
            for at in (ks, vs):
                host[0, ids[held - 1]][:, at[n[b] - (held - 1) * page:]] = fill
            c2 = T._cache(host, ids.reshape(1, -1), [n[b]], np.zeros(host.shape[1]), page, 1, d)
            c2 = repeated(c2, batch)
            only = [0] * (b + 1) + [rows[b]] * (batch - b)
            o, st = binding.kv_attention(c2, q[cu[b]:cu[b + 1]], T._i(only),
                                         T._i([ctx[b] if i == b else 0 for i in range(batch)]), max_k=4,
                                         max_context=500, window=window)
            assert int(st[b]) == 0
            out.append(o)
        outs.append(torch.cat(out))
    for o in outs[1:]:
        assert torch.equal(o.view(torch.uint8), outs[0].view(torch.uint8))
    T.check_attention(outs[0], q, [K[0][:x] for x in n[:24]], [V[0][:x] for x in n[:24]], cu[:25], ctx[:24],
                      rows[:24], dtype, d ** -0.5, window)


@pytest.mark.parametrize("num,pairs", [(64, 3), (70000, 3), (600, 150)])
def test_forks_and_compactions_captured_in_a_graph(num, pairs):
    """Fork, reserve, release and compact as one graph, replayed against eager calls on an
    equal cache, with eager work in between."""
    seqs = pairs + 2

    def make():
        cache = binding.KVCache.create(layers=2 if num < 1000 else 1, num_pages=num, page_size=16,
                                       kv_heads=1, head_dim=64, requests=seqs, max_context=128, device=DEV)
        cache.pages.copy_(torch.arange(cache.pages.numel(), device=DEV).view_as(cache.pages) % 251)
        binding.kv_reserve(cache, T._i(T._cu([40, 21] + [0] * pairs)))
        return cache

    a, b = make(), make()
    src, dst = T._i([i % 2 for i in range(pairs)]), T._i(range(2, seqs))
    cu = T._i(T._cu([1, 0] + [3] * pairs))
    give = T._i([1, 0] + [43 if i % 2 == 0 else 24 for i in range(pairs)])
    lens = T._i([40 if i % 2 == 0 else 21 for i in range(pairs)])

    def step(c):
        f = binding.kv_fork(c, src, dst, lens)
        ctx, r = binding.kv_reserve(c, cu)
        return f, ctx, r, binding.kv_release(c, give), binding.kv_compact(c)

    state = [t.clone() for t in (a.pages, a.page_table, a.seq_lens, a.ref_counts)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(a)
    for t, k in zip((a.pages, a.page_table, a.seq_lens, a.ref_counts), state):
        assert torch.equal(t, k)
    for i in range(5):
        g.replay()
        want = step(b)
        torch.cuda.synchronize()
        assert [int(x) for x in got[0]] == [0] * pairs and int(got[4]) == int(want[4])
        for u, v in zip(got, want):
            assert torch.equal(u, v), i
        for n in ("pages", "page_table", "seq_lens", "ref_counts"):
            assert torch.equal(getattr(a, n), getattr(b, n)), (i, n)
        binding.kv_compact(b)                      # (nothing left to move)
