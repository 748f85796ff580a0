"""GPU tests of attention weights, eviction and appends at offsets: the weights against
float64 with derived bounds, evictions byte for byte against plain Python, and prompts,
evictions and verify steps as a serving loop runs them."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv_budget_util as E  # noqa: E402
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
    torch.manual_seed(17)


# ------------------------------------------------------------------ weights

def check_weights(out, before, q, K, cu, ctx, rows, counts, scale, window=0, sinks=0, skip=()):
    """Every position's weight; what lies behind the last position is as `before` had it
    (`before`: what `out` held, and what was added to)."""
    o, x, old = T._f64(out), T._f64(q), T._f64(before)
    for b in range(len(rows)):
        n = ctx[b] + rows[b]
        if b in skip:
            assert np.array_equal(o[b], old[b]), b
            continue
        w, tol = E.weights(x[cu[b]:cu[b] + rows[b]], K[b], ctx[b], counts[b], scale, window, sinks)
        base = old[b].copy()
        base[:, ctx[b]:n] = 0
        assert np.array_equal(o[b][:, n:], old[b][:, n:]), b
        gap = np.abs(o[b][:, :n] - base[:, :n] - w)
        tol = tol + 2.0 ** -23 * np.abs(base[:, :n])
        assert np.all(gap <= tol), (b, gap.max(), np.unravel_index(gap.argmax(), gap.shape))


def run_weights(dtype, d, page, heads, kv, rows, ctx, *, window=0, sinks=0, seed=0, counts=None,
                max_k=None, max_context=None, loud=False, scale=None):
    cache, K, _ = T.make_attention(d, page, kv, rows, ctx, seed, loud=loud)
    cu = T._cu(rows)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(int(cu[-1]), heads * d + 5, generator=g).to(T.DTYPES[dtype]).to(DEV)
    q = q[:, :heads * d].unflatten(1, (heads, d))
    max_context = max(c + r for c, r in zip(ctx, rows)) if max_context is None else max_context
    kw = dict(max_k=max(rows) - 1 if max_k is None else max_k, max_context=max_context, window=window,
              sinks=sinks, scale=scale, row_counts=None if counts is None else T._i(counts))
    before = torch.rand(len(rows), kv, max_context + 3, generator=g).to(DEV)
    out = before.clone()
    got, st = binding.kv_attention_weights(cache, q, T._i(cu), T._i(ctx), weights=out, **kw)
    assert got is out and st.cpu().tolist() == [0] * len(rows)
    args = (q, K, cu, ctx, rows, rows if counts is None else counts, d ** -0.5 if scale is None else scale,
            window, sinks)
    check_weights(out, before, *args)
    # into other memory, and without weights before
    other = torch.zeros_like(before)
    binding.kv_attention_weights(cache, q, T._i(cu), T._i(ctx), weights=before, out=other, **kw)
    for b, (c, r) in enumerate(zip(ctx, rows)):
        assert torch.equal(other[b, :, :c + r], out[b, :, :c + r])
    assert not any(other[b, :, c + r:].any() for b, (c, r) in enumerate(zip(ctx, rows)))
    fresh, _ = binding.kv_attention_weights(cache, q, T._i(cu), T._i(ctx), **kw)
    assert fresh.shape == (len(rows), kv, max_context)
    check_weights(fresh, torch.zeros_like(fresh), *args)
    again, _ = binding.kv_attention_weights(cache, q, T._i(cu), T._i(ctx), **kw)
    assert torch.equal(fresh, again)
    return fresh


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (256, 16), (128, 32), (64, 128), (256, 256)])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 1), (6, 2)])
def test_weights_of_short_contexts(dtype, d, page, heads, kv):
    run_weights(dtype, d, page, heads, kv, [1, 1, 4, 2, 3, 1, 7, 5], [0, 15, 0, 16, 30, 31, 32, 260])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx", [200, 1500])
def test_weights_of_rows_of_every_tiling(dtype, d, ctx):
    """1 to 512 query rows per KV head: one, two and four 16-row tiles, several blocks of them,
    several groups of blocks; short contexts in one launch, longer ones in two."""
    for heads, rows in ((1, 16), (1, 17), (8, 4), (8, 5), (3, 11), (5, 13), (8, 33), (8, 64), (1, 64)):
        run_weights(dtype, d, 32, heads, 1, [rows, 1], [70, ctx], seed=rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (16, 0), (31, 4), (33, 40), (64, 32),
                                          (100, 500), (5000, 4)])
def test_weights_with_window_and_sinks(dtype, window, sinks):
    run_weights(dtype, 128, 16, 4, 2, [1, 6, 3, 8], [0, 40, 127, 333], window=window, sinks=sinks)
    run_weights(dtype, 64, 64, 2, 2, [5, 1, 2], [3000, 64, 1999], window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1000, 0), (1500, 40), (1024, 1900)])
def test_weights_in_two_launches_through_windows(dtype, d, window, sinks):
    """Windows of several chunks that hide part of the context: positions that no row sees keep
    what they have, or are 0."""
    run_weights(dtype, d, 16, 4, 2, [3, 1, 5], [4500, 33, 1601], window=window, sinks=sinks, seed=2)
    run_weights(dtype, d, 128, 8, 1, [9], [3300], window=window, sinks=sinks, seed=3, max_context=20000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_of_long_contexts(dtype):
    run_weights(dtype, 128, 16, 4, 1, [3, 1, 2], [3001, 700, 255], seed=2)
    run_weights(dtype, 64, 128, 2, 1, [1, 1], [5000, 10], seed=3, max_context=8192)
    run_weights(dtype, 256, 32, 2, 1, [2], [1500], seed=4)


def test_weights_of_chunks_of_64_tiles():
    """Calls with more than 512 chunks of 2,048 positions, some of them a few tiles."""
    rows, ctx = [1] * 70, [4200 if b % 9 == 0 else 20 + b for b in range(70)]
    run_weights("bf16", 64, 128, 8, 8, rows, ctx, seed=5, max_context=30000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_of_counted_rows_only(dtype):
    """None, some and all rows count; the rows that do not count add nothing anywhere."""
    run_weights(dtype, 128, 16, 4, 2, [7, 7, 7, 1], [90, 33, 1200, 5], counts=[0, 3, 7, 1])
    run_weights(dtype, 64, 16, 8, 1, [64, 64], [90, 10], counts=[33, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_of_peaked_scores(dtype):
    run_weights(dtype, 128, 16, 4, 2, [5, 3], [300, 0], loud=True, scale=1.0)
    run_weights(dtype, 64, 16, 2, 1, [2], [1500], loud=True, scale=2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx,at", [(70, (74, 32)), (1300, (1304, 1262))])
def test_rows_that_see_a_nan_add_nothing(dtype, d, ctx, at):
    """A K block stored as NaN, at a position that rows 4 and 5 see, then one that rows 0 and 1
    do: the others' weights are as without it.  V does not matter."""
    rows, page, window, sinks = [6], 16, 40, 2
    cache, K, _ = T.make_attention(d, page, 1, rows, [ctx], 4)
    host = cache.pages.cpu().numpy().reshape(1, -1, 1, page * (d + d // 16))
    table = cache.page_table.cpu().numpy()
    _, _, ks, vs = U.places(page, d)
    q = torch.randn(6, 2, d, device=DEV).to(T.DTYPES[dtype])
    host[0, table[0, (ctx + 1) // page], 0, vs[(ctx + 1) % page, 0]] = 255
    for t, blk, left in ((at[0], d // 32 - 1, 4), (at[1], 0, 2)):
        host[0, table[0, t // page], 0, ks[t % page, blk]] = 255
        K[0][t, 0] = np.nan
        cache.pages.copy_(torch.from_numpy(host.reshape(1, -1, host.shape[-1])))
        out, st = binding.kv_attention_weights(cache, q, T._i([0, 6]), T._i([ctx]), max_k=5,
                                               max_context=ctx + 6, window=window, sinks=sinks)
        assert st.cpu().tolist() == [0]
        check_weights(out, torch.zeros_like(out), q, K, [0, 6], [ctx], rows, [6], d ** -0.5, window, sinks)
        assert abs(float(out.sum()) - 2 * left) < 1e-3


@pytest.mark.parametrize("ctx", [50, 1300])
def test_rows_with_infinite_or_nan_queries_add_nothing(ctx):
    cache, K, _ = T.make_attention(64, 16, 1, [5], [ctx], 3)
    q = torch.randn(5, 8, 64, device=DEV)
    q[1, 3, 7], q[2, 0, 9], q[4] = float("nan"), float("inf"), float("nan")
    out, st = binding.kv_attention_weights(cache, q, T._i([0, 5]), T._i([ctx]), max_k=4,
                                           max_context=ctx + 5)
    assert st.cpu().tolist() == [0]
    check_weights(out, torch.zeros_like(out), q, K, [0, 5], [ctx], [5], [5], 0.125)
    assert abs(float(out.sum()) - 30) < 1e-3


@pytest.mark.parametrize("shift", [0, 1500])
def test_weights_statuses_and_what_is_left(shift):
    """Bad offsets, lengths, counts and pages: those requests' weights stay as they were."""
    rows, ctx = [3, 4, 2, 5, 1, 6], [10 + shift, 30, 20, 50, 8, 7]
    cache, K, _ = T.make_attention(64, 16, 1, rows, ctx, 1)
    cu = T._cu(rows)
    q = torch.randn(21, 2, 64, device=DEV)
    before = torch.rand(6, 1, 100 + shift, device=DEV)
    out = before.clone()
    cache.page_table[1, 1] = 999
    bad = [ctx[0], ctx[1], -1, 96 + shift, ctx[4], ctx[5]]
    counts = [3, 4, 2, 5, 2, 6]                            # request 4 has one row
    _, st = binding.kv_attention_weights(cache, q, T._i(cu), T._i(bad), max_k=4, max_context=100 + shift,
                                         weights=out, row_counts=T._i(counts))
    assert st.cpu().tolist() == [0, 8, 5, 5, 5, 3]
    check_weights(out, before, q, K, cu, ctx, rows, counts, 0.125, skip=(1, 2, 3, 4, 5))


@pytest.mark.parametrize("cu", [[0, 3, 2, 8], [0, 3, 9, 8], [-1, 3, 5, 8]])
def test_weights_broken_offsets_stop_there(cu):
    cache, K, _ = T.make_attention(64, 16, 1, [3, 5, 8], [4, 4, 4], 2)
    q = torch.randn(8, 1, 64, device=DEV)
    before = torch.rand(3, 1, 20, device=DEV)
    out = before.clone()
    _, st = binding.kv_attention_weights(cache, q, T._i(cu), T._i([4, 4, 4]), max_k=7, max_context=20,
                                         weights=out)
    first = 0 if cu[0] < 0 else 1
    assert st.cpu().tolist() == [0] * first + [3] * (3 - first)
    check_weights(out, before, q, K, cu, [4] * 3, [3, 5, 8], [3, 5, 8], 0.125, skip=range(first, 3))


def test_weights_do_not_depend_on_the_other_requests():
    a = run_weights("bf16", 128, 16, 4, 2, [3, 5, 1], [100, 900, 44], seed=9, max_k=7, max_context=1000)
    cache, _, _ = T.make_attention(128, 16, 2, [3, 5, 1], [100, 900, 44], 9)
    g = torch.Generator().manual_seed(9)
    q = torch.randn(9, 4 * 128 + 5, generator=g).to(torch.bfloat16).to(DEV)[:, :512].unflatten(1, (4, 128))
    out, st = binding.kv_attention_weights(cache, q, T._i([3, 3, 8, 8]), T._i([0, 900, 0]), max_k=7,
                                           max_context=1000)
    assert st.cpu().tolist() == [3, 0, 3]
    assert torch.equal(out[1], a[1])


@pytest.mark.parametrize("ctx", [30, 1500])
def test_weights_go_before_the_release(ctx):
    """Rows that do not count need their pages too: after a release that gave one back the
    request's weights stay as they were, before it they are added to."""
    rows, kept = 6, 2                                      # 4 rows are given back, over a page's end
    cache = binding.KVCache.create(layers=1, num_pages=120, page_size=16, kv_heads=1, head_dim=64,
                                   requests=1, max_context=1600, device=DEV)
    first = ctx // 16 * 16 + 14 - 3                        # the page ends after the first 3 + 2 positions
    binding.kv_reserve(cache, T._i([0, first + 3]))
    x = torch.randn(first + 3, 3, 64, device=DEV)
    binding.kv_append(cache, x[:, :1], x[:, 1:2], x[:, 2:], T._i([0, first + 3]), T._i([0]))
    cu = T._i([0, rows])
    at, _ = binding.kv_reserve(cache, cu)
    x = torch.randn(rows, 4, 64, device=DEV)
    q, st = binding.kv_append(cache, x[:, :2], x[:, 2:3], x[:, 3:], cu, at)
    before = torch.rand(1, 1, 1600, device=DEV)
    kw = dict(max_k=5, max_context=first + 9, row_counts=T._i([kept]))
    good, st = binding.kv_attention_weights(cache, q, cu, at, weights=before, out=before.clone(), **kw)
    assert st.cpu().tolist() == [0]
    assert abs(float((good[..., :first + 9] - before[..., :first + 9]).sum())
               - 2 * kept + float(before[..., first + 3:first + 9].sum())) < 1e-3
    binding.kv_release(cache, T._i([rows - kept]), at)
    late, st = binding.kv_attention_weights(cache, q, cu, at, weights=before, out=before.clone(), **kw)
    assert st.cpu().tolist() == [8] and torch.equal(late, before)


# -------------------------------------------------------------------- evict

def make_cache(lens, page, kv, d, layers, seed=0, spare=3, ld=None):
    """Random bytes in every page, shuffled: (cache, pages as numpy, table)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    num = sum(need) + spare
    ids = rng.permutation(num)
    width = max(max(need), 1) if ld is None else ld
    table = np.full((len(lens), width), -1)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    refs = np.zeros(num, np.int64)
    refs[ids[:at]] = 1
    pages = rng.integers(0, 256, (layers, num, kv, page * (d + d // 16)), dtype=np.uint8)
    return T._cache(pages, table, lens, refs, page, kv, d), pages, table, refs


def check_evict(cache, pages, table, refs, weights, before, lens, budgets, sinks, recent, page, d, skip=()):
    """Bytes, weights, tables, counts and lengths against plain Python."""
    layers, _, kv, _ = pages.shape
    want, w = pages.copy(), before.copy()
    new, tab, ref = list(lens), table.copy(), refs.copy()
    for b, (n, m) in enumerate(zip(lens, budgets)):
        if b in skip or m <= 0 or n <= m:
            continue
        held = table[b, :-(-n // page)]
        for layer in range(layers):
            for h in range(kv):
                keep = E.kept(before[layer, b, h], n, m, sinks, recent)
                want[layer, held, h] = E.evict_unit_bytes(pages[layer, held, h], page, d, keep)
                w[layer, b, h, :m] = before[layer, b, h, keep]
                w[layer, b, h, m:n] = 0
        new[b] = m
        gone = held[-(-m // page):]
        ref[gone] -= 1
        tab[b, -(-m // page):-(-n // page)] = -1
    assert cache.seq_lens.cpu().tolist() == new
    assert np.array_equal(cache.page_table.cpu().numpy(), tab)
    assert np.array_equal(cache.ref_counts.cpu().numpy(), ref)
    assert np.array_equal(weights.cpu().numpy(), w, equal_nan=True)
    assert np.array_equal(cache.pages.cpu().numpy().reshape(want.shape), want)


def run_evict(d, page, kv, layers, lens, budgets, sinks=0, recent=0, seed=0, make=None, ld_more=0):
    cache, pages, table, refs = make_cache(lens, page, kv, d, layers, seed)
    rng = np.random.default_rng(seed + 1)
    shape = (layers, len(lens), kv, max(lens) + ld_more)
    w = (np.exp(2 * rng.standard_normal(shape)) if make is None else make(rng, shape)).astype(np.float32)
    weights = torch.from_numpy(w.copy()).to(DEV)
    evicted = torch.arange(len(lens), dtype=torch.int32, device=DEV)
    st = binding.kv_evict(cache, weights, T._i(budgets), sinks=sinks, recent=recent, evicted=evicted)
    assert st.cpu().tolist() == [0] * len(lens)
    check_evict(cache, pages, table, refs, weights, w, lens, budgets, sinks, recent, page, d)
    assert evicted.cpu().tolist() == [b + max(0, n - m if m > 0 else 0)
                                      for b, (n, m) in enumerate(zip(lens, budgets))]


@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (256, 16), (128, 64), (64, 256), (256, 32)])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 8), (0, 30), (30, 0)])
def test_evict_moves_every_byte(d, page, sinks, recent):
    run_evict(d, page, 2, 2, [70, 31, 1, 0, 200, 33, 64], [30, 30, 30, 30, 60, 32, 0], sinks, recent,
              ld_more=5)


@pytest.mark.parametrize("n,m", [(2, 1), (17, 16), (1025, 1), (1025, 1024), (5000, 4097), (4097, 2049)])
def test_evict_sizes_around_the_kernels_steps(n, m):
    run_evict(64, 16, 1, 1, [n, n - 1], [m, m], seed=n)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_evict_of_many_workgroups_and_long_rows(d):
    """Small workgroups where there are many of them, with rows past what they keep in
    registers and past one list; and large ones, past what those keep."""
    run_evict(d, 64, 1, 1, [40000, 17], [9000, 16], sinks=3, recent=5, seed=d)
    lens = [4500 if b == 5 else 40 + b for b in range(130)]
    run_evict(d, 16, 8, 1, lens, [3000 if b == 5 else 33 for b in range(130)], sinks=1, recent=1, seed=d)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_of_few_from_long_rows(d, ties):
    """Most positions stay, over several lists: what the first moves write lies where weights are
    looked up again for the later ones."""
    make = (lambda r, s: r.integers(0, 40, s)) if ties else None
    run_evict(d, 64, 1, 1, [70000, 17], [67000, 16], sinks=3, recent=5, seed=d, make=make)
    lens = [9000 if b == 5 else 40 + b % 20 for b in range(130)]
    run_evict(d, 16, 8, 1, lens, [8500 if b == 5 else 33 for b in range(130)], seed=d, make=make)


@pytest.mark.parametrize("name,make", [
    ("all equal", lambda r, s: np.ones(s)),
    ("zeros and minus zeros", lambda r, s: np.where(r.random(s) < 0.5, 0.0, -0.0)),
    ("few values", lambda r, s: r.integers(0, 3, s)),
    ("negative and infinite", lambda r, s: r.choice([-np.inf, -2.0, -1e-40, 0.0, 1e-45, 3.0, np.inf], s)),
    ("some NaN", lambda r, s: np.where(r.random(s) < 0.3, np.nan, r.random(s))),
    ("all NaN", lambda r, s: np.full(s, np.nan)),
    ("one bit apart", lambda r, s: 1 + r.integers(0, 9, s) * 2.0 ** -23),
    ("falling", lambda r, s: np.broadcast_to(-np.arange(s[-1]), s)),
    ("rising", lambda r, s: np.broadcast_to(np.arange(s[-1]), s))])
def test_evict_ties_and_odd_weights(name, make):
    run_evict(64, 16, 2, 1, [1500, 90, 300], [700, 45, 13], 2, 3, make=make)


def test_evict_statuses_and_what_is_left():
    """Budgets below the protected ends, lengths past the weights or the table, missing and
    shared pages: those requests stay as they are, the others are cut."""
    lens, budgets = [80, 80, 80, 80, 80, 80], [40, 9, 40, 40, 40, 40]
    cache, pages, table, refs = make_cache(lens, 16, 1, 64, 2, ld=6)
    w = np.random.default_rng(3).random((2, 6, 1, 90)).astype(np.float32)
    weights = torch.from_numpy(w.copy()).to(DEV)
    table[2, 4] = 777                                     # outside the pool, in a page that would go
    refs[table[3, 1]] = 2                                 # shared, and written to
    refs[table[4, 4]] = 2                                 # shared, but only read from and given up
    cache.page_table.copy_(torch.from_numpy(table))
    cache.ref_counts.copy_(torch.from_numpy(refs))
    lens[5] = 97                                          # past its table row of 96 positions
    cache.seq_lens.copy_(torch.tensor(lens))
    st = binding.kv_evict(cache, weights, T._i(budgets), sinks=4, recent=6)
    assert st.cpu().tolist() == [0, 5, 8, 8, 0, 5]
    check_evict(cache, pages, table, refs, weights, w, lens, budgets, 4, 6, 16, 64, skip=(1, 2, 3, 5))
    # lengths past the weights, negative ones, budgets that do nothing
    cache.seq_lens.copy_(torch.tensor([91, -1, 10, 40, 40, 40]))
    keep = cache.pages.clone()
    st = binding.kv_evict(cache, weights, T._i([40, 40, 10, 0, -3, 41]))
    assert st.cpu().tolist() == [5, 5, 0, 0, 0, 0] and torch.equal(cache.pages, keep)
    # a batch of fewer requests than the cache has
    st = binding.kv_evict(cache, weights[:, :1].contiguous(), T._i([5]))
    assert st.cpu().tolist() == [5]


def test_evict_of_forked_sequences():
    """A fork holds its source's pages: it stays as it is until the pages are its own."""
    cache = binding.KVCache.create(layers=1, num_pages=20, page_size=16, kv_heads=1, head_dim=64, requests=2,
                                   max_context=160, device=DEV)
    cache.pages.random_(0, 256)
    binding.kv_reserve(cache, T._i([0, 100, 100]))
    binding.kv_fork(cache, T._i([0]), T._i([1]))
    before, table = cache.pages.clone(), cache.page_table.clone()
    w = torch.rand(1, 2, 1, 160, device=DEV)
    assert binding.kv_evict(cache, w, T._i([50, 50])).cpu().tolist() == [8, 8]
    assert torch.equal(cache.pages, before) and torch.equal(cache.page_table, table)
    assert cache.seq_lens.cpu().tolist() == [100, 100]
    binding.kv_release(cache, T._i([100, 0]))
    assert binding.kv_evict(cache, w, T._i([50, 50])).cpu().tolist() == [0, 0]
    assert cache.seq_lens.cpu().tolist() == [0, 50] and int(cache.ref_counts.sum()) == 4


def test_evict_with_layers_further_apart_than_their_pages():
    cache, pages, table, refs = make_cache([60, 40], 16, 2, 64, 3)
    num, size = cache.num_pages, cache.page_bytes
    wide = torch.zeros(3, num + 2, size, dtype=torch.uint8, device=DEV)
    wide[:, :num] = cache.pages
    view = binding.KVCache(pages=wide[:, :num], page_table=cache.page_table, seq_lens=cache.seq_lens,
                           ref_counts=cache.ref_counts, page_size=16, kv_heads=2, head_dim=64)
    w = np.random.default_rng(4).random((3, 2, 2, 64)).astype(np.float32)
    weights = torch.from_numpy(w.copy()).to(DEV)
    assert binding.kv_evict(view, weights, T._i([20, 30]), sinks=2).cpu().tolist() == [0, 0]
    check_evict(view, pages, table, refs, weights, w, [60, 40], [20, 30], 2, 0, 16, 64)
    assert not bool(wide[:, num:].any())


# ---------------------------------------------------------- appends at offsets

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (128, 64, True), (256, 256, False)])
def test_append_at_offsets_turns_by_the_position(dtype, d, rot, interleaved):
    """Rows at a slot with an offset have the bytes of rows whose slot is the position; with
    offsets of 0 and without any, kv_append's own."""
    heads, kv, page = 4, 2, 16
    x = torch.randn(9, heads + 2 * kv, d, device=DEV).to(T.DTYPES[dtype])
    cs = torch.from_numpy(T._rotation(300, rot)).to(DEV)
    w = torch.rand(d, device=DEV)

    def go(ctx, offsets):
        cache = binding.KVCache.create(layers=1, num_pages=40, page_size=page, kv_heads=kv, head_dim=d,
                                       requests=3, max_context=208, device=DEV)
        cache.page_table.copy_(torch.arange(39, device=DEV).view(3, 13))
        got = binding.kv_append(cache, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:],
                                T._i([0, 4, 5, 9]), T._i(ctx), cos_sin=cs, interleaved=interleaved,
                                q_weight=w, k_weight=w, want_values=True,
                                position_offsets=None if offsets is None else T._i(offsets))
        assert got[1].cpu().tolist() == [0] * 3
        return cache, got
    _, want = go([120, 7, 200], None)
    _, got = go([20, 7, 1], [100, 0, 199])
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    c0, zero = go([120, 7, 200], [0, 0, 0])
    c1, _ = go([120, 7, 200], None)
    assert torch.equal(c0.pages, c1.pages) and all(torch.equal(a, b) for a, b in zip(want, zero))
    # stored where the slot says
    c2, _ = go([20, 7, 1], [100, 0, 199])
    unit = c2.pages.view(40, kv, -1)
    ref = c1.pages.view(40, kv, -1)
    ka, va, ks, vs = U.places(page, d)
    for b, slot, pos in ((0, 20, 120), (1, 7, 7), (2, 1, 200)):
        p, r = 13 * b + slot // page, 13 * b + pos // page
        for at in (ka, va, ks, vs):
            assert torch.equal(unit[p][:, torch.from_numpy(at[slot % page])],
                               ref[r][:, torch.from_numpy(at[pos % page])])


def test_append_at_offsets_statuses():
    cache = binding.KVCache.create(layers=1, num_pages=40, page_size=16, kv_heads=1, head_dim=64, requests=3,
                                   max_context=64, device=DEV)
    cache.page_table.copy_(torch.arange(12, device=DEV).view(3, 4))
    x = torch.randn(6, 3, 64, device=DEV)
    out = torch.full((6, 1, 64), 7.0, device=DEV)
    cs = torch.from_numpy(T._rotation(100, 64)).to(DEV)
    # request 0: its second row is past the table of angles; 1: a negative offset; 2: the last angles
    _, st = binding.kv_append(cache, x[:, :1], x[:, 1:2], x[:, 2:], T._i([0, 2, 4, 6]), T._i([9, 9, 9]),
                              cos_sin=cs, position_offsets=T._i([90, -1, 89]), out=out)
    assert st.cpu().tolist() == [5, 5, 0]
    assert (out == 7.0).all((1, 2)).cpu().tolist() == [False, True, True, True, False, False]


def _rows(count, heads, kv, d, seed):
    return torch.randn(count, heads + 2 * kv, d, generator=torch.Generator().manual_seed(seed)).to(DEV)


def test_a_fork_and_a_reused_slot_after_an_eviction():
    """An evicted request is forked, and its row, then reused: with `evicted` and weights copied
    to the fork, and `evicted` back at 0 in the reused slot, new rows are turned by their own
    positions and attend to what was kept; the reused slot's bytes are those of a new cache."""
    heads, kv, d, page, n, budget, width = 4, 2, 64, 16, 90, 32, 160
    cs = torch.from_numpy(T._rotation(300, d)).to(DEV)

    def create():
        return binding.KVCache.create(layers=1, num_pages=40, page_size=page, kv_heads=kv, head_dim=d,
                                      requests=3, max_context=width, device=DEV)

    def append(cache, x, cu, ctx, **kw):
        q, st, k, v = binding.kv_append(cache, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], T._i(cu),
                                        ctx, cos_sin=cs, want_values=True, **kw)
        return q, k, v, st.cpu().tolist()
    cache, plain = create(), create()
    prompt, more, new = (_rows(c, heads, kv, d, s) for c, s in ((n, 1), (4, 2), (21, 3)))
    evicted = torch.zeros(3, dtype=torch.int32, device=DEV)
    weights = torch.zeros(1, 3, kv, width, device=DEV)
    ctx, _ = binding.kv_reserve(cache, T._i([0, n, n, n]))
    _, k0, v0, _ = append(cache, prompt, [0, n], ctx)
    w = torch.rand(kv, n, generator=torch.Generator().manual_seed(4)).to(DEV)
    weights[0, 0, :, :n] = w
    assert binding.kv_evict(cache, weights, T._i([budget, 0, 0]), sinks=2, recent=4,
                            evicted=evicted).cpu().tolist() == [0] * 3
    assert evicted.cpu().tolist() == [n - budget, 0, 0]
    # the fork: pages by kv_fork, the rest by the caller
    assert binding.kv_fork(cache, T._i([0]), T._i([2])).cpu().tolist() == [0]
    evicted[2], weights[:, 2] = evicted[0], weights[:, 0]
    # the row that was forked takes a new sequence
    assert binding.kv_release(cache, T._i([budget, 0, 0])).cpu().tolist() == [0] * 3
    evicted[0] = 0
    cu = [0, 21, 21, 25]
    ctx, st = binding.kv_reserve(cache, T._i(cu))
    assert ctx.cpu().tolist() == [0, -1, budget] and st.cpu().tolist() == [0, 3, 0]
    q, k1, v1, st = append(cache, torch.cat((new, more)), cu, ctx, position_offsets=evicted)
    assert st == [0, 3, 0]
    # as rows of positions 0 .. 20 and 90 .. 93 in a cache that nothing left
    plain.page_table.copy_(torch.arange(30, device=DEV).view(3, 10))
    pq, pk, pv, st = append(plain, torch.cat((new, more)), cu, T._i([0, 0, n]))
    assert st == [0, 3, 0]
    assert torch.equal(q, pq) and torch.equal(k1, pk) and torch.equal(v1, pv)
    kept = [E.kept(w[h].cpu().numpy(), n, budget, 2, 4) for h in range(kv)]
    out, st = binding.kv_attention(cache, q, T._i(cu), ctx, max_k=20, max_context=width)
    assert st.cpu().tolist() == [0, 3, 0]
    K = [T._f64(k1[:21]), None] + [np.stack([np.concatenate((T._f64(k0[kept[h], h]), T._f64(k1[21:, h])))
                                             for h in range(kv)], 1)]
    V = [T._f64(v1[:21]), None] + [np.stack([np.concatenate((T._f64(v0[kept[h], h]), T._f64(v1[21:, h])))
                                             for h in range(kv)], 1)]
    T.check_attention(out, q, K, V, cu, [0, 0, budget], [21, 0, 4], "f32", d ** -0.5, skip=(1,))
    # and the fork is cut by its own weights, now that its pages are its own
    binding.kv_attention_weights(cache, q, T._i(cu), ctx, max_k=20, max_context=width, weights=weights[0])
    before = weights[0, 2].cpu().numpy()
    assert binding.kv_evict(cache, weights, T._i([0, 0, 20]), recent=4,
                            evicted=evicted).cpu().tolist() == [0] * 3
    assert evicted.cpu().tolist() == [0, 0, n - 20 + 4]
    for h in range(kv):
        now = E.kept(before[h], budget + 4, 20, 0, 4)
        assert np.array_equal(weights[0, 2, h, :20].cpu().numpy(), before[h][now])


# ------------------------------------------------- streams, graphs, the binding

def _small(seed=0, ctx=(100, 1300)):
    rows = [5, 3]
    cache, K, _ = T.make_attention(128, 16, 2, rows, list(ctx), seed)
    q = torch.randn(8, 8, 128, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)
    return cache, q, T._i([0, 5, 8]), T._i(list(ctx)), dict(max_k=4, max_context=max(ctx) + 5)


@pytest.mark.parametrize("ctx", [(100, 1300), (100, 200)])
def test_weights_on_another_stream_and_of_two_threads(ctx):
    import threading
    cache, q, cu, ctx_t, kw = _small(ctx=ctx)
    want, _ = binding.kv_attention_weights(cache, q, cu, ctx_t, **kw)
    torch.cuda.synchronize()
    outs = []

    def work():
        for _ in range(10):
            outs.append(binding.kv_attention_weights(cache, q, cu, ctx_t, **kw)[0])

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        there = [binding.kv_attention_weights(cache, q, cu, ctx_t, **kw)[0] for _ in range(3)]
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(outs) == 30 and all(torch.equal(o, want) for o in outs + there)


def test_weights_in_two_captured_graphs_replayed_together():
    a, b = _small(1), _small(2)
    want = [binding.kv_attention_weights(x[0], x[1], x[2], x[3], **x[4])[0] for x in (a, b)]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    graphs = []
    for x, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.kv_attention_weights(x[0], x[1], x[2], x[3], out=o, **x[4])
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
        binding.kv_attention_weights(a[0], a[1], a[2], a[3], **a[4])      # eager work in between
        torch.cuda.synchronize()


def test_an_eviction_captured_in_a_graph():
    cache, pages, table, refs = make_cache([300, 90], 16, 2, 64, 2)
    w = np.random.default_rng(5).random((2, 2, 2, 300)).astype(np.float32)
    w0 = torch.from_numpy(w).to(DEV)
    weights, budgets = w0.clone(), T._i([100, 40])
    evicted = torch.zeros(2, dtype=torch.int32, device=DEV)
    start = [t.clone() for t in (cache.pages, cache.page_table, cache.seq_lens, cache.ref_counts)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st = binding.kv_evict(cache, weights, budgets, sinks=4, recent=4, evicted=evicted)
    for _ in range(3):
        for t, s in zip((cache.pages, cache.page_table, cache.seq_lens, cache.ref_counts), start):
            t.copy_(s)
        weights.copy_(w0)
        evicted.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert st.cpu().tolist() == [0, 0] and evicted.cpu().tolist() == [200, 50]
        check_evict(cache, pages, table, refs, weights, w, [300, 90], [100, 40], 4, 4, 16, 64)


def test_the_binding_refuses_arguments_that_do_not_fit():
    cache, q, cu, ctx, kw = _small()
    w = torch.zeros(2, 2, 1400, device=DEV)

    def call(**over):
        a = {**dict(q=q, cu=cu, ctx=ctx), **kw, **over}
        return binding.kv_attention_weights(cache, a.pop("q"), a.pop("cu"), a.pop("ctx"), **a)
    for over in (dict(q=q.half()), dict(q=q[:, :3]), dict(q=q.cpu()), dict(weights=w[:, :1]),
                 dict(weights=w[..., :1000].contiguous()), dict(weights=w.double()), dict(weights=w.cpu()),
                 dict(out=w[:, :, ::2]), dict(weights=w, out=torch.zeros(2, 2, 1500, device=DEV)),
                 dict(max_k=64), dict(max_context=0), dict(window=-1), dict(sinks=-1), dict(layer=1),
                 dict(scale=0.0), dict(row_counts=T._i([1])), dict(row_counts=torch.ones(2, device=DEV)),
                 dict(cu=cu.long()), dict(ctx=ctx[:1]),
                 dict(workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            call(**over)
    call(weights=w)
    ok = torch.zeros(1, 2, 2, 1400, device=DEV)
    for args, kws in (((ok[0], T._i([1, 1])), {}), ((ok, T._i([1])), {}), ((ok.double(), T._i([1, 1])), {}),
                      ((ok[..., ::2], T._i([1, 1])), {}), ((ok, T._i([1, 1]).long()), {}),
                      ((ok, T._i([1, 1])), dict(sinks=-1)), ((ok, T._i([1, 1])), dict(recent=1 << 31)),
                      ((ok, T._i([1, 1])), dict(evicted=T._i([0]))), ((ok.cpu(), T._i([1, 1])), {})):
        with pytest.raises(ValueError):
            binding.kv_evict(cache, *args, **kws)


@pytest.mark.parametrize("shape", [(1400,), (2, 1400), (2, 2, 1400, 1)])
def test_the_binding_refuses_results_of_another_rank(shape):
    cache, q, cu, ctx, kw = _small()
    w = torch.zeros(2, 2, 1400, device=DEV)
    odd = torch.zeros(shape, device=DEV)
    for over in (dict(weights=w, out=odd), dict(out=odd), dict(weights=odd), dict(weights=odd, out=w)):
        with pytest.raises(ValueError):
            binding.kv_attention_weights(cache, q, cu, ctx, **over, **kw)


# ------------------------------------------------------------ the calls together

@pytest.mark.parametrize("captured", [False, True])
def test_prompts_evictions_and_verify_steps(captured):
    """Prompts come in (append, prompt attention, weights of their last rows), are cut to a
    budget, and are decoded in verify steps that append at offsets, attend, verify, drain,
    count the committed rows' weights, and cut again.  A model of the cache in float64 follows:
    which positions each head kept, their K and V, and the weights."""
    layers, heads, kv, d, page, batch, vocab = 2, 4, 2, 64, 16, 3, 64
    group, budget, sinks, recent, width = heads // kv, 60, 4, 10, 256
    gen = torch.Generator().manual_seed(3)
    cache = binding.KVCache.create(layers=layers, num_pages=60, page_size=page, kv_heads=kv, head_dim=d,
                                   requests=batch, max_context=width, device=DEV)
    cs = torch.from_numpy(T._rotation(400, d)).to(DEV)
    evicted = torch.zeros(batch, dtype=torch.int32, device=DEV)
    weights = torch.zeros(layers, batch, kv, width, device=DEV)
    budgets = T._i([budget] * batch)
    held = [[[(np.zeros((0, d)), np.zeros((0, d))) for _ in range(kv)] for _ in range(batch)]
            for _ in range(layers)]

    def rows_of(count):
        return torch.randn(layers, count, heads + 2 * kv, d, generator=gen).to(DEV)

    def attend(x, cu_t, ctx, prompt, max_k):
        """Every layer's append and attention: (queries, values, outputs)."""
        got = []
        for layer in range(layers):
            q, st, k, v = binding.kv_append(cache, x[layer][:, :heads], x[layer][:, heads:heads + kv],
                                            x[layer][:, heads + kv:], cu_t, ctx, layer=layer, cos_sin=cs,
                                            want_values=True, position_offsets=evicted)
            if prompt:
                out, st2 = binding.kv_prompt_attention(cache, q, cu_t, ctx, layer=layer, max_context=width,
                                                       total_context=3 * width)
            else:
                out, st2 = binding.kv_attention(cache, q, cu_t, ctx, layer=layer, max_k=max_k,
                                                max_context=width)
            got.append((q, k, v, out, st, st2))
        return got

    def follow(got, cu):
        """The model takes the rows, and the outputs are checked against it."""
        for layer, (q, k, v, out, st, st2) in enumerate(got):
            assert st.cpu().tolist() == st2.cpu().tolist() == [0] * batch
            K, V, ctx, rows = [], [], [], []
            for b in range(batch):
                s = slice(cu[b], cu[b + 1])
                ctx.append(held[layer][b][0][0].shape[0])
                rows.append(cu[b + 1] - cu[b])
                for h in range(kv):
                    old = held[layer][b][h]
                    held[layer][b][h] = (np.concatenate((old[0], T._f64(k[s, h]))),
                                         np.concatenate((old[1], T._f64(v[s, h]))))
                K.append(np.stack([held[layer][b][h][0] for h in range(kv)], 1))
                V.append(np.stack([held[layer][b][h][1] for h in range(kv)], 1))
            T.check_attention(out, q, K, V, cu, ctx, rows, "f32", d ** -0.5)

    def cut():
        """Evicts; the model keeps what the weights say."""
        before = weights.cpu().numpy()
        lens = cache.seq_lens.cpu().tolist()
        gone = evicted.cpu().tolist()
        st = binding.kv_evict(cache, weights, budgets, sinks=sinks, recent=recent, evicted=evicted)
        assert st.cpu().tolist() == [0] * batch
        for b, n in enumerate(lens):
            assert n == held[0][b][0][0].shape[0]
            if n <= budget:
                continue
            for layer in range(layers):
                for h in range(kv):
                    keep = E.kept(before[layer, b, h], n, budget, sinks, recent)
                    held[layer][b][h] = tuple(x[keep] for x in held[layer][b][h])
        assert cache.seq_lens.cpu().tolist() == [min(n, budget) for n in lens]
        assert evicted.cpu().tolist() == [g + max(0, n - budget) for g, n in zip(gone, lens)]
        used = sum(-(-min(n, budget) // page) for n in lens)
        assert int((cache.ref_counts > 0).sum()) == used

    # the prompts
    prompts = [150, 40, 97]
    cu = T._cu(prompts).tolist()
    ctx, st = binding.kv_reserve(cache, T._i(cu))
    assert st.cpu().tolist() == [0] * batch
    got = attend(rows_of(cu[-1]), T._i(cu), ctx, True, 0)
    follow(got, cu)
    last = [min(16, p) for p in prompts]
    tail = T._cu(last).tolist()
    for layer in range(layers):
        q = torch.cat([got[layer][0][cu[b + 1] - last[b]:cu[b + 1]] for b in range(batch)])
        binding.kv_attention_weights(cache, q, T._i(tail), T._i([p - n for p, n in zip(prompts, last)]),
                                     max_k=15, max_context=width, layer=layer, out=weights[layer])
        for b in range(batch):
            k = np.stack([held[layer][b][h][0] for h in range(kv)], 1)
            w, tol = E.weights(T._f64(q[tail[b]:tail[b + 1]]), k, prompts[b] - last[b], last[b],
                               d ** -0.5, 0, 0)
            assert np.all(np.abs(T._f64(weights[layer, b, :, :prompts[b]]) - w) <= tol)
    cut()

    # verify steps, eager or replayed from one graph
    drafts = 3
    cu = T._cu([drafts + 1] * batch).tolist()
    cu_t = T._i(cu)
    x = rows_of(cu[-1]).clone()
    logits = torch.zeros(cu[-1], vocab, device=DEV)
    ids = torch.zeros(drafts * batch, dtype=torch.int32, device=DEV)

    def step():
        ctx, st = binding.kv_reserve(cache, cu_t)
        got = attend(x, cu_t, ctx, False, drafts)
        acc, tok, vst = binding.verify_greedy(logits, cu_t, ids, max_k=drafts)
        _, _, rollback = binding.drain(cu_t, acc, vst, tok)
        for layer in range(layers):
            binding.kv_attention_weights(cache, got[layer][0], cu_t, ctx, max_k=drafts, max_context=width,
                                         layer=layer, weights=weights[layer], row_counts=acc + 1)
        binding.kv_release(cache, rollback, ctx)
        return ctx, got, acc

    state = (cache.pages, cache.page_table, cache.seq_lens, cache.ref_counts, weights, evicted)
    graph = None
    if captured:
        kept = [t.clone() for t in state]
        step()                                            # (everything is loaded before the capture)
        torch.cuda.synchronize()
        for t, s in zip(state, kept):
            t.copy_(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            result = step()
        for t, s in zip(state, kept):
            t.copy_(s)
        torch.cuda.synchronize()
    for turn in range(6):
        x.copy_(rows_of(cu[-1]))
        # request b accepts (turn + b) % 4 drafts
        best = torch.randint(0, vocab, (cu[-1],), generator=gen)
        logits.copy_(torch.nn.functional.one_hot(best, vocab).float())
        flat = []
        for b in range(batch):
            for i in range(drafts):
                right = int(best[cu[b] + i])
                flat.append(right if i < (turn + b) % 4 else (right + 1) % vocab)
        ids.copy_(torch.tensor(flat))
        before = weights.cpu().numpy().astype(np.float64)
        torch.cuda.synchronize()
        if graph is not None:
            graph.replay()
            ctx, got, acc = result
        else:
            ctx, got, acc = step()
        torch.cuda.synchronize()
        taken = [(turn + b) % 4 for b in range(batch)]
        assert acc.cpu().tolist() == taken
        follow(got, cu)
        for b in range(batch):
            n = int(ctx[b])
            for layer in range(layers):
                k = np.stack([held[layer][b][h][0] for h in range(kv)], 1)
                w, tol = E.weights(T._f64(got[layer][0][cu[b]:cu[b + 1]]), k, n, taken[b] + 1, d ** -0.5, 0, 0)
                base = before[layer, b, :, :n + drafts + 1].copy()
                base[:, n:] = 0
                assert np.all(np.abs(T._f64(weights[layer, b, :, :n + drafts + 1]) - base - w)
                              <= tol + 2.0 ** -23 * base)
                for h in range(kv):
                    held[layer][b][h] = tuple(y[:n + taken[b] + 1] for y in held[layer][b][h])
        cut()
