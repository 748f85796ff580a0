"""GPU tests of prompt attention over the 4-bit paged cache: every element against float64
with bounds derived from the arithmetic, at sizes around the kernel's tiles, blocks and
splits; what never reaches a row; statuses; streams, workspaces and captured graphs."""

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
    torch.manual_seed(13)


def queries(rows, heads, d, dtype, seed, pad=5):
    """[rows, heads, d], rows `pad` elements further apart than their length."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(rows, heads * d + pad, generator=g).to(T.DTYPES[dtype]).to(DEV)
    return q[:, :heads * d].unflatten(1, (heads, d))


def check_rows(out, q, K, V, ctx, row0, picks, dtype, scale, window=0, sinks=0):
    """Chosen (row, head) pairs of one request against float64: check_attention's bounds."""
    heads = q.shape[1]
    for j, h in picks:
        got, x = T._f64(out[row0 + j, h]), T._f64(q[row0 + j, h])
        kv = h // (heads // K.shape[1])
        want, mass, slip = U.attention_row(x, K[:, kv], V[:, kv], ctx + j, scale, window, sinks)
        n, d = K.shape[0], x.shape[0]
        tol = mass * ((T.HALF["bf16"] if dtype == "bf16" else 0) + 4 * (d + 8) * 2.0 ** -24 * slip
                      + (2 * n + 128) * 2.0 ** -24 + 2.0 ** -20) + T.HALF[dtype] * np.abs(want)
        assert np.all(np.abs(got - want) <= tol + 2.0 ** -126 * np.abs(V[:, kv]).sum(0)), (j, h)


def run_prompt(dtype, d, page, heads, kv, rows, ctx, *, window=0, sinks=0, seed=0, loud=False,
               scale=None, max_context=None, total=None):
    cache, K, V = T.make_attention(d, page, kv, rows, ctx, seed, loud=loud)
    cu = T._cu(rows)
    q = queries(int(cu[-1]), heads, d, dtype, seed)
    n = [c + r for c, r in zip(ctx, rows)]
    kw = dict(max_context=max(n) if max_context is None else max_context,
              total_context=sum(n) if total is None else total, window=window, sinks=sinks, scale=scale)
    out, st = binding.kv_prompt_attention(cache, q, T._i(cu), T._i(ctx), **kw)
    again, _ = binding.kv_prompt_attention(cache, q, T._i(cu), T._i(ctx), **kw)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0] * len(rows)
    assert torch.equal(out, again)
    T.check_attention(out, q, K, V, cu, ctx, rows, dtype, d ** -0.5 if scale is None else scale,
                      window, sinks)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (256, 16), (128, 32), (64, 128), (256, 256)])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 1), (6, 2)])
def test_short_contexts(dtype, d, page, heads, kv):
    """Rows and contexts around the page half of 16 and the tile of 32."""
    run_prompt(dtype, d, page, heads, kv, [1, 1, 4, 33, 3, 1, 7, 5], [0, 15, 0, 16, 30, 31, 32, 260])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_around_waves_and_blocks(dtype, d):
    """Query rows (rows times heads per KV head) around 32, 128 and 256."""
    for heads, rows in ((1, 31), (1, 33), (1, 127), (1, 129), (3, 43), (5, 51), (8, 33), (2, 65)):
        run_prompt(dtype, d, 32, heads, 1, [rows, 1], [70, 3], seed=rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (16, 0), (31, 4), (33, 40), (64, 32),
                                          (100, 500), (5000, 4)])
def test_window_and_sinks(dtype, window, sinks):
    run_prompt(dtype, 128, 16, 4, 2, [1, 70, 3, 8], [0, 40, 127, 333], window=window, sinks=sinks)
    run_prompt(dtype, 64, 64, 2, 2, [150, 1], [0, 64], window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_contexts_split_and_joined(dtype, d):
    run_prompt(dtype, d, 16, 2, 1, [20, 1, 2], [3001, 700, 5], seed=2)
    run_prompt(dtype, d, 128, 2, 1, [3, 40], [2500, 10], seed=3, max_context=9000, total=20000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1000, 0), (1500, 40), (700, 900), (2990, 4)])
def test_split_contexts_through_windows(dtype, d, window, sinks):
    """Windows of more than a chunk of 16 tiles: parts of a row's context that it does not see, or
    sees only the first positions of, are joined."""
    run_prompt(dtype, d, 16, 2, 1, [20, 1, 2], [3001, 700, 5], seed=2, window=window, sinks=sinks)
    run_prompt(dtype, d, 128, 3, 1, [90], [2222], seed=3, max_context=9000, total=20000, window=window,
               sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 2)])
def test_nan_blocks_in_split_contexts(dtype, d, window, sinks):
    """NaN blocks of V in several chunks of a context, seen by all rows, some and none; then of K."""
    rows, ctx, page = [40], [2000], 16
    cache, K, V = T.make_attention(d, page, 1, rows, ctx, 4)
    host = cache.pages.cpu().numpy().reshape(1, -1, 1, page * (d + d // 16))
    table = cache.page_table.cpu().numpy()
    _, _, ks, vs = U.places(page, d)
    blocks = d // 32
    q = torch.randn(40, 2, d, device=DEV).to(T.DTYPES[dtype])
    args = dict(max_context=2040, total_context=2040, window=window, sinks=sinks)

    def check():
        cache.pages.copy_(torch.from_numpy(host.reshape(1, -1, host.shape[-1])))
        out, st = binding.kv_prompt_attention(cache, q, T._i([0, 40]), T._i(ctx), **args)
        assert st.cpu().tolist() == [0]
        T.check_attention(out, q, K, V, [0, 40], ctx, rows, dtype, d ** -0.5, window, sinks)
        nan = np.isnan(T._f64(out))
        assert nan.any() and not nan.all()
    for t, blk in ((1020, 0), (1500, blocks - 1), (2030, 2 % blocks)) if window else ((2030, blocks - 1),):
        host[0, table[0, t // page], 0, vs[t % page, blk]] = 255
        V[0][t, 0, 32 * blk:32 * blk + 32] = np.nan
    check()
    for t in (1010, 2035) if window else (2035,):          # rows up to 9, rows from 35 on
        host[0, table[0, t // page], 0, ks[t % page, blocks - 1]] = 255
        K[0][t, 0] = np.nan
    check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_peaked_scores(dtype):
    """Large scores: the running maximum moves, most weights underflow."""
    run_prompt(dtype, 128, 16, 4, 2, [50, 3], [300, 0], loud=True, scale=1.0)
    run_prompt(dtype, 64, 16, 2, 1, [200], [0], loud=True, scale=2.0)


@pytest.mark.parametrize("d,rows,heads,kv", [(64, 4200, 64, 1), (128, 4200, 64, 8), (256, 2100, 128, 2)])
def test_calls_of_eight_waves(d, rows, heads, kv):
    """Blocks of 256 query rows, more than 1,024 of them, ragged at the end."""
    cache, K, V = T.make_attention(d, 64, kv, [rows, 5], [33, 0], 4)
    q = queries(rows + 5, heads, d, "bf16", 4)
    out, st = binding.kv_prompt_attention(cache, q, T._i([0, rows, rows + 5]), T._i([33, 0]),
                                          max_context=rows + 33, total_context=rows + 38)
    assert st.cpu().tolist() == [0, 0] and bool(torch.isfinite(out).all())
    rng = np.random.default_rng(1)
    picks = [(0, 0), (rows - 1, heads - 1)] + [(int(rng.integers(rows)), int(rng.integers(heads)))
                                               for _ in range(150)]
    check_rows(out, q, K[0], V[0], 33, 0, picks, "bf16", d ** -0.5)
    check_rows(out, q, K[1], V[1], 0, rows, [(j, h) for j in range(5) for h in (0, heads - 1)],
               "bf16", d ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_agree_with_the_verify_rows_attention(dtype):
    """The same rows through kv_attention: each within its own bounds of float64."""
    rows, ctx = [7, 60], [500, 33]
    cache, K, V = T.make_attention(128, 16, 2, rows, ctx, 6)
    cu = T._cu(rows)
    q = queries(67, 8, 128, dtype, 6)
    a, _ = binding.kv_prompt_attention(cache, q, T._i(cu), T._i(ctx), max_context=507, total_context=600)
    b, _ = binding.kv_attention(cache, q, T._i(cu), T._i(ctx), max_k=59, max_context=507)
    for out in (a, b):
        T.check_attention(out, q, K, V, cu, ctx, rows, dtype, 128 ** -0.5)


def test_a_prompt_in_parts_gives_the_rows_of_the_whole():
    """Rows 0..299 at once, and as 100 + 200 rows with the first ones as context: each row
    within float64's bounds in both."""
    cache, K, V = T.make_attention(64, 16, 2, [300], [0], 7)
    q = queries(300, 4, 64, "bf16", 7)
    whole, _ = binding.kv_prompt_attention(cache, q, T._i([0, 300]), T._i([0]), max_context=300,
                                           total_context=300)
    first, _ = binding.kv_prompt_attention(cache, q[:100], T._i([0, 100]), T._i([0]), max_context=300,
                                           total_context=300)
    rest, _ = binding.kv_prompt_attention(cache, q[100:], T._i([0, 200]), T._i([100]), max_context=300,
                                          total_context=300)
    for out in (whole, torch.cat((first, rest))):
        T.check_attention(out, q, K, V, [0, 300], [0], [300], "bf16", 0.125)


def test_rows_do_not_depend_on_the_other_requests():
    a = run_prompt("bf16", 128, 16, 4, 2, [30, 150, 1], [100, 900, 44], seed=9, max_context=1100,
                   total=3000)
    cache, _, _ = T.make_attention(128, 16, 2, [30, 150, 1], [100, 900, 44], 9)
    q = queries(181, 4, 128, "bf16", 9)
    # request 1 alone has rows; the same sizes
    out, st = binding.kv_prompt_attention(cache, q, T._i([30, 30, 180, 180]), T._i([0, 900, 0]),
                                          max_context=1100, total_context=3000)
    assert st.cpu().tolist() == [3, 0, 3]
    assert torch.equal(out[30:180], a[30:180])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_blocks_reach_only_who_sees_them(dtype, d):
    """A V block stored as NaN: its 32 dims of the rows that see its position, nothing
    else.  A K block: the whole row.  Both at positions some rows do not see."""
    rows, ctx, page, window, sinks = [40], [70], 16, 40, 2
    cache, K, V = T.make_attention(d, page, 1, rows, ctx, 4)
    host = cache.pages.cpu().numpy().reshape(1, -1, 1, page * (d + d // 16))
    table = cache.page_table.cpu().numpy()
    _, _, ks, vs = U.places(page, d)
    blocks = d // 32
    for t, blk in ((1, 0), (33, blocks - 1), (73, 0), (50, 2 % blocks), (10, 0), (105, 1 % blocks)):
        host[0, table[0, t // page], 0, vs[t % page, blk]] = 255
        V[0][t, 0, 32 * blk:32 * blk + 32] = np.nan
    cache.pages.copy_(torch.from_numpy(host.reshape(1, -1, host.shape[-1])))
    q = torch.randn(40, 2, d, device=DEV).to(T.DTYPES[dtype])
    args = dict(max_context=110, total_context=110, window=window, sinks=sinks)
    for _ in range(2):
        out, st = binding.kv_prompt_attention(cache, q, T._i([0, 40]), T._i(ctx), **args)
        assert st.cpu().tolist() == [0]
        T.check_attention(out, q, K, V, [0, 40], ctx, rows, dtype, d ** -0.5, window, sinks)
        # keys: position 104 is seen by rows 34 on only, position 32 by rows 0 and 1
        host[0, table[0, 104 // page], 0, ks[104 % page, blocks - 1]] = 255
        host[0, table[0, 32 // page], 0, ks[32 % page, 0]] = 255
        cache.pages.copy_(torch.from_numpy(host.reshape(1, -1, host.shape[-1])))
        K[0][104, 0] = np.nan
        K[0][32, 0] = np.nan
    assert np.isfinite(T._f64(out)).any() and np.isnan(T._f64(out)).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_with_infinite_or_nan_queries_stay_alone(dtype):
    cache, K, V = T.make_attention(64, 16, 1, [50], [100], 3)
    q = torch.randn(50, 2, 64, device=DEV).to(T.DTYPES[dtype])
    clean, _ = binding.kv_prompt_attention(cache, q, T._i([0, 50]), T._i([100]), max_context=150,
                                           total_context=150)
    q[3, 1, 7] = float("nan")
    q[20, 0, 9] = float("inf")
    out, st = binding.kv_prompt_attention(cache, q, T._i([0, 50]), T._i([100]), max_context=150,
                                          total_context=150)
    assert st.cpu().tolist() == [0]
    assert torch.isnan(out[3, 1]).all() and torch.isnan(out[20, 0]).all()
    # (the moments at which a wave raises its maxima are its rows' together: to rounding)
    keep = torch.ones(50, 2, dtype=torch.bool, device=DEV)
    keep[3, 1] = keep[20, 0] = False
    assert torch.isfinite(out[keep]).all()
    K, V = [K[0]], [V[0]]
    good = T._f64(out)
    ref = T._f64(clean)
    tol = 3 * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -18) * np.abs(V[0]).max()
    assert np.abs(good - ref)[keep.cpu().numpy()].max() <= tol


@pytest.mark.parametrize("dtype,scale", [("bf16", 1e-38), ("f32", 3e-39), ("bf16", 1e-44)])
def test_the_smallest_scales_are_the_mean_of_what_is_seen(dtype, scale):
    run_prompt(dtype, 128, 16, 2, 1, [40, 3], [0, 200], scale=float(np.float32(scale)), window=50)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [10, 25, 40])
def test_scores_far_beyond_the_exponents_of_fp32(d, power):
    """Single powers of two as queries: exact scores, few weights count; from 2^30 on a row
    may be NaN, whole."""
    rows, ctx = 5, 300
    cache, K, V = T.make_attention(d, 16, 1, [rows], [ctx], power)
    x = torch.zeros(rows, 2, d)
    for j in range(rows):
        for h in range(2):
            x[j, h, (7 * j + 11 * h) % d] = (-1) ** h * 2.0 ** power
    q = x.to(DEV)
    out, st = binding.kv_prompt_attention(cache, q, T._i([0, rows]), T._i([ctx]), scale=1.0,
                                          max_context=ctx + rows, total_context=ctx + rows)
    assert st.cpu().tolist() == [0]
    o = T._f64(out)
    for j in range(rows):
        for h in range(2):
            s = (-1) ** h * K[0][:ctx + j + 1, 0, (7 * j + 11 * h) % d] * 2.0 ** power
            w = np.exp(s - s.max())
            want = w @ V[0][:ctx + j + 1, 0] / w.sum()
            if np.abs(s).max() * 1.4427 >= 2.0 ** 30 and np.isnan(o[j, h]).all():
                continue
            gap = np.minimum(s.max() - s, 200.0)
            tol = (w * (2.0 ** -20 + 2 * ctx * 2.0 ** -24 + gap * 4 * 2.0 ** -24)) @ np.abs(
                V[0][:ctx + j + 1, 0]) / w.sum() + 2.0 ** -24 * np.abs(want)
            assert np.all(np.abs(o[j, h] - want) <= tol), (j, h)


def test_statuses_and_what_is_left():
    """Bad offsets and lengths, bounds of one request and of all, missing pages; rows of no
    request."""
    rows, ctx = [3, 40, 2, 5, 6], [10, 30, 20, 50, 0]
    cache, K, V = T.make_attention(64, 16, 1, rows, ctx, 1)
    cu = [0, 3, 43, 45, 50, 56]
    q = torch.randn(60, 2, 64, device=DEV)
    out = torch.full((60, 2, 64), 7.0, device=DEV)
    kw = dict(max_context=70, total_context=300, out=out)
    table = cache.page_table.clone()
    cache.page_table[1, 2] = 999                       # position 32..47: rows of request 1 see it
    bad = [ctx[0], ctx[1], -1, 66, ctx[4]]             # request 2 negative, 3 past max_context
    _, st = binding.kv_prompt_attention(cache, q, T._i(cu), T._i(bad), **kw)
    assert st.cpu().tolist() == [0, 8, 5, 5, 0]
    assert torch.isnan(out[3:50]).all() and bool((out[56:] == 7.0).all())
    T.check_attention(out, q, K, V, cu, ctx, rows, "f32", 0.125, skip=(1, 2, 3))
    cache.page_table.copy_(table)
    # a bound of the sum that requests 0 and 1 fill: the others are past it
    out.fill_(7.0)
    _, st = binding.kv_prompt_attention(cache, q, T._i(cu), T._i(ctx), **{**kw, "total_context": 13 + 70})
    assert st.cpu().tolist() == [0, 0, 5, 5, 5]
    T.check_attention(out, q, K, V, cu, ctx, rows, "f32", 0.125, skip=(2, 3, 4))
    assert torch.isnan(out[43:56]).all()
    # a slot past the table row
    narrow = binding.KVCache(pages=cache.pages, page_table=table[:, :2].contiguous(), seq_lens=cache.seq_lens,
                             ref_counts=cache.ref_counts, page_size=16, kv_heads=1, head_dim=64)
    _, st = binding.kv_prompt_attention(narrow, q, T._i(cu), T._i(ctx), **kw)
    assert st.cpu().tolist() == [0, 8, 0, 8, 0]
    # a page that no row sees does not matter
    cache.page_table[3, 0] = -5
    _, st = binding.kv_prompt_attention(cache, q, T._i(cu), T._i(ctx), **{**kw, "window": 20})
    assert st.cpu().tolist() == [0] * 5


@pytest.mark.parametrize("cu", [[0, 3, 2, 8], [0, 3, 9, 8], [-1, 3, 5, 8], [0, 0, 0, 8]])
def test_broken_offsets_stop_there(cu):
    cache, K, V = T.make_attention(64, 16, 1, [3, 5, 8], [4, 4, 4], 2)
    q = torch.randn(8, 1, 64, device=DEV)
    out = torch.full((8, 1, 64), 7.0, device=DEV)
    _, st = binding.kv_prompt_attention(cache, q, T._i(cu), T._i([4, 4, 4]), max_context=20,
                                        total_context=40, out=out)
    first = {0: 1 if cu[1] == 3 else 0, -1: 0}[cu[0]]
    if cu == [0, 0, 0, 8]:
        assert st.cpu().tolist() == [3, 3, 0] and bool(torch.isfinite(out).all())
        return
    assert st.cpu().tolist() == [0] * first + [3] * (3 - first)
    assert bool((out[3 * first:] == 7.0).all()) and not bool((out[:3 * first] == 7.0).any())


def test_many_requests_some_without_rows():
    rng = np.random.default_rng(5)
    rows = [int(x) for x in rng.integers(1, 12, 400)]
    ctx = [int(x) for x in rng.integers(0, 40, 400)]
    cache, K, V = T.make_attention(64, 16, 1, rows, ctx, 5)
    skip = set(range(0, 400, 7))
    live = [0 if b in skip else r for b, r in enumerate(rows)]
    cu = T._cu(live)
    q = queries(int(cu[-1]), 3, 64, "bf16", 5)
    out, st = binding.kv_prompt_attention(cache, q, T._i(cu), T._i(ctx), max_context=60,
                                          total_context=400 * 60)
    assert st.cpu().tolist() == [3 if b in skip else 0 for b in range(400)]
    T.check_attention(out, q, K, V, cu, ctx, live, "bf16", 0.125, skip=skip)


def test_pages_past_32_bit_offsets():
    page, d, kv = 256, 128, 8
    unit = page * (d + d // 16) * kv
    num = (1 << 32) // unit + 40
    small, K, V = T.make_attention(d, page, kv, [300], [90], 8)
    pages = torch.zeros(1, num, unit, dtype=torch.uint8, device=DEV)
    old = small.page_table[0].cpu().tolist()
    new = [num - 1 - 3 * i for i in range(len(old))]
    for a, b in zip(old, new):
        pages[0, b] = small.pages[0, a]
    cache = T.binding.KVCache(pages=pages, page_table=T._i([new]), seq_lens=small.seq_lens,
                              ref_counts=torch.zeros(num, dtype=torch.int32, device=DEV), page_size=page,
                              kv_heads=kv, head_dim=d)
    q = queries(300, 8, d, "bf16", 8)
    out, st = binding.kv_prompt_attention(cache, q, T._i([0, 300]), T._i([90]), max_context=390,
                                          total_context=390)
    assert st.cpu().tolist() == [0]
    rng = np.random.default_rng(2)
    check_rows(out, q, K[0], V[0], 90, 0, [(int(rng.integers(300)), h) for h in range(8) for _ in range(8)],
               "bf16", d ** -0.5)


def _small(seed=0, heads=4):
    cache, K, V = T.make_attention(128, 16, 2, [40, 130], [100, 7], seed)
    q = queries(170, heads, 128, "bf16", seed)
    kw = dict(max_context=150, total_context=400)
    return cache, q, T._i([0, 40, 170]), T._i([100, 7]), kw


def test_calls_on_another_stream_and_of_two_threads():
    import threading
    cache, q, cu, ctx, kw = _small()
    want, _ = binding.kv_prompt_attention(cache, q, cu, ctx, **kw)
    torch.cuda.synchronize()
    outs = []

    def work():
        for _ in range(10):
            outs.append(binding.kv_prompt_attention(cache, q, cu, ctx, **kw)[0])

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        there = [binding.kv_prompt_attention(cache, q, cu, ctx, **kw)[0] for _ in range(3)]
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(outs) == 30 and all(torch.equal(o, want) for o in outs + there)


def test_a_workspace_of_the_callers():
    cache, q, cu, ctx, kw = _small()
    want, _ = binding.kv_prompt_attention(cache, q, cu, ctx, **kw)
    need = binding.lib().spec_kv_prompt_workspace_bytes(1, 2, 170, 4, 2, 128, 150, 400, 0, 0)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    got, _ = binding.kv_prompt_attention(cache, q, cu, ctx, workspace=ws, **kw)
    assert torch.equal(got, want)
    with pytest.raises(ValueError, match="workspace smaller"):
        binding.kv_prompt_attention(cache, q, cu, ctx, workspace=ws[:-256], **kw)
    with pytest.raises(ValueError, match="contiguous tensor"):
        binding.kv_prompt_attention(cache, q, cu, ctx, workspace=ws.cpu(), **kw)


def test_two_captured_graphs_replayed_together():
    a, b = _small(1), _small(2)
    want = [binding.kv_prompt_attention(x[0], x[1], x[2], x[3], **x[4])[0] for x in (a, b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(binding.kv_prompt_attention(x[0], x[1], x[2], x[3], **x[4])[0])
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
        binding.kv_prompt_attention(a[0], a[1], a[2], a[3], **a[4])       # eager work in between
        torch.cuda.synchronize()


def test_the_binding_refuses_arguments_that_do_not_fit():
    cache, q, cu, ctx, kw = _small()

    def call(**over):
        a = {**dict(q=q, cu_seqlens=cu, context_lens=ctx), **kw, **over}
        return binding.kv_prompt_attention(cache, a.pop("q"), a.pop("cu_seqlens"), a.pop("context_lens"), **a)
    for over in (dict(out=q), dict(q=q.half()), dict(q=q[:, :3]), dict(q=q[..., :64]), dict(q=q.cpu()),
                 dict(out=torch.empty(169, 4, 128, dtype=q.dtype, device=DEV)), dict(max_context=0),
                 dict(total_context=0), dict(total_context=(1 << 30) + 1), dict(window=-1), dict(sinks=-1),
                 dict(scale=0.0), dict(scale=float("nan")), dict(layer=1), dict(cu_seqlens=cu.long()),
                 dict(context_lens=ctx[:1]), dict(cu_seqlens=cu.cpu())):
        with pytest.raises(ValueError):
            call(**over)
    call()


@pytest.mark.parametrize("d", [64, 256])
def test_a_result_beside_its_queries(d):
    """Columns of one wider tensor share no element: the rows of a call into other memory.  A
    result that is shifted into the queries is refused, and nothing is written."""
    cache, K, V = T.make_attention(d, 16, 2, [40, 130], [100, 7], 3)
    both = torch.randn(171, 2 * 4 * d, device=DEV).to(torch.bfloat16)
    q, out = both[:170, :4 * d].unflatten(1, (4, d)), both[:170, 4 * d:].unflatten(1, (4, d))
    args = (T._i([0, 40, 170]), T._i([100, 7]))
    kw = dict(max_context=150, total_context=400)
    want, _ = binding.kv_prompt_attention(cache, q, *args, **kw)
    held = both.clone()
    for shifted in (both[:170, d:5 * d], both[1:, :4 * d], both[1:, 2 * d:6 * d], both.view(-1, 4 * d)[1:171]):
        with pytest.raises(ValueError):
            binding.kv_prompt_attention(cache, q, *args, out=shifted.unflatten(1, (4, d)), **kw)
    torch.cuda.synchronize()
    assert torch.equal(both, held)
    got, st = binding.kv_prompt_attention(cache, q, *args, out=out, **kw)
    assert st.cpu().tolist() == [0, 0] and got is out and torch.equal(out, want)
    assert torch.equal(both[:, :4 * d], held[:, :4 * d])


def test_a_prompt_of_two_million_rows():
    """2^27 query rows in one call (34 GB of queries and results), through a short window."""
    rows, heads, kv, d, page, window = 1 << 21, 64, 8, 64, 256, 70
    num = rows // page
    # pages of 64 random ones' bytes
    few, K, V = T.make_attention(d, page, kv, [64 * page], [0], 11)
    order = few.page_table[0, :64].long()
    pages = few.pages[:, order].repeat(1, num // 64, 1)
    cache = binding.KVCache(pages=pages, page_table=torch.arange(num, dtype=torch.int32, device=DEV)[None],
                            seq_lens=T._i([rows]), ref_counts=torch.ones(num, dtype=torch.int32, device=DEV),
                            page_size=page, kv_heads=kv, head_dim=d)
    q = torch.empty(rows, heads, d, dtype=torch.bfloat16, device=DEV)
    q.view(64, -1).copy_(torch.randn(rows // 64, heads * d, device=DEV).view(1, -1))
    out, st = binding.kv_prompt_attention(cache, q, T._i([0, rows]), T._i([0]), max_context=rows,
                                          total_context=rows, window=window)
    assert st.cpu().tolist() == [0]
    rng = np.random.default_rng(3)
    picks = [0, 69, 70, rows - 1, rows - 2] + [int(rng.integers(rows)) for _ in range(60)]
    for j in picks:
        h = int(rng.integers(heads))
        t = np.arange(max(0, j - window + 1), j + 1) % (64 * page)
        k, v = K[0][t, h // 8], V[0][t, h // 8]
        want, mass, slip = U.attention_row(T._f64(q[j, h]), k, v, len(t) - 1, d ** -0.5, 0, 0)
        tol = mass * (T.HALF["bf16"] + 4 * (d + 8) * 2.0 ** -24 * slip + (2 * window + 128) * 2.0 ** -24
                      + 2.0 ** -20) + T.HALF["bf16"] * np.abs(want)
        assert np.all(np.abs(T._f64(out[j, h]) - want) <= tol), (j, h)
    # nothing is left out, and rows of equal queries over equal pages are equal
    assert bool(torch.isfinite(out.view(64, -1)).all(1).all())
    block = rows // 64
    assert torch.equal(out[block + 100:block + 200], out[2 * block + 100:2 * block + 200])
