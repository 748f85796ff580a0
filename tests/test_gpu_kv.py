"""GPU tests of the 4-bit paged cache: append byte for byte, attention against
float64 with derived bounds, the page calls against Python tables, refusals on
the device, and the calls together as a serving step uses them."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv_util as U  # noqa: E402
from lossless_rejection_sampling_spec_amd import binding  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}        # half a step, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    binding.lib()
    yield


def _i(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _cache(pages, table, lens, refs, page, kv, d):
    """A KVCache of numpy state: pages [layers, num_pages, kv, unit]."""
    p = torch.from_numpy(pages.reshape(*pages.shape[:2], -1)).to(DEV)
    return binding.KVCache(pages=p, page_table=_i(table), seq_lens=_i(lens), ref_counts=_i(refs),
                           page_size=page, kv_heads=kv, head_dim=d)


def _cu(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def _f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------- append

def _rotation(n, rot):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], -1).astype(np.float32)


def run_append(dtype, d, page, heads, kv, rows, ctx, *, norm=True, rot=0, interleaved=False,
               seed=0, poke=None, shift=0, in_place=False, want_values=True):
    rng = np.random.default_rng(seed)
    batch = len(rows)
    cu = _cu(rows)
    R = int(cu[-1])
    width = max(1, max(-(-(c + r) // page) for c, r in zip(ctx, rows)))
    num = batch * width + 3
    ids = rng.permutation(num)[:batch * width].reshape(batch, width)
    unit = page * (d + d // 16)
    pages = rng.integers(0, 256, (1, num, kv, unit), dtype=np.uint8)
    # one fused projection; `shift` elements off any wide alignment
    n = (heads + 2 * kv) * d
    x = rng.standard_normal((R, n)) * np.exp(rng.uniform(-3, 3, (R, 1)))
    if poke is not None:
        poke(x.reshape(R, heads + 2 * kv, d), heads, kv)
    flat = torch.zeros(R * (n + 5) + 16, dtype=DTYPES[dtype], device=DEV)
    view = flat[shift:shift + R * (n + 5)].view(R, n + 5)[:, :n]
    view.copy_(torch.from_numpy(x))
    qkv = view.unflatten(1, (heads + 2 * kv, d))
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    xs = _f64(qkv)
    w = [(1 + 0.2 * rng.standard_normal(d)).astype(np.float32) if norm else None for _ in range(2)]
    table = _rotation(max(c + r for c, r in zip(ctx, rows)) + 2, rot) if rot else None
    cache = _cache(pages, ids, ctx, np.zeros(num), page, kv, d)
    got = binding.kv_append(
        cache, q, k, v, _i(cu), _i(ctx), eps=1e-5,
        q_weight=None if w[0] is None else torch.from_numpy(w[0]).to(DEV),
        k_weight=None if w[1] is None else torch.from_numpy(w[1]).to(DEV),
        cos_sin=None if table is None else torch.from_numpy(table).to(DEV),
        interleaved=interleaved, out=q if in_place else None, want_values=want_values)
    torch.cuda.synchronize()
    want = pages.copy()
    eps = float(np.float32(1e-5))
    for b in range(batch):
        for j in range(rows[b]):
            r, p = int(cu[b]) + j, ctx[b] + j
            yq = U.turned(xs[r, :heads], w[0], eps, table, p, interleaved)
            yk = U.turned(xs[r, heads:heads + kv], w[1], eps, table, p, interleaved)
            gq = _f64(got[0][r])
            fine = np.isfinite(yq)
            assert np.array_equal(np.isfinite(gq), fine)
            # one rounding of a float64 result (and float64's own error)
            bound = HALF[dtype] * np.abs(yq) * (1 + 1e-9) + 1e-37
            assert np.all(np.abs(gq - yq)[fine] <= bound[fine]), (b, j)
            kc, kb = U.encode(yk)
            vc, vb = U.encode(xs[r, heads + kv:])
            for h in range(kv):
                U.write_token(want[0], page, d, ids[b, p // page], h, p % page, kc[h], kb[h], vc[h],
                              vb[h])
            if want_values:
                assert np.array_equal(_f64(got[2][r]), U.decode(kc, kb), equal_nan=True)
                assert np.array_equal(_f64(got[3][r]), U.decode(vc, vb), equal_nan=True)
    have = cache.pages.cpu().numpy().reshape(want.shape)
    assert np.array_equal(have, want), np.argwhere(have != want)[:5]
    assert got[1].cpu().tolist() == [0] * batch


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 64), (256, 32), (64, 256)])
@pytest.mark.parametrize("rot,interleaved", [(0, False), ("d", False), ("d", True), (32, False),
                                             (16, True), (16, False)])
def test_append_stores_every_byte(dtype, d, page, rot, interleaved):
    run_append(dtype, d, page, 6, 2, [1, 7, 3], [0, 13, 40], rot=d if rot == "d" else rot,
               interleaved=interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 5), (3, 1)])
def test_append_head_layouts_and_no_norm(dtype, heads, kv):
    run_append(dtype, 128, 16, heads, kv, [2, 1], [15, 100], norm=False, seed=heads)
    run_append(dtype, 64, 16, heads, kv, [33], [5], rot=64, seed=heads, want_values=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 3])
def test_append_takes_any_alignment_and_writes_q_in_place(dtype, shift):
    run_append(dtype, 128, 32, 4, 2, [5, 2], [30, 0], rot=128, shift=shift)
    run_append(dtype, 256, 32, 4, 2, [5, 2], [30, 0], rot=64, shift=shift, in_place=True)


def test_append_of_a_long_ragged_prompt():
    run_append("bf16", 128, 64, 4, 1, [700, 1, 333], [0, 900, 17], rot=128, seed=5)


def test_append_of_special_values():
    def poke(x, heads, kv):
        x[0, heads + kv, :32] = 0                      # a block of zeros
        x[0, heads + kv, 32:64] = -0.0
        x[1, heads + kv, 5] = np.nan
        x[1, heads + kv, 40] = np.inf
        x[2, heads + kv, 70] = -np.inf
        x[3, heads + kv, :32] = 1e-38                  # below the smallest scale
        x[3, heads + kv, 32:64] = -1e-42
        x[3, heads + kv, 64:96] = 3.3e38               # past the largest
        x[4, heads + kv, :8] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5]
        x[4, heads + kv, 8:32] = 0
        x[4, heads + kv, 32:64] = np.linspace(-6, 6, 32)
        x[5, heads + kv] = np.arange(128) * 2.0 ** -20
        x[6, 0, 3] = np.nan                            # a query head
        x[6, heads, 3] = np.nan                        # a key head: the norm spreads it
    run_append("f32", 128, 16, 2, 1, [4, 3], [3, 50], poke=poke, norm=False)
    run_append("bf16", 128, 16, 2, 1, [4, 3], [3, 50], poke=poke, norm=False)

    def poke_norm(x, heads, kv):
        x[6, 0, 3] = np.nan
        x[6, heads, 3] = np.inf
        x[5, heads] = 0                                # a zero row under the norm
    run_append("f32", 128, 16, 2, 1, [4, 3], [3, 50], poke=poke_norm, rot=128)


def test_append_statuses_and_what_it_leaves():
    d, page, kv, heads = 128, 16, 2, 4
    rng = np.random.default_rng(7)
    pages = rng.integers(0, 256, (1, 9, kv, page * 136), dtype=np.uint8)
    table = np.array([[0, 1], [2, 9], [3, -1], [4, 5], [6, 7], [8, 8]])
    #        ok      bad page   bad page    ctx < 0  no rows   past the rotation table
    rows = [3, 20, 4, 2, 0, 3]
    ctx = [0, 2, 14, -1, 4, 18]
    cu = _cu(rows) + 1                                 # row 0 belongs to nobody
    R = int(cu[-1]) + 2                                # nor do the last two
    x = torch.randn(R, heads + 2 * kv, d, device=DEV)
    cs = torch.from_numpy(_rotation(20, 64)).to(DEV)   # positions 0 .. 19
    rot = dict(cos_sin=cs)
    ctx[1] = 0
    cache = _cache(pages, table, ctx, np.zeros(9), page, kv, d)
    out = torch.full((R, heads, d), 7.0, device=DEV)
    _, st = binding.kv_append(cache, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:],
                              _i(cu), _i(ctx), out=out, **rot)
    assert st.cpu().tolist() == [0, 8, 8, 5, 3, 5]
    o = _f64(out)
    left = [0, R - 2, R - 1] + list(range(cu[3], cu[4])) + list(range(cu[5] + 2, cu[6]))
    for r in range(R):
        assert np.all(o[r] == 7.0) == (r in left), r
    have = cache.pages.cpu().numpy().reshape(pages.shape)
    want = pages.copy()
    xs = _f64(x)
    for b, j, p in [(0, 0, 0), (0, 1, 1), (0, 2, 2)] + [(1, j, j) for j in range(16)] + \
            [(2, 0, 14), (2, 1, 15), (5, 0, 18), (5, 1, 19)]:
        r = int(cu[b]) + j
        k = U.turned(xs[r, heads:heads + kv], None, 0, _rotation(20, 64), p, False)
        kc, kb = U.encode(k)
        vc, vb = U.encode(xs[r, heads + kv:])
        for h in range(kv):
            U.write_token(want[0], page, d, table[b][p // page], h, p % page, kc[h], kb[h], vc[h],
                          vb[h])
    assert np.array_equal(have, want)


@pytest.mark.parametrize("cu", [[0, 3, 2, 8], [0, 3, 9, 8], [-1, 3, 5, 8], [5, 3, 5, 8]])
def test_append_broken_offsets_stop_there(cu):
    first = next(b for b in range(3) if cu[b] < 0 or cu[b + 1] < cu[b] or cu[b + 1] > 8)
    cache = _cache(np.zeros((1, 6, 1, 16 * 68), np.uint8), np.arange(6).reshape(3, 2), [0] * 3,
                   np.zeros(6), 16, 1, 64)
    x = torch.randn(8, 3, 64, device=DEV)
    out = torch.full((8, 1, 64), 7.0, device=DEV)
    _, st = binding.kv_append(cache, x[:, :1], x[:, 1:2], x[:, 2:], _i(cu), _i([0, 0, 0]), out=out)
    assert st.cpu().tolist() == [0] * first + [3] * (3 - first)
    written = (_f64(out) != 7.0).any((1, 2))
    want = np.zeros(8, bool)
    for b in range(first):
        want[cu[b]:cu[b + 1]] = True
    assert np.array_equal(written, want)


# ---------------------------------------------------------------- attention

def make_attention(d, page, kv, rows, ctx, seed=0, spare=2, loud=False):
    """Random K, V of every position in shuffled pages: (cache, K, V per request)."""
    rng = np.random.default_rng(seed)
    batch = len(rows)
    n = [c + r for c, r in zip(ctx, rows)]
    width = max(-(-x // page) for x in n)
    need = [-(-x // page) for x in n]
    num = sum(need) + spare
    ids = iter(rng.permutation(num))
    table = np.full((batch, width), -1)
    # what no request holds is all ones: NaN scales
    pages = np.full((1, num, kv, page * (d + d // 16)), 255, np.uint8)
    K, V = [], []
    for b in range(batch):
        kb = np.zeros((need[b] * page, kv, d))
        vb = np.zeros((need[b] * page, kv, d))
        for i in range(need[b]):
            p = table[b, i] = next(ids)
            for h in range(kv):
                k, v = rng.standard_normal((2, page, d))
                if loud:
                    k *= 4
                U.fill_unit(pages[0, p, h], page, d, k, v)
                s = slice(i * page, (i + 1) * page)
                kb[s, h], vb[s, h] = U.read_unit(pages[0, p, h], page, d)
            last = n[b] - i * page
            if last < page:                            # stale bytes behind the last position
                ka, va, ks, vs = U.places(page, d)
                for at in (ks, vs):
                    pages[0, p][:, at[last:]] = 255
        K.append(kb[:n[b]])
        V.append(vb[:n[b]])
    return _cache(pages, table, n, np.zeros(num), page, kv, d), K, V


def check_attention(out, q, K, V, cu, ctx, rows, dtype, scale, window=0, sinks=0, skip=()):
    """Every element against float64.  fp32 scores are off by at most (D + 8) 2^-24 of
    scale sum|q||k|, weights by twice that and a step of exp2, sums by a step per term;
    a bf16 row adds half a step for each weight, and the result its own rounding.
    Weights of less than 2^-126 of the largest may be 0 (fp32 ends there; the largest
    counts at least 1 in the sum they are divided by): each off by at most that."""
    o, x = _f64(out), _f64(q)
    heads, d = x.shape[1:]
    for b in range(len(rows)):
        if b in skip:
            continue
        g = heads // K[b].shape[1]
        n = K[b].shape[0]
        for j in range(rows[b]):
            for h in range(heads):
                want, mass, slip = U.attention_row(x[cu[b] + j, h], K[b][:, h // g], V[b][:, h // g],
                                                   ctx[b] + j, scale, window, sinks)
                got = o[cu[b] + j, h]
                fine = np.isfinite(want)
                assert np.array_equal(np.isfinite(got), fine), (b, j, h)
                tol = mass * ((HALF["bf16"] if dtype == "bf16" else 0) + 4 * (d + 8) * 2.0 ** -24 * slip
                              + (2 * n + 128) * 2.0 ** -24 + 2.0 ** -20) + HALF[dtype] * np.abs(want)
                tol = tol + 2.0 ** -126 * np.abs(V[b][:, h // g]).sum(0)
                bad = np.abs(got - want)[fine] > tol[fine]
                assert not bad.any(), (b, j, h, np.abs(got - want)[fine].max(), tol.min())


def run_attention(dtype, d, page, heads, kv, rows, ctx, *, window=0, sinks=0, seed=0, max_k=None,
                  max_context=None, loud=False, scale=None):
    cache, K, V = make_attention(d, page, kv, rows, ctx, seed, loud=loud)
    cu = _cu(rows)
    g = torch.Generator().manual_seed(seed)
    # rows 5 elements further apart than their length
    q = torch.randn(int(cu[-1]), heads * d + 5, generator=g).to(DTYPES[dtype]).to(DEV)
    q = q[:, :heads * d].unflatten(1, (heads, d))
    max_context = max(c + r for c, r in zip(ctx, rows)) if max_context is None else max_context
    kw = dict(max_k=max(rows) - 1 if max_k is None else max_k, max_context=max_context,
              window=window, sinks=sinks, scale=scale)
    out, st = binding.kv_attention(cache, q, _i(cu), _i(ctx), **kw)
    again, _ = binding.kv_attention(cache, q, _i(cu), _i(ctx), **kw)
    torch.cuda.synchronize()
    assert st.cpu().tolist() == [0] * len(rows)
    assert torch.equal(out, again)
    check_attention(out, q, K, V, cu, ctx, rows, dtype, d ** -0.5 if scale is None else scale,
                    window, sinks)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (256, 16), (128, 32), (64, 64), (256, 256)])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 1), (6, 2)])
def test_attention_short_contexts(dtype, d, page, heads, kv):
    """Contexts around the 16-token page half, the 32-token tile and the first split."""
    run_attention(dtype, d, page, heads, kv, [1, 1, 4, 2, 3, 1, 7, 5], [0, 15, 0, 16, 30, 31, 32, 260])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_rows_of_every_tiling(dtype, d):
    """1 to 64 rows by groups of 1 to 8: one, two, four 16-row tiles and several blocks."""
    for heads, rows in ((1, 16), (1, 17), (8, 2), (8, 3), (8, 8), (3, 11), (5, 13), (8, 64), (1, 64)):
        run_attention(dtype, d, 32, heads, 1, [rows, 1], [70, 200], seed=rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (16, 0), (31, 4), (33, 40), (64, 32),
                                          (100, 500), (5000, 4)])
def test_attention_window_and_sinks(dtype, window, sinks):
    run_attention(dtype, 128, 16, 4, 2, [1, 6, 3, 8], [0, 40, 127, 333], window=window, sinks=sinks)
    run_attention(dtype, 64, 64, 2, 2, [5, 1], [300, 64], window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_long_contexts_split_and_joined(dtype):
    run_attention(dtype, 128, 16, 4, 1, [3, 1, 2], [3001, 700, 255], seed=2)
    run_attention(dtype, 64, 128, 2, 1, [1, 1], [5000, 10], seed=3, max_context=8192)
    run_attention(dtype, 256, 32, 2, 1, [2], [1500], seed=4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_peaked_scores(dtype):
    """Large scores: the running maximum moves, most weights underflow."""
    run_attention(dtype, 128, 16, 2, 1, [4, 1], [400, 90], loud=True, scale=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,heads", [(64, 8), (128, 4), (256, 2)])
def test_attention_of_many_short_items(dtype, d, heads):
    """More items than the device holds at once, none split: the planned launch with two
    waves per workgroup, rows of 1 to 4 tiles, with and without a window."""
    rng = np.random.default_rng(d)
    rows = [int(x) for x in rng.integers(0, 6, 520)]
    rows[:3] = [6, 1, 5]
    ctx = [int(x) for x in rng.integers(0, 90, 520)]
    check_many(dtype, d, heads, 2, rows, ctx, 100, 0, 0, range(0, 520, 7))
    check_many(dtype, d, heads, 2, rows, ctx, 100, 20, 3, range(3, 520, 7))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,batch,max_context", [(16, 300, 100), (8, 300, 100), (16, 520, 100),
                                                     (8, 520, 100), (16, 60, 20000),
                                                     (8, 60, 20000)])
def test_attention_of_many_items_with_rows_of_every_tiling(dtype, d, heads, batch, max_context):
    """Up to 32 and 64 rows per KV head where items are many: with and without a plan,
    two and four waves per workgroup, whole and split."""
    rng = np.random.default_rng(batch + heads)
    rows = [int(x) for x in rng.integers(1, 9, batch)]
    rows[:4] = [8, 1, 7, 3]
    ctx = [int(x) for x in rng.integers(0, 90, batch)]
    if max_context > 100:
        ctx[1], ctx[7], ctx[39] = 2047, 4100, 2500
    check_many(dtype, d, heads, 2, rows, ctx, max_context, 0, 0,
               range(0, 8) if max_context > 100 else range(0, batch, 29))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [4, 16, 32])
def test_attention_of_a_full_batch_in_fp32(d, heads):
    """1,024 requests over 4 KV heads: as many items as a call of fp32 rows takes two
    waves per workgroup for; 8, 32 and 64 rows each."""
    rng = np.random.default_rng(heads)
    rows = [int(x) for x in rng.integers(0, 9, 1024)]
    ctx = [int(x) for x in rng.integers(0, 60, 1024)]
    rows[1], rows[37] = 8, 0
    check_many("f32", d, heads, 4, rows, ctx, 68, 0, 0, range(0, 1024, 111))


def check_many(dtype, d, heads, kv, rows, ctx, max_context, window, sinks, some):
    """Pages of random codes; the requests `some` are compared."""
    page, rng, some = 16, np.random.default_rng(1), set(some)
    n = [c + max(r, 1) for c, r in zip(ctx, rows)]
    need = [-(-x // page) for x in n]
    pages = rng.integers(0, 256, (1, sum(need) + 2, kv, page * (d + d // 16)), np.uint8)
    pages[..., page * d:] = rng.integers(122, 128, pages[..., page * d:].shape, np.uint8)
    ids, table = rng.permutation(sum(need)), np.full((len(rows), max(need)), -1)
    ks, vs = U.places(page, d)[2:]
    K, V = [None] * len(rows), [None] * len(rows)
    for b, first in enumerate(np.cumsum([0] + need[:-1])):
        mine = table[b, :need[b]] = ids[first:first + need[b]]
        for at in (ks, vs):                      # stale bytes behind the last position
            pages[0, mine[-1]][:, at[n[b] - (need[b] - 1) * page:]] = 255
        if b in some:
            units = [[U.read_unit(pages[0, p, h], page, d) for h in range(kv)] for p in mine]
            K[b], V[b] = (np.concatenate([np.stack([u[i] for u in p], 1) for p in units])[:n[b]]
                          for i in (0, 1))
    cache = _cache(pages, table, n, np.zeros(pages.shape[1]), page, kv, d)
    cu = _cu(rows)
    q = torch.randn(int(cu[-1]), heads, d, device=DEV).to(DTYPES[dtype])
    out, st = binding.kv_attention(cache, q, _i(cu), _i(ctx), max_k=7, max_context=max_context,
                                   window=window, sinks=sinks)
    assert st.cpu().tolist() == [0 if r else 3 for r in rows]
    assert not torch.isnan(out).any()
    check_attention(out, q, K, V, cu, ctx, rows, dtype, d ** -0.5, window, sinks,
                    skip=set(range(len(rows))) - some)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_many_items_some_of_them_split(dtype, d):
    """The planned launch with chunks: few long requests among many short ones, bad ones
    between them, the same rows as calls that are not planned."""
    rng = np.random.default_rng(d)
    rows = [int(x) for x in rng.integers(1, 4, 60)]
    ctx = [int(x) for x in rng.integers(0, 60, 60)]
    for b, c in ((5, 6200), (17, 2049), (40, 4095), (59, 2047)):
        ctx[b] = c
    cache, K, V = make_attention(d, 32, 4, rows, ctx, 2)
    ctx[8] = -1
    ctx[9] = 2 ** 31 - 1
    cache.page_table[30, 0] = -5
    cache.page_table[40, 100] = 1 << 29
    cu = _cu(rows)
    q = torch.randn(int(cu[-1]), 8, d, device=DEV).to(DTYPES[dtype])
    out, st = binding.kv_attention(cache, q, _i(cu), _i(ctx), max_k=3, max_context=20000)
    want = [0] * 60
    want[8], want[9], want[30], want[40] = 5, 5, 8, 8
    assert st.cpu().tolist() == want
    o = _f64(out)
    for b in (8, 9, 30, 40):
        assert np.isnan(o[cu[b]:cu[b + 1]]).all()
    check_attention(out, q, K, V, cu, ctx, rows, dtype, d ** -0.5, skip=(8, 9, 30, 40))
    again, _ = binding.kv_attention(cache, q, _i(cu), _i(ctx), max_k=3, max_context=20000)
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))


def test_attention_does_not_depend_on_the_other_requests():
    a = run_attention("bf16", 128, 16, 4, 2, [3, 5, 1], [100, 900, 44], seed=9, max_k=7,
                      max_context=1000)
    cache, _, _ = make_attention(128, 16, 2, [3, 5, 1], [100, 900, 44], 9)
    g = torch.Generator().manual_seed(9)
    q = torch.randn(9, 4 * 128 + 5, generator=g).to(torch.bfloat16).to(DEV)[:, :512].unflatten(1, (4, 128))
    # request 1 alone has rows; the same sizes
    out, st = binding.kv_attention(cache, q, _i([3, 3, 8, 8]), _i([0, 900, 0]), max_k=7,
                                   max_context=1000)
    assert st.cpu().tolist() == [3, 0, 3]
    assert torch.equal(out[3:8], a[3:8])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_nan_blocks_reach_only_who_sees_them(dtype, d):
    """A V block stored as NaN: its 32 dims of the rows that see its position, nothing
    else.  A K block: the whole row.  Both at positions some rows do not see."""
    rows, ctx, page, window, sinks = [6], [70], 16, 40, 2
    cache, K, V = make_attention(d, page, 1, rows, ctx, 4)
    host = cache.pages.cpu().numpy().reshape(1, -1, 1, page * (d + d // 16))
    table = cache.page_table.cpu().numpy()
    _, _, ks, vs = U.places(page, d)
    blocks = d // 32
    for t, blk in ((1, 0), (33, blocks - 1), (73, 0), (50, 2 % blocks), (10, 0)):
        host[0, table[0, t // page], 0, vs[t % page, blk]] = 255
        V[0][t, 0, 32 * blk:32 * blk + 32] = np.nan
    cache.pages.copy_(torch.from_numpy(host.reshape(1, -1, host.shape[-1])))
    q = torch.randn(6, 2, d, device=DEV).to(DTYPES[dtype])
    args = dict(max_k=5, max_context=80, window=window, sinks=sinks)
    out, st = binding.kv_attention(cache, q, _i([0, 6]), _i(ctx), **args)
    assert st.cpu().tolist() == [0]
    check_attention(out, q, K, V, [0, 6], ctx, rows, dtype, d ** -0.5, window, sinks)
    assert np.isfinite(_f64(out)).any() and np.isnan(_f64(out)).any()
    # keys: position 74 is seen by rows 4 and 5 only, position 32 by rows 0 and 1
    host[0, table[0, 74 // page], 0, ks[74 % page, blocks - 1]] = 255
    host[0, table[0, 32 // page], 0, ks[32 % page, 0]] = 255
    cache.pages.copy_(torch.from_numpy(host.reshape(1, -1, host.shape[-1])))
    K[0][74, 0] = np.nan
    K[0][32, 0] = np.nan
    out, _ = binding.kv_attention(cache, q, _i([0, 6]), _i(ctx), **args)
    check_attention(out, q, K, V, [0, 6], ctx, rows, dtype, d ** -0.5, window, sinks)
    o = _f64(out)
    assert np.isnan(o[[0, 4, 5]]).all() and np.isfinite(o[2:4]).any()


def test_attention_rows_with_infinite_or_nan_queries_stay_alone():
    cache, K, V = make_attention(128, 16, 1, [4], [60], 1)
    q = torch.randn(4, 2, 128, device=DEV)
    clean, _ = binding.kv_attention(cache, q, _i([0, 4]), _i([60]), max_k=3, max_context=64)
    q[1, 0, 5] = float("nan")
    q[2, 1, 7] = float("inf")
    out, _ = binding.kv_attention(cache, q, _i([0, 4]), _i([60]), max_k=3, max_context=64)
    assert torch.isnan(out[1, 0]).all() and torch.isnan(out[2, 1]).all()
    for j, h in ((0, 0), (0, 1), (1, 1), (2, 0), (3, 0), (3, 1)):
        assert torch.equal(out[j, h], clean[j, h])


@pytest.mark.parametrize("dtype,scale,shift", [("bf16", 1e-38, 0), ("bf16", 2e38, 120),
                                               ("f32", 1e-38, 0), ("f32", 1.5e32, 100)])
def test_attention_scales_from_the_smallest_to_the_largest(dtype, scale, shift):
    """The smallest gives the mean of V; the largest meet queries so small that the
    scores stay in range."""
    cache, K, V = make_attention(64, 16, 1, [2], [70], 3)
    q = (torch.randn(2, 4, 64, device=DEV) * 2.0 ** -shift).to(DTYPES[dtype])
    out, st = binding.kv_attention(cache, q, _i([0, 2]), _i([70]), max_k=1, max_context=72, scale=scale)
    assert st.cpu().tolist() == [0]
    check_attention(out, q, K, V, [0, 2], [70], [2], dtype, float(np.float32(scale)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("max_context", [1200, 20000])
def test_attention_writes_over_its_queries(dtype, d, max_context):
    """Several row blocks, whole and split, planned and not: out = q gives the same bits."""
    rng = np.random.default_rng(d)
    batch = 4 if max_context == 1200 else 40
    rows = [int(x) for x in rng.integers(1, 9, batch)]
    ctx = [int(x) for x in rng.integers(0, 1100, batch)]
    cache, _, _ = make_attention(d, 64, 1, rows, ctx, 7)
    q = torch.randn(sum(rows), 20, d, device=DEV).to(DTYPES[dtype])
    kw = dict(max_k=7, max_context=max_context)
    out, _ = binding.kv_attention(cache, q, _i(_cu(rows)), _i(ctx), **kw)
    for _ in range(3):
        x = q.clone()
        same, st = binding.kv_attention(cache, x, _i(_cu(rows)), _i(ctx), out=x, **kw)
        assert same is x and st.cpu().tolist() == [0] * batch
        assert torch.equal(x, out)


def test_attention_statuses_and_what_it_leaves():
    d, page = 64, 16
    rows, ctx = [2, 2, 2, 3, 2, 2], [20, 30, 40, 30, 30, 30]
    cache, K, V = make_attention(d, page, 1, rows, ctx, 5)
    table = cache.page_table.clone()
    table[1, 1] = -1                         # a page row 0 and 1 see
    table[2, 0] = 1 << 20                    # out of the pool
    cache.page_table.copy_(table)
    cu = _cu(rows) + 2
    q = torch.randn(int(cu[-1]) + 1, 2, d, device=DEV)
    out = torch.full_like(q, 7.0)
    ctx2 = list(ctx)
    ctx2[4] = -1
    _, st = binding.kv_attention(cache, q, _i(cu), _i(ctx2), max_k=1, max_context=64, out=out)
    assert st.cpu().tolist() == [0, 8, 8, 3, 5, 0]          # request 3 has 2 drafts, max_k 1
    o = _f64(out)
    for r, kind in enumerate("--vvnnnn---nnvv-"):
        row = o[r]
        assert {"-": (row == 7).all(), "v": np.isfinite(row).all() and (row != 7).all(),
                "n": np.isnan(row).all()}[kind], r
    check_attention(out[2:], q[2:], K, V, _cu(rows), ctx, rows, "f32", d ** -0.5, skip=(1, 2, 3, 4))
    # behind a window the pages may be gone
    table[1, 1] = -1
    _, st = binding.kv_attention(cache, q, _i(cu), _i([20, 64, 40, 0, 30, 60]), max_k=2,
                                 max_context=66, window=8, out=out)
    assert st.cpu().tolist()[1] == 8                         # past its table row
    cache2, K, V = make_attention(d, page, 1, [3], [70], 6)
    cache2.page_table[0, :3] = -1
    q = torch.randn(3, 2, d, device=DEV)
    out, st = binding.kv_attention(cache2, q, _i([0, 3]), _i([70]), max_k=2, max_context=73,
                                   window=20)
    assert st.cpu().tolist() == [0]
    check_attention(out, q, K, V, [0, 3], [70], [3], "f32", d ** -0.5, 20)
    out, st = binding.kv_attention(cache2, q, _i([0, 3]), _i([70]), max_k=2, max_context=73,
                                   window=20, sinks=1)
    assert st.cpu().tolist() == [8] and torch.isnan(out).all()
    # more context than the call's bound
    out, st = binding.kv_attention(cache2, q, _i([0, 3]), _i([70]), max_k=2, max_context=72)
    assert st.cpu().tolist() == [5] and torch.isnan(out).all()
    # a page id outside the pool in one chunk of several
    cache3, _, _ = make_attention(d, page, 1, [1], [2000], 6)
    cache3.page_table[0, 90] = 1 << 30
    out, st = binding.kv_attention(cache3, q[:1], _i([0, 1]), _i([2000]), max_k=0, max_context=2001)
    assert st.cpu().tolist() == [8] and torch.isnan(out).all()


@pytest.mark.parametrize("cu", [[0, 3, 2, 8], [0, 3, 9, 8], [-1, 3, 5, 8]])
def test_attention_broken_offsets_stop_there(cu):
    first = next(b for b in range(3) if cu[b] < 0 or cu[b + 1] < cu[b] or cu[b + 1] > 8)
    cache, _, _ = make_attention(64, 16, 1, [8, 8, 8], [0, 0, 0], 1)
    q = torch.randn(8, 1, 64, device=DEV)
    out = torch.full_like(q, 7.0)
    _, st = binding.kv_attention(cache, q, _i(cu), _i([0, 0, 0]), max_k=7, max_context=8, out=out)
    assert st.cpu().tolist() == [0] * first + [3] * (3 - first)
    written = (_f64(out) != 7.0).any((1, 2))
    want = np.zeros(8, bool)
    for b in range(first):
        want[cu[b]:cu[b + 1]] = True
    assert np.array_equal(written, want)


def test_pages_past_32_bit_offsets():
    """A pool of more than 4 GiB whose used pages lie at its end."""
    d, page, kv = 256, 256, 8
    n = binding.kv_page_bytes(kv, d, page)
    num = (9 << 29) // n + 8
    pool = torch.empty(1, num, n, dtype=torch.uint8, device=DEV)
    assert pool.numel() > 1 << 32
    cache = binding.KVCache(pages=pool, page_table=_i([[num - 1, num - 2]]), seq_lens=_i([300]),
                            ref_counts=torch.zeros(num, dtype=torch.int32, device=DEV),
                            page_size=page, kv_heads=kv, head_dim=d)
    x = torch.randn(300, 3 * kv, d, device=DEV).to(torch.bfloat16)
    q, _, k, v = binding.kv_append(cache, x[:, :kv], x[:, kv:2 * kv], x[:, 2 * kv:], _i([0, 300]),
                                   _i([0]), want_values=True)
    out, st = binding.kv_attention(cache, q[-2:], _i([0, 2]), _i([298]), max_k=1, max_context=300)
    assert st.cpu().tolist() == [0]
    check_attention(out, q[-2:], [_f64(k)], [_f64(v)], [0, 2], [298], [2], "bf16", d ** -0.5)


# -------------------------------------------------------------------- pages

class World:
    """A cache and its Python tables, page contents as random bytes."""

    def __init__(self, seqs, width, num, page, layers=2, seed=0):
        self.rng = np.random.default_rng(seed)
        self.t = U.Tables(seqs, width, num, page)
        self.cache = binding.KVCache.create(layers=layers, num_pages=num, page_size=page, kv_heads=1,
                                            head_dim=64, requests=seqs, max_context=width * page,
                                            device=DEV)
        self.cache.pages.random_(0, 256)
        self.host = self.cache.pages.cpu().numpy().copy()
        self.dead = np.zeros(num, bool)        # contents no longer defined by the tables

    def check(self):
        c, t = self.cache, self.t
        assert c.seq_lens.cpu().tolist() == t.lens
        assert c.ref_counts.cpu().tolist() == t.refs
        table = c.page_table.cpu().numpy()
        for b, r in enumerate(t.rows):
            assert table[b, :len(r)].tolist() == r, b
        assert np.array_equal(c.pages.cpu().numpy(), self.host)

    def reserve(self, rows):
        cu = _cu(np.maximum(rows, 0))
        ctx, st = binding.kv_reserve(self.cache, _i(cu))
        rc, rs, copies = self.t.reserve(list(rows))
        for s, d in copies:
            self.host[:, d] = self.host[:, s]
        assert ctx.cpu().tolist() == rc and st.cpu().tolist() == rs
        self.check()
        return rs

    def release(self, give, ctx=None):
        st = binding.kv_release(self.cache, _i(give), None if ctx is None else _i(ctx))
        assert st.cpu().tolist() == self.t.release(list(give), ctx)
        self.check()

    def fork(self, pairs):
        s, d, n = (list(x) for x in zip(*pairs))
        whole = all(x is None for x in n)
        st = binding.kv_fork(self.cache, _i(s), _i(d), None if whole else _i(n))
        assert st.cpu().tolist() == self.t.fork(pairs)
        self.check()

    def compact(self):
        live = binding.kv_compact(self.cache)
        want, moves = self.t.compact()
        for s, d in moves:
            self.host[:, d] = self.host[:, s]
        assert live.cpu().tolist() == [want]
        self.check()


@pytest.mark.parametrize("seqs,width,num,page", [(1, 4, 3, 16), (7, 9, 40, 16), (40, 30, 500, 32),
                                                 (300, 12, 9000, 16), (1024, 6, 4097, 256),
                                                 (50, 900, 70001, 16)])
def test_page_calls_in_random_order(seqs, width, num, page):
    w = World(seqs, width, num, page, layers=1 if num > 1000 else 2, seed=num)
    rng = w.rng
    for step in range(24 if seqs < 300 else 10):
        op = int(rng.integers(0, 6))
        if op <= 1:
            w.reserve(rng.integers(-1, int(rng.choice([3, 2 * page, width * page])), seqs).tolist())
        elif op == 2:
            w.release([int(rng.integers(0, min(n, 40) + 1)) for n in w.t.lens])
        elif op == 3:
            w.release([n if rng.random() < 0.4 else 0 for n in w.t.lens])
        elif op == 4:
            empty = [b for b, n in enumerate(w.t.lens) if n == 0]
            full = [b for b, n in enumerate(w.t.lens) if n]
            if empty and full:
                pairs = [(int(rng.choice(full)), int(d), None) for d in empty[:200]]
                if rng.random() < 0.5:
                    pairs = [(s, d, int(rng.integers(0, w.t.lens[s] + 1))) for s, d, _ in pairs]
                w.fork(pairs)
        else:
            w.compact()
    w.compact()


@pytest.mark.parametrize("num", [9000, 65535, 65536, 65537])
def test_prompts_that_take_thousands_of_pages(num):
    """Admissions next to single steps, with shared tails to copy, up to a full pool."""
    width = num // 20
    w = World(40, width, num, 16, layers=1, seed=num)
    w.reserve([5] * 10 + [0] * 30)
    w.fork([(i, 10 + i, None) for i in range(10)])
    w.reserve([16 * (width - 1)] * 7 + [1] * 13 + [0] * 20)      # both holders copy
    w.release([0, 16 * width // 2] + [0] * 38)
    w.reserve([0] * 20 + [16 * width - 3] * 20)                  # the pool ends among these
    w.reserve([0] * 8 + [1] * 12 + [0] * 20)
    w.compact()


def test_shared_tails_are_copied_once_per_holder_and_freed():
    w = World(4, 4, 12, 16)
    w.reserve([20, 0, 0, 0])
    w.fork([(0, 1, 20), (0, 2, 18), (0, 3, 16)])
    w.reserve([3, 1, 40, 2])               # every holder copies: the first tail is nobody's
    assert w.t.refs[0] == 4 and w.t.refs[1] == 0
    w.release([4, 0, 42, 2])
    w.reserve([1, 0, 0, 1])
    w.compact()


def test_reserve_fails_whole_and_lets_small_requests_through():
    w = World(5, 3, 4, 16)
    assert w.reserve([16, 33, 10, 5, 49]) == [0, 0, 7, 7, 7]
    assert w.reserve([0, 15, 0, 0, 0]) == [3, 0, 3, 3, 3]   # needs no page
    w.release([16, 0, 0, 0, 0])
    assert w.reserve([0, 1, 16, 0, 0]) == [3, 7, 0, 3, 3]   # past its table row
    w.release([0, 48, 16, 0, 0])
    assert sum(w.t.refs) == 0


def test_release_and_fork_refuse_on_the_device():
    w = World(6, 4, 20, 16)
    w.reserve([20, 40, 0, 0, 0, 0])
    w.release([21, -1, 1, 0, 0, 0])                          # all refused
    w.release([5, 3, 0, 0, 0, 0], [-1, 0, -1, 0, 0, 0])      # request 0 is skipped
    w.fork([(0, 2, None), (1, 2, None), (0, 1, None), (3, 3, None), (6, 4, None), (0, -1, None),
            (2, 4, None), (0, 5, None)])
    w.fork([(0, 3, 21), (0, 4, -1), (1, 3, 0)])
    w.fork([(3, 4, None)])                                   # an empty sequence
    # ids outside the pool
    w.cache.page_table[1, 1] = 20
    st = binding.kv_fork(w.cache, _i([1]), _i([3]))
    assert st.cpu().tolist() == [8] and w.cache.seq_lens.cpu().tolist()[3] == 0
    ctx, st = binding.kv_reserve(w.cache, _i([0, 0, 1]))
    assert st.cpu().tolist() == [3, 0] and ctx.cpu().tolist() == [-1, 37]
    w.cache.page_table[1, 2] = -7
    ctx, st = binding.kv_reserve(w.cache, _i([0, 0, 1]))
    assert st.cpu().tolist() == [3, 8] and ctx.cpu().tolist() == [-1, -1]
    st = binding.kv_release(w.cache, _i([0, 30]))
    assert st.cpu().tolist() == [0, 8] and w.cache.seq_lens.cpu().tolist()[:2] == [20, 8]


@pytest.mark.parametrize("cu", [[0, 3, 2, 8], [-1, 3, 5, 8]])
def test_reserve_broken_offsets_stop_there(cu):
    first = 1 if cu[0] == 0 else 0
    w = World(3, 4, 12, 16)
    ctx, st = binding.kv_reserve(w.cache, _i(cu))
    assert st.cpu().tolist() == [0] * first + [3] * (3 - first)
    w.t.reserve([3 if b < first else 0 for b in range(3)])
    w.check()


def test_compact_of_empty_full_and_one_page_pools():
    for num in (1, 5, 4096, 4100):
        w = World(3, 2100, num, 16, layers=1)
        w.compact()
        w.reserve([1, 0, 0])
        w.compact()
        w.reserve([0, (num - 1) * 16 if num > 1 else 0, 0])
        w.compact()
        w.release([1, 0, 0])
        w.compact()


def test_fork_of_lengths_past_the_table_row():
    """A length that its table row cannot hold is refused, also where many pairs share it."""
    w = World(300, 3, 40, 16, layers=1)
    w.reserve([40] + [0] * 299)
    w.cache.seq_lens[0] = 16 * 64
    st = binding.kv_fork(w.cache, _i([0] * 299), _i(range(1, 300)))
    assert st.cpu().tolist() == [8] * 299
    st = binding.kv_fork(w.cache, _i([0] * 299), _i(range(1, 300)), _i([40] * 299))
    assert st.cpu().tolist() == [0] * 299
    assert w.cache.ref_counts.cpu().tolist()[:4] == [300, 300, 300, 0]


# ------------------------------------------------------- streams and graphs

def test_calls_of_two_threads_on_one_stream():
    """The launches of a call do not mix with another thread's on the same stream."""
    import threading
    cache, q, cu, ctx, kw = _small()
    want, _ = binding.kv_attention(cache, q, cu, ctx, **kw)
    torch.cuda.synchronize()
    outs = []

    def work():
        for _ in range(20):
            outs.append(binding.kv_attention(cache, q, cu, ctx, **kw)[0])

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(outs) == 60 and all(torch.equal(o, want) for o in outs)


def test_a_workspace_of_the_callers():
    cache, q, cu, ctx, kw = _small()
    want, _ = binding.kv_attention(cache, q, cu, ctx, **kw)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)     # any contents
    out, _ = binding.kv_attention(cache, q, cu, ctx, workspace=ws, **kw)
    assert torch.equal(out, want)
    for bad in (ws[:64], ws[8:], ws[::2], ws.cpu()):
        with pytest.raises(ValueError):
            binding.kv_attention(cache, q, cu, ctx, workspace=bad, **kw)
    w = World(3, 4, 12, 16)
    for bad in (ws[:16], ws.cpu()):
        with pytest.raises(ValueError):
            binding.kv_reserve(w.cache, _i([0, 1, 1, 1]), workspace=bad)
        with pytest.raises(ValueError):
            binding.kv_compact(w.cache, workspace=bad)


def test_the_binding_refuses_arguments_that_do_not_fit():
    cache, q, cu, ctx, kw = _small()
    x = torch.randn(9, 8, 128, device=DEV, dtype=torch.bfloat16)
    ok = dict(q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], cu_seqlens=cu, context_lens=ctx)
    binding.kv_append(cache, **ok)
    cs = torch.zeros(800, 64, device=DEV)
    for change in (dict(q=x[:, :3]), dict(k=x[:, 4:7]), dict(v=x[:8, 6:]), dict(q=x[:, :4].float()),
                   dict(q=x[:, :4, :64]), dict(q=x[:, 0:8:2]), dict(q=x[:, :4].cpu()),
                   dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu[:1]), dict(context_lens=ctx[:2]),
                   dict(context_lens=ctx.float()), dict(q_weight=torch.ones(64, device=DEV)),
                   dict(k_weight=torch.ones(128, device=DEV, dtype=torch.bfloat16)),
                   dict(cos_sin=cs[:, :40]), dict(cos_sin=cs.double()), dict(cos_sin=cs[0]),
                   dict(cos_sin=cs[:, :24].contiguous()), dict(layer=1), dict(layer=-1),
                   dict(out=x[:8, :4]), dict(eps=-1.0), dict(q=x[0:1, :4].expand(9, -1, -1)),
                   dict(cu_seqlens=torch.zeros(9, dtype=torch.int32, device=DEV)),
                   dict(q=x[:0, :4], k=x[:0, 4:6], v=x[:0, 6:])):
        with pytest.raises(ValueError):
            binding.kv_append(cache, **{**ok, **change})
    ok = dict(q=q, cu_seqlens=cu, context_lens=ctx, **kw)
    for change in (dict(q=q.half()), dict(q=q[:, :3]), dict(max_k=64), dict(max_context=0),
                   dict(window=-1), dict(scale=0.0), dict(layer=2), dict(out=q.float()),
                   dict(context_lens=ctx[:1])):
        with pytest.raises(ValueError):
            binding.kv_attention(cache, **{**ok, **change})
    with pytest.raises(ValueError):
        binding.kv_release(cache, torch.zeros(4, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        binding.kv_release(cache, _i([0, 0]), _i([0]))
    with pytest.raises(ValueError):
        binding.kv_fork(cache, _i([0, 1]), _i([2]))
    for name, bad in (("pages", cache.pages[:, :, :-16]), ("page_table", cache.page_table.long()),
                      ("seq_lens", cache.seq_lens[:1]), ("ref_counts", cache.ref_counts[:2])):
        with pytest.raises(ValueError):
            binding.KVCache(**{**{n: getattr(cache, n) for n in (
                "pages", "page_table", "seq_lens", "ref_counts", "page_size", "kv_heads",
                "head_dim")}, name: bad})

def _small(seed=0, batch=3):
    rows, ctx = [3, 1, 5][:batch], [40, 7, 700][:batch]
    cache, K, V = make_attention(128, 16, 2, rows, ctx, seed)
    q = torch.randn(sum(rows), 4, 128, device=DEV, dtype=torch.bfloat16)
    return cache, q, _i(_cu(rows)), _i(ctx), dict(max_k=4, max_context=705)


def test_calls_on_another_stream():
    cache, q, cu, ctx, kw = _small()
    want, _ = binding.kv_attention(cache, q, cu, ctx, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    with torch.cuda.stream(s):
        for _ in range(3):
            outs.append(binding.kv_attention(cache, q, cu, ctx, **kw)[0])
    here = [binding.kv_attention(cache, q, cu, ctx, **kw)[0] for _ in range(3)]
    torch.cuda.synchronize()
    for o in outs + here:
        assert torch.equal(o, want)


def test_two_captured_graphs_replayed_together():
    a, b = _small(1), _small(2)
    want = [binding.kv_attention(x[0], x[1], x[2], x[3], **x[4])[0] for x in (a, b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(binding.kv_attention(x[0], x[1], x[2], x[3], **x[4])[0])
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
        binding.kv_attention(a[0], a[1], a[2], a[3], **a[4])          # eager work in between
        torch.cuda.synchronize()


# ------------------------------------------------------------ the whole step

class Step:
    """A serving loop's verify step on two layers: reserve, append and attention per
    layer, greedy verify, drain, release."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.layers, self.heads, self.kv, self.d, self.page, self.V = 2, 4, 2, 64, 16, 64
        self.batch, self.k = 4, 3
        self.cache = binding.KVCache.create(layers=2, num_pages=64, page_size=16, kv_heads=2,
                                            head_dim=64, requests=self.batch, max_context=256,
                                            device=DEV)
        self.w = torch.randn(2, self.heads + 2 * self.kv, 64, 64, generator=g).to(DEV) * 0.3
        self.embed = torch.randn(self.V, 64, generator=g).to(DEV)
        self.head = torch.randn(self.heads * 64, self.V, generator=g).to(DEV)
        self.cs = torch.from_numpy(_rotation(256, 64)).to(DEV)
        self.nw = (1 + 0.1 * torch.randn(64, generator=g)).to(DEV)

    def forward(self, tokens, cu, ctx, max_k):
        x = self.embed[tokens.long()]
        h = None
        for layer in range(self.layers):
            qkv = (x[:, None, None] @ self.w[layer]).squeeze(2).contiguous()
            q, _ = binding.kv_append(self.cache, qkv[:, :self.heads],
                                     qkv[:, self.heads:self.heads + self.kv],
                                     qkv[:, self.heads + self.kv:], cu, ctx, layer=layer,
                                     q_weight=self.nw, k_weight=self.nw, cos_sin=self.cs)
            h, _ = binding.kv_attention(self.cache, q, cu, ctx, layer=layer, max_k=max_k,
                                        max_context=256)
            x = x + h.sum(1)
        return h.flatten(1) @ self.head

    def greedy(self, prompts, steps, drafts_of):
        """Verify steps with the given drafter; the committed tokens of each request."""
        cu = _i(_cu([len(p) for p in prompts]))
        ctx, st = binding.kv_reserve(self.cache, cu)
        toks = torch.tensor([t for p in prompts for t in p], device=DEV)
        logits = self.forward(toks, cu, ctx, max(len(p) for p in prompts) - 1)
        last = logits[cu[1:].long() - 1].argmax(-1)
        out = [[int(t)] for t in last.cpu()]
        for step in range(steps):
            drafts = [drafts_of(b, len(out[b]), step) for b in range(len(prompts))]
            rows = [[out[b][-1]] + list(drafts[b]) for b in range(len(prompts))]
            cu = _i(_cu([len(r) for r in rows]))
            ctx, st = binding.kv_reserve(self.cache, cu)
            assert st.cpu().tolist() == [0] * len(prompts)
            logits = self.forward(torch.tensor([t for r in rows for t in r], device=DEV), cu, ctx,
                                  max(len(r) for r in rows) - 1)
            flat = [t for d in drafts for t in d]
            acc, tok, vst = binding.verify_greedy(logits, cu, _i(flat) if flat else
                                                  torch.empty(0, dtype=torch.int32, device=DEV),
                                                  max_k=8)
            committed, offs, rollback = binding.drain(cu, acc, vst, tok)
            st = binding.kv_release(self.cache, rollback, ctx)
            assert st.cpu().tolist() == [0] * len(prompts)
            offs, committed = offs.cpu().tolist(), committed.cpu().tolist()
            for b in range(len(prompts)):
                out[b] += committed[offs[b]:offs[b + 1]]
        lens = self.cache.seq_lens.cpu().tolist()
        assert lens == [len(p) + len(o) - 1 for p, o in zip(prompts, out)]
        return out


def test_speculation_commits_what_plain_decoding_does():
    """Wrong, right and partly right drafts at different places every step: the
    committed tokens are those of one-token decoding (rejected positions were given
    back and written over), for sequences of different lengths."""
    rng = np.random.default_rng(5)
    prompts = [rng.integers(0, 64, n).tolist() for n in (1, 17, 30, 45)]
    plain = Step().greedy(prompts, 24, lambda b, n, s: [])

    def drafts(b, n, step):
        k = (b + step) % 5
        right = plain[b][n:n + k]
        wrong = (step * 7 + b) % (k + 1)
        return [t if i != wrong else (t + 1) % 64 for i, t in enumerate(right)]

    spec = Step().greedy(prompts, 8, drafts)
    for b in range(4):
        n = min(len(plain[b]), len(spec[b]))
        assert n > 8 and spec[b][:n] == plain[b][:n], b


def test_forked_sequences_continue_like_their_source():
    s = Step(3)
    cu = _i(_cu([37, 0, 0, 0]))
    toks = torch.randint(0, 64, (37,), device=DEV)
    ctx, _ = binding.kv_reserve(s.cache, cu)
    s.forward(toks, cu, ctx, 36)
    st = binding.kv_fork(s.cache, _i([0, 0]), _i([1, 2]), _i([37, 32]))
    assert st.cpu().tolist() == [0, 0]
    # the second fork appends the source's last five tokens itself
    rows = [2, 2, 7, 0]
    cu = _i(_cu(rows))
    nxt = torch.tensor([5, 9], device=DEV)
    ctx, st = binding.kv_reserve(s.cache, cu)
    assert st.cpu().tolist() == [0, 0, 0, 3] and ctx.cpu().tolist() == [37, 37, 32, -1]
    logits = s.forward(torch.cat([nxt, nxt, toks[32:], nxt]), cu, ctx, 6)
    assert torch.equal(logits[0:2], logits[2:4])
    # (its rows 5 and 6 share a tile with others: the same bits too)
    assert torch.allclose(logits[9:11], logits[0:2], rtol=1e-4, atol=1e-3)
    live = binding.kv_compact(s.cache)
    refs = s.cache.ref_counts.cpu().numpy()
    assert (refs[:int(live)] > 0).all() and (refs[int(live):] == 0).all()
    q = torch.randn(3, 4, 64, device=DEV)
    out, st = binding.kv_attention(s.cache, q[:1].expand(3, -1, -1).contiguous(), _i([0, 1, 2, 3]),
                                   _i([38, 38, 38]), max_k=0, max_context=64)
    assert st.cpu().tolist() == [0, 0, 0]
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


def test_a_step_captured_in_a_graph():
    """Reserve, append, attention and release as one graph, replayed against eager calls
    on an equal cache, eager work between the replays."""
    a, b = Step(1), Step(1)
    cu0 = _i(_cu([5, 20, 1, 33]))
    toks = torch.randint(0, 64, (59,), device=DEV)
    for s in (a, b):
        ctx, _ = binding.kv_reserve(s.cache, cu0)
        s.forward(toks, cu0, ctx, 32)
    cu = _i(_cu([4, 3, 1, 2]))
    give = _i([2, 0, 1, 1])
    x = torch.randn(10, 8, 64, device=DEV)

    def step(s, x):
        ctx, st = binding.kv_reserve(s.cache, cu)
        q, _ = binding.kv_append(s.cache, x[:, :4], x[:, 4:6], x[:, 6:], cu, ctx, layer=1,
                                 q_weight=s.nw, k_weight=s.nw, cos_sin=s.cs)
        out, _ = binding.kv_attention(s.cache, q, cu, ctx, layer=1, max_k=3, max_context=256)
        return out, st, binding.kv_release(s.cache, give, ctx)

    keep = [t.clone() for t in (a.cache.pages, a.cache.page_table, a.cache.seq_lens,
                                a.cache.ref_counts)]
    g = torch.cuda.CUDAGraph()
    xin = x.clone()
    with torch.cuda.graph(g):
        got = step(a, xin)
    for t, k in zip((a.cache.pages, a.cache.page_table, a.cache.seq_lens, a.cache.ref_counts), keep):
        assert torch.equal(t, k)                             # capture runs nothing
    for i in range(6):
        new = torch.randn(10, 8, 64, device=DEV)
        xin.copy_(new)
        g.replay()
        want = step(b, new)
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v), i
        for n in ("pages", "seq_lens", "ref_counts"):
            assert torch.equal(getattr(a.cache, n), getattr(b.cache, n)), (i, n)
