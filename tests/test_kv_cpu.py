"""The cache operators on the CPU: what the references the GPU tests compare
with are pinned by, every refusal of the C entry points (each call fails
validation on the host, so no GPU is touched), and the binding's own checks."""

import numpy as np
import pytest
import torch

import kv_util as U
from lossless_rejection_sampling_spec_amd import binding

F = 0x1000        # a 16-byte aligned non-NULL pointer value that validation never reads


# ------------------------------------------------------------ the references

def test_every_code_and_scale_reads_back_as_itself():
    for byte in (1, 2, 100, 127, 200, 252):
        code = np.arange(32, dtype=np.uint8) & 15
        code[code == 8] = 0                                  # minus zero is stored as zero
        v = U.decode(code[None], np.array([[byte]], np.uint8))
        c2, b2 = U.encode(v)
        assert np.array_equal(c2[0], code) and b2[0, 0] == byte


def test_encoding_is_nearest_with_the_smallest_scale_that_fits():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 64)) * np.exp(rng.uniform(-20, 20, (200, 1)))
    code, byte = U.encode(x)
    v = U.decode(code, byte)
    s = np.repeat(np.ldexp(1.0, byte.astype(int) - 127), 32, -1)
    amax = np.repeat(np.abs(x.reshape(200, 2, 32)).max(-1), 32, -1)
    assert np.all(amax <= 6 * s) and np.all(amax > 3 * s)
    grid = np.concatenate([U.LEVELS, -U.LEVELS])
    nearest = np.abs(x[..., None] - s[..., None] * grid).min(-1)
    assert np.array_equal(np.abs(x - v), nearest)


def test_ties_go_to_the_even_code_and_bad_blocks_read_as_nan():
    x = np.zeros((1, 32))
    x[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    code, byte = U.encode(x)
    assert code[0, :8].tolist() == [7, 0, 2, 2, 4, 4, 6, 6] and byte[0, 0] == 127
    x[0, 9] = np.inf
    code, byte = U.encode(x)
    assert byte[0, 0] == 255 and np.isnan(U.decode(code, byte)).all()


@pytest.mark.parametrize("page", [16, 32, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_layout_fills_a_unit_without_overlap(page, d):
    at = np.concatenate([a.ravel() for a in U.places(page, d)])
    assert np.array_equal(np.sort(at), np.arange(page * (d + d // 16)))
    assert binding.kv_page_bytes(3, d, page) == 3 * at.size


def test_reference_attention_is_a_softmax():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 9, 64))
    q = rng.standard_normal(64)
    out, _, _ = U.attention_row(q, k, v, 5, 0.1, 0, 0)
    w = np.exp(0.1 * k[:6] @ q)
    assert np.allclose(out, (w[:, None] * v[:6]).sum(0) / w.sum(), rtol=1e-13)
    out, _, _ = U.attention_row(q, k, v, 8, 0.1, 2, 1)
    keep = [0, 7, 8]
    w = np.exp(0.1 * k[keep] @ q)
    assert np.allclose(out, (w[:, None] * v[keep]).sum(0) / w.sum(), rtol=1e-13)


def test_reference_tables_keep_their_counts():
    rng = np.random.default_rng(3)
    t = U.Tables(12, 20, 90, 16)
    for _ in range(200):
        op = rng.integers(0, 4)
        if op == 0:
            t.reserve(rng.integers(0, 40, 12).tolist())
        elif op == 1:
            t.release([int(rng.integers(0, n + 1)) for n in t.lens])
        elif op == 2:
            t.fork([(int(rng.integers(0, 12)), int(rng.integers(0, 12)), None)])
        else:
            live, _ = t.compact()
            assert all(t.refs[:live]) and not any(t.refs[live:])
        refs = [0] * 90
        for r, n in zip(t.rows, t.lens):
            assert len(r) == t.pages(n)
            for p in r:
                refs[p] += 1
        assert refs == t.refs


# ------------------------------------------------------------ refusals

def _append(**kw):
    a = dict(q=F, ldq=512, k=F, ldk=256, v=F, ldv=256, dt=1, qw=None, kw=None, eps=1e-6, cs=None,
             maxp=0, rot=0, inter=0, cu=F, ctx=F, batch=2, rows=6, heads=4, kv=2, d=128, pages=F,
             num=10, page=16, table=F, ldt=4, qo=F, ldo=512, kv_=None, vv_=None, st=F, stream=None)
    a.update(kw)
    return binding.lib().spec_kv_append(*a.values())


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(cu=None), 1),
    (dict(ctx=None), 1), (dict(pages=None), 1), (dict(table=None), 1), (dict(qo=None), 1),
    (dict(st=None), 1), (dict(rot=64), 1), (dict(kv_=F), 1), (dict(vv_=F), 1),
    (dict(dt=2), 3), (dict(batch=0), 2), (dict(batch=1025), 2), (dict(rows=0), 2),
    (dict(heads=3), 2), (dict(heads=1), 2), (dict(kv=0), 2), (dict(heads=1026), 2),
    (dict(d=96), 2), (dict(d=0), 2), (dict(page=8), 2), (dict(page=48), 2), (dict(page=512), 2),
    (dict(num=0), 2), (dict(num=(1 << 24) + 1), 2), (dict(ldt=0), 2),
    (dict(ldt=(1 << 26) + 1), 2), (dict(ldq=511), 2), (dict(ldk=255), 2), (dict(ldv=255), 2),
    (dict(ldo=511), 2), (dict(cs=F, rot=24, maxp=4), 2), (dict(cs=F, rot=144, maxp=4), 2),
    (dict(cs=F, rot=-16, maxp=4), 2), (dict(cs=F, rot=64, maxp=0), 2), (dict(eps=-1.0), 2),
    (dict(eps=float("nan")), 2), (dict(eps=2.0), 2), (dict(pages=F + 8), 2),
    (dict(rows=1 << 28), 2)])
def test_append_refuses(kw, rc):
    assert _append(**kw) == rc


def _attention(**kw):
    a = dict(q=F, ldq=512, dt=1, cu=F, ctx=F, batch=2, rows=6, max_k=3, heads=4, kv=2, d=128,
             pages=F, num=10, page=16, table=F, ldt=4, maxc=64, scale=0.1, window=0, sinks=0,
             out=F, ldo=512, st=F, ws=F, wsb=1 << 40, stream=None)
    a.update(kw)
    return binding.lib().spec_kv_attention(*a.values())


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), 1), (dict(cu=None), 1), (dict(ctx=None), 1), (dict(pages=None), 1),
    (dict(table=None), 1), (dict(out=None), 1), (dict(st=None), 1), (dict(dt=7), 3),
    (dict(batch=0), 2), (dict(batch=1025), 2), (dict(rows=0), 2), (dict(max_k=-1), 2),
    (dict(max_k=64), 2), (dict(heads=3), 2), (dict(heads=0), 2), (dict(kv=0), 2),
    (dict(d=32), 2), (dict(page=24), 2), (dict(num=0), 2), (dict(num=1 << 31), 2),
    (dict(ldt=0), 2), (dict(ldt=(1 << 26) + 1), 2), (dict(ldq=511), 2), (dict(ldo=511), 2),
    (dict(maxc=0), 2), (dict(maxc=(1 << 30) + 1), 2), (dict(scale=0.0), 2),
    (dict(scale=-1.0), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(scale=2.1e38), 2),
    (dict(window=-1), 2), (dict(sinks=-1), 2), (dict(pages=F + 4), 2),
    (dict(maxc=100000, ws=None), 1), (dict(maxc=100000, ws=F + 4), 1),
    (dict(maxc=100000, wsb=64), 4)])
def test_attention_refuses(kw, rc):
    assert _attention(**kw) == rc


def test_attention_workspace_sizes():
    f = binding.lib().spec_kv_attention_workspace_bytes
    assert f(1, 1, 0, 8, 8, 128, 40, 0, 0) == 16             # a short context is not split
    assert f(1, 1, 0, 32, 8, 128, 40000, 0, 0) > 1 << 16
    assert f(1, 1, 0, 32, 8, 128, 40000, 64, 4) == 16        # a window is short
    for bad in ((2, 1, 0, 8, 8, 128, 40, 0, 0), (1, 0, 0, 8, 8, 128, 40, 0, 0),
                (1, 1, 64, 8, 8, 128, 40, 0, 0), (1, 1, 0, 9, 8, 128, 40, 0, 0),
                (1, 1, 0, 8, 8, 100, 40, 0, 0), (1, 1, 0, 8, 8, 128, 0, 0, 0),
                (1, 1, 0, 8, 8, 128, 40, -1, 0), (1, 1, 0, 8, 8, 128, 40, 0, -1)):
        assert f(*bad) == 0


def _reserve(**kw):
    a = dict(cu=F, batch=4, page=16, lens=F, table=F, ldt=8, refs=F, num=100, pages=F, pb=4352,
             layers=2, lb=435200, ctx=F, st=F, ws=F, wsb=1 << 20, stream=None)
    a.update(kw)
    return binding.lib().spec_kv_reserve(*a.values())


def _compact(**kw):
    a = dict(seqs=4, page=16, lens=F, table=F, ldt=8, refs=F, num=100, pages=F, pb=4352, layers=2,
             lb=435200, live=F, ws=F, wsb=1 << 20, stream=None)
    a.update(kw)
    return binding.lib().spec_kv_compact(*a.values())


@pytest.mark.parametrize("call", [_reserve, _compact])
@pytest.mark.parametrize("kw,rc", [
    (dict(lens=None), 1), (dict(table=None), 1), (dict(refs=None), 1), (dict(pages=None), 1),
    (dict(ws=None), 1), (dict(page=20), 2), (dict(ldt=0), 2), (dict(num=0), 2),
    (dict(num=1 << 25), 2), (dict(pb=0), 2), (dict(pb=4350), 2), (dict(layers=0), 2),
    (dict(layers=70000), 2), (dict(lb=435199), 2), (dict(lb=400000), 2), (dict(pages=F + 1), 2),
    (dict(ws=F + 4), 2), (dict(wsb=15), 4)])
def test_reserve_and_compact_refuse(call, kw, rc):
    assert call(**kw) == rc


def test_the_other_page_calls_refuse():
    assert _reserve(cu=None) == 1 and _reserve(ctx=None) == 1 and _reserve(st=None) == 1
    assert _reserve(batch=0) == 2 and _reserve(batch=1025) == 2
    assert _compact(live=None) == 1 and _compact(seqs=0) == 2 and _compact(seqs=1025) == 2
    L = binding.lib()

    def release(give=F, ctx=None, batch=4, page=16, lens=F, table=F, ldt=8, refs=F, num=100, st=F):
        return L.spec_kv_release(give, ctx, batch, page, lens, table, ldt, refs, num, st, None)

    for name in ("give", "lens", "table", "refs", "st"):
        assert release(**{name: None}) == 1
    for kw in (dict(batch=0), dict(batch=1025), dict(page=1), dict(ldt=0), dict(num=0)):
        assert release(**kw) == 2

    def fork(src=F, dst=F, lens=None, pairs=3, seqs=8, page=16, sl=F, table=F, ldt=8, refs=F,
             num=100, st=F):
        return L.spec_kv_fork(src, dst, lens, pairs, seqs, page, sl, table, ldt, refs, num, st,
                              None)

    for name in ("src", "dst", "sl", "table", "refs", "st"):
        assert fork(**{name: None}) == 1
    for kw in (dict(pairs=0), dict(pairs=1025), dict(seqs=0), dict(seqs=1025), dict(page=0),
               dict(ldt=0), dict(num=0)):
        assert fork(**kw) == 2
    assert L.spec_kv_pages_workspace_bytes(4, 0) == 0
    assert L.spec_kv_pages_workspace_bytes(0, 4) == 0
    assert L.spec_kv_pages_workspace_bytes(1024, 1 << 24) > 3 << 26
    for bad in ((0, 128, 16), (1, 96, 16), (1, 128, 8), (1, 128, 24)):
        assert L.spec_kv_page_bytes(*bad) == 0


def test_header_arity_and_status_strings():
    import re
    from test_abi import HEADER, _declared
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(spec_kv_\w+)\s*\(", src)))
    assert len(names) == 9
    for name in names:
        m = re.search(name + r"\s*\(([^;]*)\);", src, flags=re.S)
        assert len(getattr(binding.lib(), name).argtypes) == len(m.group(1).split(",")), name
    assert not set(names) & set(_declared())
    for code in (binding.ROW_NO_PAGES, binding.ROW_BAD_PAGE):
        assert binding.status_string(100 + code).startswith("row")


def test_the_cache_refuses_host_tensors_and_bad_sizes():
    with pytest.raises(ValueError):
        binding.KVCache.create(layers=1, num_pages=4, page_size=16, kv_heads=2, head_dim=96,
                               requests=2, max_context=64, device="cpu")
    with pytest.raises(ValueError):                          # host tensors
        binding.KVCache.create(layers=1, num_pages=4, page_size=16, kv_heads=2, head_dim=128,
                               requests=2, max_context=64, device="cpu")
    with pytest.raises(ValueError):
        binding.KVCache(pages=torch.zeros(1, 4, 100, dtype=torch.uint8),
                        page_table=torch.zeros(2, 4, dtype=torch.int32),
                        seq_lens=torch.zeros(2, dtype=torch.int32),
                        ref_counts=torch.zeros(4, dtype=torch.int32), page_size=16, kv_heads=2,
                        head_dim=128)
