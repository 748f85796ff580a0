"""Prompt attention, attention weights, eviction and appends at offsets on the CPU: every
refusal of the C entry points (each call fails validation on the host, so no GPU is touched),
the workspace sizes, the reference of an eviction, and that no kernel of theirs spills."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

import kv_budget_util as E
from lossless_rejection_sampling_spec_amd import binding, build
from test_kernel_registers import spills

F = 0x1000        # a 16-byte aligned non-NULL pointer value that validation never reads
BIG = 1 << 40     # more workspace than any call here needs


def _prompt(**kw):
    a = dict(q=F, ldq=512, dt=1, cu=F, ctx=F, batch=2, rows=6, heads=4, kv=2, d=128, pages=F, num=10,
             page=16, table=F, ldt=4, maxc=64, total=128, scale=0.1, window=0, sinks=0, out=2 * F,
             ldo=512, st=F, ws=F, wsb=BIG, stream=None)
    a.update(kw)
    return binding.lib().spec_kv_prompt_attention(*a.values())


def _weights(**kw):
    a = dict(q=F, ldq=512, dt=1, cu=F, ctx=F, counts=None, batch=2, rows=6, max_k=5, heads=4, kv=2,
             d=128, pages=F, num=10, page=16, table=F, ldt=4, maxc=64, scale=0.1, window=0, sinks=0,
             win=None, wout=F, ldw=64, st=F, ws=F, wsb=BIG, stream=None)
    a.update(kw)
    return binding.lib().spec_kv_attention_weights(*a.values())


def _evict(**kw):
    a = dict(budgets=F, batch=2, sinks=0, recent=0, weights=F, ldw=64, kv=2, d=128, page=16, lens=F,
             table=F, ldt=4, refs=F, num=10, pages=F, layers=1, layer_bytes=1 << 20, evicted=None, st=F,
             stream=None)
    a.update(kw)
    return binding.lib().spec_kv_evict(*a.values())


COMMON = [(dict(q=None), 1), (dict(cu=None), 1), (dict(ctx=None), 1), (dict(pages=None), 1),
          (dict(table=None), 1), (dict(st=None), 1), (dict(ws=None), 1), (dict(ws=F + 8), 1),
          (dict(dt=2), 3), (dict(batch=0), 2), (dict(batch=1025), 2), (dict(rows=0), 2),
          (dict(heads=3), 2), (dict(heads=1), 2), (dict(kv=0), 2), (dict(heads=1026), 2), (dict(d=96), 2),
          (dict(page=8), 2), (dict(page=48), 2), (dict(num=0), 2), (dict(ldt=0), 2),
          (dict(ldt=(1 << 26) + 1), 2), (dict(ldq=511), 2), (dict(maxc=0), 2), (dict(maxc=(1 << 30) + 1), 2),
          (dict(scale=0.0), 2), (dict(scale=-1.0), 2), (dict(scale=float("nan")), 2),
          (dict(scale=float("inf")), 2), (dict(window=-1), 2), (dict(sinks=-1), 2), (dict(pages=F + 4), 2),
          (dict(wsb=0), 4)]


@pytest.mark.parametrize("kw,rc", COMMON + [
    (dict(out=None), 1), (dict(out=F), 2), (dict(ldo=511), 2), (dict(total=0), 2),
    (dict(total=(1 << 30) + 1), 2), (dict(rows=1 << 29), 2), (dict(total=1 << 30, maxc=1 << 30), 2)])
def test_prompt_refusals(kw, rc):
    assert _prompt(**kw) == rc


# q: 6 rows of 1,024 bytes at Q
Q = 1 << 20


@pytest.mark.parametrize("kw", [
    dict(out=Q + 1024), dict(out=Q - 1024), dict(out=Q + 256), dict(out=Q - 2), dict(out=Q + 5 * 1024 + 1022),
    dict(out=Q + 1022, ldq=1024, ldo=1024),            # the last element of a row, rows 2,048 bytes apart
    dict(out=Q + 5 * 2048 - 1022, ldq=1024, ldo=1024), dict(out=Q - 4 * 2048 + 1026, ldq=1024, ldo=1024),
    dict(out=Q + 1024, ldq=1024, ldo=600),             # rows at other distances
    dict(dt=0, out=Q + 6 * 1024), dict(dt=0, out=Q + 2044, ldq=1024, ldo=1024)])
def test_prompt_refuses_a_result_that_overlaps_its_queries(kw):
    assert _prompt(**{"q": Q, **kw}) == 2


def test_overlap_of_strided_rows(tmp_path):
    """The host's check of two strided arrays against every byte of them."""
    source = tmp_path / "rows.cpp"
    source.write_text('#include "row_ranges.h"\nextern "C" int meet(long long a, long long la, long long b, '
                      'long long lb, long long rows, long long width) {\n  return svk::rows_overlap((void*)a, la, '
                      '(void*)b, lb, rows, width); }\n')
    lib = tmp_path / "rows.so"
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(build.PKG, "csrc"), str(source),
                    "-o", str(lib)], check=True)
    meet = ctypes.CDLL(str(lib)).meet
    meet.argtypes = [ctypes.c_longlong] * 6
    seen = set()
    for rows in (1, 2, 5):
        for width in (1, 3):
            for la in range(width, 7):
                mine = {i * la + x for i in range(rows) for x in range(width)}
                for lb in range(width, 7):
                    for gap in range(-32, 33):
                        want = any(gap + j * lb + x in mine for j in range(rows) for x in range(width))
                        seen.add(want)
                        assert meet(1000, la, 1000 + gap, lb, rows, width) == want, (rows, width, la, lb, gap)
    assert seen == {True, False}
    # the largest sizes
    assert meet(1 << 40, 1 << 40, (1 << 40) + 8192, 1 << 40, (1 << 31) - 1, 8192) == 0
    assert meet(1 << 40, 1 << 40, (1 << 40) + 8191, 1 << 40, (1 << 31) - 1, 8192) == 1
    assert meet(1 << 40, (1 << 62) - 1, 1 << 41, (1 << 62) - 2, 1 << 20, 8192) == 0


@pytest.mark.parametrize("kw,rc", COMMON + [
    (dict(wout=None), 1), (dict(max_k=-1), 2), (dict(max_k=64), 2), (dict(ldw=63), 2),
    (dict(win=F + 16), 2), (dict(wout=F + 16, win=F), 2), (dict(win=F + 2 * 2 * 64 * 4 - 16), 2),
    (dict(batch=1024, heads=1024, kv=1024, ldq=1024 * 128, maxc=1 << 14, ldw=1 << 14), 2)])
def test_weights_refusals(kw, rc):
    assert _weights(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(budgets=None), 1), (dict(weights=None), 1), (dict(lens=None), 1), (dict(table=None), 1),
    (dict(refs=None), 1), (dict(pages=None), 1), (dict(st=None), 1), (dict(batch=0), 2),
    (dict(batch=1025), 2), (dict(sinks=-1), 2), (dict(recent=-1), 2), (dict(ldw=0), 2), (dict(kv=0), 2),
    (dict(d=32), 2), (dict(page=24), 2), (dict(ldt=0), 2), (dict(num=0), 2), (dict(num=(1 << 24) + 1), 2),
    (dict(pages=F + 8), 2), (dict(layers=0), 2), (dict(layers=65536), 2), (dict(layer_bytes=24), 2),
    (dict(layers=2, layer_bytes=16), 2), (dict(layers=2048, batch=1024), 2)])
def test_evict_refusals(kw, rc):
    assert _evict(**kw) == rc


def test_append_at_refuses_what_append_does():
    L = binding.lib()

    def call(**kw):
        a = dict(q=F, ldq=512, k=F, ldk=256, v=F, ldv=256, dt=1, qw=None, kw=None, eps=1e-6, cs=None,
                 maxp=0, rot=0, inter=0, cu=F, ctx=F, offs=None, batch=2, rows=6, heads=4, kv=2, d=128,
                 pages=F, num=10, page=16, table=F, ldt=4, qo=F, ldo=512, kv_=None, vv_=None, st=F,
                 stream=None)
        a.update(kw)
        return L.spec_kv_append_at(*a.values())
    for kw, rc in ((dict(q=None), 1), (dict(rot=64), 1), (dict(kv_=F), 1), (dict(dt=2), 3), (dict(d=96), 2),
                   (dict(rows=0), 2), (dict(rot=64, cs=F, maxp=0), 2), (dict(offs=F, heads=3), 2)):
        assert call(**kw) == rc


def test_the_binding_has_the_headers_arity():
    import os
    import re
    from test_abi import ROOT
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "specverify_cache.h")).read(), flags=re.S)
    found = re.findall(r"\b(spec_kv_\w+)\s*\(([^;]*)\);", src, flags=re.S)
    assert len(found) == 6
    for name, args in found:
        assert len(getattr(binding.lib(), name).argtypes) == len(args.split(",")), name


def test_workspace_sizes():
    L = binding.lib()
    prompt = dict(dt=1, batch=4, rows=1000, heads=32, kv=8, d=128, maxc=4000, total=9000, window=0, sinks=0)

    def size(**kw):
        return L.spec_kv_prompt_workspace_bytes(*{**prompt, **kw}.values())
    # the requests' cache in bf16 (a tile more per request), and less than 64 MiB besides
    wide = 4 * 128 * 8 * (9000 + 4 * 32)
    assert wide - 4 * 128 * 8 * 32 * 4 <= size() <= wide + (64 << 20)
    assert size(total=18000) > size() > size(window=64)
    for kw in (dict(dt=2), dict(batch=0), dict(batch=1025), dict(rows=0), dict(heads=30), dict(d=96),
               dict(maxc=0), dict(total=0), dict(total=(1 << 30) + 1), dict(window=-1), dict(sinks=-1),
               dict(rows=1 << 30)):
        assert size(**kw) == 0
    weights = dict(dt=1, batch=4, max_k=6, heads=32, kv=8, d=128, maxc=4000, window=0, sinks=0)

    def wsize(**kw):
        return L.spec_kv_weights_workspace_bytes(*{**weights, **kw}.values())
    assert 0 < wsize(maxc=100) < wsize() < wsize(max_k=63)
    for kw in (dict(dt=2), dict(batch=0), dict(max_k=-1), dict(max_k=64), dict(heads=30), dict(d=32),
               dict(maxc=0), dict(window=-1), dict(sinks=-1)):
        assert wsize(**kw) == 0


def test_prompt_sizes_at_their_limits():
    """Both sides of what one launch takes, and of the tiles' numbers; refusals and sizes agree."""
    L = binding.lib()

    def fits(**kw):
        a = dict(dt=1, batch=1, rows=1 << 20, heads=128, kv=8, d=128, maxc=1 << 20, total=1 << 20, window=0,
                 sinks=0)
        a.update(kw)
        size = L.spec_kv_prompt_workspace_bytes(*a.values())
        rc = _prompt(**{"ldq": a["heads"] * a["d"], "ldo": a["heads"] * a["d"], "wsb": 0, **a})
        assert rc == (4 if size else 2), kw                # no workspace, or sizes
        return size > 0
    assert fits() and fits(window=64) and fits(dt=0)
    assert fits(d=256) and fits(rows=1 << 21, heads=64, d=64)
    one = dict(heads=1, kv=1, maxc=4096, total=4096)
    assert fits(**one, rows=(1 << 31) - 256) and not fits(**one, rows=(1 << 31) - 255)
    assert fits(**one, d=256, rows=(1 << 30) - 256) and not fits(**one, d=256, rows=(1 << 30) - 255)
    assert fits(**one, dt=0, rows=(1 << 31) - 128) and not fits(**one, dt=0, rows=(1 << 31) - 127)
    # (many requests of short contexts: blocks of 128, one for each request besides)
    assert fits(**one, batch=1024, rows=(1 << 31) - 1024 * 127 - 1)
    assert not fits(**one, batch=1024, rows=(1 << 31) - 1024 * 127)
    assert not fits(rows=1 << 24) and fits(rows=(1 << 24) - 1 - 64)
    few = dict(rows=1000, heads=8)
    assert fits(**few, total=(1 << 26) - 33) and not fits(**few, total=(1 << 26) - 32)
    assert fits(**few, total=1 << 30, maxc=1 << 30, window=100)


def test_reference_of_what_stays():
    """Against sorting by hand; protected ends, ties, NaN and -0."""
    w = np.array([0.0, 5, -0.0, 3, 3, np.nan, 9, 3, 1, 0], np.float32)
    assert E.kept(w, 10, 4, 0, 0) == [1, 3, 4, 6]
    assert E.kept(w, 10, 5, 1, 1) == [0, 1, 3, 6, 9]
    assert E.kept(w, 10, 4, 2, 2) == [0, 1, 8, 9]
    assert E.kept(w, 10, 9, 0, 0) == [0, 1, 2, 3, 4, 6, 7, 8, 9]       # NaN goes first
    assert E.kept(np.zeros(6, np.float32), 6, 3, 0, 1) == [0, 1, 5]
    w = np.array([-1, -np.inf, np.nan, np.inf, -2], np.float32)
    assert [E.kept(w, 5, m, 0, 0) for m in (1, 2, 3, 4)] == [[3], [0, 3], [0, 3, 4], [0, 1, 3, 4]]


def test_reference_weights_sum_to_the_counted_rows():
    rng = np.random.default_rng(0)
    k = rng.standard_normal((20, 2, 64))
    q = rng.standard_normal((4, 6, 64))
    w, tol = E.weights(q, k, 16, 3, 0.1, 0, 0)
    assert np.allclose(w.sum(-1), 9) and w.shape == (2, 20) and not w[:, 19].any()
    assert np.all(tol >= 0) and np.all(tol < 1e-4)


@pytest.mark.parametrize("source,kernels", [
    ("kvprompt.hip", {"8k_prompt": 9, "16k_prompt_prepare": 3, "13k_prompt_join": 6}),
    ("kvbudget.hip", {"9k_weights": 54, "7k_evict": 6, "14k_evict_tables": 1})])
def test_no_kernel_spills(source, kernels, tmp_path):
    flags = [f for f in build.HIPCC_FLAGS if f != "-shared"]
    path = next(s for s in build.SRC if s.endswith(source))
    done = subprocess.run([build.hipcc(), *flags, "-I", build.INC, "--cuda-device-only", "-c", path, "-o",
                           str(tmp_path / "x.o"), "-Rpass-analysis=kernel-resource-usage"],
                          capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]
    found = spills(done.stderr)
    for kernel, count in kernels.items():
        names = [n for n in found if f"{kernel}I" in n or f"{kernel}E" in n]
        assert len(names) == count, (kernel, names)
    assert not {n: v for n, v in found.items() if v != (0, 0)}


def test_direct_loads_to_lds_are_waited_for_before_they_are_shared(tmp_path):
    """Every instance of k_prompt waits for its own loads to LDS, by an instruction of the source,
    right before the barriers that hand the first and each next stage of tiles to the other
    waves: not only where the compiler happens to put a wait."""
    flags = [f for f in build.HIPCC_FLAGS if f != "-shared"]
    path = next(s for s in build.SRC if s.endswith("kvprompt.hip"))
    out = tmp_path / "x.s"
    subprocess.run([build.hipcc(), *flags, "-I", build.INC, "--cuda-device-only", "-S", path, "-o", str(out)],
                   check=True, capture_output=True)
    kernels, name = {}, None
    for line in out.read_text().splitlines():
        text = line.strip()
        if line.startswith("_ZN3svk6prompt8k_promptI"):
            name = line.split(":")[0]
            kernels[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name and (text.startswith(";;#ASM") or text and text[0] not in ".;_" and not text.endswith(":")):
            kernels[name].append(text.split()[0] if text.startswith(";;#ASM") else text)
    assert len(kernels) == 9
    for name, code in kernels.items():
        waits = [i for i in range(1, len(code) - 1) if code[i].startswith("s_waitcnt vmcnt(0)")
                 and code[i - 1] == ";;#ASMSTART" and code[i + 1] == ";;#ASMEND"]
        assert len(waits) >= 2, name
        for at in waits:
            barrier = next(i for i in range(at, len(code)) if code[i].startswith("s_barrier"))
            assert not any("load_lds" in x for x in code[at:barrier]), name
        # a wait behind the first tiles' loads, and one behind the next ones'
        loads = [i for i, x in enumerate(code) if "load_lds" in x]
        between = [i for i in waits if any(l < i for l in loads) and any(l > i for l in loads)]
        assert loads and between and waits[-1] > loads[-1], name
