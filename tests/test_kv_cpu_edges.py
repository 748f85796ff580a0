"""CPU tests of the cache calls' return codes and sizes at the ends of what they accept."""

import pytest

torch = pytest.importorskip("torch")

import test_kv_cpu as C  # noqa: E402


def test_a_misaligned_workspace_has_the_code_the_header_states():
    for off in (1, 4, 8):
        assert C._attention(maxc=100000, ws=C.F + off) == 1
        assert C._reserve(ws=C.F + off) == 2
        assert C._compact(ws=C.F + off) == 2
    for call in (C._reserve, C._compact):
        assert call(ws=None) == 1
    assert C._attention(maxc=100000, ws=None) == 1


def _workspace(dtype, batch, k, heads, kv, d, bound, window=0, sinks=0):
    return C.binding.lib().spec_kv_attention_workspace_bytes(dtype, batch, k, heads, kv, d, bound, window,
                                                             sinks)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,kv", [(8, 8), (32, 8), (64, 8), (64, 1), (128, 128)])
@pytest.mark.parametrize("k", [0, 6, 63])
def test_the_attention_workspace_stops_growing_with_the_bound(dtype, d, heads, kv, k):
    """512 MiB, or 8 places per request, KV head and block of rows (at most 16 rows more
    than there are), and 32 bytes per place for the plan."""
    per = (d + 2) * 4 * 64 + 32
    for batch in (1, 7, 64, 256, 1024):
        blocks = batch * kv * -(-(k + 1) * (heads // kv) // 16)
        most = max((512 << 20) * 1.02, 8 * blocks * per) + 64
        sizes = [_workspace(dtype, batch, k, heads, kv, d, 1 << s) for s in (5, 10, 14, 17, 20, 24, 30)]
        assert all(0 < x <= most for x in sizes), (batch, sizes)
    # the sizes the header names
    assert _workspace(1, 256, 6, 32, 8, 128, 1 << 17) < 500 << 20
    assert _workspace(1, 1024, 6, 32, 8, 128, 1 << 17) < 1050 << 20


def test_a_call_of_more_workgroups_than_a_launch_takes_is_refused():
    big = dict(batch=1024, max_k=63, heads=1024, kv=1024, d=256, ldq=1 << 18, ldo=1 << 18, rows=1024)
    assert _workspace(0, 1024, 63, 1024, 1024, 256, 1 << 20) == 0
    assert C._attention(dt=0, maxc=1 << 20, **big) == 2


def test_page_bytes_of_sizes_past_32_bits():
    assert C.binding.kv_page_bytes(2, 128, 16) == 2 * 16 * 136
    for i in range(3):
        sizes = [2, 128, 16]
        sizes[i] += 1 << 32
        assert C.binding.kv_page_bytes(*sizes) == 0
