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
