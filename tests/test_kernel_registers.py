"""The cache kernels keep their values in registers: no vector register is spilled.

A spill is more than slow here.  hipcc 7.2.0 (clang 22.0.0git, roc-7.2.0) parts the four
words of an operand that it spills between scratch and accumulation registers, and in
an attention kernel of 32 rows at D=256 with two tiles on their way it stored all four
words of a query operand and reloaded three: the second row tile of every request came
out wrong, the same way each time, with no warning."""

import re
import subprocess

import pytest

from lossless_rejection_sampling_spec_amd import build


def spills(remarks: str) -> dict:
    """Per kernel what the compiler's resource remarks say: (scratch bytes, spilled VGPRs)."""
    found, name = {}, None
    for line in remarks.splitlines():
        if m := re.search(r"Function Name: (\S+)", line):
            name = m.group(1)
            found[name] = [None, None]
        elif m := re.search(r"ScratchSize \[bytes/lane\]: (\d+)", line):
            found[name][0] = int(m.group(1))
        elif m := re.search(r"VGPRs Spill: (\d+)", line):
            found[name][1] = int(m.group(1))
    return {k: tuple(v) for k, v in found.items()}


@pytest.mark.parametrize("source,kernels", [("kvattn.hip", {"k_attn": 41, "k_attn_join": 13,
                                                            "k_attn_join_rows": 13,
                                                            "k_attn_plan": 1}),
                                            ("kvcache.hip", {"k_append": 6})])
def test_no_cache_kernel_spills(source, kernels, tmp_path):
    flags = [f for f in build.HIPCC_FLAGS if f != "-shared"]
    path = next(s for s in build.SRC if s.endswith(source))
    done = subprocess.run([build.hipcc(), *flags, "-I", build.INC, "--cuda-device-only", "-c", path, "-o",
                           str(tmp_path / "x.o"), "-Rpass-analysis=kernel-resource-usage"],
                          capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]
    found = spills(done.stderr)
    for kernel, count in kernels.items():
        names = [n for n in found if f"svk{len(kernel)}{kernel}I" in n or f"svk{len(kernel)}{kernel}E" in n]
        assert len(names) == count, (kernel, names)
    assert not {n: v for n, v in found.items() if v != (0, 0)}


def test_the_remarks_of_a_kernel_that_spills_are_found():
    text = """x.hip:1:0: remark: Function Name: _ZN3svk6k_attnILi256E [-Rpass-analysis=kernel-resource-usage]
x.hip:1:0: remark:     VGPRs: 256 [-Rpass-analysis=kernel-resource-usage]
x.hip:1:0: remark:     ScratchSize [bytes/lane]: 400 [-Rpass-analysis=kernel-resource-usage]
x.hip:1:0: remark:     SGPRs Spill: 3 [-Rpass-analysis=kernel-resource-usage]
x.hip:1:0: remark:     VGPRs Spill: 113 [-Rpass-analysis=kernel-resource-usage]
"""
    assert spills(text) == {"_ZN3svk6k_attnILi256E": (400, 113)}
