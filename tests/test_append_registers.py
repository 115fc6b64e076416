"""The append kernels of calls without norms keep their rows in registers (CPU: what the
compiler reports when it builds them)."""
import os
import re
import subprocess

import pytest

from speculative_decoding_verify_split_gb300 import build


@pytest.fixture(scope="module")
def spills(tmp_path_factory):
    """(kind of cache, interleaved rotation, with norms) -> bytes of spill stores and loads."""
    cmd = [build.nvcc(), *build.ARCH, *build.COMMON, "-Xptxas", "-v", "-c", os.path.join(build.CSRC, "va_append.cu"), "-o",
           str(tmp_path_factory.mktemp("append") / "va_append.o")]
    text = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    found = re.findall(r"Compiling entry function '\w*?16va_append_kernelILi(\d)ELb(\d)ELb(\d)E.*?(\d+) bytes spill stores, (\d+) bytes spill loads", text,
                       re.S)
    return {tuple(map(int, f[:3])): tuple(map(int, f[3:])) for f in found}


@pytest.mark.parametrize("kind,interleaved,most", [
    (0, 0, (0, 0)), (0, 1, (0, 0)), (1, 0, (0, 0)), (1, 1, (0, 0)),     # bf16, e4m3
    (2, 0, (56, 28)), (2, 1, (16, 8)),                                  # page scales: older tokens' codes beside the rows
])
def test_spills_without_norms(spills, kind, interleaved, most):
    assert len(spills) == 12
    assert all(got <= allowed for got, allowed in zip(spills[kind, interleaved, 0], most)), spills
