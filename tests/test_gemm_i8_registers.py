"""The int8 tiles keep their sums in accumulation registers that only the
MFMAs written in assembly touch. Spilled values in the same registers would be
moved between those MFMAs without the distances the hardware needs, so every
instance must have exactly its sums there, and nothing in scratch memory. Asks
the compiler (CPU only)."""

import os
import re
import subprocess

import pytest

from memory_bound_w8a8_amd import build


@pytest.fixture(scope="module")
def usage(tmp_path_factory):
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("registers") / "gemm_i8.o")
    proc = subprocess.run([hipcc, *build.HIPCC_FLAGS, "--offload-device-only", "-c", "-w",
                           "-Rpass-analysis=kernel-resource-usage", os.path.join(build.CSRC, "gemm_i8.hip"), "-o", out],
                          capture_output=True, text=True)
    assert proc.returncode == 0, proc.stderr[-2000:]
    found, name = {}, None
    for line in proc.stderr.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            name = m.group(1)
            found[name] = {}
        m = re.search(r"\s(AGPRs|ScratchSize \[bytes/lane\]): (\d+)", line)
        if m:
            found[name][m.group(1)] = int(m.group(2))
    return found


def test_accumulation_registers_hold_the_sums_alone(usage):
    tiles = {n: u for n, u in usage.items() if "gemm_i8_tiled_kernel" in n}
    assert len(tiles) == 10  # nine tile shapes and the one that splits K
    for name, u in tiles.items():
        bm, bn, wm, wn, _ = (int(x) for x in re.search(r"ILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name).groups())
        assert u["AGPRs"] == (bm // wm) * (bn // wn) // 64, name
        assert u["ScratchSize [bytes/lane]"] == 0, name
