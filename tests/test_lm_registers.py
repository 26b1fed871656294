"""The tiled products keep their sums in the matrix instructions' registers through the whole K loop and into the
epilogue: an accumulator array that the compiler cannot resolve to registers goes to memory, with results as right
as before and a K loop ten times as slow.  Compiled for gfx950 (no GPU needed) and read from the compiler's kernel
metadata: no kernel has scratch memory or spilled registers."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
@pytest.mark.parametrize("src", ["lm_nt.hip", "lm_nn.hip", "lm_tn.hip", "lm_rows.hip", "lm_small.hip"])
def test_no_scratch_and_no_spills(tmp_path, src):
    out = tmp_path / "kernels.s"
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S",
           os.path.join(ROOT, "allgather_gemm_amd", "csrc", src), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    blocks = out.read_text().split("  - .agpr_count")[1:]
    assert blocks
    for block in blocks:
        value = {k: int(re.search(r"\.%s:\s+(\d+)" % k, block).group(1))
                 for k in ("private_segment_fixed_size", "vgpr_spill_count", "group_segment_fixed_size")}
        name = re.search(r"\.name:\s+(\S+)", block).group(1)
        assert value["private_segment_fixed_size"] == 0 and value["vgpr_spill_count"] == 0, (name, value)
        assert value["group_segment_fixed_size"] <= 160 * 1024, (name, value)
