"""Facts about the compiled kernels that the launches rest on, from the
assembler's own report (no GPU)."""
import os
import re
import subprocess

from denoise_step_token_gb300 import _build


def test_tile_kernels_have_the_registers_they_share_out(tmp_path):
    """kv4_tile_kernel shares out 128 registers per thread between its warps, and
    its launch refuses any other number: a compiler that gives it fewer takes
    attention of more than 32 rows away, and is noticed here."""
    src = os.path.join(_build.CSRC, "kv4_tile.cu")
    run = subprocess.run([_build.nvcc_path(), *_build.ARCH_FLAGS, *_build.NVCC_FLAGS, "-Xptxas", "-v", "-c", src, "-o",
                          str(tmp_path / "kv4_tile.o")], capture_output=True, text=True, check=True)
    found = re.findall(r"Compiling entry function '\S*?(kv4_\w+?_kernel)I\S*'.*?Used (\d+) registers",
                       run.stdout + run.stderr, re.S)
    tile = [int(regs) for name, regs in found if name.endswith("kv4_tile_kernel")]
    assert tile == [128] * 4, found
