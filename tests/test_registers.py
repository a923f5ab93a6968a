"""Registers that grids count on, as the assembler reports them; no GPU."""
import os
import re
import subprocess

from tile_signaled_grouped_gb300 import build as B

SM_REGISTERS = 65536


def registers(source, kernel):
    """{mangled template arguments: registers a thread} of the kernels of that name in a source."""
    out = subprocess.run([B.nvcc(), *B._flags(()), "-Xptxas=-v", "-c", os.path.join(B.CSRC, source), "-o", os.devnull],
                         capture_output=True, text=True, check=True).stderr
    return {m[1]: int(m[2]) for m in re.finditer(
        rf"Compiling entry function '\S*{kernel}I(\w+?)EEEv\S*'.*?Used (\d+) registers", out, re.S)}


def test_eight_ctas_of_the_gradient_by_columns_fit_an_sm():
    """dz and db of features that are no multiple of 8: the ranges of rows are cut for eight CTAs of 256 threads
    an SM. With fewer there is a second wave, and twice the time."""
    found = registers("linear.cu", "act_grad_kernel")
    # act, vectors, z in 8 bits, x restored beside
    plain = {k: v for k, v in found.items() if k.endswith("ELb0ELb0ELb0")}
    assert len(plain) == 5, found
    for k, v in plain.items():
        assert -(-v // 8) * 8 * 256 * 8 <= SM_REGISTERS, (k, v)
