"""The recurrence of gated_delta_prefill moves registers between its warpgroups, and the entry point refuses a
build whose kernels do not hold exactly the number that the shares add up to: this build has it."""
import os
import re
import subprocess


def test_recurrence_registers(tmp_path):
    from bit_quantized_linear_q8_gb300 import build
    src = os.path.join(build.CSRC, "gated_delta_prefill.cu")
    with open(src) as f:
        want = int(re.search(r"constexpr int GC_REGS = (\d+);", f.read()).group(1))
    r = subprocess.run([build._nvcc(), "-c", src, "-o", str(tmp_path / "x.o"), "-Xptxas", "-v"] + build.NVCC_FLAGS,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    used = re.findall(r"Compiling entry function '(\S*gated_delta_recur_kernel\S*)'.*?Used (\d+) registers", r.stdout + r.stderr,
                      re.DOTALL)
    assert len(used) == 2, r.stderr
    assert all(int(n) == want for _, n in used), used
