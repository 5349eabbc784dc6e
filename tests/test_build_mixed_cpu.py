"""Register budgets of the AdamW, norm and conversion kernels, checked on the CPU
with ptxas (no GPU needed): each gets few enough registers for the thread
blocks per SM that its grid is sized for, and the AdamW kernel does not
spill."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "muon_optimizer_step_02_b200", "csrc")


def _constant(name):
    text = "".join(open(os.path.join(CSRC, f)).read()
                   for f in ("k_adamw_mixed.cuh", "k_grad_norm.cuh"))
    return int(re.search(rf"\b{name} = (\d+)", text).group(1))


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc is not available")
    out = tmp_path_factory.mktemp("ptxas") / "mixed_api.o"
    res = subprocess.run(
        [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17",
         "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-Xptxas", "-v",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", "-o", str(out),
         os.path.join(CSRC, "mixed_api.cu")], capture_output=True, text=True, timeout=900)
    assert res.returncode == 0, res.stderr[-3000:]
    return res.stdout + res.stderr


@pytest.mark.parametrize("kernel, threads, resident", [
    ("adamw_mixed_kernel", "kMixThreads", "kMixResident"),
    ("grad_norm_kernel", "kNormThreads", "kNormResident"),
    ("adam8_write_kernel", "kMixThreads", "kA8WriteResident"),
    ("adam8_read_kernel", "kMixThreads", "kA8ReadResident")])
def test_registers_leave_room_for_the_grid(report, kernel, threads, resident):
    found = re.findall(rf"Function properties for _Z\w*{kernel}\w*\s*\n"
                       r"\s*\d+ bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill "
                       r"loads\s*\n.*?Used (\d+) registers", report)
    assert len(found) >= 2      # a short and a long tensor table at least
    for stores, loads, used in found:
        per_thread = -(-int(used) // 8) * 8      # registers are given out in eights
        assert per_thread * _constant(threads) * _constant(resident) <= 65536
        if kernel == "adamw_mixed_kernel":
            assert (stores, loads) == ("0", "0")


def test_tables_fit_the_kernel_parameters():
    """The limit is 32,764 bytes; each kernel's table and its scalars."""
    assert _constant("kMixMaxSegs") * 76 + 4 + 62 * 8 + 200 <= 32764
    assert _constant("kNormMaxSegs") * 20 + 64 <= 32764
    assert _constant("kA8MaxSegs") * 52 + 64 <= 32764
