"""Register and local-memory budget of the kernels around the linears of a
served block, from the compiler's own report (CPU): norms and rotary append
must not spill; the attention kernel is launched with 96 registers a thread,
which its roles share out, and may keep a few values in local memory."""
import os
import shutil
import subprocess

import pytest

from test_kernel_resources import CSRC, entries, nvcc_flags


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = tmp_path_factory.mktemp("ptxas")
    procs = [subprocess.Popen([nvcc] + nvcc_flags() + ["-Xptxas", "-v", "-c", os.path.join(CSRC, src), "-o",
                                                       str(out / (src + ".o"))],
                              stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for src in ("norm.cu", "rope_append.cu", "chunk_attention.cu")]
    logs = []
    for p in procs:
        log, _ = p.communicate(timeout=900)
        assert p.returncode == 0, log[-2000:]
        logs.append(log)
    return entries("\n".join(logs))


def test_norms_and_append_do_not_spill(report):
    seen = [e for e in report if "residual_norm" in e[0] or "rope_append" in e[0] or "combine" in e[0]]
    assert len(seen) >= 22
    for name, _, stores, loads in seen:
        assert (stores, loads) == (0, 0), name


def test_staying_norms_fill_an_sm(report):
    seen = [e for e in report if "residual_norm_stay" in e[0]]
    assert len(seen) == 4
    for name, regs, _, _ in seen:
        assert regs * 512 <= 65536, name          # 512 threads an SM


def test_attention_kernel(report):
    seen = [e for e in report if "chunk_attn_kernel" in e[0]]
    assert len(seen) == 2
    for name, regs, stores, loads in seen:
        assert regs == 96, name                    # 640 threads: 5 x 96 = 2 x 136 + 2 x 80 + 48
        assert stores <= 32 and loads <= 64, name
