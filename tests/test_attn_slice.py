"""The slices of attn_cache_evict's warps, walked on the host."""
import os
import subprocess

from block_scaled_fp4_softmax_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_slices_on_host(tmp_path):
    """csrc/attn_slice.h for lengths up to the largest by tests/attn_slice_check.cu."""
    exe = tmp_path / "attn_slice_check"
    cmd = [build._nvcc(), "-std=c++17", "-O2", "-gencode", "arch=compute_103a,code=sm_103a", "-I", build.CSRC, "-o", str(exe),
           os.path.join(HERE, "attn_slice_check.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and ", 0 failed" in r.stdout, r.stdout[-3000:]


def test_the_kernel_takes_its_slots_from_there():
    """No loop of the selection over slots steps past its slice by a whole cluster's
    threads: near the largest length that sum does not fit an int."""
    text = open(os.path.join(build.CSRC, "attn_evict.cu")).read()
    select = text[text.index("select_kernel("):text.index("constexpr int kMoveThreads")]
    assert "C * kThreads" not in select
    assert "slice_begin" in select
    # nor is a slice's size or end formed anywhere else
    assert "j0 + sub" not in text and "* sub" not in select.replace("warp * sub;", "") and "+ 127" not in text
