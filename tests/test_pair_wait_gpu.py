"""The bounded wait of a pair of CTAs: where it gives up in one, both know, so
that neither stores sums that the other's wait had to vouch for."""
import os
import subprocess

import pytest

from softmax_cross_entropy_pass_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


def compiled(path):
    cmd = [_build._nvcc()] + _build.ARCH + _build.NVCC_FLAGS + [os.path.join(HERE, "pair_wait.cu"), "-o", str(path)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(path)


@pytest.mark.gpu
def test_a_wait_that_gives_up_is_known_in_both_ctas(tmp_path):
    r = subprocess.run([compiled(tmp_path / "pair_wait")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0
    assert r.stdout.split("\n")[:3] == ["1 1", "1 1", "0 0"]


def test_pair_kernel_waits_for_both():
    """No wait of the 8-bit product's pair kernel, but for the drains at its end, keeps to its own CTA's flag."""
    with open(os.path.join(_build.CSRC, "fp8_gemm.cu")) as f:
        text = f.read()
    kernel = text[text.index("fp8_pair_kernel(const __grid_constant__"):text.index("cudaError_t allow_smem")]
    alone = [line for line in kernel.split("\n") if "mbar_wait_polled" in line or "mbar_wait_bounded" in line]
    assert kernel.count("mbar_wait_pair(") == 4
    assert all("drain_abort" in line for line in alone), alone


@pytest.mark.parametrize("name,commit", [("fp8_few_kernel(const", "mma_commit(smem_u32(&done))"),
                                         ("fp8_pair_kernel(const", "mma_commit_pair_mc(smem_u32(&done), 0x1)")])
def test_products_wait_for_their_mmas_before_they_leave(name, commit):
    """Tensor memory is given back behind a wait of the issuer for all of its MMAs: an epilogue whose own waits gave
    up may be there first."""
    with open(os.path.join(_build.CSRC, "fp8_gemm.cu")) as f:
        text = f.read()
    kernel = text[text.index(name):]
    end = kernel.index("tmem_dealloc")
    at = kernel.index(commit)
    wait = kernel.index("mbar_wait_polled(smem_u32(&done), 0, &drain_abort[1])")
    assert kernel.rindex("mma_e4m3", 0, end) < at < wait < kernel.rindex("__syncthreads", 0, end) < end
