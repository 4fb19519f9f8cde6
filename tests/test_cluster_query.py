"""rowops_add_rmsnorm_bwd where the runtime cannot say how many clusters run at once."""
import ctypes
import os
import subprocess

from row_wise_softmax_warp_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_failed_query_is_no_failed_launch(tmp_path):
    """The call goes on with the grid that its sizes give: both kernels are launched, and no error is left for others."""
    out = str(tmp_path / "probe.so")
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-Xptxas", "-O0", "-Xcicc", "-O1", "-I", build.CSRC, "-shared", "-o", out,
                    os.path.join(HERE, "csrc", "cluster_query_probe.cu")], check=True, capture_output=True)
    got = (ctypes.c_int * 4)()
    ctypes.CDLL(out).run_cluster_query_probe(got)
    assert list(got) == [0, 2, 152, 0]  # 76 clusters of two
