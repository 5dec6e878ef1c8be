"""The bounded waits of the kernels (csrc/barrier.cuh): a wait that nothing ends gives up and is reported, one whose
copy has arrived does not."""
import ctypes
import os
import subprocess

import pytest

from bit_plane_key_b200 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def waits():
    """tests/waits.cu as a library, built again when it or a header is newer."""
    src, lib = os.path.join(HERE, "waits.cu"), os.path.join(HERE, "_build", "libwaits.so")
    deps = [src, os.path.join(B.CSRC, "barrier.cuh"), os.path.join(B.CSRC, "fathom_internal.cuh"), os.path.join(B.INCLUDE, "fathom.h")]
    if not os.path.exists(lib) or any(os.path.getmtime(p) > os.path.getmtime(lib) for p in deps):
        os.makedirs(os.path.dirname(lib), exist_ok=True)
        tmp = lib + ".tmp%d" % os.getpid()
        subprocess.check_call([B.NVCC] + B.NVCC_FLAGS + ["-shared", src, "-o", tmp])
        os.replace(tmp, lib)
    return lib


def test_the_waits_compile_by_themselves(waits):
    assert os.path.exists(waits)


@pytest.mark.gpu
@pytest.mark.parametrize("nothing", [0, 1])
def test_a_wait_ends_and_reports(waits, nothing):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from bit_plane_key_b200 import fathom as F
    L = ctypes.CDLL(waits)
    out = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert L.waits_run(nothing, ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(status.data_ptr())) == 0
    torch.cuda.synchronize()
    assert out.tolist() == [nothing, 0, 0, 0]
    assert status.item() == (F.DEV_TIMEOUT if nothing else 0)
