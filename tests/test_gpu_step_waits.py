"""Calls launched dependently behind a kernel that lets them start and then runs for longer
than their waits' limit (2 s): the limit counts from that kernel's end."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

# One thread that sleeps in steps of at most a millisecond until `ns` have passed (64 ns at least a step: it ends).
SOURCE = """
#include <cuda_runtime.h>
__global__ void pause_kernel(unsigned long long ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    for (long long i = 0; i < 100000000; ++i) {
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (t - t0 > ns) break;
        __nanosleep(1000000);
    }
}
extern "C" int pause_launch(unsigned long long ns, void* stream) {
    pause_kernel<<<1, 1, 0, (cudaStream_t)stream>>>(ns);
    return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_weight_quantized_w4a8_gb300 as m
    m.build()
    assert m.w4a8_device_error() == 0
    return m


@pytest.fixture(scope="module")
def pause(tmp_path_factory):
    d = tmp_path_factory.mktemp("pause")
    (d / "pause.cu").write_text(SOURCE)
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    nvcc = nvcc if os.path.exists(nvcc) else shutil.which("nvcc")
    so = str(d / "pause.so")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static",
                    "-o", so, str(d / "pause.cu")], check=True)
    f = ctypes.CDLL(so).pause_launch
    f.argtypes, f.restype = [ctypes.c_ulonglong, ctypes.c_void_p], ctypes.c_int

    def call():
        assert f(2_400_000_000, torch.cuda.current_stream().cuda_stream) == 0

    call()
    torch.cuda.synchronize()
    return call


@pytest.mark.parametrize("M,K,N", [(1, 3584, 512), (2, 4096, 9000), (40, 2048, 300), (100, 512, 256), (300, 512, 9000)])
def test_f8_linear_behind_a_long_kernel(w4, pause, M, K, N):
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).cuda()
    w = w4.f8_quantize_weights(torch.from_numpy((0.05 * rng.standard_normal((N, K))).astype(np.float32)).cuda())
    want = w4.f8_linear(x, *w)
    y = torch.zeros_like(want)
    ws = torch.empty(w4.f8_linear_workspace_bytes(M, K, N), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    pause()
    w4.f8_linear(x, *w, Y=y, ws=ws, flags=w4.LAUNCH_PDL)
    assert w4.w4a8_device_error() == 0
    assert torch.equal(y, want)


@pytest.mark.parametrize("M,K,N", [(16, 3584, 512), (40, 18944, 300), (64, 4096, 4096)])
def test_w4a8_linear_behind_a_long_kernel(w4, pause, M, K, N):
    """The tensor-core kernel, whose weights' way through its stages waits for the activation's."""
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float16)).cuda()
    w = w4.w4_quantize_weights(torch.from_numpy((0.05 * rng.standard_normal((N, K))).astype(np.float32)).cuda())
    assert w4.w4a8_plan_info(M, K, N)["kernel"] == 1
    ws = torch.zeros(w4.w4a8_workspace_bytes(M, K, N), dtype=torch.uint8, device="cuda")
    want = w4.w4a8_linear(x, *w, ws=ws)
    y = torch.zeros_like(want)
    torch.cuda.synchronize()
    pause()
    w4.w4a8_linear(x, *w, Y=y, ws=ws, flags=w4.LAUNCH_PDL)
    assert w4.w4a8_device_error() == 0
    assert torch.equal(y, want)
