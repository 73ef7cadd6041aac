"""Kernels are configured per device (CPU): the launchers' helper against a fake of the calls that it makes.

csrc/kvc_configured.cuh is compiled as host code with the runtime's three calls replaced; two devices that hold
different numbers of CTAs, one that refuses the query, and none at all."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "paged_kv_cache_kvc_gb300", "csrc", "kvc_configured.cuh")

PROGRAM = r"""
#include <cstdio>
#include <cuda_runtime.h>
static int device = 0, queries = 0;
static const int holds[3] = {3, 5, -1};
static cudaError_t fake_get_device(int *d) { *d = device; return device < 0 ? cudaErrorNoDevice : cudaSuccess; }
static cudaError_t fake_set(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
static cudaError_t fake_occupancy(int *n, const void *, int, size_t)
{
    ++queries;
    *n = holds[device];
    return holds[device] < 0 ? cudaErrorInvalidValue : cudaSuccess;
}
#define cudaGetDevice fake_get_device
#define cudaFuncSetAttribute fake_set
#define cudaOccupancyMaxActiveBlocksPerMultiprocessor fake_occupancy
#include "%s"
struct A {};
struct B {};
int main()
{
    const int order[] = {1, 0, 1, 2, 0, 2, -1};
    for (int d : order) {
        device = d;
        const kvc::DecodeKernel k = kvc::configured<A>(&device, 64, 288, false);
        printf("%%d %%d %%d\n", k.fn != nullptr, k.ctas_per_sm, k.threads);
    }
    printf("%%d\n", queries);
    device = 0;
    kvc::configured<B>(&queries, 0, 32, true);   // another kernel asks for itself
    printf("%%d\n", queries);
    return 0;
}
"""


def test_each_device_has_its_own_configuration(tmp_path):
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    nvcc = nvcc if os.path.exists(nvcc) else shutil.which("nvcc")
    if not nvcc:
        pytest.skip("nvcc not available")
    (tmp_path / "conf.cu").write_text(PROGRAM % HEADER)
    subprocess.check_call([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr",
                           "-I" + os.path.join(ROOT, "include"), "-o", str(tmp_path / "conf"), str(tmp_path / "conf.cu")], cwd=tmp_path)
    out = subprocess.check_output([str(tmp_path / "conf")], text=True).splitlines()
    rows = [tuple(map(int, line.split())) for line in out[:7]]
    assert [r[1] for r in rows] == [5, 3, 5, 0, 3, 0, 0]   # a refused query is no configuration, and no device none
    assert [r[0] for r in rows] == [1, 1, 1, 1, 1, 1, 0] and all(r[2] == 288 for r in rows[:6])
    assert out[7:] == ["3", "4"]                           # asked once a device and kernel
