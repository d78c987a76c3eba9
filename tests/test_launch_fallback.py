"""The launch helper against a driver that refuses programmatic dependent launches:
the kernel is launched without the attribute, in its cluster, and the refusal is
remembered; an error of another kind is returned and is not."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

SRC = r"""
#include <cstdio>
#include "k3_launch.cuh"
static int calls, dependent, cluster, refuse, broken;
extern "C" cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *, void **)
{
    calls++, dependent = 0, cluster = 1;
    for (unsigned i = 0; i < c->numAttrs; i++) {
        if (c->attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization) dependent = 1;
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = (int)c->attrs[i].val.clusterDim.x;
    }
    return broken || (refuse && dependent) ? cudaErrorInvalidValue : cudaSuccess;
}
extern "C" cudaError_t cudaGetLastError() { return cudaSuccess; }
namespace k3 {
static int noted;
void note_weight_writes(cudaStream_t) noexcept { noted++; }
bool weights_settled(cudaStream_t s) noexcept { return s == nullptr; }
}
static void one(int) {}
static void two(long) {}
static void three(float) {}
#define CHECK(x) if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; }
int main()
{
    using namespace k3;
    const dim3 g(8), b(32);
    CHECK(launch_dependent(true, 2, one, g, b, 0, nullptr, 1) == cudaSuccess && calls == 1 && dependent && cluster == 2);
    broken = 1, calls = 0;
    CHECK(launch_dependent(true, 2, one, g, b, 0, nullptr, 1) != cudaSuccess && calls == 2);
    broken = 0, calls = 0;
    CHECK(launch_dependent(true, 4, one, g, b, 0, nullptr, 1) == cudaSuccess && calls == 1 && dependent && cluster == 4);
    CHECK(launch_dependent(false, 4, one, g, b, 0, nullptr, 1) == cudaSuccess && !dependent && cluster == 4);
    refuse = 1, calls = 0;
    CHECK(launch_dependent(true, 8, two, g, b, 0, nullptr, 1L) == cudaSuccess && calls == 2 && !dependent && cluster == 8);
    calls = 0;
    CHECK(launch_dependent(true, 8, two, g, b, 0, nullptr, 1L) == cudaSuccess && calls == 1 && !dependent && cluster == 8);
    refuse = 0;
    CHECK(launch_pdl_weights(three, g, b, 0, nullptr, 1.f) == cudaSuccess && dependent && cluster == 1);
    CHECK(launch_pdl_weights(three, g, b, 0, (cudaStream_t)8, 1.f) == cudaSuccess && !dependent);
    CHECK(launch_pdl(three, g, b, 0, (cudaStream_t)8, 1.f) == cudaSuccess && dependent && noted == 0);
    // a launch that failed behind a writer leaves its note for the next
    broken = 1;
    CHECK(launch_pdl_weights(three, g, b, 0, nullptr, 1.f) != cudaSuccess && noted == 0);
    CHECK(launch_pdl_weights(three, g, b, 0, (cudaStream_t)8, 1.f) != cudaSuccess && noted == 1);
    puts("ok");
    return 0;
}
"""


def test_a_refused_attribute(tmp_path):
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    if not os.path.exists(nvcc) and shutil.which(nvcc) is None:
        pytest.skip("no nvcc")
    src, exe = tmp_path / "launch.cpp", tmp_path / "launch"
    src.write_text(SRC)
    csrc = os.path.join(ROOT, "mxfp4_routed_expert_select_gb300", "csrc")
    subprocess.run([nvcc, "-std=c++17", "-cudart", "none", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
