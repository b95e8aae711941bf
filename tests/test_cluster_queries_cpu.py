"""CPU: how often the host code asks the driver how many clusters run at once, and what it keeps of the answers:
csrc/host_common.cuh compiled by g++ on a runtime of fakes."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

PROGRAM = r"""
#include <utility>
#include "host_common.cuh"

static int queries, device, answer = 148;  // answer: SMs that clusters may take; < 0: every query fails
static bool fail_large;                    // queries of clusters above 8 fail
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return ""; }
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *c) {
    ++queries;
    const int cl = (int)c->attrs[0].val.clusterDim.x;
    if (answer < 0 || (fail_large && cl > 8)) return cudaErrorUnknown;
    *n = answer / cl;
    return cudaSuccess;
}
}
static char kernels[80];

#define EXPECT(x) do { if (!(x)) { printf("line %d: %s (queries %d)\n", __LINE__, #x, queries); return 1; } } while (0)
int main() {
    using namespace q8;
    auto find = [](int slot, int64_t n) { return cluster_for(slot, n, kernels + slot, 512, 1000, 148, 16, 1); };
    // a failed query is asked again, and its answer not kept
    answer = -1;
    EXPECT(find(0, 1) == 1 && max_active_clusters(kernels, 1, 1, 2) == 0);
    answer = 148;
    EXPECT(find(0, 1) == 16 && max_active_clusters(kernels, 1, 1, 2) == 74);
    fail_large = true;
    EXPECT(find(1, 2) == 8);
    fail_large = false;
    EXPECT(find(1, 2) == 16);
    // every slot and batch on four devices: asked once each, and none of it in the planners' cache
    for (device = 0; device < 4; ++device)
        for (int slot = 0; slot < 4; ++slot)
            for (int n = 1; n <= 160; ++n) find(slot, n);
    queries = 0;
    for (device = 0; device < 4; ++device)
        for (int slot = 0; slot < 4; ++slot)
            for (int n = 1; n <= 160; ++n) EXPECT(find(slot, n) == (n > 148 ? 1 : 148 / n < 16 ? 148 / n : 16));
    EXPECT(queries == 0);
    device = 0;
    EXPECT(find(0, 161) == 1 && cluster_for(0, 16, kernels, 512, 1000, 148, 16, 4) == 9 && queries == 0);
    for (int pass = 0; pass < 2; ++pass)
        for (int i = 1; i < 60; ++i) EXPECT(max_active_clusters(kernels + i, 256, 4096, 4) == 37);
    EXPECT(queries == 59);
    return 0;
}
"""


def test_cluster_sizes_are_found_once_and_leave_the_planners_cache_alone(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA headers not available")
    src, exe = tmp_path / "queries.cpp", tmp_path / "queries"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-I", os.path.join(ROOT, "q8_block_quantized_02_b200", "csrc"), "-I",
                    os.path.join(CUDA, "include"), "-Wl,--unresolved-symbols=ignore-all", "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
