"""Launch shapes of the kernels over rows of logits (csrc/lm_shape.h), compiled
on the host with stand-ins for the runtime's calls: what is remembered of a
device is that device's, and the shapes follow from its number of SMs."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include "lm_shape.h"

static int device = 0, asked = 0;

extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int d)
{
    ++asked;
    *v = 100 + d;
    return d == 7 ? cudaErrorInvalidDevice : cudaSuccess;
}

int main()
{
    using namespace dpz;
    static PerDevice<3> per;
    const int order[] = {0, 1, 0, 1, 70, 70, 7};
    for (int d : order) {
        device = d;
        int sms = 0;
        const cudaError_t e = sm_count(&sms);
        std::printf("sms %d %d %d %d\n", d, (int)e, sms, asked);
    }
    for (int d = 0; d < 2; ++d)
        for (int key = 0; key < 3; ++key)
            for (int again = 0; again < 2; ++again) {
                device = d;
                int v = 0, calls = 0;
                per.get(key, &v, [&](int dev, int* n) {
                    ++calls;
                    *n = 10 * dev + key + 1;
                    return cudaSuccess;
                });
                std::printf("per %d %d %d %d\n", d, key, v, calls);
            }
    for (int sms : {76, 152})
        for (int T = 1; T <= 700; ++T)
            for (int64_t bytes : {2000, 16384, 16385, 49152, 49153, 100514, 600000, 2400000}) {
                int threads = 0;
                by_row_threads(T, bytes, sms, [&](auto n) { threads = n; return cudaSuccess; });
                std::printf("row %d %d %lld %d %u\n", sms, T, (long long)bytes, threads,
                            row_cluster(T, bytes, threads, sms));
            }
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None or not os.path.isdir(cuda):
        pytest.skip("needs a C++ compiler and the CUDA headers")
    d = tmp_path_factory.mktemp("shape")
    src, exe = d / "shape.cpp", d / "shape"
    src.write_text(PROGRAM)
    subprocess.check_call([cxx, "-std=c++17", "-I", cuda, "-I", os.path.join(ROOT, "include"), "-I",
                           os.path.join(ROOT, "gradient_reduction_zero_gb300", "csrc"), str(src),
                           "-o", str(exe)])
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return [s.split() for s in out.splitlines()]


def test_figures_are_the_devices_own(lines):
    got = [list(map(int, s[1:])) for s in lines if s[0] == "sms"]
    # device, error, SMs, how often the runtime was asked: once per device up to 63
    assert got[:6] == [[0, 0, 100, 1], [1, 0, 101, 2], [0, 0, 100, 2], [1, 0, 101, 2],
                       [70, 0, 170, 3], [70, 0, 170, 4]]
    assert got[6][1] != 0
    per = [list(map(int, s[1:])) for s in lines if s[0] == "per"]
    assert per == [[d, k, 10 * d + k + 1, 1 - again] for d in range(2) for k in range(3)
                   for again in range(2)]


def test_shapes_follow_the_number_of_sms(lines):
    rows = {tuple(map(int, s[1:4])): (int(s[4]), int(s[5])) for s in lines if s[0] == "row"}
    for (sms, T, size), (threads, n) in rows.items():
        assert threads == (256 if T <= 2 * sms or size > 49152 else 64 if size <= 16384 else 128)
        assert n in (1, 2, 4, 8)
        assert n == 1 or T * n <= (2 if size < n * (256 << 10) else 4) * sms
        assert n == 1 or size >= n * threads * 16             # a vector for every thread
        if sms == 152 and T % 2 == 0:                         # half the GPU, half the rows
            assert rows[76, T // 2, size] == (threads, n)
