"""The optimiser's roots and reciprocals (csrc/roots.cuh) at every float of the
ranges that they are for, against CUDA's correctly rounded functions."""
import ctypes
import os
import subprocess

import pytest
import torch

from transformer_xl_relative_rel_gb300 import _build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "roots.cuh"
using namespace txl;

// bad[0]: how many of the floats with the bits first .. last differ; bad[1]: one of them
__device__ void compare(float got, float want, uint32_t bits, unsigned long long *bad)
{
    if (__float_as_uint(got) == __float_as_uint(want)) return;
    atomicAdd(bad, 1ull);
    atomicExch(bad + 1, (unsigned long long)bits);
}

__global__ void reciprocals(uint32_t first, uint32_t last, unsigned long long *bad)
{
    for (uint64_t i = first + (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i <= last; i += (uint64_t)gridDim.x * blockDim.x)
        compare(exact_reciprocal(__uint_as_float((uint32_t)i)), __frcp_rn(__uint_as_float((uint32_t)i)), (uint32_t)i, bad);
}

// each float by itself, beside one far from it
__global__ void pairs(uint32_t first, uint32_t last, unsigned long long *bad)
{
    for (uint64_t i = first + (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i <= last; i += (uint64_t)gridDim.x * blockDim.x) {
        const float x = __uint_as_float((uint32_t)i), y = __uint_as_float(first + (last - (uint32_t)i));
        float a, b;
        unpair(pair_sqrt(pair(x, y)), a, b);
        compare(a, __fsqrt_rn(x), (uint32_t)i, bad);
        compare(b, __fsqrt_rn(y), __float_as_uint(y), bad);
    }
}

// eight neighbours, the last of them replaced by `other`
__global__ void eights(uint32_t first, uint32_t last, float other, unsigned long long *bad)
{
    for (uint64_t i = first + 8 * ((uint64_t)blockIdx.x * blockDim.x + threadIdx.x); i + 7 <= last;
         i += 8 * (uint64_t)gridDim.x * blockDim.x) {
        float x[8];
        uint64_t v[4], root[4];
        for (int j = 0; j < 8; ++j) x[j] = j == 7 && other >= 0.f ? other : __uint_as_float((uint32_t)i + j);
        for (int k = 0; k < 4; ++k) v[k] = pair(x[2 * k], x[2 * k + 1]);
        eight_sqrt(v, root);
        for (int k = 0; k < 4; ++k) {
            float a, b;
            unpair(root[k], a, b);
            compare(a, __fsqrt_rn(x[2 * k]), __float_as_uint(x[2 * k]), bad);
            compare(b, __fsqrt_rn(x[2 * k + 1]), __float_as_uint(x[2 * k + 1]), bad);
        }
    }
}

extern "C" int run(int which, uint32_t first, uint32_t last, float other, void *bad, void *stream)
{
    cudaStream_t s = (cudaStream_t)stream;
    unsigned long long *b = (unsigned long long *)bad;
    if (which == 0) reciprocals<<<1216, 256, 0, s>>>(first, last, b);
    else if (which == 1) pairs<<<1216, 256, 0, s>>>(first, last, b);
    else eights<<<1216, 256, 0, s>>>(first, last, other, b);
    return (int)cudaGetLastError();
}
"""

BITS = lambda e: (127 + e) << 23      # of 2^e
INFINITY = 0x7f800000


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    at = tmp_path_factory.mktemp("roots")
    src, lib = os.path.join(at, "roots.cu"), os.path.join(at, "roots.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    cmd = [_build.nvcc(), *_build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", _build.CSRC, "-o", lib, src]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    f = ctypes.CDLL(lib).run
    f.argtypes = [ctypes.c_int, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]

    def call(which, first, last, other=-1.0):
        bad = torch.zeros(2, dtype=torch.int64, device="cuda")
        assert f(which, first, last, other, bad.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        n, bits = bad.tolist()
        assert n == 0, f"{n} differ, {bits:#x} for one"
    return call


def test_reciprocals(run):
    """A block's largest moment: from 2^-100 to below 2^126."""
    run(0, BITS(-100), BITS(126) - 1)


def test_roots_of_pairs(run):
    """From 2^-100 to the largest number, and 0."""
    run(1, BITS(-100), INFINITY - 1)
    run(1, 0, 0)


@pytest.mark.parametrize("other", [-1.0, 0.0, 1.0, 1e-40, 3e38, float("inf")])
def test_roots_of_eight(run, other):
    """Every number from 0 to infinity, beside its neighbours, and beside one
    that may take the eight the other way."""
    run(2, 0, INFINITY - 1, other)
    run(2, 1, INFINITY, other)
