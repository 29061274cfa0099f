"""Refusals, sizes and builds of code lookup, group norm and AdamW at the ends of their ranges, on the host (no GPU needed)."""
import ctypes as C
import os
import re
import shutil
import subprocess
import sys
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from gaussian_splatting_gb300 import _native as N  # noqa: E402

P = 1 << 30  # an address that is never followed: the checks come first


@pytest.fixture(scope="module")
def lib():
    from gaussian_splatting_gb300 import build
    build.build()
    return N.load()


# arrays of a tensor of 1,000 values: their bytes with 32-bit and with 8-bit moments
ARRAYS = {"param": (4000, 4000), "grad": (4000, 4000), "exp_avg": (4000, 1000), "exp_avg_sq": (4000, 1000),
          "exp_avg_scale": (0, 16), "exp_avg_sq_scale": (0, 16), "copy": (2000, 2000)}


def _tensors(bits, apart):
    """Three tensors, arrays 8 KB from each other: tensor by tensor (the last one first), or each kind `apart` from the others."""
    out, at = [N.AdamWTensor(n=1000, lr=1e-3) for _ in range(3)], P
    kinds = [(k, t) for k in ARRAYS for t in out] if apart else [(k, t) for t in reversed(out) for k in ARRAYS]
    for k, t in kinds:
        size = ARRAYS[k][bits == 8]
        setattr(t, k, at if size else None)
        at += 8192
    return out


def _step(lib, bits, tensors):
    d = N.AdamWDesc(0.9, 0.999, 1e-8, 1, N.GS_F32, bits, 0)
    arr = (N.AdamWTensor * len(tensors))(*tensors)
    return lib.gs_adamw(C.addressof(d), C.addressof(arr), len(tensors), None, 0, None)


@pytest.mark.parametrize("apart", [True, False])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("one", list(ARRAYS))
@pytest.mark.parametrize("other", list(ARRAYS))
def test_adamw_refuses_arrays_that_overlap(lib, one, other, bits, apart):
    """An array of the second tensor whose last element is the first element of one of the third's, and the other way round."""
    sizes = {k: v[bits == 8] for k, v in ARRAYS.items()}
    if not sizes[one] or not sizes[other] or one == other == "grad":
        pytest.skip("no such arrays, or both only read")
    for forward in (True, False):
        t = _tensors(bits, apart)
        a, b = (one, other) if forward else (other, one)
        end = getattr(t[2], b) + (sizes[b] - 4 if not forward else 4)
        setattr(t[1], a, end // 4 * 4 - (sizes[a] // 4 * 4 if forward else 0))
        assert _step(lib, bits, t) == N.GS_ERR_INVALID
        assert b"overlap" in lib.gs_last_error()


@pytest.mark.parametrize("name", ["adamw", "embedding", "groupnorm"])
def test_no_function_spills(name):
    """Not the kernels alone: what they call out of line neither."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    from gaussian_splatting_gb300 import build
    with tempfile.TemporaryDirectory() as out:
        r = subprocess.run([nvcc, *build.NVCC_FLAGS, "-Xptxas", "-v", "-c", os.path.join(build.CSRC, name + ".cu"), "-o",
                            os.path.join(out, "o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    seen, spilling, function = 0, [], None
    for line in (r.stdout + r.stderr).splitlines():
        m = re.search(r"Function properties for (\S+)", line)
        function = m.group(1) if m else function
        m = re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", line)
        if m and "warning" not in line:
            seen += 1
            if m.group(1) != "0" or m.group(2) != "0":
                spilling.append((function, line.strip()))
    assert seen and not spilling, spilling


HARNESS = r"""
#include <cuda_runtime_api.h>
#include <cstdio>
static int calls = 0, device = 0;
static cudaError_t answer = cudaSuccess;
extern "C" {
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { ++calls; return answer; }
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return ""; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 1; return cudaSuccess; }
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
}
namespace gs { cudaError_t max_dynamic_smem(const void* fn, int bytes); }
static char kernels[100];
static void all(int bytes) {  // driver calls for a launch of each kernel
  const int before = calls;
  for (char& k : kernels) gs::max_dynamic_smem(&k, bytes);
  printf("%d ", calls - before);
}
int main() {
  answer = cudaErrorInvalidValue;
  all(100);  // a refused size is not remembered
  answer = cudaSuccess;
  all(100), all(100), all(50), all(200), all(100);
  device = 1;
  all(200), all(200);
}
"""


def test_shared_memory_of_a_kernel_is_raised_once(tmp_path):
    """The driver is called once for a kernel and device, however many kernels there are, and again for more bytes."""
    nvcc, gxx = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc", shutil.which("g++")
    if not os.path.exists(nvcc) or not gxx:
        pytest.skip("nvcc or g++ not available")
    from gaussian_splatting_gb300 import build
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    (tmp_path / "harness.cpp").write_text(HARNESS)
    obj, exe = str(tmp_path / "api.o"), str(tmp_path / "harness")
    for cmd in ([nvcc, *build.NVCC_FLAGS, "-c", os.path.join(build.CSRC, "api.cu"), "-o", obj],
                [gxx, "-std=c++17", "-I", include, str(tmp_path / "harness.cpp"), obj, "-o", exe, "-lpthread"]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.stdout.split() == ["100", "100", "0", "0", "100", "0", "100", "0"]


@pytest.mark.parametrize("bits", [16, 32])
@pytest.mark.parametrize("width", [1, 4, 27, 64, 100, 600])
def test_embedding_gradient_workspace_is_bounded(lib, bits, width):
    """Besides sums, 20 bytes a row (lists of the sort, twice 8, and its counts; or pairs and theirs), a bit a code, the sums at the
    ends of the sort's parts (a quarter of dy's values at most) and a few MB."""
    padded = (width + 7) // 8 * 8
    for rows in (9_000, 100_000, 1_572_864, 2_000_000, 4_000_001, 11_000_000, 50_000_000, 400_000_000):
        for n in (1, 257, 5_000, 70_000, 300_000, 1_000_001, 1 << 21, (1 << 22) - 3, 1 << 22, 20_000_000):
            d = N.EmbeddingDesc(rows, n, width, width, width, N.GS_BF16 if bits == 16 else N.GS_F32, 32, 1.0)
            need = lib.gs_embedding_bwd_workspace_size(C.addressof(d))
            dy = rows * width * bits // 8
            of_rows = min(n + 2048 + rows // 24, rows * 3 // 8)
            sums = max(64 << 20, dy // 4, 4 * padded * of_rows)
            ends = rows * padded if rows < 1 << 21 or n > 1 << 22 else 0
            assert need <= sums + 20 * rows + n // 8 + ends + (8 << 20), (rows, n, need, sums)
