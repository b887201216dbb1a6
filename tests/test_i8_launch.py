"""What the row quantiser launches (no GPU): its launching code compiled for the
host alone, against stand-ins for HIP's launch functions that write down every
launch.  A direction of a grid has fewer than 2^32 threads."""
from __future__ import annotations

import ctypes
import re
import subprocess
from pathlib import Path

import pytest

from tests import test_lds_poison_build as poison

STANDINS = r"""
#include <hip/hip_runtime.h>
#include <vector>

#include "i8.h"

#define HERE extern "C"

struct Launch { long long grid, block, x, M, K, codes, scales; };
static std::vector<Launch> launches;
static dim3 grid_, block_;

HERE void **__hipRegisterFatBinary(const void *) { static void *p; return &p; }
HERE void __hipRegisterFunction(void **, const void *, char *, const char *, unsigned, void *, void *, void *, void *, int *) {}
HERE void __hipUnregisterFatBinary(void **) {}
HERE hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t, hipStream_t) { grid_ = g; block_ = b; return hipSuccess; }
HERE hipError_t __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *n, hipStream_t *s)
{
    *g = grid_; *b = block_; *n = 0; *s = nullptr;
    return hipSuccess;
}
HERE hipError_t hipGetLastError() { return hipSuccess; }
HERE hipError_t hipLaunchKernel(const void *, dim3 g, dim3 b, void **a, size_t, hipStream_t)
{
    if (g.y != 1 || g.z != 1 || b.y != 1 || b.z != 1) return hipErrorInvalidValue;
    auto word = [&](int i) { return *static_cast<long long *>(a[i]); };
    launches.push_back(Launch{g.x, b.x, word(0), word(1), word(2), word(3), word(4)});
    return hipSuccess;
}

extern "C" int quant_launches(long long x, int bf16, long long M, long long K, long long codes, long long scales, Launch *out, int most)
{
    launches.clear();
    if (dbs::launch_quant_i8(reinterpret_cast<void *>(x), bf16, M, K, reinterpret_cast<int8_t *>(codes),
                             reinterpret_cast<float *>(scales), nullptr) != hipSuccess)
        return -1;
    for (int i = 0; i < most && i < (int)launches.size(); ++i) out[i] = launches[i];
    return (int)launches.size();
}
"""


class Launch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_longlong) for n in ("grid", "block", "x", "M", "K", "codes", "scales")]


@pytest.fixture(scope="module")
def quant_launches(tmp_path_factory):
    if not Path(poison.HIPCC).exists():
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("i8_launch")
    (out / "standins.hip").write_text(STANDINS)
    flags = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-fPIC", f"-I{poison.ROOT / 'include'}",
             f"-I{poison.CSRC}"]
    objects = []
    for unit in (poison.CSRC / "i8_quant.hip", out / "standins.hip"):
        objects.append(str(out / (unit.stem + ".o")))
        subprocess.run([poison.HIPCC, *flags, "-c", str(unit), "-o", objects[-1]], check=True)
    # the device code that a host-only unit has no copy of
    names = subprocess.run(["nm", "-u", *objects], check=True, capture_output=True, text=True).stdout
    absent = [f"-Wl,--defsym={n}=0" for n in sorted(set(re.findall(r"__hip_fatbin\w*", names)))]
    lib = out / "launches.so"
    # (only the one function is seen outside: the stand-ins must not serve the process's own HIP calls)
    (out / "exports").write_text("{ global: quant_launches; local: *; };")
    subprocess.run(["g++", "-shared", f"-Wl,--version-script={out / 'exports'}", *absent, *objects, "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).quant_launches
    f.argtypes = [ctypes.c_longlong, ctypes.c_int] + [ctypes.c_longlong] * 4 + [ctypes.POINTER(Launch), ctypes.c_int]

    def run(x, bf16, M, K, codes, scales):
        got = (Launch * 64)()
        n = f(x, bf16, M, K, codes, scales, got, 64)
        assert 0 < n <= 64
        return got[:n]

    return run


X, CODES, SCALES = 1 << 40, 1 << 48, 1 << 52          # (addresses, never read)


@pytest.mark.parametrize("K", [1, 5, 8, 17, 512, 1024, 1032, 2048, 2056, 4096, 8192, 16384, 1 << 21])
@pytest.mark.parametrize("bf16", [0, 1])
def test_rows_are_launched_once_in_grids_that_hip_takes(quant_launches, K, bf16):
    row = K * (2 if bf16 else 4)
    for M in (1, 4097, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, 3 * (1 << 23) + 5, 1 << 25):
        for off in (0, 4):
            done = 0
            for g in quant_launches(X + off, bf16, M, K, CODES, SCALES):
                assert g.grid * g.block < 1 << 32, (M, off)
                assert (g.x, g.codes, g.scales, g.K) == (X + off + done * row, CODES + done * K, SCALES + 4 * done, K)
                # a row to a workgroup, or to each of its four waves
                assert g.block == 256 and g.M > 0 and g.grid in (g.M, -(-g.M // 4))
                done += g.M
            assert done == M
