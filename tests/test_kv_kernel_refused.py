"""When the attention kernel of many query rows cannot run (its roles share out a fixed number of
registers), only the calls that need it are refused. CPU only: the CUDA runtime's calls are
answered by a fake that is loaded before it, in a process of its own."""
import json
import os
import re
import shutil
import subprocess
import sys

import pytest

from nvfp4_expert_ffn_b200 import binding as B

CSRC = os.path.join(os.path.dirname(os.path.abspath(B.__file__)), "csrc")

FAKE = r"""
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>
static int launches, asked;
int fake_launches(void) { int n = launches; launches = 0; return n; }
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
  (void)d;
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrMultiProcessorCount ? 148 : 0;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) { (void)f; (void)a; (void)v; return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes* at, const void* f) {
  (void)f;
  char text[64];
  memset(at, 0, sizeof *at);
  strncpy(text, getenv("FAKE_REGISTERS"), sizeof text - 1);
  char* p = text;
  for (int i = 0; i < asked && strchr(p, ','); ++i) p = strchr(p, ',') + 1;
  ++asked;
  at->numRegs = atoi(p);
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void* s) { (void)s; *p = (void*)0x100; return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** a) { (void)c; (void)f; (void)a; ++launches; return cudaSuccess; }
"""

CALLS = r"""
import ctypes, json, sys
lib, fake = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(None)
i64, P = ctypes.c_int64, ctypes.c_void_p
lib.moe_last_error.restype = ctypes.c_char_p
class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_pages", "page", "Hkv", "D")] + [(n, P) for n in "abcdef"]
class Prep(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("eps", ctypes.c_double), ("f", P), ("rot", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("m", ctypes.c_double)]
p, out = P(0x10000), []
def say(status):
    out.append([status, fake.fake_launches(), lib.moe_last_error().decode() if status else ""])
say(lib.moe_qk_norm_rope(p, i64(512), p, i64(256), 4, 4, 2, 128, p, ctypes.byref(Prep(None, None, 1e-6, None, 0, 0, 1.0)), p, p, None))
for D in (64, 128, 256):
    c = Cache(64, 64, 2, D, *[0x10000] * 6)
    for T, n_seqs, max_q, pages in ((2, 2, 1, 60), (2000, 1, 2000, 60)):  # single tokens, a prompt
        say(lib.nvfp4_kv_attention(p, i64(4 * D), T, 4, p, p, p, n_seqs, pages, max_q, ctypes.byref(c), ctypes.c_float(0.1), 1, p,
                                   None, p, ctypes.c_size_t(1 << 40), None))
print(json.dumps(out))
"""


def _registers():
    two = re.search(r"launch_regs = pair \? (\d+) : (\d+)", open(os.path.join(CSRC, "kv_attn_tc.cu")).read())
    return f"{two[2]},{two[2]},{two[1]}"  # in the order of the checks: D = 64, 128, 256


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    cc = shutil.which("gcc") or shutil.which("cc")
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if cc is None or not os.path.exists(os.path.join(include, "cuda_runtime_api.h")):
        pytest.skip("needs a C compiler and CUDA's headers")
    tmp = tmp_path_factory.mktemp("fake")
    (tmp / "fake.c").write_text(FAKE)
    (tmp / "calls.py").write_text(CALLS)
    subprocess.run([cc, "-shared", "-fPIC", "-I", include, "-o", str(tmp / "fake.so"), str(tmp / "fake.c")], check=True)
    B.lib()  # built, and its runtime found
    runtime = [line.split()[-1] for line in open("/proc/self/maps") if "libcudart" in line][0]

    def run(registers):
        env = dict(os.environ, LD_PRELOAD=str(tmp / "fake.so"), FAKE_REGISTERS=registers,
                   LD_LIBRARY_PATH=os.path.dirname(runtime) + ":" + os.environ.get("LD_LIBRARY_PATH", ""))
        r = subprocess.run([sys.executable, str(tmp / "calls.py"), B.LIB_PATH], env=env, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        return json.loads(r.stdout)
    return run


def test_all_calls_launch_when_the_registers_are_right(calls):
    assert [x[:2] for x in calls(_registers())] == [[0, 1]] + [[0, 2], [0, 4]] * 3


def test_only_the_kernel_of_many_rows_is_refused_when_they_are_not(calls):
    got = calls("8")
    assert [x[:2] for x in got] == [[0, 1]] + [[0, 2], [3, 0]] * 3
    assert all("many query rows" in x[2] for x in got if x[0])
