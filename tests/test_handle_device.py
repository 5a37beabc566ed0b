"""An attention handle belongs to the device it was made on, whichever is
current when it is asked for its status or destroyed.

Two devices, on the host: the few calls of the CUDA runtime that these entry
points make are answered by a small fake, loaded before the real one in a
process of its own, which writes down the current device of each."""
import subprocess
import sys

from tests.conftest import ROOT

FAKE = r"""
#include <stdlib.h>
#include <string.h>
#include <stdio.h>
static int current = 0;
static char text[4096];
static void note(const char* what) {
  char line[64];
  snprintf(line, sizeof line, "%s@%d ", what, current);
  strncat(text, line, sizeof text - strlen(text) - 1);
}
const char* fake_log(void) { return text; }
void fake_clear(void) { text[0] = 0; }
int cudaGetDevice(int* d) { *d = current; return 0; }
int cudaSetDevice(int d) { if (d < 0 || d > 1) return 101; current = d; return 0; }
int cudaDeviceGetAttribute(int* v, int attr, int d) { *v = attr == 75 ? 10 : attr == 76 ? 3 : 152; return 0; }
int cudaFuncSetAttribute(const void* f, int attr, int v) { return 0; }
int cudaMalloc(void** p, size_t n) { note("malloc"); *p = malloc(n < 4096 ? n : 4096); return 0; }
int cudaFree(void* p) { note("free"); free(p); return 0; }
int cudaMemset(void* p, int v, size_t n) { note("memset"); memset(p, v, n); return 0; }
int cudaMemcpy(void* d, const void* s, size_t n, int kind) { note("memcpy"); memcpy(d, s, n); return 0; }
int cudaDeviceSynchronize(void) { note("sync"); return 0; }
"""

CHILD = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[2])
fake = ctypes.CDLL(sys.argv[1])
fake.fake_log.restype = ctypes.c_char_p
from weight_streaming_expert_gb300 import native as N
L = N.lib()
def log():
    got = fake.fake_log().decode().split()
    fake.fake_clear()
    return got
def current():
    d = ctypes.c_int()
    fake.cudaGetDevice(ctypes.byref(d))
    return d.value
fake.cudaSetDevice(1)
h = ctypes.c_void_p(L.moe_attn_create(8, 2, 64))
assert h, N.last_error()
assert all(x.endswith("@1") for x in log())
fake.cudaSetDevice(0)
assert L.moe_attn_get_status(h) == N.MOE_OK
assert log() == ["sync@1", "memcpy@1", "memset@1"] and current() == 0
a = N.moe_attn_args_t(dtype=0, batch=1, n_tokens=1, max_q_len=1, scale=1.0, q=16, q_token_stride=512, q_head_stride=64,
                      k_cache=16, v_cache=16, k_page_stride=2048, k_row_stride=128, v_page_stride=2048,
                      v_row_stride=128, n_pages=4, page_size=16, block_table=16, table_stride=4, q_starts=16,
                      kv_lens=16, out=16, out_token_stride=512, out_head_stride=64)
assert L.moe_attn_forward(h, ctypes.byref(a), None) == N.MOE_ERR_INVALID_ARG
assert "device" in N.last_error(), N.last_error()
L.moe_attn_destroy(h)
got = log()
assert got[0] == "sync@1" and got[1:] == ["free@1"] * 4 and current() == 0, got
print("done")
"""


def test_status_and_destroy_go_to_the_handles_device(tmp_path):
    from weight_streaming_expert_gb300 import native as N
    N.lib()  # built
    source, lib = tmp_path / "fake.c", tmp_path / "fake.so"
    source.write_text(FAKE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-w", "-o", str(lib), str(source)], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, str(lib), ROOT], env={"LD_PRELOAD": str(lib), "PATH": "/usr/bin:/bin"},
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr
