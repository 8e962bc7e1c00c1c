"""The 8-bit latent cache's calls on more than one device of a process, on the CPU: a C program links the library and
answers its runtime calls itself. Its launches fail, as the runtime's do, where a kernel's dynamic shared memory is above
48 KB and was not allowed for that kernel on the current device."""
import os
import subprocess

import pytest

from mla_block_diffusion_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stdio.h>
#include <string.h>
#include "dspark.h"

static int device, launches, refuse;
static struct { const void *f; int dev, bytes; } allowed[64];
static int n_allowed;

cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr a, int d) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *f, enum cudaFuncAttribute a, int value) {
  if (a != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
  if (refuse) return cudaErrorInvalidDevice;
  allowed[n_allowed].f = f; allowed[n_allowed].dev = device; allowed[n_allowed++].bytes = value;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **args) {
  int i, ok = c->dynamicSmemBytes <= 48 * 1024;
  for (i = 0; i < n_allowed; ++i) ok |= allowed[i].f == f && allowed[i].dev == device && c->dynamicSmemBytes <= (size_t)allowed[i].bytes;
  launches += ok;
  return ok ? cudaSuccess : cudaErrorInvalidValue;
}
static CUresult encode(CUtensorMap *m) { memset(m, 0, sizeof *m); return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *name, void **f, unsigned v, unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult *q) {
  *f = (void *)encode; *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
#define P(k) ((void *)(size_t)(0x100000 + 0x1000 * (k)))  /* never dereferenced */

static int append(const dspark_qcache_t *c, int type) {
  return dspark_qcache_append(c, P(30), type, 576, 0, P(31), 4, P(32), 2, P(50), 1024, NULL);
}
static int attend(const dspark_qcache_t *c) {
  dspark_qattn_t a = {P(20), 64 * 576, P(21), P(22), 64, 7, 0, 0.1f, P(23), 64 * 512, NULL};
  return dspark_qcache_attend(c, 0, &a, 1, P(60), (size_t)1 << 40, NULL);
}
int main(void) {
  const int order[] = {0, 0, 1, 0, 3, 1, 63};
  dspark_qcache_t c;
  memset(&c, 0, sizeof c);
  c.kv_lora = 512; c.d_rope = 64; c.page_size = 64; c.n_layers = 1; c.codes[0] = P(1); c.scales[0] = P(2);
  c.n_pages = 8; c.page_table = P(3); c.max_pages = 4;
  refuse = 1;  /* a failed attempt is not taken for a done one */
  printf("%d %d\n", append(&c, DSPARK_ENTRY_BF16), attend(&c));
  refuse = 0;
  for (int i = 0; i < (int)(sizeof order / sizeof *order); ++i) {
    device = order[i];
    printf("%d %d %d\n", append(&c, DSPARK_ENTRY_BF16), append(&c, DSPARK_ENTRY_FP32), attend(&c));
  }
  printf("%d launches, %d attributes\n", launches, n_allowed);
  return 0;
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    lib, cuda = B.build(), os.path.dirname(os.path.dirname(B._nvcc()))
    d = tmp_path_factory.mktemp("devices")
    (d / "p.c").write_text(PROGRAM)
    subprocess.run(["gcc", "-rdynamic", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(cuda, "include"), str(d / "p.c"),
                    "-o", str(d / "p"), lib, f"-Wl,-rpath,{os.path.dirname(lib)}", f"-Wl,-rpath-link,{os.path.join(cuda, 'lib64')}"],
                   check=True)
    env = dict(os.environ, LD_LIBRARY_PATH=os.path.join(cuda, "lib64") + ":" + os.environ.get("LD_LIBRARY_PATH", ""))
    return subprocess.run([str(d / "p")], capture_output=True, text=True, check=True, env=env).stdout.splitlines()


def test_every_device_is_set_up(lines):
    assert lines[0] == "5 5"
    assert lines[1:8] == ["0 0 0"] * 7


def test_each_device_is_set_up_once(lines):
    # three kernels on devices 0, 1, 3 and 63; 7 x (two appends, the attention and its combine) launches
    assert lines[8] == f"{7 * 4} launches, {3 * 4} attributes"
