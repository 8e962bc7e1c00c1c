"""The 8-bit layers' calls on the CPU: a C program links the library and answers its runtime calls itself. What the runtime says
of clusters that fit a device, and on which devices kernels have been set up, decides the launches."""
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

static int device, fits, fail, queries, grid, cluster, launches;
static struct { const void *f; int dev, bytes; } allowed[1024];
static int n_allowed;

cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr a, int d) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *f, enum cudaFuncAttribute a, int value) {
  if (a != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
  allowed[n_allowed].f = f; allowed[n_allowed].dev = device; allowed[n_allowed++].bytes = value;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *f, const cudaLaunchConfig_t *c) {
  ++queries;
  if (fail) return cudaErrorNotReady;
  *n = fits / (int)c->attrs[0].val.clusterDim.x;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **args) {
  int ok = c->dynamicSmemBytes <= 48 * 1024;
  for (int i = 0; i < n_allowed; ++i) ok |= allowed[i].f == f && allowed[i].dev == device && c->dynamicSmemBytes <= (size_t)allowed[i].bytes;
  if (!ok) return cudaErrorInvalidValue;
  ++launches;
  grid = (int)c->gridDim.x, cluster = 0;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = (int)c->attrs[i].val.clusterDim.x;
  return cudaSuccess;
}
static CUresult encode(CUtensorMap *m) { memset(m, 0, sizeof *m); return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *name, void **f, unsigned v, unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult *q) {
  *f = (void *)encode; *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
#define P(k) ((void *)(size_t)(0x100000000ull * (k)))  /* never dereferenced */

static int matmul(int m, int n, int k) {
  dspark_qrows_t x = {m, k, P(1), P(2), m};
  dspark_qweight_t w = {n, k, P(3), P(4)};
  grid = cluster = 0;
  return dspark_qlinear_matmul(&x, &w, NULL, 0, P(5), DSPARK_ENTRY_FP32, n, P(6), 1024, NULL);
}
static int gated(int m, int n, int k) {
  dspark_qrows_t x = {m, k, P(1), P(2), m}, h = {m, n, P(7), P(8), m};
  dspark_qweight_t g = {n, k, P(3), P(4)}, u = {n, k, P(9), P(10)};
  grid = cluster = 0;
  return dspark_qlinear_gated(&x, &g, &u, &h, P(6), 1024, NULL);
}
static int quantise(void) {
  dspark_qrows_t x = {7, 512, P(1), P(2), 7};
  return dspark_qlinear_quantise(P(5), DSPARK_ENTRY_FP32, 512, &x, NULL);
}
static void say(const char *name, int status) { printf("%s %d grid %d cluster %d\n", name, status, grid, cluster); }

int main(void) {
  /* a query that fails fails the call, and the next call asks again */
  fits = 152, fail = 1;
  say("few failed", matmul(1, 128, 1536));
  say("many failed", matmul(65, 256, 512));
  fail = 0;
  say("few", matmul(1, 128, 1536));
  say("many", matmul(65, 25600, 512));
  int asked = queries;
  say("few again", matmul(1, 128, 1536));
  say("many again", matmul(65, 25600, 512));
  printf("asked again %d\n", queries - asked);
  /* a device that holds no cluster of two */
  device = 1, fits = 1;
  say("few alone", matmul(1, 128, 1536));
  say("gated alone", gated(17, 128, 1536));
  say("many alone", matmul(65, 256, 512));
  /* three of them */
  device = 2, fits = 3;
  say("few of three", matmul(1, 128, 1536));
  say("few of three tiles", matmul(1, 384, 1536));
  /* every device is set up, those behind the 64th on every call */
  fits = 152;
  launches = 0;
  const int order[] = {0, 5, 63, 64, 0, 100, 64};
  for (int i = 0; i < 7; ++i) {
    device = order[i];
    printf("%d %d %d %d\n", quantise(), matmul(7, 272, 512), matmul(300, 272, 512), gated(300, 272, 512));
  }
  printf("launches %d\n", launches);
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


def test_a_failed_query_is_not_an_answer(lines):
    assert lines[0] == "few failed 5 grid 0 cluster 0"
    assert lines[1] == "many failed 5 grid 0 cluster 0"
    assert lines[2] == "few 0 grid 4 cluster 4"            # twelve blocks of k, three to a CTA
    assert lines[3] == "many 0 grid 152 cluster 2"


def test_an_answer_is_kept(lines):
    assert lines[4:7] == ["few again 0 grid 4 cluster 4", "many again 0 grid 152 cluster 2", "asked again 0"]


def test_clusters_that_do_not_fit(lines):
    assert lines[7] == "few alone 0 grid 1 cluster 1"
    assert lines[8] == "gated alone 0 grid 1 cluster 1"
    assert lines[9] == "many alone 5 grid 0 cluster 0"
    assert lines[10] == "few of three 0 grid 3 cluster 3"
    assert lines[11] == "few of three tiles 0 grid 3 cluster 1"


def test_every_device_is_served(lines):
    assert lines[12:19] == ["0 0 0 0"] * 7  # also those behind the 64 that answers are kept for
    assert lines[19] == "launches 28"


def test_every_kernel_of_the_library_is_launched():
    """The quantiser of rows has one form for fp32, two for bf16."""
    out = subprocess.run(["nm", "-C", B.build()], capture_output=True, text=True, check=True).stdout
    forms = {line.split("quantise_rows_kernel<")[1].split(">")[0] for line in out.splitlines() if "quantise_rows_kernel<" in line}
    assert forms == {"__nv_bfloat16, 1", "__nv_bfloat16, 2", "float, 1"}
