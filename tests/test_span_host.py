"""The host side of the span calls, without a GPU: what it computes on the way to the launches.  The sources are compiled
with the device queries answered and the launches left out, so nothing is launched on a machine that has a GPU either."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cuda_runtime.h>
#include <stdio.h>
#include <stdlib.h>

#include "kev_internal.cuh"
#include "kev_span.cuh"
#define cudaGetDevice(p) (*(p) = 0, cudaSuccess)
#define cudaDeviceGetAttribute(p, attribute, device) (*(p) = 152, cudaSuccess)
#define cudaFuncSetAttribute(kernel, attribute, value) ((void)(kernel), cudaSuccess)
static volatile size_t shared_bytes;
#define launch_pdl(kernel, grid, block, smem, ...) ((void)(kernel), shared_bytes = (smem), cudaSuccess)
#include "kev_span_api.cu"
#include "kev_span_plan.cu"

namespace kev {
static int attends = 0;
bool span_small_copy(const SpanArgs& a) { return a.T <= 512; }
cudaError_t launch_span_write(const SpanArgs&, bool, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_span_read(const SpanArgs&, void*, void*, bool, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_span_simt(const SpanArgs&, cudaStream_t) { ++attends; return cudaSuccess; }
cudaError_t launch_span_tc(const SpanArgs&, cudaStream_t) { ++attends; return cudaSuccess; }
cudaError_t launch_span_rows(const SpanArgs&, bool, cudaStream_t) { ++attends; return cudaSuccess; }
cudaError_t launch_span_merge(const SpanArgs&, int, cudaStream_t) { return cudaSuccess; }
int span_rows_ctas(int, int) { return 1; }
}  // namespace kev

int main(int argc, char** argv) {
  int at = 0;
  auto next = [&] { return atoi(argv[++at]); };
  const int h_q = next(), h_kv = next(), dtype = next(), pool = next(), T = next(), n = next(), max_chunk = next();
  const kev_attn_shape shape = {h_q, h_kv, 128, dtype, 0.f};
  void* p = reinterpret_cast<void*>(0x100000);  // never read
  void* out = reinterpret_cast<void*>(0x100000000ull);
  const kev_paged_cache cache = {p, p, static_cast<float*>(p), static_cast<float*>(p), static_cast<int32_t*>(p), 4, 64, pool};
  const kev_interval* iv = static_cast<const kev_interval*>(p);
  const int32_t* pre = static_cast<const int32_t*>(p);
  const size_t bytes = (size_t)1 << 40;
  const int a = kev_chunk_attn_paged(p, p, p, T, iv, n, pre, max_chunk, &cache, 0, 0, out, &shape, p, bytes, nullptr, nullptr);
  const int b = kev_chunk_attn_paged(p, nullptr, nullptr, T, iv, n, pre, max_chunk, &cache, 9, 2, out, &shape, p, bytes, nullptr, nullptr);
  const int c = kev_prefill_attn_window(p, p, p, T, iv, n, 9, 2, out, &shape, p, bytes, nullptr, nullptr);
  const int d = kev_paged_write(p, p, T, iv, n, pre, &cache, &shape, p, bytes, nullptr, nullptr);
  const int e = kev_paged_read(p, p, T, iv, n, pre, &cache, &shape, p, bytes, nullptr, nullptr);
  printf("%d %d %d %d %d, %d\n", a, b, c, d, e, kev::attends);
  return 0;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    d = tmp_path_factory.mktemp("span_host")
    src, exe = str(d / "host.cu"), str(d / "host")
    with open(src, "w") as f:
        f.write(SOURCE)
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-gencode", "arch=compute_103a,code=sm_103a",
                        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "packed_question_isolated_gb300", "csrc"),
                        src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return lambda *a: subprocess.run([exe, *map(str, a)], capture_output=True, text=True, timeout=60)


HEADS = [(4, 4), (8, 2), (7, 1), (16, 2), (9, 1), (12, 1), (16, 1), (30, 2)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,pool", [(0, 0), (0, 2), (1, 1), (1, 2)])
def test_calls_without_tokens(host, heads, dtype, pool):
    """A round whose questions are all dropped, at every group size (16 / G tokens fit a tile of the kernel for few rows)."""
    for n in (0, 1, 40):
        for max_chunk in (0, 1, 5):
            r = host(*heads, dtype, pool, 0, n, max_chunk)
            assert r.returncode == 0 and r.stdout.startswith("0 0 0 0 0,"), (n, max_chunk, r.returncode, r.stdout)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,pool", [(0, 0), (0, 2), (1, 1)])
def test_calls_with_tokens(host, heads, dtype, pool):
    for T, n, max_chunk in ((1, 1, 0), (1, 1, 1), (40, 40, 1), (40, 0, 1), (700, 5, 0), (100000, 4096, 0), (3, 2, 2)):
        r = host(*heads, dtype, pool, T, n, max_chunk)
        assert r.returncode == 0 and r.stdout.startswith("0 0 0 0 0,"), (T, n, max_chunk, r.returncode, r.stdout)
