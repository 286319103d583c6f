"""The bounded waits of the dense paged attention, in a kernel of their own: two warps wait on barriers
of shared memory that nothing, or another warp, arrives at."""
import ctypes
import os
import subprocess

import pytest

from dsa_sparse_attention_mla_gb300 import _build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include <cuda_runtime.h>
#include "dsa_paged_wait.cuh"
using namespace dsa;
using namespace dsa::paged;

__device__ void pause(uint64_t ns) {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < ns) __nanosleep(1000);
}

// Warp 0 waits on barrier 0 for limit0, warp 1, which follows the counter, on barrier 1 for limit1. Warp 2 arrives at barrier 1 after
// `arrive` ns (0: never), and counts until then if `step` is set: once every `step` ns. A warp whose wait
// runs out sets the flag. out: [2][result, us].
__global__ void waits(long long* out, uint64_t limit0, uint64_t limit1, uint64_t arrive, uint64_t step) {
  __shared__ uint64_t bars[2];
  __shared__ int flag, count;
  const uint32_t bar = (uint32_t)__cvta_generic_to_shared(bars);
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
    flag = count = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  const uint64_t t0 = globaltimer_ns();
  if (warp < 2) {
    const bool ok = __all_sync(0xffffffffu, warp == 0 ? bar_wait(bar, 0, &flag, limit0)
                                                      : bar_wait_row(bar + 8, 0, &flag, &count, limit1));
    if ((threadIdx.x & 31) == 0) {
      if (!ok) *(volatile int*)&flag = 1;
      out[2 * warp] = ok;
      out[2 * warp + 1] = (long long)(globaltimer_ns() - t0) / 1000;
    }
  } else if (arrive) {
    if (step) {
      for (uint64_t t = 0; t < arrive; t += step) {
        pause(step);
        if (threadIdx.x == 64) *(volatile int*)&count = (int)(t / step) + 1;
      }
    } else {
      pause(arrive);
    }
    if (threadIdx.x == 64) mbar_arrive(bar + 8);
  }
}

extern "C" __attribute__((visibility("default"))) int run(long long* host, unsigned long long limit0,
                                                              unsigned long long limit1, unsigned long long arrive,
                                                              unsigned long long step) {
  long long* dev = nullptr;
  cudaError_t e = cudaMalloc(&dev, 32);
  if (e != cudaSuccess) return e;
  waits<<<1, 96>>>(dev, limit0, limit1, arrive, step);
  e = cudaMemcpy(host, dev, 32, cudaMemcpyDeviceToHost);
  cudaFree(dev);
  return e;
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory, gpu):
    d = tmp_path_factory.mktemp("wait")
    (d / "wait.cu").write_text(SOURCE)
    subprocess.run([_build._nvcc(), *_build.NVCC_FLAGS, "-I", _build.CSRC, "-shared", str(d / "wait.cu"), "-o",
                    str(d / "wait.so")], check=True, capture_output=True)
    lib = ctypes.CDLL(str(d / "wait.so"))

    def call(limit0, limit1, arrive=0, step=0):
        """((result, us) of warp 0, of warp 1); times in milliseconds."""
        out = (ctypes.c_longlong * 4)()
        assert lib.run(out, *(ctypes.c_ulonglong(int(x * 1e6)) for x in (limit0, limit1, arrive, step))) == 0
        return (out[0], out[1]), (out[2], out[3])

    return call


def test_a_wait_runs_out(run):
    (r0, t0), (r1, t1) = run(30, 30)
    assert (r0, r1) == (0, 0) and 29000 <= max(t0, t1) < 200000


def test_a_wait_ends_with_the_arrival(run):
    (_, _), (r1, t1) = run(400, 400, arrive=20)
    assert r1 == 1 and 19000 <= t1 < 100000


def test_the_others_leave_with_the_first(run):
    """Nobody waits out a limit of its own once another's has run out."""
    (r0, t0), (r1, t1) = run(30, 1500)
    assert (r0, r1) == (0, 0) and t0 >= 29000 and t1 < 300000


def test_progress_restarts_the_limit(run):
    """A wait of many limits holds as long as the block gets on, and runs out once it does not."""
    (_, _), (r1, t1) = run(2000, 60, arrive=300, step=10)
    assert r1 == 1 and 290000 <= t1 < 900000
    (_, _), (r1, t1) = run(2000, 60, arrive=300)
    assert r1 == 0 and 59000 <= t1 < 290000
