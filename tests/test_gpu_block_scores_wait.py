"""Block scores whose units outlast the limit of a wait: the kernel built with a limit of 2 ms instead of
2 s, over units of some 20 ms. Queries and weights of the next unit wait for all tiles of the one before."""
import ctypes
import os
import subprocess

import pytest
import torch

import dsa_sparse_attention_mla_gb300 as dsa
from dsa_sparse_attention_mla_gb300 import _build

pytestmark = pytest.mark.gpu

HOST = r"""
#include "dsa_block_scores.cu"
namespace dsa {
dsa_status_t cuda_fail(cudaError_t) { return DSA_ERR_CUDA; }
dsa_status_t current_device(DeviceInfo* out) {
  out->device = 0;
  return cudaDeviceGetAttribute(&out->sm_count, cudaDevAttrMultiProcessorCount, 0) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
}  // namespace dsa
"""


@pytest.fixture(scope="module")
def short_waits(tmp_path_factory, gpu):
    d = tmp_path_factory.mktemp("scores")
    for name in os.listdir(_build.CSRC):
        if name.endswith((".h", ".cuh")) or name == "dsa_block_scores.cu":
            with open(os.path.join(_build.CSRC, name)) as f:
                text = f.read()
            if name == "dsa_paged_wait.cuh":
                assert text.count("kWaitNs = 2000000000ull") == 1
                text = text.replace("kWaitNs = 2000000000ull", "kWaitNs = 2000000ull")
            (d / name).write_text(text)
    (d / "host.cu").write_text(HOST)
    subprocess.run([_build._nvcc(), *_build.NVCC_FLAGS, "-I", str(d), "-shared", str(d / "host.cu"), "-o", str(d / "scores.so")],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(str(d / "scores.so"))
    lib.dsa_block_scores.argtypes = dsa.load_library().dsa_block_scores.argtypes
    return lib.dsa_block_scores


@pytest.mark.parametrize("weights", [False, True])
def test_long_units(gpu, short_waits, weights):
    sms = torch.cuda.get_device_properties(gpu).multi_processor_count
    H, width, pages = 128, 2_000_000, 500  # two tokens a group, a group a unit, two units an SM and a few more
    T = 4 * sms + 10
    gen = torch.Generator(device=gpu).manual_seed(1)
    q = torch.randn((T, H, 256), generator=gen, device=gpu).to(torch.bfloat16)
    w = torch.randn((T, H), generator=gen, device=gpu) if weights else None
    summary = torch.randn((pages, 256), generator=gen, device=gpu).to(torch.bfloat16)
    table = torch.randint(0, pages, (1, width), generator=gen, device=gpu, dtype=torch.int32)
    lens = torch.full((T,), width, dtype=torch.int32, device=gpu)
    req = torch.zeros(T, dtype=torch.int32, device=gpu)
    out = torch.full((T, width), 7.0, device=gpu)
    err = torch.zeros(1, dtype=torch.int32, device=gpu)
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    st = short_waits(at(q), H * 256, 256, T, H, at(summary), pages, at(table), width, 1, width, 1, at(req), at(lens), 0.125,
                     at(w), at(out), width, width, at(err), torch.cuda.current_stream().cuda_stream)
    end.record()
    torch.cuda.synchronize()
    assert st == 0 and err.item() == 0
    assert begin.elapsed_time(end) > 3 * 6  # three units in turn, each of them several limits long
    # every block of a page has the score of that page
    small = dsa.dsa_block_scores(q, summary, torch.arange(pages, dtype=torch.int32, device=gpu)[None],
                                 torch.full_like(lens, pages), 0.125, page_size=1, req_of_token=req, weights=w)
    for t in range(0, T, 7):
        assert torch.equal(out[t], small[t][table[0].long()]), t
    del out
    torch.cuda.empty_cache()
