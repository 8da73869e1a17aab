"""The codec where one launch cannot hold the work: 2^32 threads and more."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # the CPU suite deselects these with -m "not gpu"
    pytest.skip("no GPU", allow_module_level=True)

import ggml_iq_codebook_amd as iq  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def needs(gib):
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip("needs %d GiB of GPU memory" % gib)


@pytest.mark.parametrize("fmt", ["iq1_s", "iq2_xs", "iq1_m"])
def test_decode(fmt):
    """2^26 + 4096 blocks of 64 threads, the payload of 4096 blocks again and again."""
    needs(80)
    grid = workloads.iq2xs_grid() if fmt == "iq2_xs" else workloads.iq1s_grid()
    weight = workloads.normal_weight((64, 64 * 256), 3)
    some = iq.encode(torch.from_numpy(weight).to(DEV), torch.from_numpy(grid).to(DEV), fmt=fmt)
    want = torch.from_numpy(oracle.decode(fmt, some.cpu().numpy(), grid).astype(np.float32)).to(DEV)
    times = 2 ** 26 // 4096 + 1
    packed = some.repeat(times, 1, 1)
    out = torch.full((packed.shape[0], want.shape[1]), 7.0, device=DEV)
    iq.dequant(packed, torch.from_numpy(grid).to(DEV), fmt=fmt, out=out)
    out = out.view(times, *want.shape)
    for first in range(0, times, 1024):
        assert bool((out[first:first + 1024] == want).all()), first


def test_choice_search():
    """2^27 + 40 rows, 32 threads each, of one candidate of zeros: every pick is that one,
    and so is every entry of the trace."""
    needs(160)
    rows, groups, sweeps = 2 ** 27 + 40, 8, 1
    H = torch.eye(256, device=DEV)
    cand = torch.zeros((rows, 256), device=DEV)
    picks = torch.full((rows, groups), 7, dtype=torch.int32, device=DEV)
    trace = torch.full((sweeps + 1, rows, groups), 7, dtype=torch.int32, device=DEV)
    P = ctypes.c_void_p
    code = iq.load().iq_choice_search(P(H.data_ptr()), P(cand.data_ptr()), rows, groups, 1, sweeps,
                                      P(picks.data_ptr()), P(trace.data_ptr()),
                                      P(torch.cuda.current_stream().cuda_stream))
    assert code == 0
    assert not picks.any() and not trace.any()
