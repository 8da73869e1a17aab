"""What autograd has to know of the 4-bit weights and the router."""

import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # the CPU suite deselects these with -m "not gpu"
    pytest.skip("no GPU", allow_module_level=True)

import ggml_iq_codebook_amd as iq  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write("\n[gpu] %s\n" % request.node.nodeid)
    sys.__stderr__.flush()
    yield


def normal(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def test_values_are_not_written_into_a_recorded_tensor():
    codes, scale = iq.quantize_groups(normal((6, 64), 1))
    want = iq.dequantize_groups(codes, scale)
    leaf = normal((6, 64), 2).requires_grad_()
    before = leaf.detach().clone()
    computed = leaf * 2.0
    for out in (leaf, computed, computed[:, :64]):
        with pytest.raises(ValueError, match="out cannot be given"):
            iq.dequantize_groups(codes, scale, out=out)
    assert torch.equal(leaf.detach(), before)
    computed.sum().backward()
    assert torch.equal(leaf.grad, torch.full_like(leaf, 2.0))
    # where nothing is recorded they are, as torch's own results
    with torch.no_grad():
        assert iq.dequantize_groups(codes, scale, out=leaf) is leaf
    assert torch.equal(leaf.detach(), want)
