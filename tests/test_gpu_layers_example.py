"""The training step of examples/expert_layer.py, every output against 64 bits."""

import numpy as np
import pytest
import torch

from tests import layers_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # the CPU suite deselects these with -m "not gpu"
    pytest.skip("no GPU", allow_module_level=True)

from examples import expert_layer  # noqa: E402
from tests.test_gpu_layers import DEV, DTYPES, IDS, gen, normal, routing, within  # noqa: E402


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("tokens,top_k,experts,width,dropped", [(70, 2, 4, 512, 0.0), (33, 5, 7, 300, 0.2)])
def test_train_step(dtype, tokens, top_k, experts, width, dropped):
    """Experts that double their rows, which is exact.  The answers are rounded as combine's are;
    the gradient of a token sums rows that were rounded once before, so each term may be off by a
    rounding of the type; the gradient of a weight is one dot product in fp32."""
    c = routing(tokens, top_k, experts, 9, dropped)
    _, position, offsets = ref.sort(c.numpy(), experts)
    x, g = normal((tokens, width), 1, dtype), normal((tokens, width), 2, dtype)
    weights = torch.rand((tokens, top_k), generator=gen(3)).to(DEV)
    out, x_grad, w_grad = expert_layer.train_step(x, c.to(DEV), weights, lambda rows, _: rows * 2.0,
                                                  lambda rows, _: rows * 2.0, g, experts)
    x64, g64, w64 = (ref.to64(t) for t in (x, g, weights))
    y = 2.0 * ref.dispatch(x64, position, offsets)
    want, size = ref.combine(y, position, offsets, w64)
    within(out, want, ref.combine_bound(want, size, top_k, dtype))
    gy, gw, dots = ref.combine_backward(g64, y, position, offsets, w64)
    within(w_grad, gw, ref.dot_bound(dots, width))
    gx, size = ref.combine(2.0 * gy, position, offsets, np.ones_like(w64))
    within(x_grad, gx, ref.combine_bound(gx, size, top_k, dtype)
           + (size * ref.ROUND[dtype] + 2 * top_k * ref.TINY[dtype]) * (1 + 2.0 ** -6))
