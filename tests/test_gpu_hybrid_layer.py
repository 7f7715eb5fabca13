"""The example layer: speculative decoding step by step against one prompt over the same tokens.

The two ways round differently.  The prompt's q and k are rounded twice (after the conv and after
the norm), the drafts' once; states and outputs pass the same products in another order.  Each
rounding is off by at most 2^-8 of its value: three for q, three for k (through the state as
well), one for each output of the attention on either side, so the outputs differ by at most
8 * 2^-8 of their norm, the gated norm and the one behind it take that over (their divisors may
double it), and their own roundings and the products between them add 2^-8 each: 20 * 2^-8.
"""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("hybrid_layer", os.path.join(ROOT, "examples", "hybrid_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("heads", [(4, 8, 64, 64), (2, 6, 128, 128), (3, 3, 96, 72)], ids=str)
def test_steps_agree_with_one_prompt(example, heads):
    print("[case] layer", heads, flush=True)
    q_heads, v_heads, dk, dv = heads
    layer = example.HybridLayer(dim=256, q_heads=q_heads, v_heads=v_heads, dk=dk, dv=dv)
    out, want = example.serve(layer, [5, 200, 64, 1, 129])
    assert torch.isfinite(out.float()).all()
    off = (out.float() - want.float()).norm() / want.float().norm()
    print("[case] off", off.item(), flush=True)
    assert off <= 20 * 2.0 ** -8
