"""The example model's run together: prompts, drafts, verdicts and commits step by step against one
prompt over what was kept.

The two ways pass the same products in another order and round the same tensors, so their logits differ by
bf16 roundings (2^-8 each) that are not the same ones.  On the way are the conv's output, the scan's inputs
(two products), its output, the product behind it, the residual sum, the norm, q, k and v and their rotation,
the attention's output, its product, the sum, the norm and the head's product: 16 roundings on either side,
each taken over by a norm that may double it: 2 * 16 * 2 * 2^-8 = 64 * 2^-8 of the logits' norm, and no more
than half of that where they are as unrelated as roundings are, in root of their number: 8 * 2 * 2^-8."""

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
    spec = importlib.util.spec_from_file_location("speculative_model", os.path.join(ROOT, "examples", "speculative_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("sizes", [dict(), dict(dim=128, d_inner=264, d_state=24, heads=2, head_dim=96, rot=48, T=9, vocab=333),
                                   dict(T=2, d_state=64, heads=1, head_dim=128, rot=128)], ids=str)
def test_steps_agree_with_one_prompt(example, sizes):
    print("[case] model", sizes, flush=True)
    model = example.SpeculativeModel(**sizes)
    prompts = [5, 200, 64, 1, 129]
    rows, counts, stepped, whole = example.write(model, prompts)
    assert all(1 <= c <= model.T for step in counts for c in step)
    for i, p in enumerate(prompts):
        assert len(rows[i]) == p + sum(step[i] for step in counts) == int(model.lengths[i])
        assert bool(((rows[i] >= 0) & (rows[i] < model.vocab)).all())
    assert torch.isfinite(stepped.float()).all()
    off = ((stepped.float() - whole.float()).norm() / whole.float().norm()).item()
    print("[case] off", off, "kept", counts, flush=True)
    assert off <= 16 * 2.0 ** -8
