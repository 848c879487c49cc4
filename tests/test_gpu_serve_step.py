"""The example's layer: prefill and decode through the adapted projection and the
experts, each operator against its plain 64-bit form on what it was handed."""
import importlib.util
import os

import pytest
import torch

import serving_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_step.py")
    spec = importlib.util.spec_from_file_location("serve_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def bf16_step(v):
    """The rounding of a residual sum kept in bf16."""
    return v.abs() * 2.0 ** -8 * 1.01


@pytest.mark.parametrize("rows", [1, 7, 100])
def test_layer(example, rows):
    say("serve_step", rows)
    layer = example.Layer(256, 96, 12, 3, 5, 16)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, 256, device="cuda", generator=g).bfloat16()
    ids = torch.randint(-1, 5, (rows,), device="cuda", generator=g, dtype=torch.int32)
    n = example.norm(x)
    w = R.dequant(layer.w, layer.w_sf) / layer.gs_w.double()

    def projected(base_x, got):
        ref, bound = R.adapters(base_x @ w.t(), base_x.abs() @ w.abs().t(), 256, n, layer.lora_a, layer.lora_b, ids,
                                layer.scaling, None)
        # 1 / gs in fp32, twice at most; then the residual sum
        bound = bound + ref.abs() * 2.0 ** -22
        assert R.worst(got, ref + x.double(), bound + bf16_step((ref + x.double()).abs() + bound)) <= 1.0

    y = layer.project_decode(x, ids)
    projected(n.double(), y)
    codes, sf, gs, _ = example.ops.nvfp4_quantize_alpha(n, layer.gs_w)
    projected(R.dequant(codes, sf) / gs.double(), layer.project_prefill(x, ids))

    z = layer.experts(y)
    m = example.norm(y)
    ref, bound, _, _ = R.moe(m, m.float() @ layer.router.t(), layer.w13, layer.w13_sf, layer.alpha13, layer.w2, layer.w2_sf,
                             layer.alpha2, 3, "softmax", True)
    assert R.worst(z, ref + y.double(), bound + bf16_step((ref + y.double()).abs() + bound)) <= 1.0
    assert torch.equal(z, layer.decode(x, ids))


def test_example_runs(example):
    say("serve_step main")
    token = example.main(h=512, inter=128, experts=8, top_k=2, adapters=3, r=8, prompts=(9, 1, 70), steps=2)
    assert token.shape == (3, 512) and bool(torch.isfinite(token).all())
