"""One layer of a server that holds many customers' low-rank adapters over shared
NVFP4 weights, with a mixture of experts behind the projection:

    y = x + W norm(x) + adapter(norm(x))          (adapted projection)
    z = y + experts(norm(y); router(norm(y)))     (mixture of experts)

A prefill step takes the rows of several prompts at once: the activation is
quantized and multiplied on the block-scaled GEMM, each row with its request's
adapter.  A decode step takes one row a request, unquantized, in four launches.
The workspaces are kept from step to step; calls on one stream may share them.

    python examples/serve_step.py        (needs an MI355X)
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_block_scaled_04_amd import ops, serving  # noqa: E402

MOE_TOKENS = 64  # most tokens of one nvfp4_moe_small call


def norm(x):
    f = x.float()
    return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Layer:
    """Random weights of a layer: hidden size h, `experts` experts of inner size
    inter, `adapters` adapters of rank r."""

    def __init__(self, h, inter, experts, top_k, adapters, r, seed=0, max_rows=4096):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape, scale=1.0):
            return torch.randn(*shape, device="cuda", generator=g) * scale

        def pack(n, k):  # a weight as it is kept: codes, swizzled scales, global scale
            return ops.nvfp4_quantize(rand(n, k, scale=k ** -0.5).bfloat16())

        self.h, self.inter, self.top_k, self.r = h, inter, top_k, r
        self.w, self.w_sf, self.gs_w = pack(h, h)
        self.alpha_w = 1 / self.gs_w
        self.lora_a = rand(adapters, r, h, scale=h ** -0.5).bfloat16()
        self.lora_b = rand(adapters, h, r, scale=0.3).bfloat16()
        self.scaling = torch.rand(adapters, device="cuda", generator=g) + 0.5
        self.router = rand(experts, h, scale=h ** -0.5)
        self.w13, self.w13_sf, gs = (torch.stack(p) for p in zip(*(pack(2 * inter, h) for _ in range(experts))))
        self.alpha13 = 1 / gs.view(-1)
        self.w2, self.w2_sf, gs = (torch.stack(p) for p in zip(*(pack(h, inter) for _ in range(experts))))
        self.alpha2 = 1 / gs.view(-1)
        need = max(serving.adapters_ws_bytes(max_rows, r, split=True),
                   serving.moe_small_ws_bytes(MOE_TOKENS, top_k, h, inter))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")

    def project_prefill(self, x, adapter):
        n = norm(x)
        codes, sf, _, alpha = ops.nvfp4_quantize_alpha(n, self.gs_w)
        return x + serving.nvfp4_gemm_adapters(codes, self.w, sf, self.w_sf, alpha, n, self.lora_a, self.lora_b, adapter,
                                               scaling=self.scaling, workspace=self.workspace)

    def project_decode(self, x, adapter):
        return x + serving.nvfp4_linear_adapters(norm(x), self.w, self.w_sf, self.alpha_w, self.lora_a, self.lora_b, adapter,
                                                 scaling=self.scaling, workspace=self.workspace)

    def experts(self, y):
        n = norm(y)
        logits = n.float() @ self.router.t()
        out = torch.empty_like(y)
        for i in range(0, y.shape[0], MOE_TOKENS):
            s = slice(i, i + MOE_TOKENS)
            serving.nvfp4_moe_small(n[s], logits[s], self.w13, self.w13_sf, self.alpha13, self.w2, self.w2_sf, self.alpha2,
                                    self.top_k, out=out[s], workspace=self.workspace)
        return y + out

    def prefill(self, x, adapter):
        return self.experts(self.project_prefill(x, adapter))

    def decode(self, x, adapter):
        return self.experts(self.project_decode(x, adapter))


def main(h=4096, inter=1024, experts=32, top_k=4, adapters=8, r=16, prompts=(37, 5, 96, 1, 61), steps=16):
    layer = Layer(h, inter, experts, top_k, adapters, r)
    g = torch.Generator(device="cuda").manual_seed(1)
    # a request's adapter; -1: the shared weights alone
    request = torch.tensor([i % (adapters + 1) - 1 for i in range(len(prompts))], dtype=torch.int32, device="cuda")
    lengths = torch.tensor(prompts, device="cuda")
    x = torch.randn(sum(prompts), h, device="cuda", generator=g).bfloat16()
    z = layer.prefill(x, request.repeat_interleave(lengths))
    token = z[lengths.cumsum(0) - 1]  # each request's last row
    token = layer.decode(token, request)  # first step, untimed
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(steps):
        token = layer.decode(norm(token), request)
    torch.cuda.synchronize()
    print(f"prefill of {sum(prompts)} rows, {len(prompts)} requests; {(time.perf_counter() - t0) / steps * 1e6:.0f} us a "
          f"decode step (launches from Python); finite: {bool(torch.isfinite(token).all())}")
    return token


if __name__ == "__main__":
    main()
