"""One layer of a server that holds many customers' low-rank adapters over shared
NVFP4 weights, with a mixture of experts behind the projection:

    y = x + W norm(x) + adapter(norm(x))          (adapted projection)
    z = y + experts(norm(y); router(norm(y)))     (mixture of experts)

With --attention an attention block comes first,

    x <- x + Wo attention(rope(Wqkv norm(x)))

over a paged cache of keys and values in NVFP4: a prompt's rows are appended to it and
attend to each other in bf16, a decode step attends to the cache.

A prefill step takes the rows of several prompts at once: the activation is
quantized and multiplied on the block-scaled GEMM, each row with its request's
adapter.  A decode step takes one row a request, unquantized, in four launches.
The workspaces are kept from step to step; calls on one stream may share them.

    python examples/serve_step.py [--attention]        (needs an MI355X)
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_block_scaled_04_amd import attention, ops, serving  # noqa: E402

MOE_TOKENS = 64  # most tokens of one nvfp4_moe_small call


def norm(x):
    f = x.float()
    return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Cache:
    """Pages of keys and values in NVFP4 for `requests` requests of up to `most` tokens."""

    def __init__(self, requests, most, heads, d, page=64, k_max=16.0, v_max=16.0):
        per = -(-most // page)
        self.page = page
        self.kv = torch.empty(requests * per, 2, heads, page, d // 2, dtype=torch.uint8, device="cuda")
        self.kv_sf = torch.empty(requests * per, 2, heads, d // 16, page, dtype=torch.uint8, device="cuda")
        self.kv_gs = torch.tensor([2688 / k_max, 2688 / v_max], device="cuda")  # calibrated: the largest key and value
        order = torch.randperm(requests * per, device="cuda").int()
        self.block_table = order.view(requests, per).contiguous()
        self.lengths = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def slots(self, request, position):
        """Slots of tokens at `position` of their requests."""
        return self.block_table[request, position // self.page] * self.page + (position % self.page).int()


class Attention:
    """Grouped-query attention with NVFP4 projections: h hidden, q_heads and heads of width d."""

    def __init__(self, h, q_heads, heads, d, max_requests, seed=0, sections=None, base=1e4):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def pack(n, k):
            return ops.nvfp4_quantize((torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).bfloat16())

        self.q_heads, self.heads, self.d = q_heads, heads, d
        self.wqkv, self.wqkv_sf, self.gs_qkv = pack((q_heads + 2 * heads) * d, h)
        self.wo, self.wo_sf, self.gs_o = pack(h, q_heads * d)
        self.sections = sections or (d // 2,)
        self.inv_freq = (base ** -(torch.arange(d // 2, device="cuda", dtype=torch.float64) / (d // 2))).float()
        self.workspace = torch.empty(attention.attention_ws_bytes(max_requests, d), dtype=torch.uint8, device="cuda")

    def qkv(self, x, position, project):
        """Rotated q, rotated k and v of rows x: parts of one projection's output."""
        y = project(norm(x), self.wqkv, self.wqkv_sf, self.gs_qkv).view(len(x), -1, self.d)
        turned = y[:, : self.q_heads + self.heads]
        attention.rope_axes(turned, position.int().expand(len(self.sections), -1).contiguous(), self.inv_freq, self.sections, out=turned)
        return y[:, : self.q_heads], turned[:, self.q_heads:], y[:, self.q_heads + self.heads:]

    def prefill(self, x, lengths, cache):
        """Whole prompts of `lengths`, one after the other; each is a request of the cache."""
        request = torch.arange(len(lengths), device="cuda").repeat_interleave(lengths)
        cu = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)]).int()
        position = torch.arange(len(x), device="cuda") - cu[request]
        q, k, v = self.qkv(x, position, wide)
        attention.nvfp4_kv_append(k, v, cache.slots(request, position), cache.kv_gs, cache.kv, cache.kv_sf)
        cache.lengths.copy_(lengths)
        out = attention.attention_prefill(q, k, v, cu)
        return x + wide(out.view(len(x), -1), self.wo, self.wo_sf, self.gs_o)

    def decode(self, x, cache):
        """One more token of every request."""
        position = cache.lengths.long()
        q, k, v = self.qkv(x, position, narrow)
        request = torch.arange(len(x), device="cuda")
        attention.nvfp4_kv_append(k, v, cache.slots(request, position), cache.kv_gs, cache.kv, cache.kv_sf)
        cache.lengths += 1
        out = attention.nvfp4_attention_decode(q[:, None], cache.kv, cache.kv_sf, cache.kv_gs, cache.block_table,
                                               cache.lengths, workspace=self.workspace)
        return x + narrow(out.view(len(x), -1), self.wo, self.wo_sf, self.gs_o)


def wide(x, w, sf, gs):
    """Many rows: quantized, then the block-scaled product."""
    codes, x_sf, _, alpha = ops.nvfp4_quantize_alpha(x.contiguous(), gs)
    return ops.nvfp4_gemm(codes, w, x_sf, sf, alpha)


def narrow(x, w, sf, gs):
    """Few rows, unquantized."""
    return ops.nvfp4_gemm_w4a16(x.contiguous(), w, sf, 1 / gs)


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


def main(h=4096, inter=1024, experts=32, top_k=4, adapters=8, r=16, prompts=(37, 5, 96, 1, 61), steps=16, attend=None):
    """attend: None, or (q_heads, heads, width) of an attention block before the layer."""
    layer = Layer(h, inter, experts, top_k, adapters, r)
    if attend:
        block = Attention(h, *attend, max_requests=len(prompts))
        cache = Cache(len(prompts), max(prompts) + steps + 1, attend[1], attend[2])
    g = torch.Generator(device="cuda").manual_seed(1)
    # a request's adapter; -1: the shared weights alone
    request = torch.tensor([i % (adapters + 1) - 1 for i in range(len(prompts))], dtype=torch.int32, device="cuda")
    lengths = torch.tensor(prompts, device="cuda")
    x = torch.randn(sum(prompts), h, device="cuda", generator=g).bfloat16()

    def step(token):
        return layer.decode(block.decode(token, cache) if attend else token, request)

    x = block.prefill(x, lengths, cache) if attend else x
    z = layer.prefill(x, request.repeat_interleave(lengths))
    token = z[lengths.cumsum(0) - 1]  # each request's last row
    token = step(token)  # first step, untimed
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(steps):
        token = step(norm(token))
    torch.cuda.synchronize()
    print(f"prefill of {sum(prompts)} rows, {len(prompts)} requests; {(time.perf_counter() - t0) / steps * 1e6:.0f} us a "
          f"decode step (launches from Python); finite: {bool(torch.isfinite(token).all())}")
    return token


if __name__ == "__main__":
    main(attend=(32, 8, 128) if "--attention" in sys.argv[1:] else None)
