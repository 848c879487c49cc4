"""The attention operators together, as a server uses them: prompts, decode steps, a prompt
behind a cached prefix, each against its 64-bit form on what it was handed; captured and
replayed steps; calls on several streams; the example's block."""
import importlib.util
import os

import pytest
import torch

import attention_ref as A
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def att():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from nvfp4_block_scaled_04_amd import attention
    return attention


class Server:
    """Requests with tokens of a fused projection's output, and their cache."""

    def __init__(self, att, lens, q_heads, heads, d, page, room, seed):
        self.att, self.q_heads, self.heads, self.d, self.page = att, q_heads, heads, d, page
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.b, self.lens = len(lens), list(lens)
        per = -(-(max(lens) + room) // page)
        pages = self.b * per + 1
        self.kv = torch.full((pages, 2, heads, page, d // 2), 0xFF, dtype=torch.uint8, device="cuda")
        self.sf = torch.full((pages, 2, heads, d // 16, page), 0xFF, dtype=torch.uint8, device="cuda")
        self.gs = torch.tensor([2688 / 6.0, 2688 / 5.0], device="cuda")
        self.table = torch.randperm(pages, device="cuda", generator=self.g)[: self.b * per].int().view(self.b, per).contiguous()
        self.sections = (d // 4, d // 8, d // 8)
        self.freq = (1e4 ** -(torch.arange(d // 2, device="cuda", dtype=torch.float64) / (d // 2))).float()
        self.scale = d ** -0.5

    def rows(self, request, position):
        """qkv of tokens, rotated in place: (q, k, v), parts of one tensor; slots."""
        n = len(position)
        qkv = torch.randn(n, self.q_heads + 2 * self.heads, self.d, device="cuda", generator=self.g).bfloat16()
        turned = qkv[:, : self.q_heads + self.heads]
        plain = turned.clone()
        pos = torch.stack([position, position // 3, position % 7]).int()
        self.att.rope_axes(turned, pos, self.freq, self.sections, out=turned)
        ref = A.rope(plain, pos, self.freq, self.sections, False)
        assert ((turned.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + (plain.double().abs().amax() * 2.0 ** -19)).all()
        slots = self.table[request, position // self.page] * self.page + (position % self.page).int()
        return qkv[:, : self.q_heads], turned[:, self.q_heads:], qkv[:, self.q_heads + self.heads:], slots.int()

    def cached(self, i, which):
        j = torch.arange(self.lens[i], device="cuda")
        slots = self.table[i, j // self.page].long() * self.page + j % self.page
        return A.rows(self.kv, self.sf, which, slots) / self.gs[which].double()

    def check(self, q, k, v, out, seen, half_step, tiny):
        """One sequence's rows of out against the 64-bit form."""
        group = self.q_heads // self.heads
        for h in range(self.q_heads):
            ref, _, bound, _ = A.attend(q[:, h].double(), k[:, h // group].double(), v[:, h // group].double(), self.scale, seen,
                                        half_step, tiny)
            assert A.worst(out[:, h], ref, bound) <= 1.0, h


@pytest.mark.parametrize("lens,q_heads,heads,d,page", [((37, 5, 130, 1), 8, 2, 128, 16), ((300, 64), 6, 6, 64, 64), ((65, 190, 2), 10, 2, 96, 32)])
def test_prompts_then_steps_then_a_prefix(att, lens, q_heads, heads, d, page):
    say("attention step", lens, q_heads, heads, d, page)
    s = Server(att, lens, q_heads, heads, d, page, 40, sum(lens))
    lengths = torch.tensor(lens, device="cuda")
    request = torch.arange(s.b, device="cuda").repeat_interleave(lengths)
    cu = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)]).int()
    position = torch.arange(sum(lens), device="cuda") - cu[request]
    q, k, v, slots = s.rows(request, position)
    att.nvfp4_kv_append(k, v, slots, s.gs, s.kv, s.sf)
    out = att.attention_prefill(q, k, v, cu)
    at = cu.tolist()
    for i, n in enumerate(lens):
        r = slice(at[i], at[i + 1])
        j = torch.arange(n, device="cuda")
        s.check(q[r], k[r], v[r], out[r], j <= j[:, None], 2.0 ** -8, 0.0)

    held = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(att.attention_ws_bytes(s.b, d), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        q, k, v, slots = s.rows(torch.arange(s.b, device="cuda"), held.long())
        att.nvfp4_kv_append(k, v, slots, s.gs, s.kv, s.sf)
        held += 1
        s.lens = held.tolist()
        out = att.nvfp4_attention_decode(q[:, None], s.kv, s.sf, s.gs, s.table, held, workspace=ws)
        for i, n in enumerate(s.lens):
            seen = torch.ones(1, n, dtype=torch.bool, device="cuda")
            s.check(q[i:i + 1], s.cached(i, 0), s.cached(i, 1), out[i], seen, 2.0 ** -11, 2.0 ** -25)

    # a longer prompt for every request behind what the cache holds: its prefix is read back
    # beside the new rows, one call for all of them
    more = [7 + 3 * i for i in range(s.b)]
    cu_q = torch.tensor([0] + more, device="cuda").cumsum(0).int()
    cu_k = torch.tensor([0] + [a + n for a, n in zip(s.lens, more)], device="cuda").cumsum(0).int()
    request = torch.arange(s.b, device="cuda").repeat_interleave(torch.tensor(more, device="cuda"))
    position = torch.arange(sum(more), device="cuda") - cu_q[request] + held.long()[request]
    q, k, v, slots = s.rows(request, position)
    kk = torch.zeros(int(cu_k[-1]), heads, d, dtype=torch.bfloat16, device="cuda")
    vv = torch.zeros_like(kk)
    where = torch.full((len(kk),), -1, dtype=torch.int32, device="cuda")
    for i, n in enumerate(s.lens):
        j = torch.arange(n, device="cuda")
        where[cu_k[i] + j] = s.table[i, j // page] * page + (j % page).int()
        kk[cu_k[i] + n: cu_k[i + 1]], vv[cu_k[i] + n: cu_k[i + 1]] = k[cu_q[i]:cu_q[i + 1]], v[cu_q[i]:cu_q[i + 1]]
    att.nvfp4_kv_read(where, s.gs, s.kv, s.sf, k=kk, v=vv)
    out = att.attention_prefill(q, kk, vv, cu_q, cu_k)
    for i, n in enumerate(s.lens):
        kr, vr = kk[cu_k[i]:cu_k[i + 1]], vv[cu_k[i]:cu_k[i + 1]]
        assert torch.equal(kr[:n], s.cached(i, 0).float().bfloat16()) and torch.equal(vr[:n], s.cached(i, 1).float().bfloat16())
        j = torch.arange(len(kr), device="cuda")
        r = slice(int(cu_q[i]), int(cu_q[i + 1]))
        s.check(q[r], kr, vr, out[r], j <= (n + torch.arange(more[i], device="cuda"))[:, None], 2.0 ** -8, 0.0)


def capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g


def step_of(att, s, ws, t):
    """A step's buffers and the calls on them: t new tokens of every request."""
    b = s.b
    bufs = dict(qkv=torch.zeros(b * t, s.q_heads + 2 * s.heads, s.d, dtype=torch.bfloat16, device="cuda"),
                pos=torch.zeros(3, b * t, dtype=torch.int32, device="cuda"), slots=torch.full((b * t,), -1, dtype=torch.int32, device="cuda"),
                held=torch.zeros(b, dtype=torch.int32, device="cuda"), q=torch.zeros(b, t, s.q_heads, s.d, dtype=torch.bfloat16, device="cuda"),
                out=torch.zeros(b, t, s.q_heads, s.d, dtype=torch.bfloat16, device="cuda"), lse=torch.zeros(b, t, s.q_heads, device="cuda"))

    def run():
        y = bufs["qkv"]
        att.rope_axes(y[:, : s.q_heads], bufs["pos"], s.freq, s.sections, out=bufs["q"].view(b * t, s.q_heads, s.d))
        k = att.rope_axes(y[:, s.q_heads: s.q_heads + s.heads], bufs["pos"], s.freq, s.sections)
        att.nvfp4_kv_append(k, y[:, s.q_heads + s.heads:], bufs["slots"], s.gs, s.kv, s.sf)
        att.nvfp4_attention_decode(bufs["q"], s.kv, s.sf, s.gs, s.table, bufs["held"], out=bufs["out"], lse=bufs["lse"], workspace=ws)

    return bufs, run


def next_inputs(s, bufs, held, t):
    """The step's inputs for requests that hold `held` tokens before it."""
    position = (held[:, None] + torch.arange(t, device="cuda")).view(-1)
    request = torch.arange(s.b, device="cuda").repeat_interleave(t)
    bufs["qkv"].copy_(torch.randn(bufs["qkv"].shape, device="cuda", generator=s.g).bfloat16())
    bufs["pos"].copy_(torch.stack([position, position // 3, position % 7]).int())
    bufs["slots"].copy_(s.table[request, position // s.page] * s.page + (position % s.page).int())
    bufs["held"].copy_(held + t)


@pytest.mark.parametrize("t", [1, 3])
def test_captured_steps_replay(att, t):
    """Two captured steps that share a workspace, replayed in turn while lengths grow by leaps, with
    eager work between: every replay as the eager calls."""
    say("attention graph", t)
    servers = [Server(att, (900, 3, 0, 40), 8, 2, 128, 16, 3000, 1), Server(att, (60,), 21, 3, 64, 32, 5000, 2)]
    ws = torch.empty(max(att.attention_ws_bytes(s.b, s.d) for s in servers), dtype=torch.uint8, device="cuda")
    steps = [step_of(att, s, ws, t) for s in servers]
    graphs = [capture(run) for _, run in steps]
    for leap in (0, 1, 260, 2000):
        for s, (bufs, run), g in zip(servers, steps, graphs):
            held = torch.tensor([n + leap if n else 0 for n in s.lens], device="cuda")
            s.kv.random_(0, 256)
            s.sf.random_(0, 0x70)
            next_inputs(s, bufs, held, t)
            before = s.kv.clone(), s.sf.clone()
            run()
            want = bufs["out"].clone(), bufs["lse"].clone(), s.kv.clone(), s.sf.clone()
            s.kv.copy_(before[0])
            s.sf.copy_(before[1])
            ws.fill_(0xFF)
            bufs["out"].fill_(float("nan"))
            torch.cuda.synchronize()
            for _ in range(2):
                g.replay()
                torch.cuda.synchronize()
                got = bufs["out"], bufs["lse"], s.kv, s.sf
                assert all(torch.equal(a, b) for a, b in zip(got, want)), leap
                torch.randn(1000, 1000, device="cuda") @ torch.randn(1000, 1000, device="cuda")


def test_captured_prefill_replays(att):
    """Offsets that change between the replays, of a graph of the same tensors."""
    say("attention prefill graph")
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(1500, h, 128, device="cuda", generator=g).bfloat16() for h in (8, 2, 2))
    cu = torch.tensor([0, 700, 1500], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    run = lambda: att.attention_prefill(q, k, v, cu, out=out)  # noqa: E731
    graph = capture(run)
    for cut in (700, 1, 1499, 0, 1500, 64):
        cu[1] = cut
        out.fill_(float("nan"))
        run()
        want = out.clone()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), cut


def test_captured_prefix_replays(att):
    """The same where workgroups share the keys."""
    say("attention prefix graph")
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(150, 8, 128, device="cuda", generator=g).bfloat16()
    k, v = (torch.randn(6000, 2, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
    need = att.attention_prefill_ws_bytes(150, 6000, 8, 2, 2, 128)
    assert need > 0
    cu_q, cu_k = (torch.tensor([0, 70, n], dtype=torch.int32, device="cuda") for n in (150, 6000))
    out, ws = torch.zeros_like(q), torch.empty(need, dtype=torch.uint8, device="cuda")
    run = lambda: att.attention_prefill(q, k, v, cu_q, cu_k, out=out, workspace=ws)  # noqa: E731
    graph = capture(run)
    for a, b in ((70, 3000), (1, 5999), (149, 200), (0, 0), (150, 6000), (64, 1)):
        cu_q[1], cu_k[1] = a, b
        out.fill_(float("nan"))
        run()
        want = out.clone()
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and bool(out.isfinite().all()), (a, b)


def test_streams(att):
    """Calls on two streams at once, with a workspace each, and tensors made on another stream."""
    say("attention streams")
    servers = [Server(att, (2500, 800), 8, 2, 128, 64, 10, 4), Server(att, (3000,), 16, 2, 64, 16, 10, 5)]
    steps = []
    for s in servers:
        s.kv.random_(0, 256)
        s.sf.random_(0, 0x70)
        ws = torch.empty(att.attention_ws_bytes(s.b, s.d), dtype=torch.uint8, device="cuda")
        bufs, run = step_of(att, s, ws, 1)
        next_inputs(s, bufs, torch.tensor(s.lens, device="cuda"), 1)
        run()
        steps.append((bufs, run, bufs["out"].clone()))
        bufs["out"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for (bufs, run, _), st in zip(steps, streams):
            with torch.cuda.stream(st):
                run()
    torch.cuda.synchronize()
    for bufs, _, want in steps:
        assert torch.equal(bufs["out"], want)


def test_example_with_attention():
    say("serve_step with attention")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_step.py")
    spec = importlib.util.spec_from_file_location("serve_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    token = mod.main(h=512, inter=128, experts=8, top_k=2, adapters=3, r=8, prompts=(9, 1, 70), steps=2, attend=(8, 2, 64))
    assert token.shape == (3, 512) and bool(torch.isfinite(token).all())
