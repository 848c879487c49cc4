"""The attention operators' measured cases: what a prompt or a decode step hands
them, their plain torch forms and their definitions in 64 bits.

The operators (nvfp4_block_scaled_04_amd.attention):
  * rope    -- rotary positions with several axes (text, or time, height and
               width of a video), in place on the heads of a projection's output.
  * append  -- new keys and values quantized to NVFP4 into the slots of a paged
               cache, and read back as bf16 (the two calls of a cached prefix).
  * decode  -- attention of one or a few tokens a sequence over the 4-bit cache,
               grouped heads, sequences of any length.
  * prefill -- attention over whole prompts packed one after the other, causal or
               full, grouped heads, with or without a prefix.

The cache: kv [pages, 2, heads, page, d/2] packed e2m1 (K then V, element 2i in the
low nibble of byte i), kv_sf [pages, 2, heads, d/16, page] ue4m3 scales of 16
elements, kv_gs [2] the global scales; slot = page index * page size + position.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
SCRATCH = 64 << 20            # bytes of workspace a serving program keeps for all its calls
CACHED = 64 * 9000 * 8 * 128  # cached tokens x heads x width of the largest decode case
PAIRS = 40 * 8192 * 8192      # heads x rows x keys of the largest prefill case
WIDE = 20280 * 48 * 128       # elements of the largest rope case


# ---- the cases ----------------------------------------------------------------

def listed():
    return [
        # one decode step of 16 conversations: text positions on a vision-language
        # model's three axes, pairs in halves; latency
        {"name": "rope 16 tokens", "op": "rope", "t": 16, "heads": 40, "pad": 8, "d": 128, "rot": 128, "style": "halves",
         "sections": "16,24,24", "base": 1e6, "grid": "text"},
        # a clip of 13 x 30 x 52 patches, q and k of 24 heads: a whole forward pass
        {"name": "rope 20280 video patches", "op": "rope", "t": 20280, "heads": 48, "pad": 24, "d": 128, "rot": 128,
         "style": "pairs", "sections": "22,21,21", "base": 1e4, "grid": "video"},
        # the tokens of one decode step into the cache
        {"name": "append 16 tokens", "op": "append", "t": 16, "heads": 8, "d": 128, "page": 64, "skip": False},
        # a prompt of odd length into scattered pages, a few rows of padding without a slot
        {"name": "append 8003 rows", "op": "append", "t": 8003, "heads": 8, "d": 128, "page": 16, "skip": True},
        # one long conversation: its cache has to be spread over the whole card
        {"name": "decode 1 of 32768", "op": "decode", "b": 1, "new": 1, "q": 32, "kv": 8, "d": 128, "page": 64,
         "most": 32768, "even": True, "lse": False},
        # a batch of unequal conversations on small pages
        {"name": "decode 16 to 8192", "op": "decode", "b": 16, "new": 1, "q": 40, "kv": 8, "d": 128, "page": 16,
         "most": 8192, "even": False, "lse": False},
        # odd sizes: three draft tokens to check, narrow heads, an empty sequence
        {"name": "decode 7 x 3 drafts, odd sizes", "op": "decode", "b": 7, "new": 3, "q": 21, "kv": 3, "d": 64, "page": 32,
         "most": 2001, "even": False, "lse": True},
        # the largest batch: half a billion cached elements a tensor
        {"name": "decode 64 to 16384", "op": "decode", "b": 64, "new": 1, "q": 64, "kv": 8, "d": 128, "page": 64,
         "most": 16384, "even": False, "lse": False},
        # a short question: latency
        {"name": "prefill 1 prompt of 61", "op": "prefill", "b": 1, "q": 32, "kv": 8, "d": 128, "most": 61, "prefix": 0,
         "even": True, "causal": True, "lse": False},
        # many prompts of unequal, odd length with cached prefixes, narrow heads
        {"name": "prefill 23 ragged, prefixes", "op": "prefill", "b": 23, "q": 12, "kv": 4, "d": 64, "most": 701,
         "prefix": 519, "even": False, "causal": True, "lse": True},
        # the patches of two clips, every patch sees its whole clip
        {"name": "prefill 2 clips, full", "op": "prefill", "b": 2, "q": 24, "kv": 24, "d": 128, "most": 4680, "prefix": 0,
         "even": True, "causal": False, "lse": False},
        # the large prompt
        {"name": "prefill 1 prompt of 8192", "op": "prefill", "b": 1, "q": 40, "kv": 8, "d": 128, "most": 8192, "prefix": 0,
         "even": True, "causal": True, "lse": False},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("rope", "append", "decode", "decode", "prefill", "prefill"))
    d = rng.choice((64, 80, 96, 128, 128, 128, 256))
    if op == "rope":
        heads, rot = _log(rng, 1, 48), rng.choice((d, d, d // 2))
        axes = rng.choice((1, 2, 3, 3))
        cut = [rot // 2 * (a + 1) // axes for a in range(axes)]
        return {"op": op, "t": _log(rng, 1, WIDE // (heads * d)), "heads": heads, "pad": rng.choice((0, 1, 8)), "d": d,
                "rot": rot, "style": rng.choice(("halves", "pairs")),
                "sections": ",".join(str(b - a) for a, b in zip([0] + cut, cut)), "base": rng.choice((1e4, 5e5, 1e6)),
                "grid": rng.choice(("text", "video"))}
    if op == "append":
        return {"op": op, "t": _log(rng, 1, 8192), "heads": _log(rng, 1, 8), "d": min(d, 128),
                "page": rng.choice((16, 32, 64, 128)), "skip": rng.random() < 0.5}
    kv = _log(rng, 1, 8)
    group = _log(rng, 1, 16)
    if op == "decode":
        b = _log(rng, 1, 64)
        return {"op": op, "b": b, "new": rng.choice((1, 1, 1, 2, 5)), "q": kv * group, "kv": kv, "d": d,
                "page": rng.choice((16, 32, 64, 128)), "most": _log(rng, 16, min(65536, CACHED // (b * kv * d))),
                "even": rng.random() < 0.3, "lse": rng.random() < 0.5}
    most = _log(rng, 1, 4096)
    q = kv * max(1, min(group, 40 // kv))
    prefix = rng.choice((0, 0, 1)) * _log(rng, 1, 4096)
    b = _log(rng, 1, max(1, min(64, PAIRS // (q * most * (most + prefix) * 2))))
    return {"op": op, "b": b, "q": q, "kv": kv, "d": d, "most": most, "prefix": prefix, "even": rng.random() < 0.3,
            "causal": rng.random() < 0.7, "lse": rng.random() < 0.5}


# ---- inputs -------------------------------------------------------------------

def _lengths(c, rng=None):
    """A case's sequences, (new or cached tokens, prefix) each; `rng` gives their order.  Unequal ones have one of
    the longest; batches of more than four have one without tokens (decode) or of a single one (prefill)."""
    fixed = random.Random(c["b"] * 65537 + c["most"])
    prefix = c.get("prefix", 0)
    if c["even"]:
        some = [(c["most"], prefix)] * c["b"]
    else:
        n = [c["most"]] + [fixed.randint(max(1, c["most"] // 8), c["most"]) for _ in range(c["b"] - 1)]
        if c["b"] > 4:
            n[-1] = 0 if c["op"] == "decode" else 1
        some = [(v, fixed.randint(0, prefix)) for v in n]
    return rng.sample(some, len(some)) if rng else some


def _codes(x, gs):
    """NVFP4 of x [..., 16 n] with a global scale: codes (one a byte) and ue4m3 bytes, in the library's fp32 steps."""
    b = x.float().unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / 6 * gs).clamp(max=448).to(torch.float8_e4m3fn)
    d = s.float()[..., None]
    v = torch.where(d == 0, torch.zeros_like(b), b * (gs / d))
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    return (code | (v < 0).to(torch.uint8) << 3).flatten(-2), s.view(torch.uint8)


def _keys(shape, g):
    """Keys ~ N(0, 1), one channel of sixteen four times as large (the same for all tokens of a head)."""
    k = torch.randn(shape, generator=g, device=DEV)
    return k * (1 + 3 * (torch.rand(shape[-2:], generator=g, device=DEV) < 1 / 16).float())


def _cache(pages, kv, page, d, g):
    k, v = _keys((pages, page, kv, d), g), torch.randn((pages, page, kv, d), generator=g, device=DEV)
    gs = torch.stack([2688 / k.abs().amax(), 2688 / v.abs().amax()])
    pair = []
    for x, s in ((k, gs[0]), (v, gs[1])):
        code, sf = _codes(x, s)
        pair.append(((code[..., 0::2] | code[..., 1::2] << 4).transpose(1, 2).contiguous(), sf.permute(0, 2, 3, 1).contiguous()))
    return torch.stack([pair[0][0], pair[1][0]], 1), torch.stack([pair[0][1], pair[1][1]], 1), gs


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = random.Random(seed)
    byte = torch.arange(256, device=DEV)
    signed = torch.tensor(E2M1 + [-v for v in E2M1], device=DEV)
    s = {"case": c, "table": torch.stack([signed[byte & 15], signed[byte >> 4]], -1)}   # byte -> its two values
    d = c["d"]
    if c["op"] == "rope":
        t, cuts = c["t"], [int(v) for v in c["sections"].split(",")]
        at = torch.arange(t, device=DEV)
        if c["grid"] == "video":   # time, height and width of a patch, 30 x 52 patches a frame
            pos = [at // 1560, at % 1560 // 52, at % 52][3 - len(cuts):]
        else:                      # far into a long conversation
            far = torch.randint(0, 1 << 20, (t,), generator=g, device=DEV)
            pos = [far + a for a in range(len(cuts))]
        freq = torch.cat([c["base"] ** -(torch.arange(n, device=DEV, dtype=torch.float64) / n) for n in cuts])
        # a projection's output: the rotated heads, then `pad` others that stay as they are
        s.update(sections=cuts, inv_freq=freq.float(), positions=torch.stack(pos).int(),
                 x=torch.randn(t, c["heads"] + c["pad"], d, generator=g, device=DEV).bfloat16(),
                 out=torch.empty(t, c["heads"], d, dtype=torch.bfloat16, device=DEV))
        return s
    if c["op"] == "append":
        t, heads, page = c["t"], c["heads"], c["page"]
        pages = -(-t // page) + 3
        kv, kv_sf, gs = _cache(pages, heads, page, d, g)
        order = torch.tensor(rng.sample(range(pages), pages), device=DEV)
        at = torch.arange(t, device=DEV)
        slots = order[at // page] * page + at % page
        if c["skip"]:
            slots[t - t // 16:] = -1
        s.update(kv=kv, kv_sf=kv_sf, kv_gs=gs, slots=slots.int(), k=_keys((t, heads, d), g).bfloat16(),
                 v=torch.randn(t, heads, d, generator=g, device=DEV).bfloat16(),
                 k_out=torch.zeros(t, heads, d, dtype=torch.bfloat16, device=DEV),
                 v_out=torch.zeros(t, heads, d, dtype=torch.bfloat16, device=DEV))
        return s
    if c["op"] == "decode":
        b, page = c["b"], c["page"]
        lens = [n for n, _ in _lengths(c, rng)]
        per = -(-c["most"] // page)
        pages = sum(-(-n // page) for n in lens) + 5
        order, table = rng.sample(range(pages), pages), []
        for n in lens:
            mine = [order.pop() for _ in range(-(-n // page))]
            table.append(mine + [0] * (per - len(mine)))
        kv, kv_sf, gs = _cache(pages, c["kv"], page, d, g)
        s.update(kv=kv, kv_sf=kv_sf, kv_gs=gs, lengths=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 block_table=torch.tensor(table, dtype=torch.int32, device=DEV), scale=d ** -0.5,
                 q=torch.randn(b, c["new"], c["q"], d, generator=g, device=DEV).bfloat16(),
                 out=torch.empty(b, c["new"], c["q"], d, dtype=torch.bfloat16, device=DEV),
                 lse=torch.empty(b, c["new"], c["q"], device=DEV) if c["lse"] else None,
                 scratch=torch.empty(SCRATCH, dtype=torch.uint8, device=DEV))
        return s
    lq, lk = zip(*((n, n + p) for n, p in _lengths(c, rng)))
    cu = [torch.tensor([0, *n], device=DEV).cumsum(0).int() for n in (lq, lk)]
    tq, tk = sum(lq), sum(lk)
    s.update(cu_q=cu[0], cu_k=cu[1], most_q=max(lq), most_k=max(lk), scale=d ** -0.5,
             q=torch.randn(tq, c["q"], d, generator=g, device=DEV).bfloat16(), k=_keys((tk, c["kv"], d), g).bfloat16(),
             v=torch.randn(tk, c["kv"], d, generator=g, device=DEV).bfloat16(),
             out=torch.empty(tq, c["q"], d, dtype=torch.bfloat16, device=DEV),
             lse=torch.empty(tq, c["q"], device=DEV) if c["lse"] else None)
    return s


# ---- the plain forms -----------------------------------------------------------

def _rope_plain(s):
    c = s["case"]
    half = c["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=DEV), torch.tensor(s["sections"], device=DEV))
    angle = s["positions"][axis].t().double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = s["x"][:, :c["heads"]].float()
    out = x.clone()
    if c["style"] == "halves":
        x1, x2 = x[..., :half], x[..., half:2 * half]
        out[..., :half], out[..., half:2 * half] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    else:
        x1, x2 = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return out.bfloat16()


def _values(codes, sf, table):
    """fp32 values (before the global scale) of rows of codes [..., d/2] with scales [..., d/16]."""
    v = table[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    return (v * sf.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _append_plain(s):
    page = s["case"]["page"]
    live = (s["slots"] >= 0).nonzero()[:, 0]
    at, off = s["slots"][live].long() // page, s["slots"][live].long() % page
    out = {"k": s["k_out"], "v": s["v_out"]}

    def one(which, x, to):
        code, sf = _codes(x[live], s["kv_gs"][which])
        s["kv"][at, which, :, off] = code[..., 0::2] | code[..., 1::2] << 4
        s["kv_sf"][at, which, :, :, off] = sf
        back = _values(s["kv"][at, which, :, off], s["kv_sf"][at, which, :, :, off], s["table"])
        to[live] = (back / s["kv_gs"][which]).bfloat16()

    one(0, s["k"], out["k"])
    one(1, s["v"], out["v"])
    return out


def _softmax(sc, seen, v):
    """(softmax of the scores that are seen) @ v and the log of the sum; rows that see nothing are zeros and -inf."""
    sc = torch.where(seen, sc, torch.full_like(sc, -math.inf))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(sc - top)
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, torch.ones_like(total), total), (top + total.log())[..., 0]


def _decode_plain(s):
    c = s["case"]
    b, new, kv, d, group = c["b"], c["new"], c["kv"], c["d"], c["q"] // c["kv"]
    codes = s["kv"][s["block_table"].long()]       # [b, pages, 2, kv, page, d/2]
    sf = s["kv_sf"][s["block_table"].long()].transpose(-1, -2)
    k = _values(codes[:, :, 0], sf[:, :, 0], s["table"]).transpose(1, 2).reshape(b, kv, -1, d) / s["kv_gs"][0]
    v = _values(codes[:, :, 1], sf[:, :, 1], s["table"]).transpose(1, 2).reshape(b, kv, -1, d) / s["kv_gs"][1]
    q = s["q"].float().view(b, new, kv, group, d).transpose(1, 2).reshape(b, kv, new * group, d)
    sc = (q @ k.transpose(-1, -2) * s["scale"]).view(b, kv, new, group, -1)
    last = s["lengths"][:, None] - (new - 1 - torch.arange(new, device=DEV))
    seen = torch.arange(sc.shape[-1], device=DEV) < last[:, None, :, None, None]
    o, lse = _softmax(sc, seen, v[:, :, None])
    out = o.transpose(1, 2).reshape(b, new, c["q"], d).bfloat16()
    return {"out": out, "lse": lse.transpose(1, 2).reshape(b, new, c["q"])} if c["lse"] else out


def _prefill_plain(s):
    c = s["case"]
    kv, d, group, b = c["kv"], c["d"], c["q"] // c["kv"], c["b"]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    iq, ik = torch.arange(s["most_q"], device=DEV), torch.arange(s["most_k"], device=DEV)
    # the sequences side by side, padded to the longest
    q = s["q"].float()[(cq[:-1, None] + iq).clamp(max=len(s["q"]) - 1)].view(b, -1, kv, group, d).permute(0, 2, 3, 1, 4)
    at = (ck[:-1, None] + ik).clamp(max=len(s["k"]) - 1)
    k, v = s["k"].float()[at].transpose(1, 2), s["v"].float()[at].transpose(1, 2)
    sc = (q.reshape(b, kv, -1, d) @ k.transpose(-1, -2) * s["scale"]).view(b, kv, group, len(iq), len(ik))
    seen = (ik < lk[:, None])[:, None]
    if c["causal"]:
        seen = seen & (ik <= iq[:, None] + (lk - lq)[:, None, None])
    o, lse = _softmax(sc, seen[:, None, None], v[:, :, None])
    rows = (iq < lq[:, None]).nonzero()
    out = o.permute(0, 3, 1, 2, 4).reshape(b, -1, c["q"], d)[rows[:, 0], rows[:, 1]].bfloat16()
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(b, -1, c["q"])[rows[:, 0], rows[:, 1]]} if c["lse"] else out


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rope": _rope_plain, "append": _append_plain, "decode": _decode_plain, "prefill": _prefill_plain}[c["op"]](s)
    from nvfp4_block_scaled_04_amd import attention
    if c["op"] == "rope":
        return attention.rope_axes(s["x"][:, :c["heads"]], s["positions"], s["inv_freq"], s["sections"],
                                   interleaved=c["style"] == "pairs", out=s["out"])
    if c["op"] == "append":
        attention.nvfp4_kv_append(s["k"], s["v"], s["slots"], s["kv_gs"], s["kv"], s["kv_sf"])
        k, v = attention.nvfp4_kv_read(s["slots"], s["kv_gs"], s["kv"], s["kv_sf"], k=s["k_out"], v=s["v_out"])
        return {"k": k, "v": v}
    if c["op"] == "decode":
        out = attention.nvfp4_attention_decode(s["q"], s["kv"], s["kv_sf"], s["kv_gs"], s["block_table"], s["lengths"],
                                               scale=s["scale"], out=s["out"], lse=s["lse"], workspace=s["scratch"])
    else:
        out = attention.attention_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"],
                                          scale=s["scale"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": s["lse"]} if c["lse"] else out


# ---- work and the definitions in 64 bits ------------------------------------------

def work(case):
    c = case
    d = c["d"]
    if c["op"] == "rope":
        return {"bytes": 4 * c["t"] * c["heads"] * d + 4 * c["t"] * len(c["sections"].split(",")),
                "flops": 3 * c["t"] * c["heads"] * c["rot"]}
    if c["op"] == "append":   # bf16 in and out, the codes and scales written and read
        n = 2 * (c["t"] - (c["t"] // 16 if c["skip"] else 0)) * c["heads"] * d
        return {"bytes": n * (4 + 2 * 9 / 16), "flops": 4 * n}
    some = _lengths(c)
    if c["op"] == "decode":
        n = sum(v for v, _ in some)
        return {"bytes": n * c["kv"] * d * 9 / 8 + 4 * c["b"] * c["new"] * c["q"] * d,
                "flops": 4 * n * c["new"] * c["q"] * d}
    pairs = sum(n * p + (n * (n + 1) / 2 if c["causal"] else n * n) for n, p in some)
    return {"bytes": 4 * d * sum(n * c["q"] + (n + p) * c["kv"] for n, p in some), "flops": 4 * pairs * c["q"] * d}


def _exact_rows(x, gs):
    """What the cache holds of rows x [..., d], as float64: nearest codes by search, ties to the even code."""
    b = x.double().unflatten(-1, (-1, 16))
    want = (b.abs().amax(-1) / 6).float().double().mul(gs.double()).float().double()
    every = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()

    def nearest(v, table):
        hi = torch.searchsorted(table, v).clamp(max=len(table) - 1)
        lo = (hi - 1).clamp(min=0)
        up, down = table[hi] - v, v - table[lo]
        return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)

    s = every[nearest(want, every)][..., None]
    r = torch.where(s == 0, torch.zeros_like(s), (gs.double() / s).float().double())
    y = (b * r).float().double()
    mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    return (mag[nearest(y.abs(), mag)] * y.sign() * s / gs.double()).flatten(-2)


def _wide(kv, kv_sf, which, head, pages, gs):
    """The cached rows of one head on these pages, as float64 [tokens, d]."""
    codes = kv[pages, which, head].reshape(-1, kv.shape[-1])
    sf = kv_sf[pages, which, head].view(torch.float8_e4m3fn).double().transpose(1, 2).reshape(len(codes), -1)
    mag = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=DEV)
    v = torch.empty(len(codes), 2 * codes.shape[1], dtype=torch.float64, device=DEV)
    v[:, 0::2], v[:, 1::2] = mag[(codes & 15).long()], mag[(codes >> 4).long()]
    return v * sf.repeat_interleave(16, 1) / gs[which].double()


def _attend(q, k, v, scale, seen):
    """q [rows, d], k, v [keys, d] in float64, row r sees the first seen[r] keys."""
    sc = q @ k.t() * scale
    sc.masked_fill_(torch.arange(len(k), device=DEV) >= seen[:, None], -math.inf)
    lse = torch.logsumexp(sc, -1)
    p = torch.exp_(sc.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None]))
    return p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    d = c["d"]
    if c["op"] == "rope":
        half = c["rot"] // 2
        out = s["x"][:, :c["heads"]].double()
        first = 0
        for a, n in enumerate(s["sections"]):
            turn = torch.polar(torch.ones(c["t"], n, dtype=torch.float64, device=DEV),
                               s["positions"][a].double()[:, None] * s["inv_freq"][first:first + n].double())[:, None]
            for i in range(n):
                p = first + i
                at = (p, p + half) if c["style"] == "halves" else (2 * p, 2 * p + 1)
                z = torch.complex(out[..., at[0]], out[..., at[1]]) * turn[..., i]
                out[..., at[0]], out[..., at[1]] = z.real, z.imag
            first += n
        return out
    if c["op"] == "append":
        dead = (s["slots"] < 0)[:, None, None]
        return {n: _exact_rows(s[n], s["kv_gs"][i]).masked_fill(dead, 0.0) for i, n in enumerate(("k", "v"))}
    group = c["q"] // c["kv"]
    q = s["q"].double()
    out, lse = torch.zeros_like(q), torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=DEV)
    if c["op"] == "decode":
        for i, n in enumerate(s["lengths"].tolist()):
            if n:
                pages = s["block_table"][i, : -(-n // c["page"])].long()
                seen = n - (c["new"] - 1 - torch.arange(c["new"], device=DEV))
                for h in range(c["kv"]):
                    k, v = (_wide(s["kv"], s["kv_sf"], w, h, pages, s["kv_gs"])[:n] for w in (0, 1))
                    for j in range(h * group, (h + 1) * group):
                        out[i, :, j], lse[i, :, j] = _attend(q[i, :, j], k, v, s["scale"], seen)
    else:
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        for i in range(c["b"]):
            n, m = cq[i + 1] - cq[i], ck[i + 1] - ck[i]
            seen = torch.arange(n, device=DEV) + 1 + m - n if c["causal"] else torch.full((n,), m, device=DEV)
            for j in range(c["q"]):
                k, v = (s[w][ck[i]:ck[i + 1], j // group].double() for w in ("k", "v"))
                out[cq[i]:cq[i + 1], j], lse[cq[i]:cq[i + 1], j] = _attend(q[cq[i]:cq[i + 1], j], k, v, s["scale"], seen)
    return {"out": out, "lse": lse} if c["lse"] else out
