"""The attention operators' C ABI and binding without a GPU: every argument error is
returned before any HIP call (no device pointer here is dereferenced), the binding's names,
argument counts and workspace sizes are the header's."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4_attention.h")
LIB = os.path.join(ROOT, "nvfp4_block_scaled_04_amd", "libnvfp4_amd.so")
NULLP, SHAPE, MISAL, UNSUP = 1, 2, 3, 6
P = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def att():
    if not os.path.exists(LIB):
        pytest.fail(f"{LIB} not built; run __graft_entry__.build()")
    from nvfp4_block_scaled_04_amd import attention
    return attention


def test_header_and_binding_agree(att):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    decl = {name: args.count(",") + 1 for name, args in re.findall(r"^int\s+(\w+)\s*\((.*?)\);", src, flags=re.M | re.S)}
    assert sorted(decl) == sorted(att.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True).stdout
    for name, n in decl.items():
        assert re.search(rf"\bT {name}$", out, flags=re.M), name
        assert len(getattr(att._lib, name).argtypes) == n, name


def sec(*v):
    return (ctypes.c_int32 * len(v))(*v)


ROPE = dict(x=P, xs=512, out=P, outs=512, t=4, heads=4, d=128, pos=P, freq=P, sections=sec(24, 20, 20), axes=3, inter=0, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({n: None}, NULLP) for n in ("x", "out", "pos", "freq", "sections")],
    ({"t": 0}, SHAPE), ({"t": -1}, SHAPE), ({"heads": 0}, SHAPE), ({"d": 120}, SHAPE), ({"d": 0}, SHAPE), ({"xs": 504}, SHAPE), ({"outs": 508}, SHAPE),
    ({"xs": 516}, SHAPE), ({"xs": (1 << 22) + 8}, SHAPE), ({"axes": 0}, SHAPE), ({"axes": 5, "sections": sec(8, 8, 8, 8, 8)}, UNSUP),
    ({"heads": 1, "d": 1040, "xs": 1040, "outs": 1040}, UNSUP), ({"sections": sec(24, 20, 28)}, SHAPE), ({"sections": sec(24, 20, 19)}, SHAPE),
    ({"sections": sec(24, -8, 8)}, SHAPE), ({"sections": sec(0, 0, 0)}, SHAPE), ({"x": P + 8}, MISAL), ({"out": P + 2}, MISAL),
    ({"pos": P + 2}, MISAL), ({"freq": P + 1}, MISAL), ({"t": (1 << 27) + 1}, UNSUP),
])
def test_rope_validation(att, change, status):
    assert att._lib.rope_axes(*{**ROPE, **change}.values()) == status


CACHE = [
    ({"pages": 0}, SHAPE), ({"page": 8}, SHAPE), ({"page": 48}, SHAPE), ({"page": 8192}, UNSUP), ({"page": 0}, SHAPE), ({"page": -16}, SHAPE),
    ({"d": 8}, SHAPE), ({"d": 0}, SHAPE), ({"d": 88}, SHAPE), ({"d": 272}, UNSUP), ({"heads": 0}, SHAPE), ({"heads": 1 << 20}, UNSUP),
    ({"kv": P + 8}, MISAL), ({"sf": P + 4}, MISAL), ({"gs": P + 2}, MISAL),
]
APPEND = dict(k=P, ks=512, v=P, vs=512, t=4, heads=4, d=128, slots=P, gs=P, kv=P, sf=P, pages=10, page=64, stream=None)
READ = dict(kv=P, sf=P, gs=P, pages=10, page=64, slots=P, t=4, heads=4, d=128, k=P, ks=512, v=P, vs=512, stream=None)


@pytest.mark.parametrize("call,base", [("nvfp4_kv_append", APPEND), ("nvfp4_kv_read", READ)])
@pytest.mark.parametrize("change,status", [
    *[({n: None}, NULLP) for n in ("k", "v", "slots", "gs", "kv", "sf")], *CACHE, ({"t": 0}, SHAPE), ({"ks": 500}, SHAPE), ({"vs": 516}, SHAPE),
    ({"t": 1 << 30, "heads": 512, "ks": 1 << 16, "vs": 1 << 16}, UNSUP), ({"t": (1 << 26) + 1}, UNSUP), ({"k": P + 8}, MISAL), ({"v": P + 2}, MISAL), ({"slots": P + 2}, MISAL),
])
def test_rows_validation(att, call, base, change, status):
    assert getattr(att._lib, call)(*{**base, **change}.values()) == status


DEC = dict(q=P, qs=2048, b=2, t=1, hq=16, kv=P, sf=P, gs=P, heads=4, d=128, pages=10, page=64, table=P, per=5, lens=P, scale=0.1, out=P, lse=None,
           ws=P, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({n: None}, NULLP) for n in ("q", "kv", "sf", "gs", "table", "lens", "out", "ws")], *CACHE, ({"b": 0}, SHAPE), ({"t": 0}, SHAPE), ({"hq": 18}, SHAPE),
    ({"hq": 0}, SHAPE), ({"qs": 2040}, SHAPE), ({"qs": 2052}, SHAPE), ({"qs": (1 << 22) + 8}, SHAPE), ({"per": 0}, SHAPE), ({"t": 65}, UNSUP), ({"b": 65537}, UNSUP), ({"scale": 0.0}, UNSUP), ({"scale": -1.0}, UNSUP),
    ({"scale": float("nan")}, UNSUP), ({"scale": float("inf")}, UNSUP), ({"per": (1 << 24) + 1}, UNSUP), ({"hq": 1 << 16, "qs": 1 << 22}, SHAPE),
    ({"scale": 2.1e38}, UNSUP), ({"b": 65536, "t": 1, "hq": 132, "qs": 132 * 128}, UNSUP), ({"b": 65536, "t": 64, "hq": 16384, "heads": 8192, "qs": 1 << 21}, UNSUP),
    ({"wsb": 256 + 2048 * 64 * 130 - 1}, SHAPE), ({"q": P + 8}, MISAL), ({"out": P + 4}, MISAL), ({"ws": P + 8}, MISAL), ({"table": P + 1}, MISAL),
    ({"lens": P + 2}, MISAL), ({"lse": P + 2}, MISAL),
])
def test_decode_validation(att, change, status):
    assert att._lib.nvfp4_attention_decode(*{**DEC, **change}.values()) == status


PRE = dict(q=P, qs=2048, k=P, ks=512, v=P, vs=512, tq=9, tk=9, hq=16, heads=4, d=128, cq=P, ck=P, b=2, scale=0.1, causal=1, out=P, outs=2048, lse=None, ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({n: None}, NULLP) for n in ("q", "k", "v", "cq", "ck", "out")], ({"tq": 0}, SHAPE), ({"tk": 0}, SHAPE), ({"hq": 18}, SHAPE), ({"heads": 0}, SHAPE),
    ({"d": 0}, SHAPE), ({"d": 120}, SHAPE), ({"b": 0}, SHAPE), ({"qs": 2040}, SHAPE), ({"ks": 508}, SHAPE), ({"vs": 516}, SHAPE), ({"outs": 0}, SHAPE),
    ({"d": 272, "qs": 1 << 14, "ks": 1 << 14, "vs": 1 << 14, "outs": 1 << 14}, UNSUP), ({"scale": 0.0}, UNSUP), ({"scale": float("nan")}, UNSUP), ({"b": 65537}, UNSUP), ({"scale": 2.1e38}, UNSUP),
    ({"b": 65536, "hq": 128, "qs": 1 << 14, "outs": 1 << 14}, UNSUP), ({"tq": 1 << 30, "hq": 64, "qs": 8192, "outs": 8192}, UNSUP), ({"q": P + 2}, MISAL), ({"k": P + 8}, MISAL), ({"v": P + 4}, MISAL), ({"out": P + 8}, MISAL), ({"cq": P + 2}, MISAL),
    ({"ck": P + 1}, MISAL), ({"lse": P + 2}, MISAL),
])
def test_prefill_validation(att, change, status):
    assert att._lib.attention_prefill(*{**PRE, **change}.values()) == status


def test_workspace_sizes(att, tmp_path):
    shapes = [(1, 32), (64, 64), (33, 96), (1000, 128), (7, 160), (65536, 256)]
    src = tmp_path / "ws.c"
    src.write_text('#include <stdio.h>\n#include "nvfp4_attention.h"\nint main(void) {\n' + "".join(
        f'  printf("%lld\\n", (long long)NVFP4_ATTENTION_WS_BYTES({b}, {d}));\n' for b, d in shapes) + "  return 0;\n}\n")
    exe = tmp_path / "ws"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out] == [att.attention_ws_bytes(b, d) for b, d in shapes]


def test_host_tensors_refused(att):
    """The binding takes device tensors only; nothing falls back to the host."""
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 2, dtype=torch.int32)
    kv, sf = torch.zeros(3, 2, 4, 16, 32, dtype=torch.uint8), torch.zeros(3, 2, 4, 4, 16, dtype=torch.uint8)
    gs = torch.ones(2)
    with pytest.raises(ValueError):
        att.rope_axes(x, i, torch.ones(32), (32,))
    with pytest.raises(ValueError):
        att.nvfp4_kv_append(x, x, i[0], gs, kv, sf)
    with pytest.raises(ValueError):
        att.nvfp4_kv_read(i[0], gs, kv, sf)
    with pytest.raises(ValueError):
        att.nvfp4_attention_decode(x[:, None], kv, sf, gs, i.view(2, 1), i[0])
    with pytest.raises(ValueError):
        att.attention_prefill(x, x, x, i[0])


def test_prefill_workspace_sizes(att, tmp_path):
    """The binding asks for what the library checks, and the header's bound holds for it."""
    src = tmp_path / "w.c"
    src.write_text('#include <stdio.h>\n#include "nvfp4_attention.h"\n'
                   'int main(void) { printf("%lld %lld %lld\\n", (long long)NVFP4_ATTENTION_PREFILL_WS_BYTES(64), '
                   '(long long)NVFP4_ATTENTION_PREFILL_WS_BYTES(80), (long long)NVFP4_ATTENTION_PREFILL_WS_BYTES(256)); return 0; }\n')
    exe = tmp_path / "w"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    bound = dict(zip((64, 80, 256), map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())))
    some = 0
    for d in (64, 80, 256):
        for q_heads, heads in ((1, 1), (3, 3), (32, 8), (32, 32), (40, 1), (127, 127), (128, 2), (128, 128), (129, 3)):
            for b in (1, 2, 7, 64):
                for tq in (1, 16, 127, 128, 129, 300, 8191):
                    for tk in (1, 1535, 1536, 20000, 1 << 20):
                        need = att.attention_prefill_ws_bytes(tq, tk, q_heads, heads, b, d)
                        assert 0 <= need <= bound[d]
                        if need and some < 200:
                            some += 1
                            a = {**PRE, "tq": tq, "tk": tk, "hq": q_heads, "heads": heads, "b": b, "d": d, "qs": q_heads * d, "outs": q_heads * d, "ks": heads * d, "vs": heads * d,
                                 "ws": P}
                            assert att._lib.attention_prefill(*{**a, "wsb": need - 1}.values()) == SHAPE
                            assert att._lib.attention_prefill(*{**a, "ws": P + 8, "wsb": need}.values()) == MISAL
    assert some == 200
