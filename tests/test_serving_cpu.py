"""The serving operators' C ABI and binding without a GPU: every argument error
is returned before any HIP call (no pointer here is dereferenced), the binding's
names, argument counts and workspace sizes are the header's."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4_serving.h")
LIB = os.path.join(ROOT, "nvfp4_block_scaled_04_amd", "libnvfp4_amd.so")
NULLP, SHAPE, MISAL, RANK, DTYPE, UNSUP = 1, 2, 3, 4, 5, 6
P = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def serving():
    if not os.path.exists(LIB):
        pytest.fail(f"{LIB} not built; run __graft_entry__.build()")
    from nvfp4_block_scaled_04_amd import serving as _s
    return _s


def test_header_and_binding_agree(serving):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    decl = {name: args.count(",") + 1 for name, args in re.findall(r"^int\s+(\w+)\s*\((.*?)\);", src, flags=re.M | re.S)}
    assert sorted(decl) == sorted(serving.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True).stdout
    for name, n in decl.items():
        assert re.search(rf"\bT {name}$", out, flags=re.M), name
        assert len(getattr(serving._lib, name).argtypes) == n, name


MOE = dict(x=P, t=4, h=64, logits=P, dt=1, E=8, k=2, score=0, renorm=1, w13=P, sf13=P, al13=P, w2=P, sf2=P, al2=P, inter=32,
           out=P, ids=P, wts=P, ws=P, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({n: None}, NULLP) for n in ("x", "logits", "w13", "sf13", "al13", "w2", "sf2", "al2", "out", "ids", "wts", "ws")],
    ({"dt": 2}, DTYPE), ({"t": 0}, SHAPE), ({"t": -1}, SHAPE), ({"t": 65}, UNSUP), ({"E": 0}, SHAPE), ({"E": 257}, UNSUP),
    ({"k": 0}, SHAPE), ({"k": 9}, SHAPE), ({"E": 64, "k": 17}, UNSUP), ({"h": 0}, SHAPE), ({"h": 40}, SHAPE),
    ({"inter": 8}, SHAPE), ({"inter": 0}, SHAPE), ({"score": 2}, UNSUP), ({"h": 1 << 24, "inter": 256}, UNSUP),
    ({"wsb": 4 * 4 * 2 * 32 + 4096 + 4096 * 128 + 32 - 1}, SHAPE), ({"x": P + 8}, MISAL), ({"w13": P + 4}, MISAL), ({"w2": P + 8}, MISAL),
    ({"sf13": P + 8}, MISAL), ({"sf2": P + 8}, MISAL), ({"logits": P + 4}, MISAL), ({"out": P + 2}, MISAL),
    ({"ws": P + 8}, MISAL), ({"ids": P + 2}, MISAL), ({"wts": P + 1}, MISAL), ({"al13": P + 2}, MISAL), ({"al2": P + 3}, MISAL),
])
def test_moe_small_validation(serving, change, status):
    assert serving._lib.nvfp4_moe_small(*{**MOE, **change}.values()) == status


LIN = dict(x=P, b=P, sf=P, alpha=P, la=P, lb=P, ad=P, sc=None, bias=None, out=P, m=4, n=32, k=64, r=16, L=3, ws=P, wsb=256,
           stream=None)
GEMM = dict(a=P, b=P, asf=P, sf=P, alpha=P, x=P, la=P, lb=P, ad=P, sc=None, bias=None, out=P, m=4, n=32, k=64, r=16, L=3,
            ws=P, wsb=256, stream=None)
COMMON = [
    *[({n: None}, NULLP) for n in ("x", "b", "sf", "alpha", "la", "lb", "ad", "out", "ws")],
    ({"r": 0}, RANK), ({"r": -8}, RANK), ({"r": 12}, RANK), ({"r": 264}, RANK), ({"m": 0}, SHAPE), ({"n": 0}, SHAPE),
    ({"k": 8}, SHAPE), ({"k": 72}, SHAPE), ({"L": 0}, SHAPE), ({"wsb": 255}, SHAPE), ({"m": 1 << 21, "wsb": 1 << 40}, SHAPE),
    ({"n": 1 << 24, "k": 1 << 12}, UNSUP), ({"n": 1 << 29, "k": 16}, UNSUP), ({"k": (1 << 23) + 16}, UNSUP),
    ({"x": P + 8}, MISAL), ({"la": P + 8}, MISAL), ({"lb": P + 2}, MISAL),
    ({"ad": P + 2}, MISAL), ({"sc": P + 2}, MISAL), ({"bias": P + 2}, MISAL), ({"ws": P + 4}, MISAL), ({"b": P + 8}, MISAL),
    ({"sf": P + 8}, MISAL), ({"alpha": P + 2}, MISAL), ({"out": P + 8}, MISAL),
]


@pytest.mark.parametrize("change,status", COMMON)
def test_linear_adapters_validation(serving, change, status):
    assert serving._lib.nvfp4_linear_adapters(*{**LIN, **change}.values()) == status


@pytest.mark.parametrize("change,status", COMMON + [({"a": None}, NULLP), ({"asf": None}, NULLP), ({"a": P + 8}, MISAL),
                                                    ({"asf": P + 8}, MISAL)])
def test_gemm_adapters_validation(serving, change, status):
    assert serving._lib.nvfp4_gemm_adapters(*{**GEMM, **change}.values()) == status


@pytest.mark.parametrize("call,base", [("nvfp4_linear_adapters", LIN), ("nvfp4_gemm_adapters", GEMM)])
def test_adapters_row_limit(serving, call, base):
    """Any m up to 2^20 (checked before the misaligned weight), none beyond."""
    f, big = getattr(serving._lib, call), {"wsb": 1 << 40, "n": 16, "k": 16, "r": 8}
    for m in (1048560, 1048561, 1 << 20):
        assert f(*{**base, **big, "m": m, "b": P + 8}.values()) == MISAL
    assert f(*{**base, **big, "m": (1 << 20) + 1, "b": P + 8}.values()) == SHAPE


def test_workspace_sizes(serving, tmp_path):
    shapes = [(1, 1, 16), (64, 16, 8192), (7, 3, 48)]   # (t, top_k, h), inter = 2 h; (m, ., r)
    src = tmp_path / "ws.c"
    lines = ["#include <stdio.h>", '#include "nvfp4_serving.h"', "int main(void) {"]
    for a, b, c in shapes:
        lines.append(f'  printf("%lld %lld\\n", (long long)NVFP4_MOE_SMALL_WS_BYTES({a}, {b}, {c}, {2 * c}), '
                     f"(long long)NVFP4_ADAPTERS_WS_BYTES({a}, {c}));")
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "ws"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    for (a, b, c), line in zip(shapes, out):
        assert [int(v) for v in line.split()] == [serving.moe_small_ws_bytes(a, b, c, 2 * c), serving.adapters_ws_bytes(a, c)]
    assert serving.adapters_ws_bytes(5, 24, split=True) == serving.adapters_ws_bytes(5, 24) + 33554432


def test_host_tensors_refused(serving):
    """The binding takes device tensors only; nothing falls back to the host."""
    x, lg = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 4)
    z = torch.zeros(4, 64, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        serving.nvfp4_moe_small(x, lg, z, z, lg[0], z, z, lg[0], 1)
    with pytest.raises(ValueError):
        serving.nvfp4_linear_adapters(x, z[0], z, lg[0], z, z, lg[0])
    with pytest.raises(ValueError):
        serving.nvfp4_gemm_adapters(z[0], z[0], z, z, lg[0], x, z, z, lg[0])


def test_reference_bound_admits_the_rounded_reference():
    """A bf16 output that is the 64-bit value correctly rounded differs from it by
    up to 2^-8 of itself: 1 + 2^-8 lies halfway between two bf16 values."""
    v = torch.tensor([1 + 2.0 ** -8, 3 + 2.0 ** -7], dtype=torch.float64)
    assert ((v.bfloat16().double() - v).abs() / v > 2.0 ** -9).all()
    w = torch.rand(100000, dtype=torch.float64) + 1
    assert ((w.bfloat16().double() - w).abs() / w <= 2.0 ** -8).all()
