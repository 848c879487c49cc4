"""Which kernels the attention calls run, by their sizes: csrc/attention_plan.h, compiled by itself, on
the cases of attention_cases.py.  Every variant that any sizes reach is run by one of them, with
several tiles of rows and of keys wherever the variant takes such."""
import itertools
import os
import subprocess

import pytest

import attention_cases as C

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_block_scaled_04_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "attention_plan.h"
using namespace nvfp4;
int main() {
    char what[16];
    long long a[8];
    while (scanf("%15s %lld %lld %lld %lld %lld %lld %lld %lld", what, a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6, a + 7) == 9) {
        if (!strcmp(what, "prefill")) {
            const PrefillPlan p = prefill_plan(a[0], a[1], a[2], a[3], a[4], a[5], a[6] != 0, a[7] != 0);
            printf("%d %d %d %d %d %d\n", p.width, p.keys, p.waves, p.split, p.parts > 1, p.pack);
        } else if (!strcmp(what, "decode")) {
            const DecodePlan p = decode_plan(a[0], a[1], a[2], a[3], a[4], a[5]);
            printf("%d %d %d %d %d\n", p.width, p.two ? 2 : 1, p.once, p.packed, p.join ? p.join_waves : 0);
        } else if (!strcmp(what, "rope")) {
            const RopePlan p = rope_plan(a[0], a[1], a[2], a[3]);
            printf("%d %d\n", p.stream, p.width);
        } else {
            printf("%d\n", kv_rows_threads(a[0]));
        }
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(at / "plan.cpp"), "-o", str(at / "plan")], check=True)

    def ask(what, lines):
        text = "".join(" ".join(map(str, [what, *map(int, v), *[0] * (8 - len(v))])) + "\n" for v in lines)
        out = subprocess.run([str(at / "plan")], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == len(lines)
        return [tuple(map(int, o.split())) for o in out]
    return ask


def test_prefill(plan):
    sizes = [(tq, tk, q, h, d, b, causal, ws)
             for tq, tk, (q, h), d, b, causal, ws in itertools.product(
                 (1, 50, 200, 700, 2000, 9000), (60, 500, 1800, 9000, 40000), ((1, 1), (8, 2), (8, 8), (40, 8), (64, 64), (128, 4)), (64, 128, 256), (1, 3, 20, 200), (0, 1), (0, 1))
             if tk >= tq]
    reached = set(plan("prefill", sizes))
    assert len(reached) == 16
    # the binding hands a workspace over exactly where the plan has parts
    for causal in (0, 1):
        mine = plan("prefill", [(sum(lq), sum(lk), q, h, d, len(lq), causal, 1) for lq, lk, q, h, d in C.PREFILL])
        assert set(mine) == reached, sorted(reached - set(mine))
        for v in reached:
            width, keys, waves, split, parts, pack = v
            rows = 32 * waves // split
            cases = [c for c, m in zip(C.PREFILL, mine) if m == v]
            assert any(n * (c[2] // c[3] if pack else 1) > rows for c in cases for n in c[0]), (v, "one tile of rows")
            assert any(m >= 3 * keys * split for c in cases for m in c[1]), (v, "few tiles of keys")


def test_decode(plan):
    sizes = list(itertools.product((1, 2, 30, 400), (1, 3, 7), (8, 64), (1, 2, 8), (16, 48, 64, 80, 96, 128, 144, 160, 256), (64, 1024, 5000, 1 << 18)))
    reached = set(plan("decode", sizes))
    mine = plan("decode", [(len(lens), new, q, h, d, max(wide, (-(-max(lens) // page) + 1) * page)) for lens, new, q, h, d, page, wide in C.DECODE])
    kernels, joins = {v[:4] for v in reached}, {(*v[:2], v[4]) for v in reached}
    assert len(kernels) == 20 and len(joins) == 10 + 5   # (five: no join)
    assert {v[:4] for v in mine} == kernels, sorted(kernels - {v[:4] for v in mine})
    missing = {j for j in joins if j[2]} - {(*v[:2], v[4]) for v in mine}
    assert not missing, missing
    assert any(v[4] == 0 for v in mine)


def test_rope_and_rows(plan):
    reached = set(plan("rope", list(itertools.product((1, 300000), (1, 8), (80, 128), (2, 4, 8, 20, 40)))))
    mine = plan("rope", [(t, h, d, sum(s)) for t, h, d, s in C.ROPE])
    assert len(reached) == 6 and set(mine) == reached
    mine = plan("rows", [(t * h * (d // 16),) for t, h, d, _ in C.ROWS])
    assert set(mine) == {(256,), (512,)}
