"""Inline assembly tells the compiler every register that it changes by name."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_block_scaled_04_amd", "csrc")


def statements(src):
    """(template, what follows it) of each asm statement."""
    for m in re.finditer(r"\basm\b\s*(?:volatile)?\s*\(", src):
        depth, at = 1, m.end()
        while depth:
            quoted = re.match(r'"(?:[^"\\]|\\.)*"', src[at:])
            if quoted:
                at += quoted.end()
                continue
            depth += {"(": 1, ")": -1}.get(src[at], 0)
            at += 1
        body = src[m.end():at - 1]
        template = re.match(r'(?:\s*"(?:[^"\\]|\\.)*")+', body)
        yield template.group(0), body[template.end():]


def undeclared(src):
    """Registers that a statement moves into and does not list among what it clobbers."""
    bad = []
    for template, rest in statements(src):
        text = template.replace("\\n", "\n").replace("\\t", " ")
        written = {m.group(1) for m in re.finditer(r"(?:^|[\n\"])\s*[sv]_\w+ +(m0|vcc|exec|scc|[sv]\d+|[sv]\[\d+:\d+\])\b", text)}
        parts = re.split(r':(?=(?:[^"]*"[^"]*")*[^"]*$)', rest)
        clobbers = set(re.findall(r'"([^"]*)"', parts[3])) if len(parts) > 3 else set()
        bad += sorted(written - clobbers)
    return bad


def test_the_check_sees_what_is_missing():
    good = 'asm volatile("s_mov_b32 m0, %1\\n\\tbuffer_load_dwordx4 %0, %2, 0 offen lds" ::"v"(a), "s"(b), "s"(c) : "memory", "m0");'
    assert undeclared(good) == []
    assert undeclared(good.replace(', "m0"', "")) == ["m0"]
    assert undeclared('asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); asm("v_mov_b32 v7, 0" ::);') == ["v7"]


def test_every_statement():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if path.endswith((".hip", ".h", ".cpp")):
            src = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
            seen += sum(1 for _ in statements(src))
            assert undeclared(src) == [], os.path.basename(path)
    assert seen > 10
