"""Reads the generated gfx950 assembly of the adapters' kernels: on no path is a matrix
instruction's result read or overwritten by another instruction before it is written.  (The
compiler places the waits; behind a uniform branch between a matrix instruction and the read of its
result it has left too few, and two of four result registers came out wrong.  The kernels have no
such branch; this keeps it so, whatever the compiler makes of a change.)"""
import os
import re
import subprocess

import pytest

from bit_diffusion_amd import build as b

WAIT = 8        # wait states from a 16x16x32 bf16 product to a read of its result, 7 to a write


def regs(text):
    out = set()
    for m in re.finditer(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        if m.group(1):
            out |= {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
        else:
            out.add((m.group(4), int(m.group(5))))
    return out


def functions(text):
    funcs, cur = {}, None
    for line in text.splitlines():
        line = line.split(";")[0].rstrip()
        m = re.match(r"^(_Z\w+):", line)
        if m:
            cur = funcs.setdefault(m.group(1), [])
            continue
        m = re.match(r"^(\.LBB\w+):", line)
        if cur is None:
            continue
        if m:
            cur.append(("label", m.group(1)))
        elif line.strip() and not line.strip().startswith("."):
            cur.append(("code", line.strip()))
    return funcs


def early_uses(ins):
    """(product, instruction, wait states) of every use that comes too early."""
    labels = {x[1]: i for i, x in enumerate(ins) if x[0] == "label"}
    found, products = [], 0
    for i, (kind, text) in enumerate(ins):
        if kind != "code" or not text.startswith("v_mfma"):
            continue
        products += 1
        dst = regs(text.split(None, 1)[1].split(", ")[0])
        todo, seen = [(i + 1, 0)], {}
        while todo:
            j, w = todo.pop()
            while j < len(ins) and w < WAIT and seen.get(j, WAIT) > w:
                seen[j] = w
                kind2, t = ins[j]
                j += 1
                if kind2 == "label":
                    continue
                m = re.match(r"s_nop (\d+)", t)
                if m:
                    w += int(m.group(1)) + 1
                    continue
                if t.startswith("s_endpgm"):
                    break
                ops = t.split(None, 1)[1].split(", ") if " " in t else []
                if t.startswith("v_mfma"):
                    if (regs(ops[1]) | regs(ops[2])) & dst:
                        found.append((text, t, w))
                        break
                    if regs(ops[0]) == dst:      # accumulates on it, or its own result comes later
                        break
                elif not t.startswith("s_"):
                    reads = regs(", ".join(ops[1:])) if t.startswith("v_") else regs(", ".join(ops))
                    if reads & dst or (w < WAIT - 1 and regs(", ".join(ops)) & dst):
                        found.append((text, t, w))
                        break
                if t.startswith("s_branch"):
                    j = labels[t.split()[1]]
                elif t.startswith("s_cbranch"):
                    todo.append((labels[t.split()[1]], w + 1))
                w += 1
    return products, found


def test_the_reader_finds_an_early_use():
    text = "\n".join(["_Zk:", " v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]", " s_cbranch_vccnz .LBB0_2",
                      " s_nop 7", ".LBB0_2:", " v_add_f32_e32 v5, v5, v2", " s_endpgm"])
    products, found = early_uses(functions(text)["_Zk"])
    assert products == 1 and len(found) == 1 and found[0][2] == 1
    ok = text.replace(" v_add", " s_nop 6\n v_add")
    assert early_uses(functions(ok)["_Zk"])[1] == []


@pytest.mark.parametrize("source", ["lora_batch.hip"])
def test_no_product_is_used_before_it_is_there(source, tmp_path):
    if not os.path.exists(b.HIPCC):
        pytest.skip("no hipcc")
    out = str(tmp_path / "k.s")
    subprocess.run([b.HIPCC, *b.FLAGS, *b.EXTRA.get(source, []), "--cuda-device-only", "-S",
                    os.path.join(b.CSRC, source), "-o", out], check=True, capture_output=True)
    total = 0
    for name, ins in functions(open(out).read()).items():
        products, found = early_uses(ins)
        total += products
        assert not found, (name, found[:3])
    assert total > 100
