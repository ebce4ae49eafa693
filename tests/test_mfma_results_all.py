"""The check of test_mfma_results (no matrix instruction's result is read or overwritten before it
is written) on the other sources with matrix instructions.  A result stands after the product's
passes and 4 more wait states: 4 passes for the 16x16 products of these sources, 8 for the 32x32
ones."""
import os
import re
import subprocess

import pytest

import test_mfma_results as reader
from bit_diffusion_amd import build as b

WAITS = {"16x16": 8, "32x32": 12}
SOURCES = ["gemm_int4_fp6.hip", "gemm_nvfp4.hip", "gemm_int4.hip", "quant.hip", "awq.hip"]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    if not os.path.exists(b.HIPCC):
        pytest.skip("no hipcc")
    d = tmp_path_factory.mktemp("assembly")
    runs = {s: subprocess.Popen([b.HIPCC, *b.FLAGS, *b.EXTRA.get(s, []), "--cuda-device-only", "-S", os.path.join(b.CSRC, s),
                                 "-o", str(d / s)], stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL) for s in SOURCES}
    assert {s: r.wait() for s, r in runs.items()} == {s: 0 for s in SOURCES}
    return {s: open(d / s).read() for s in SOURCES}


def early(ins, monkeypatch):
    found, products = [], set()
    for shape, wait in WAITS.items():
        monkeypatch.setattr(reader, "WAIT", wait)
        found += [f for f in reader.early_uses(ins)[1] if shape in f[0]]
    for kind, text in ins:
        if kind == "code" and text.startswith("v_mfma"):
            products.add(re.search(r"_(\d+x\d+)x", text).group(1))
    return products, found


def test_the_reader_knows_both_shapes(monkeypatch):
    text = "\n".join(["_Zk:", " v_mfma_f32_32x32x16_bf16 v[0:15], v[20:23], v[24:27], v[0:15]", " s_nop 7",
                      " v_add_f32_e32 v30, v31, v3", " s_endpgm"])
    products, found = early(reader.functions(text)["_Zk"], monkeypatch)
    assert products == {"32x32"} and len(found) == 1 and found[0][2] == 8
    assert early(reader.functions(text.replace("s_nop 7", "s_nop 11"))["_Zk"], monkeypatch)[1] == []
    assert early(reader.functions(text.replace("32x32x16", "16x16x32").replace("v[0:15]", "v[0:3]"))["_Zk"], monkeypatch)[1] == []


@pytest.mark.parametrize("source", SOURCES)
def test_no_product_is_used_before_it_is_there(source, assembly, monkeypatch):
    shapes = set()
    for name, ins in reader.functions(assembly[source]).items():
        products, found = early(ins, monkeypatch)
        shapes |= products
        assert not found, (name, found[:3])
    assert shapes and shapes <= set(WAITS)
