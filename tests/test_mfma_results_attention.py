"""The check of test_mfma_results (no matrix instruction's result is read or overwritten before it
is written) on the attention's kernels: 32x32 products of 8 passes, whose results stand 4 wait states
after them."""
import os
import subprocess

import pytest

import test_mfma_results as reader
from bit_diffusion_amd import build as b

WAIT = 12
SOURCE = "attention.hip"


def test_no_product_is_used_before_it_is_there(tmp_path, monkeypatch):
    if not os.path.exists(b.HIPCC):
        pytest.skip("no hipcc")
    out = str(tmp_path / "k.s")
    subprocess.run([b.HIPCC, *b.FLAGS, *b.EXTRA[SOURCE], "--cuda-device-only", "-S", os.path.join(b.CSRC, SOURCE), "-o", out],
                   check=True, capture_output=True)
    monkeypatch.setattr(reader, "WAIT", WAIT)
    total = 0
    for name, ins in reader.functions(open(out).read()).items():
        products, found = reader.early_uses(ins)
        total += products
        assert not found, (name, found[:3])
        assert not any(k == "code" and t.startswith("scratch_") for k, t in ins), (name, "spills")
    assert total > 500
