"""The launches of svdq_layer_norm, svdq_rotary and svdq_attention over their documented ranges start
fewer than 2^32 threads: a dispatch counts them in 32 bits, and the runtime refuses more."""
import os
import random
import shutil
import subprocess

import pytest

from bit_diffusion_amd import build as b

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "launches")
SOURCES = ("layer_norm.hip", "rotary.hip", "attention.hip")
pytestmark = pytest.mark.skipif(not (os.path.exists(b.HIPCC) and shutil.which("g++")), reason="needs hipcc and g++")


@pytest.fixture(scope="module")
def threads(tmp_path_factory):
    d = tmp_path_factory.mktemp("threads")
    objs = [str(d / (s + ".o")) for s in SOURCES]
    runs = [subprocess.Popen([b.HIPCC, *[f for f in b.FLAGS if f != "-O3"], "-O1", "-w", "--offload-host-only", "-include",
                              os.path.join(HERE, "threads.hpp"), "-c", os.path.join(b.CSRC, s), "-o", o])
            for s, o in zip(SOURCES, objs)]
    assert [r.wait() for r in runs] == [0] * len(runs)
    exe = str(d / "threads")
    subprocess.run(["g++", "-std=c++17", "-w", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", b.CSRC,
                    os.path.join(HERE, "threads_driver.cpp"), *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", exe], check=True)

    def run(calls):
        out = subprocess.run([exe], input="".join(c + "\n" for c in calls), capture_output=True, text=True, check=True).stdout
        return [[int(n) for n in line.split()[1:]] for line in out.splitlines()]

    return run


def check(calls, launches):
    assert len(calls) == len(launches)
    for c, ls in zip(calls, launches):
        assert all(0 < n < 1 << 32 for n in ls), (c, ls)


def test_rotary(threads):
    calls = [f"rotary {M} {q} {k} {D} {halves} {vec} {word}" for M in (1, 65537, (1 << 23) + 1, (1 << 24) - 1, 1 << 24)
             for q, k in ((1, 0), (0, 1), (24, 24), (128, 0), (255, 1), (256, 256), (1 << 16, 1 << 16)) for D in (2, 8, 64, 128, 256)
             for halves, vec, word in ((0, 1, 1), (0, 0, 1), (0, 0, 0), (1, 1, 0), (1, 0, 0)) if not vec or D % (16 if halves else 8) == 0]
    launches = threads(calls)
    assert all(len(ls) == 1 for ls in launches)
    check(calls, launches)


def test_layer_norm(threads):
    calls = [f"layer {M} {C} {vec} {xb}" for M in (1, 8192, 8193, (1 << 30) - 1, 1 << 30) for C, vec in ((1, 1), (8192, 1), (2, 2), (8192, 2), (4, 4), (16384, 4))
             for xb in (0, 1)]
    launches = threads(calls)
    assert all(len(ls) == 1 for ls in launches)
    check(calls, launches)


def test_attention(threads):
    r = random.Random(5)
    calls = [f"attn {Mq} {Mk} {H} {G} {D} {n}" for Mq in (1, 511, 4096, 1 << 20, (1 << 24) - 1, 1 << 24) for Mk in (1, 70000, 1 << 30)
             for H, G in ((1, 1), (2, 1), (24, 24), (1 << 16, 1), (1 << 16, 1 << 15), (1 << 16, 1 << 16)) for D in (8, 128) for n in (1, 64, 65, 1 << 16)]
    for _ in range(3000):
        G = 1 << r.randint(0, 12)
        calls.append(f"attn {int(2 ** r.uniform(0, 24))} {int(2 ** r.uniform(0, 30))} {G * r.randint(1, 16)} {G} {8 * r.randint(1, 16)} {int(2 ** r.uniform(0, 16))}")
    launches = threads(calls)
    assert sum(bool(ls) for ls in launches) > 1000
    check(calls, launches)
