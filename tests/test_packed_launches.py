"""The host side of svdq_layer_norm, svdq_rotary and svdq_attention without a GPU: every kernel that
their launch code can start is run by a GPU test's case (launches that only record their kernel), both
sides of the splits' limits, and argument checks, size query and launch choices under sanitizers."""
import os
import random
import shutil
import subprocess

import pytest

import test_gpu_attention as attn
import test_gpu_layer_norm as layer
import test_gpu_rotary as rot
from bit_diffusion_amd import build as b

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCES = ("layer_norm.hip", "rotary.hip", "attention.hip")
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1")
pytestmark = pytest.mark.skipif(not (os.path.exists(b.HIPCC) and shutil.which("g++")), reason="needs hipcc and g++")


def start(exe, calls):
    r = subprocess.run([exe], input="".join(c + "\n" for c in calls), capture_output=True, text=True, env=ENV, timeout=120)
    assert r.returncode == 0 and "runtime error" not in r.stderr, (r.stdout + r.stderr)[-2000:]
    return [line.split("|") for line in r.stdout.splitlines()]


@pytest.fixture(scope="module")
def trace(tmp_path_factory):
    d = tmp_path_factory.mktemp("packed_launches")
    here = os.path.join(HERE, "launches")
    objs = [str(d / (s + ".o")) for s in SOURCES]
    runs = [subprocess.Popen([b.HIPCC, *[f for f in b.FLAGS if f != "-O3"], "-O1", "-g", "-w", "--offload-host-only",
                              "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
                              "-include", os.path.join(here, "trace.hpp"), "-c", os.path.join(b.CSRC, s), "-o", o])
            for s, o in zip(SOURCES, objs)]
    assert [r.wait() for r in runs] == [0] * len(runs)
    exe = str(d / "launches")
    # the kernels' device code, which nothing here loads, is left out
    subprocess.run(["g++", "-std=c++17", "-g", "-w", "-fsanitize=undefined", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                    "-I", b.CSRC, os.path.join(here, "packed_driver.cpp"), *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", exe],
                   check=True, capture_output=True)

    def run(calls):
        """The kernels that can be launched, those of each call, and the attention calls' workspaces."""
        lines = start(exe, calls)
        return ({p[1] for p in lines if p[0] == "all"}, [p[1:] for p in lines if p[0] == "call"],
                [(int(p[1]), int(p[2])) for p in lines if p[0] == "bytes"])

    return run


def layer_call(starts, C, tail=0, xd=layer.BF, yd=layer.BF, od=layer.BF, md=layer.F32, residual=True, mod=True, gate=True, xpad=0,
               ypad=0, opad=0, shift=0, **_):
    ms = 3 * C + (4 if C % 4 == 0 else 2 - C % 2)

    def takes(n):
        strides = [C, C + xpad, C + opad, shift] + ([C + ypad] if residual else []) + ([ms] if mod or (gate and residual) else [])
        return all(s % n == 0 for s in strides)

    vec = 4 if takes(4) else 2 if takes(2) else 1
    return f"layer {starts[-1] + tail} {C} {vec} {int(xd == layer.BF)} {int(residual and yd == layer.BF)} {int(od == layer.BF)}"


def rotary_call(M, H, G, pairs, halves=False, xd=rot.BF, od=rot.BF, pad=0, opad=0, shift=0, **_):
    D = 2 * sum(pairs)
    xe, oe = xd.itemsize, od.itemsize
    ins, outs = (H + 2 * G) * D + pad, [H * D + opad + shift] * (H > 0) + [G * D + opad + shift] * (G > 0)
    # where q and k begin, and the outputs
    at = [shift] * (H > 0) + [shift + H * D] * (G > 0)
    vec = D % (16 if halves else 8) == 0 and all(v * xe % 16 == 0 for v in [ins, *at]) and all(v * oe % 16 == 0 for v in [*outs, shift])
    word = not halves and all(v % 2 == 0 for v in [ins, *at, *outs, shift])
    return f"rotary {M} {H} {G} {D} {int(halves)} {int(vec)} {int(word)} {int(xd == rot.BF)} {int(od == rot.BF)}"


def attn_call(qs, H, G, D, ks=None, tail=0, cap=0.0, bias=False, **_):
    Mq, Mk = qs[-1] + tail, (qs if ks is None else ks)[-1] + (tail if ks is None else 0)
    return f"attn {Mq} {Mk} {H} {G} {D} {len(qs) - 1} {int(cap > 0)} {int(bias)}"


def test_every_kernel_is_launched_by_a_case(trace):
    types = [dict(starts=layer.cut(11, 0, 6), C=C, tail=2, xd=xd, yd=yd, od=od)
             for C in (200, 1200, 3072, 5000, 9000, 122, 1170, 2050, 4102, 63, 333, 2001, 3001)
             for xd in (layer.BF, layer.F32) for yd in (layer.BF, layer.F32) for od in (layer.BF, layer.F32)]
    calls = [layer_call(**c) for c in [*layer.CASES.values(), *types]] + [rotary_call(**c) for c in [*rot.CASES.values(), *rot.TYPES]] \
        + [attn_call(**c) for c in attn.CASES.values()]
    known, launched, _ = trace(calls)
    assert len(known) > 150 and all(launched)
    assert known - {k for c in launched for k in c} == set()


def test_splits(trace):
    """Few rows over many keys are split, and joined, by four waves a row or one; short keys, and two
    workgroups a CU without, are not."""
    split = {"attn 1 1024 1 1 64 1 0 0": 0, "attn 1 1025 1 1 64 1 0 0": 4, "attn 512 100000 512 512 64 512 0 0": 0,
             "attn 511 100000 1 1 64 511 0 0": 0, "attn 255 100000 1 1 64 255 0 0": 4,
             "attn 4096 1500 8 8 64 1 0 0": 0, "attn 4096 9000 8 8 64 1 0 0": 1, "attn 1023 4000 4 4 64 1 0 0": 4,
             "attn 1024 4000 4 4 64 1 0 0": 1, "attn 8 9000 8 8 128 8 0 0": 4, "attn 8 9000 64 64 128 8 0 0": 0}
    _, launched, sizes = trace(list(split))
    for c, ks, (_, b), per in zip(split, launched, sizes, split.values()):
        assert (b > 0) == (per > 0) and len(ks) == 1 + (per > 0), (c, ks, b)
        assert not per or ks[1] == f"attention_join_kernel<{per}>", (c, ks)


def test_launch_choices_at_every_size(trace):
    r = random.Random(11)

    def log(lo, hi):
        return int(round(2 ** r.uniform(lo, hi)))

    calls = []
    for _ in range(700):
        vec = r.choice([1, 2, 4])
        calls.append(f"layer {log(0, 30)} {vec * log(0, 14 if vec == 4 else 13) // vec * vec or vec} {vec} {r.randint(0, 1)} {r.randint(0, 1)} {r.randint(0, 1)}")
        halves, D = r.randint(0, 1), 2 * log(0, 7)
        vec = int(D % (16 if halves else 8) == 0 and r.random() < 0.7)
        calls.append(f"rotary {log(0, 24)} {log(0, 16)} {log(0, 16)} {D} {halves} {vec} {int(not halves and r.random() < 0.5)} {r.randint(0, 1)} {r.randint(0, 1)}")
        G = log(0, 10)
        calls.append(f"attn {log(0, 24)} {log(0, 30)} {G * log(0, 6)} {G} {8 * r.randint(1, 16)} {log(0, 16)} {r.randint(0, 1)} {r.randint(0, 1)}")
    _, launched, sizes = trace(calls)
    assert len(launched) == len(calls) and all(0 <= s < 1 << 34 for fits, s in sizes if fits)


def test_argument_checks_and_size_query(tmp_path):
    objs = [os.path.join(b.OBJ_DIR, os.path.splitext(s)[0] + ".o") for s in b.SOURCES if s != "api.hip"]
    if not all(os.path.exists(o) for o in objs):
        b.build()
    api, exe = str(tmp_path / "api.o"), str(tmp_path / "packed")
    subprocess.run([b.HIPCC, *b.FLAGS, "-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-sanitize-recover=all",
                    "-c", os.path.join(b.CSRC, "api.hip"), "-o", api], check=True, capture_output=True)
    subprocess.run(["g++", "-std=c++17", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "sanitize", "packed_driver.cpp"), api, *objs, "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", exe], check=True, capture_output=True)
    assert ["0 failures"] in start(exe, [])
