"""The host side of svdq_lora_batch and svdq_group_norm under sanitizers: the argument checks and size
queries of the C ABI (AddressSanitizer and UBSan), and the choice of kernels, grids and cuts for
sizes up to the calls' limits (UBSan; the launches only record their kernel).  CPU only."""
import os
import random
import shutil
import subprocess

import pytest

from bit_diffusion_amd import build as b

HERE = os.path.dirname(os.path.abspath(__file__))
HIPCC = "/opt/rocm/bin/hipcc"
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1")
pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and shutil.which("g++")), reason="needs hipcc and g++")


def run(exe, text=""):
    r = subprocess.run([exe], input=text, capture_output=True, text=True, env=ENV, timeout=120)
    assert r.returncode == 0, (r.stdout + r.stderr)[-2000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-2000:]
    return r.stdout


def test_argument_checks_and_size_queries(tmp_path):
    objs = [os.path.join(b.OBJ_DIR, os.path.splitext(s)[0] + ".o") for s in b.SOURCES if s != "api.hip"]
    if not all(os.path.exists(o) for o in objs):
        b.build()
    api, exe = str(tmp_path / "api.o"), str(tmp_path / "batch")
    subprocess.run([HIPCC, *b.FLAGS, "-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-sanitize-recover=all",
                    "-c", os.path.join(b.CSRC, "api.hip"), "-o", api], check=True, capture_output=True)
    subprocess.run(["g++", "-std=c++17", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "sanitize", "batch_driver.cpp"), api, *objs, "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib", "-o", exe], check=True, capture_output=True)
    assert "0 failures" in run(exe)


def sizes():
    r = random.Random(7)

    def log(lo, hi):
        return int(round(2 ** r.uniform(lo, hi)))

    calls = ["lora 4194304 16777216 1 128 65536 2147483647 1", "lora 4194304 64 256 16 1 1 0"]
    while len(calls) < 1000:
        M, n, N = log(0, 22), log(0, 16), log(0, 30)
        tiles = min((M + n * 15) // 16, M) + 8
        if tiles < 1 << 19 and tiles * ((N + 127) // 128) < 1 << 24:
            calls.append(f"lora {M} {64 * log(0, 18)} {N} {16 * r.randint(1, 8)} {n} {r.randint(0, 5)} {r.randint(0, 1)}")
    for C, G in ((65536, 1), (65536, 65536), (65536, 32), (65535, 5)):
        calls += [f"norm 65535 1073741824 {C} {G} {half} 0 {vec} 0" for half in (0, 1) for vec in (0, 1)]
    while len(calls) < 2500:
        G, cg = log(0, 16), log(0, 16)
        if G * cg <= 65536:
            flags = " ".join(str(r.randint(0, 1)) for _ in range(4))
            calls.append(f"norm {min(log(0, 16), 65535)} {log(0, 30)} {G * cg} {G} {flags}")
    return calls


def test_launch_choices_at_every_size(tmp_path):
    here = os.path.join(HERE, "launches")
    objs = [str(tmp_path / (s + ".o")) for s in ("lora_batch.hip", "group_norm.hip")]
    runs = [subprocess.Popen([HIPCC, *[f for f in b.FLAGS if f != "-O3"], "-O1", "-g", "-w", "--offload-host-only",
                              "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
                              "-include", os.path.join(here, "trace.hpp"), "-c", os.path.join(b.CSRC, s), "-o", o])
            for s, o in zip(("lora_batch.hip", "group_norm.hip"), objs)]
    assert [r.wait() for r in runs] == [0, 0]
    exe = str(tmp_path / "launches")
    # the kernels' device code, which nothing here loads, is left out
    subprocess.run(["g++", "-std=c++17", "-g", "-w", "-fsanitize=undefined", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                    "-I", b.CSRC, os.path.join(here, "driver.cpp"), *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", exe],
                   check=True, capture_output=True)
    calls = sizes()
    lines = run(exe, "".join(c + "\n" for c in calls)).splitlines()
    assert sum(x.startswith("call|") for x in lines) == len(calls)
