"""Every kernel of the batched adapters and the group norm is run by a test: their launch code,
built for the host with launches that only record their kernel, is given the sizes of the GPU
tests' cases, and what they launch is all that it can launch."""
import os
import shutil
import subprocess

import pytest

import test_gpu_group_norm
import test_gpu_lora_batch
import test_gpu_variants
from bit_diffusion_amd import build as b

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "launches")
SOURCES = ("lora_batch.hip", "group_norm.hip")
pytestmark = pytest.mark.skipif(not (os.path.exists(b.HIPCC) and shutil.which("g++")), reason="needs hipcc and g++")


@pytest.fixture(scope="module")
def trace(tmp_path_factory):
    d = tmp_path_factory.mktemp("launches")
    objs = [str(d / (s + ".o")) for s in SOURCES]
    runs = [subprocess.Popen([b.HIPCC, *[f for f in b.FLAGS if f != "-O3"], "-O1", "-w", "--offload-host-only", "-include",
                              os.path.join(HERE, "trace.hpp"), "-c", os.path.join(b.CSRC, s), "-o", o])
            for s, o in zip(SOURCES, objs)]
    assert [r.wait() for r in runs] == [0] * len(runs)
    exe = str(d / "launches")
    subprocess.run(["g++", "-std=c++17", "-w", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", b.CSRC,
                    os.path.join(HERE, "driver.cpp"), *objs, "-o", exe], check=True)

    def run(calls):
        """The kernels that can be launched, and those of each call."""
        out = subprocess.run([exe], input="".join(c + "\n" for c in calls), capture_output=True, text=True, check=True).stdout
        lines = [line.split("|") for line in out.splitlines()]
        return {p[1] for p in lines if p[0] == "all"}, [p[1:] for p in lines if p[0] == "call"]

    return run


def lora(M, K, N, R, starts, ids, bf=True, S=3, **_):
    return f"lora {M} {K} {N} {R} {len(ids)} {S} {int(bf)}"


def norm(B, rows, C, G, xd=test_gpu_group_norm.BF, od=test_gpu_group_norm.BF, xpad=0, opad=0, shift=0, in_place=0, **_):
    sizes = [xd.itemsize, od.itemsize]
    vec = all(n * e % 16 == 0 for n, e in zip((C + xpad, C + opad), sizes)) and all(shift * e % 16 == 0 for e in sizes)
    return f"norm {B} {rows} {C} {G} {int(xd.itemsize == 2)} {int(od.itemsize == 2)} {int(vec)} {in_place}"


def calls():
    return ([lora(**c) for t in (test_gpu_lora_batch.CASES, test_gpu_variants.LORA) for c in t.values()]
            + [norm(**c) for t in (test_gpu_group_norm.CASES, test_gpu_variants.NORM) for c in t.values()])


def test_every_kernel_is_launched_by_a_case(trace):
    known, launched = trace(calls())
    assert len(known) > 50 and all(launched)
    assert known - {k for c in launched for k in c} == set()


# both sides of a limit are two launches of different kernels, or of different numbers of them
@pytest.mark.parametrize("last,first", [
    ("the last below 32 MB", "the first of 32 MB"), ("fp32, the one launch's last", "fp32, the two launches' first"),
    ("reads, the one launch's last", "reads, the two launches' first"), ("one row, the last", "four rows, the first")])
def test_limits_of_the_norm(trace, last, first):
    _, (one, other) = trace([norm(**test_gpu_variants.NORM[n]) for n in (last, first)])
    assert one != other
    assert abs(test_gpu_variants.NORM[last]["rows"] - test_gpu_variants.NORM[first]["rows"]) + \
        abs(test_gpu_variants.NORM[last]["B"] - test_gpu_variants.NORM[first]["B"]) == 1


def test_names_and_launch_counts(trace):
    for name, table in (("large", test_gpu_variants.NORM), ("two launches", test_gpu_variants.NORM), ("four rows", test_gpu_variants.NORM)):
        picked = {n: norm(**c) for n, c in table.items() if n.startswith(name)}
        _, launched = trace(list(picked.values()))
        for n, ks in zip(picked, launched):
            if name == "four rows":
                assert len(ks) == 1 and ", 4" in ks[0], (n, ks)
            else:
                assert len(ks) == 2, (n, ks)
            if name == "large":
                assert ks[1].endswith("true>"), (n, ks)


def test_in_place_takes_two_launches_where_a_slab_has_several_workgroups(trace):
    _, (apart, in_place, small) = trace([norm(1, 1024, 64, 8), norm(1, 1024, 64, 8, in_place=1), norm(1, 60, 64, 8, in_place=1)])
    assert len(apart) == 1 and len(in_place) == 2 and len(small) == 1


def test_an_empty_pool_has_no_down_projection(trace):
    _, (full, empty) = trace(["lora 9000 64 64 64 2 3 1", "lora 9000 64 64 64 2 0 1"])
    assert len(full) == 2 and len(empty) == 1 and empty[0] == full[1]


@pytest.mark.parametrize("K,R,rows", [(512, 64, 4096), (2048, 64, 6144), (4096, 64, 8192), (12288, 48, 8192),
                                      (512, 128, 2304), (2048, 128, 4096), (4096, 112, 6144), (12288, 128, 6144)])
def test_rows_from_which_the_wide_down_projection_is_taken(trace, K, R, rows):
    _, (narrow, wide) = trace([f"lora {m} {K} 1024 {R} 4 3 1" for m in (rows - 1, rows)])
    assert narrow[0].startswith("lora_down_kernel<") and wide[0].startswith("lora_down_wide_kernel<")


@pytest.mark.parametrize("R,K", [(16, 16384), (32, 4096), (48, 2048), (64, 1536)])
def test_longest_k_of_one_launch(trace, R, K):
    _, (one, two) = trace([f"lora 4 {k} 1024 {R} 1 3 1" for k in (K, K + 64)])
    assert len(one) == 1 and len(two) == 2
