"""The rules by which the launchers choose a kernel (csrc/aa_rules.h), compiled
for the host and checked on the CPU: the launchers use the same functions."""
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "associative_algebra_block_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "host_rules")


def compiled(tmp_path, name):
    cxx = shutil.which("g++") or shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"
    exe = str(tmp_path / name)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"),
                        os.path.join(HERE, name + ".cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


def test_a_turned_append_fits_a_grid(tmp_path):
    r = subprocess.run([compiled(tmp_path, "append_driver")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "append rule holds" in r.stdout, (r.stdout, r.stderr)


def test_every_kernel_of_the_experts_layer_is_tested(tmp_path):
    """The GPU cases of the mixture-of-experts layer reach every kernel that the
    rule can take: each gate/up kernel with both orders of the pairs, each down
    kernel with both output types, and the two-strip ones with a last strip
    alone."""
    from tests.test_gpu_moe import CASES, KERNEL_CASES
    cases = CASES + KERNEL_CASES
    lines = "".join(f"{int(law == 'Q2xQ2')} {q} {D} {F} {k} {M}\n" for law, q, D, F, E, k, M, *_ in cases)
    r = subprocess.run([compiled(tmp_path, "moe_driver")], input=lines, capture_output=True, text=True, timeout=60)
    got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    assert r.returncode == 0 and len(got) == len(cases)
    up = {(ws, eight) for ws, eight, *_ in got}
    assert {ws for ws, _ in up} == {1, 2, 4, 8} and {eight for _, eight in up} == {0, 1}, up
    down = {(ns, nw, alone, c[8]) for (_, _, ns, nw, alone), c in zip(got, cases)}
    for ns, nw in ((1, 4), (1, 16), (2, 4), (2, 8)):
        for alone in (0, 1) if ns == 2 else (0,):
            assert {(ns, nw, alone, "f32"), (ns, nw, alone, "bf16")} <= down, (ns, nw, alone, down)
