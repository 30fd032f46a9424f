"""The tile kernel's plan on the CPU: the kernel's own source of it, compiled with the CTA's threads and warps emulated
(plan_on_cpu.cpp).  All CTAs together must hold every block of every tile once, and find its parts where they were stored."""
import os
import random
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "bit_routed_expert_gb300", "csrc", "kv_tree.cu")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src = open(SOURCE).read()
    part = src[src.index("// Tiles: the list is cut"):src.index("// The queries as two E4M3 terms")]
    consts = re.findall(r"^constexpr int (?:TT_THREADS|TT_WARPS|COST_ONE)\b.*?;", src, flags=re.M)
    assert len(consts) == 3
    at = tmp_path_factory.mktemp("plan")
    (at / "shares.inc").write_text("\n".join(consts) + "\n" + part)
    exe = str(at / "plan")
    subprocess.run([cxx, "-O2", "-std=c++17", "-w", f'-DSHARES="{at / "shares.inc"}"', os.path.join(HERE, "plan_on_cpu.cpp"), "-o", exe], check=True)

    def run(runs, G, H, N=4096, ctas=24):
        """runs: (first position, tokens) of a sequence each; a negative position: padding."""
        seq = [b for b, (_, n) in enumerate(runs) for _ in range(n)]
        pos = [p + i if p >= 0 else -1 for p, n in runs for i in range(n)]
        text = " ".join(map(str, [G, H, N, ctas, len(seq), *seq, *pos]))
        return subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
    return run


@pytest.mark.parametrize("runs,G,H", [
    ([(0, 2048)] * 2, 8, 4), ([(0, 512)] * 8, 8, 4), ([(8192, 1024)] * 2, 8, 8),
    ([(16384, 512), (0, 512), (8000, 512), (100, 512)], 8, 4),       # runs that end where a round of the plan does
    ([(8192, 16)] * 32 + [(1024, 16)] * 32, 8, 4),                   # equal drafts, long contexts before short ones
    ([(9000, 512), (-1, 100), (70, 3)], 4, 2),                       # padding that begins there
    ([(-1, 512), (9000, 40)], 4, 2),
    ([(5000, 500), (300, 12), (7, 600)], 1, 1), ([(5000, 1100)], 16, 2), ([(3000, 33)] * 20, 3, 2),
    ([(20000, 1)], 8, 1), ([(0, 1)] * 513, 8, 1), ([(64 * i % 977, 1 + i % 50) for i in range(60)], 5, 2)])
def test_blocks_are_held_once(plan, runs, G, H):
    assert plan(runs, G, H) == ""


def test_lists_of_more_rounds_than_are_kept(plan):
    """Beyond 16,384 tokens a share's place is searched from every second round on."""
    assert plan([(40 * i % 9001, 33) for i in range(560)], 8, 1, ctas=6) == ""


def test_random_batches(plan):
    """Sequences of the same number of drafts, or tokens of any number, behind contexts of any length."""
    rng = random.Random(4)
    for i in range(12):
        G, H = rng.choice([1, 3, 4, 8, 8, 16]), rng.choice([1, 2, 4])
        n = rng.choice([8, 16, 32, 64, 128, 256, 512])
        runs, left = [], 1500
        while left > 0:
            m = n if i % 2 else min(left, rng.randint(1, 600))
            runs.append((-1 if rng.random() < 0.1 else rng.randint(0, 16000), m))
            left -= m
        assert plan(runs, G, H, ctas=rng.choice([7, 24, 60])) == "", (G, H, runs)


def test_as_many_ctas_as_the_gpu_has(plan):
    assert plan([(random.Random(7).randint(0, 16000), 16) for _ in range(64)], 8, 4, ctas=152) == ""
