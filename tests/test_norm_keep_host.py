"""The gradient norm's share of the last-level cache
(precision_state_amd/csrc/norm_keep.h) on the host: only whole chunks stay
there, so only they are counted."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHUNK, KEEP = 8192, 256 << 20


def expected(chunk, keep, tensors):
    """Chunk by chunk from the last one: parts of a chunk are free, a whole chunk takes its bytes of what is left."""
    chunks = [(min(chunk, n - o) == chunk, size) for n, size in tensors for o in range(0, n, chunk)]
    i = len(chunks)
    while i and (not chunks[i - 1][0] or chunk * chunks[i - 1][1] <= keep):
        i -= 1
        keep -= chunk * chunks[i][1] if chunks[i][0] else 0
    return i


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = tmp_path_factory.mktemp("keep") / "norm_keep"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-fsanitize=address,undefined",
                    "-I", os.path.join(ROOT, "precision_state_amd", "csrc"),
                    os.path.join(ROOT, "tests", "norm_keep_host_test.cpp"), "-o", str(exe)], check=True)

    def call(cases):
        text = "\n".join(f"{c} {k} {len(t)} " + " ".join(f"{n} {s}" for n, s in t) for c, k, t in cases)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return [int(x) for x in r.stdout.split()]
    return call


def test_small_tensors_take_nothing_from_large_ones(run):
    large, small = (200_000_000, 2), [(4096, 2)] * 1000
    got = run([(CHUNK, KEEP, [large]), (CHUNK, KEEP, [large] + small)])
    assert got[0] == got[1] == expected(CHUNK, KEEP, [large])
    assert got[0] == 200_000_000 // CHUNK - KEEP // (CHUNK * 2)


def test_against_a_count_chunk_by_chunk(run):
    rng = random.Random(1)
    cases = [(8, 64, []), (8, 64, [(1, 4)]), (8, 64, [(8, 4), (8, 4)]), (8, 63, [(8, 4), (8, 4)]), (8, 0, [(20, 2), (3, 4)])]
    for _ in range(400):
        chunk = rng.choice([4, 8, 32])
        t = [(rng.randint(1, 6 * chunk), rng.choice([2, 4])) for _ in range(rng.randint(0, 12))]
        cases.append((chunk, rng.randint(0, 40 * chunk), t))
    assert run(cases) == [expected(*c) for c in cases]
