"""CPU tests of the token operators' host code: where each call's parts of the workspace lie, and its
argument checks under the sanitizers."""
import os
import shutil
import subprocess

import pytest

import expert_cache_ffn_amd as ecf
import tokens_host
from tokens_host import WS, overlaps


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    return tokens_host.build(tmp_path_factory.mktemp("tokens_host"))


def sort_parts(q):
    parts = [] if q["itself"] else [("segments", q["segments"], q["n_segments"] * (q["e"] + 1) * 4)]
    sizes = {"counts": q["e"], "offsets": q["e"] + 1, "tiles": q["e"] + 2, "order": q["t"] * q["k"], "place": q["t"] * q["k"]}
    return parts + [(name, q[name], 4 * n) for name, n in sizes.items() if q[name] >= WS]


TOKENS = (1, 16, 64, 65, 66, 700, 4096, 8193, 100000, 1 << 22)


@pytest.mark.parametrize("K,N", [(1, 1), (64, 4096), (257, 130), (2048, 4096), (4096, 2048), (16384, 8), (5, 1 << 20)])
def test_adapters_workspace(host, K, N):
    """Everything that a call writes behind d_ws lies in the bytes that the size query gave, apart from all else."""
    for T in TOKENS:
        for r, n in ((1, 1), (16, 64), (100, 1024), (256, 3)):
            for back in (False, True):
                for order in (False, True):
                    for od in (ecf.ECF_BF16, ecf.ECF_F32):
                        calls, ws = host.adapters(T, K, N, r, n, back, order, od)
                        parts, slots = [], {}
                        for q in calls:
                            if q["kind"] == "sort":
                                parts += sort_parts(q)
                            elif q["kind"] in ("shrink", "few_shrink"):
                                parts.append(("part", q["part"], q["splits"] * T * r * 4))
                            elif q["kind"] == "expand" and q["h"] >= WS:
                                parts.append(("g", q["h"], T * r * 4))
                            elif q["kind"] == "outer" and q["chunks"] > 1:
                                parts.append(("slots", q["slots"], q["chunks"] * 2 * q["w"] * r * 4))
                        assert not overlaps(parts, ws), (T, r, n, back, order)


def test_every_split_has_work(host):
    """The blocks of a split with no k would write zeros, which every block of the expand reads back."""
    for K in [1, 7, 128, 129, 256, 257, 300, 513, 1000, 1330, 2000, 2048, 2049, 2304, 4096, 8192, 1 << 20] + list(range(64, 5000, 97)):
        for T in (65, 100, 700, 4096, 8192, 30000, 100000):
            for back in (False, True):
                (q,) = [q for q in host.adapters(T, 8 if back else K, K if back else 8, 16, 8, back)[0] if q["kind"] == "shrink"]
                assert q["k"] == K and q["split_k"] % 128 == 0 and 1 <= q["splits"] <= 7
                assert (q["splits"] - 1) * q["split_k"] < K <= q["splits"] * q["split_k"], (T, q)


def test_sort_and_norm_workspace(host):
    for T in TOKENS:
        for k, E in ((1, 1), (6, 256), (8, 1024), (16, 60)):
            calls, ws = host.sort(T, k, E)
            assert not overlaps([p for p in sort_parts(calls[0]) if p[0] == "segments"], ws), (T, k, E)
        for d in (1, 1000, 2048, 4096, 16384, 20000):
            (q,), ws = host.norm_backward(T, d)
            assert q["partial"] == WS and q["parts"] * d * 4 <= ws


def test_grids(host):
    """A block for each row of the most tokens (of 1024 threads) and for every four of the most choices: fewer than 2^32 threads
    in a dimension, and no more blocks than complete the last line."""
    for blocks in (1, 2, 1000, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, (1 << 22) - 3, 1 << 22, (1 << 24) - 1, 1 << 24):
        x, y = host.grid(blocks)
        assert x * 1024 < 1 << 32 and y < 1 << 16 and x * y >= blocks and x * (y - 1) < blocks
        assert (y == 1 or x == 1 << 21) and x * y * 4 + blocks < 1 << 32  # (numbers of choices behind the last fit 32 bits)


def test_host_code_under_sanitizers(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "tokens_checks")
    subprocess.run(["g++", *tokens_host.FLAGS, "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                    *tokens_host.SOURCES, os.path.join(tokens_host.HERE, "sanitize", "tokens_checks.cpp"), "-o", exe], check=True)
    p = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    assert p.returncode == 0 and "token checks passed" in p.stdout, p.stdout[-4000:]
    for bad in ("ERROR: AddressSanitizer", "runtime error:"):
        assert bad not in p.stdout, p.stdout[-4000:]
