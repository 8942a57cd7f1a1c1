"""Attention over selected pages on the host: the workspace that callers are told to bring."""
import os
import subprocess

import numpy as np
import pytest

from flash_attention_backward_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def decode(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("decode") / "decode")
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "-I", B.INCLUDE, os.path.join(HERE, "decode_pages_host.cu"), "-o", exe], check=True)

    def run(cases):
        text = "".join(" ".join(map(str, c)) + "\n" for c in cases)
        out = subprocess.run([exe], input=text, stdout=subprocess.PIPE, text=True, check=True).stdout
        return [tuple(int(x) for x in row.split()) for row in out.strip().split("\n")]
    return run


def test_the_workspace_that_is_asked_for_does_for_every_call(decode):
    """fa_paged_decode_workspace_size() does for fa_paged_decode() and for fa_paged_decode_pages() of any K: all head
    sizes and types, batches with few and many items, tables of one page and of long sequences."""
    rng = np.random.default_rng(3)
    cases = []
    for D in (64, 128, 256):
        for Dv in (64, 128, 256):
            for kt in range(4):
                for vt in range(4):
                    batches = [(48, 1, 1, 512, 16, 64), (8, 8, 8, 512, 64, 64)]  # B, Hkv, H, max_pages, page_size, K
                    for _ in range(40):
                        n, Hkv, G, wide, page, K = (int(np.exp(rng.uniform(0, np.log(m)))) for m in (2000, 16, 20, 5000, 300, 6000))
                        batches.append((n, Hkv, G * Hkv, wide, page, K))
                    cases += [(D, Dv, kt, vt, n, Hkv, H, 1000, page, wide, k, sms) for n, Hkv, H, wide, page, K in batches
                              for k in (0, K) for sms in (152, 1)]
    for case, (need, rc) in zip(cases, decode(cases)):
        assert need > 0 and rc == 0, (case, need, rc)


@pytest.fixture(scope="module")
def position(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("position") / "position")
    checks = [x for f in ("-fsanitize=undefined", "-fno-sanitize-recover=all") for x in ("-Xcompiler", f)]
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", *checks, "-I", B.INCLUDE, os.path.join(HERE, "selected_position_host.cu"), "-o", exe], check=True)

    def run(page, max_pages, at, sel):
        r = subprocess.run([exe], input=" ".join(map(str, [page, max_pages, at, *sel])) + "\n", capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return int(r.stdout)
    return run


@pytest.mark.parametrize("L, page, K, sel", [
    (100, 40, 64, [2, 0, 1]),            # three pages, of 64 entries three are read; 120 keys end inside a tile
    (9, 5, 21, [1, -1]),
    (3, 12, 7, [0]),
    (70, 1, 40, list(range(69, 29, -1))),
    (300, 16, 4, [2 ** 31 - 1, 3, -2 ** 31, 18]),
])
def test_positions_of_selected_keys(position, L, page, K, sel):
    """At most min(K, ceil(L / page)) entries of a list are read, for the places behind its last key in a tile of 16 too,
    and entries that are no page of the sequence (any number) do not leave the range of an int."""
    n = -(-L // page)
    assert len(sel) == min(K, n)
    keys = len(sel) * page
    for at in sorted({0, 1, page - 1, keys // 2, keys - 1, keys, keys + (-keys) % 16, -(-keys // 16) * 16 - 1}):
        got = position(page, n + 2, at, sel)
        if at < keys and 0 <= sel[at // page] < n:
            assert got == sel[at // page] * page + at % page, at
