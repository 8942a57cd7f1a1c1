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
