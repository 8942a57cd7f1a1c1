"""Host side of fa_paged.h: exports, argument checks before any launch, the frequency table, and the
refusals of the Python wrappers."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

import flash_attention_backward_gb300 as fb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fa_paged.h")


@pytest.fixture(scope="module", autouse=True)
def L():
    from flash_attention_backward_gb300 import build
    build.build()
    return fb.lib()


def test_declared_functions_are_exported_and_bound(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(["fa_rope_frequencies", "fa_qk_norm_rope", "fa_qk_norm_rope_backward_workspace_size",
                            "fa_qk_norm_rope_backward", "fa_cache_append", "fa_cache_read",
                            "fa_paged_decode_workspace_size", "fa_paged_decode"])
    for n in names:
        assert hasattr(L, n) and hasattr(fb, n), n
    assert fb.fa_back_status_string(10) != fb.fa_back_status_string(99) and fb.STATUS[10] == "FA_ERR_PAGE"


def cache(**kw):
    c = dict(k=0x10000, v=0x20000, page_table=0x30000, k_type=2, v_type=2, num_pages=8, page_size=16, B=2, max_pages=4,
             Hkv=2, D=128, Dv=128)
    c.update({f: kw.pop(f) for f in list(kw) if f in dict(fb.fa_paged_cache._fields_)})
    return fb.fa_paged_cache(**c), kw


CACHE_ERRORS = [
    (dict(k_type=4), "FA_ERR_TYPE"),
    (dict(v_type=-1), "FA_ERR_TYPE"),
    (dict(num_pages=-1), "FA_ERR_SHAPE"),
    (dict(page_size=0), "FA_ERR_SHAPE"),
    (dict(B=-1), "FA_ERR_SHAPE"),
    (dict(max_pages=-1), "FA_ERR_SHAPE"),
    (dict(Hkv=0), "FA_ERR_SHAPE"),
    (dict(D=96), "FA_ERR_UNSUPPORTED"),
    (dict(Dv=512), "FA_ERR_UNSUPPORTED"),
    (dict(Hkv=512), "FA_ERR_UNSUPPORTED"),
    (dict(max_pages=1 << 27), "FA_ERR_UNSUPPORTED"),  # 2^31 positions
    (dict(page_size=1, Hkv=1), "FA_ERR_ALIGN"),  # a page of 136 bytes
    (dict(k=None), "FA_ERR_NULL"),
    (dict(v=None), "FA_ERR_NULL"),
    (dict(page_table=None), "FA_ERR_NULL"),
    (dict(k=0x10008), "FA_ERR_ALIGN"),
    (dict(page_table=0x30002), "FA_ERR_ALIGN"),
]


def append(**kw):
    c, kw = cache(**kw)
    a = dict(k=0x40000, v=0x50000, x_type=0, views=None, cache=c, seq=0x60000, pos=0x70000, T=5, k_norm=None, eps=1e-6,
             rope=None, stream=None)
    a.update({("k" if f == "xk" else "v" if f == "xv" else f): x for f, x in kw.items()})
    return fb.STATUS[fb.fa_cache_append(**a)]


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + [
    (dict(x_type=3), "FA_ERR_TYPE"),
    (dict(T=-1), "FA_ERR_SHAPE"),
    (dict(eps=-1.0), "FA_ERR_SHAPE"),
    (dict(eps=float("nan")), "FA_ERR_SHAPE"),
    (dict(views=fb.fa_kv_views(-1, 0, 0, 0)), "FA_ERR_SHAPE"),
    (dict(xk=None), "FA_ERR_NULL"),
    (dict(xv=None), "FA_ERR_NULL"),
    (dict(seq=None), "FA_ERR_NULL"),
    (dict(pos=None), "FA_ERR_NULL"),
    (dict(xk=0x40002), "FA_ERR_ALIGN"),
    (dict(seq=0x60001), "FA_ERR_ALIGN"),
    (dict(rope=fb.fa_rope(0x80000, 130, 1)), "FA_ERR_SHAPE"),
    (dict(rope=fb.fa_rope(0x80000, 7, 0)), "FA_ERR_SHAPE"),
    (dict(rope=fb.fa_rope(0x80000, 64, 2)), "FA_ERR_SHAPE"),
    (dict(rope=fb.fa_rope(0x80000, 24, 1)), "FA_ERR_UNSUPPORTED"),
    (dict(rope=fb.fa_rope(0x80004, 64, 1)), "FA_ERR_ALIGN"),
    (dict(cache=None), "FA_ERR_NULL"),
])
def test_append_argument_errors(kw, code):
    assert append(**dict(kw)) == code


def read(**kw):
    c, kw = cache(**kw)
    a = dict(cache=c, seq=0x60000, pos=0x70000, T=5, y_type=0, k_out=0x80000, v_out=0x90000, stream=None)
    a.update(kw)
    return fb.STATUS[fb.fa_cache_read(**a)]


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + [
    (dict(y_type=4), "FA_ERR_TYPE"),
    (dict(T=-1), "FA_ERR_SHAPE"),
    (dict(seq=None), "FA_ERR_NULL"),
    (dict(k_out=0x80008), "FA_ERR_ALIGN"),
])
def test_read_argument_errors(kw, code):
    assert read(**dict(kw)) == code


def decode(**kw):
    c, kw = cache(**kw)
    a = dict(q=0x40000, act=0, q_row=1024, q_head=128, cache=c, seq_lens=0x50000, H=8, scale=0.1, alibi_slopes=None,
             softcap=0.0, sinks=None, O=0x60000, lse=0x70000, workspace=0x100000, workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    return fb.STATUS[fb.fa_paged_decode(**a)]


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + [
    (dict(act=3), "FA_ERR_TYPE"),
    (dict(H=7), "FA_ERR_SHAPE"),
    (dict(H=0), "FA_ERR_SHAPE"),
    (dict(q_row=-1), "FA_ERR_SHAPE"),
    (dict(softcap=-1.0), "FA_ERR_SHAPE"),
    (dict(softcap=float("inf")), "FA_ERR_SHAPE"),
    (dict(q=None), "FA_ERR_NULL"),
    (dict(O=None), "FA_ERR_NULL"),
    (dict(seq_lens=None), "FA_ERR_NULL"),
    (dict(q=0x40002), "FA_ERR_ALIGN"),
    (dict(O=0x60008), "FA_ERR_ALIGN"),
    (dict(sinks=0x3), "FA_ERR_ALIGN"),
])
def test_decode_argument_errors(kw, code):
    assert decode(**dict(kw)) == code


def test_decode_workspace_size():
    c, _ = cache()
    n = fb.fa_paged_decode_workspace_size(c, 8)
    assert n > 0 and fb.fa_paged_decode_workspace_size(c, 7) == 0
    assert fb.fa_paged_decode_workspace_size(cache(D=96)[0], 8) == 0
    # it does not depend on how long the sequences may get, only on the heads and the batch
    assert fb.fa_paged_decode_workspace_size(cache(max_pages=1 << 16)[0], 8) <= 64 << 20


def norm(back=False, **kw):
    a = dict(q=0x10000, k=0x20000, x_type=0, views=None, wq=0x30000, wk=0x31000, eps=1e-6, pos=0x32000,
             rope=fb.fa_rope(0x33000, 128, 1), N=5, H=4, Hkv=2, D=128, y_type=0, stream=None)
    a.update(dict(gq=0x40000, gk=0x50000, dq=0x60000, dk=0x70000, dwq=0x80000, dwk=0x81000, workspace=0x90000,
                  workspace_bytes=1 << 24) if back else dict(q_out=0x40000, k_out=0x50000))
    a.update(kw)
    return fb.STATUS[(fb.fa_qk_norm_rope_backward if back else fb.fa_qk_norm_rope)(**a)]


NORM_ERRORS = [
    (dict(x_type=3), "FA_ERR_TYPE"),
    (dict(y_type=-1), "FA_ERR_TYPE"),
    (dict(N=-1), "FA_ERR_SHAPE"),
    (dict(H=0), "FA_ERR_SHAPE"),
    (dict(Hkv=-1), "FA_ERR_SHAPE"),
    (dict(eps=-1e-6), "FA_ERR_SHAPE"),
    (dict(D=80), "FA_ERR_UNSUPPORTED"),
    (dict(views=fb.fa_qk_views(0, 0, 0, -1)), "FA_ERR_SHAPE"),
    (dict(q=None), "FA_ERR_NULL"),
    (dict(k=None), "FA_ERR_NULL"),
    (dict(pos=None), "FA_ERR_NULL"),
    (dict(q=0x10001), "FA_ERR_ALIGN"),
    (dict(wq=0x30002), "FA_ERR_ALIGN"),
    (dict(rope=fb.fa_rope(0x33000, 256, 1)), "FA_ERR_SHAPE"),
    (dict(rope=fb.fa_rope(0x33000, 40, 1)), "FA_ERR_UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,code", NORM_ERRORS + [
    (dict(q_out=None), "FA_ERR_NULL"),
    (dict(k_out=None), "FA_ERR_NULL"),
    (dict(k_out=0x50008), "FA_ERR_ALIGN"),
])
def test_norm_argument_errors(kw, code):
    assert norm(**dict(kw)) == code


@pytest.mark.parametrize("kw,code", NORM_ERRORS + [
    (dict(gq=None), "FA_ERR_NULL"),
    (dict(dk=None), "FA_ERR_NULL"),
    (dict(gk=0x50004), "FA_ERR_ALIGN"),
    (dict(dwk=0x81001), "FA_ERR_ALIGN"),
])
def test_norm_backward_argument_errors(kw, code):
    assert norm(back=True, **dict(kw)) == code


def test_valid_calls_reach_the_device_query():
    """Arguments that are in order stop at the device (none here), before anything is enqueued."""
    if fb.lib() and os.environ.get("CUDA_VISIBLE_DEVICES") != "" and __import__("torch").cuda.is_available():
        pytest.skip("made-up addresses are not run on a GPU")
    stops = ("FA_ERR_CUDA", "FA_ERR_DEVICE")
    assert append() in stops and read() in stops and read(k_out=None) in stops and decode() in stops
    assert norm() in stops and norm(back=True) in stops and norm(Hkv=0, k=None, k_out=None) in stops
    assert norm(back=True, q=None, k=None, wq=None, wk=None) in stops  # a rotation's gradient needs no x
    assert decode(page_size=2, Hkv=4) in stops and decode(page_size=1, Hkv=4) in stops


def test_rope_frequencies_definition_and_errors():
    import torch
    f = fb.rope_frequencies(64, 500000.0, scale=0.25, factors=[1.0 + 0.1 * i for i in range(32)], device="cpu")
    for i in range(32):
        factor = float(np.float32(1.0 + 0.1 * i))
        turns = 0.25 * 500000.0 ** (-2.0 * i / 64) / factor / (2 * math.pi)
        assert abs(int(f[i]) / 2.0 ** 64 - turns) <= 2.0 ** -50 * turns + 2.0 ** -64  # cut off to whole units of 2^-64
    # more than a turn per position: whole turns drop out
    g = fb.rope_frequencies(2, 10000.0, scale=2 * math.pi * 1.75, device="cpu")
    assert abs((int(g[0]) % 2 ** 64) / 2.0 ** 64 - 0.75) < 1e-15
    assert fb.rope_frequencies(0, device="cpu").shape == (0,)
    out = (ctypes.c_uint64 * 4)()
    bad = (ctypes.c_float * 4)(1.0, 0.0, 1.0, 1.0)
    for args in ((7, 1e4, 1.0, None), (-2, 1e4, 1.0, None), (8, 0.0, 1.0, None), (8, 1e4, float("inf"), None),
                 (8, 1e4, 1.0, ctypes.addressof(bad))):
        assert fb.STATUS[fb.fa_rope_frequencies(*args, ctypes.addressof(out))] == "FA_ERR_SHAPE"
    assert fb.STATUS[fb.fa_rope_frequencies(8, 1e4, 1.0, None, None)] == "FA_ERR_NULL"
    with pytest.raises(fb.FaBackError):
        fb.rope_frequencies(8, factors=[1.0], device="cpu")
    assert f.dtype == torch.int64


def test_wrappers_refuse_what_the_kernels_do_not_take():
    torch = pytest.importorskip("torch")
    k = torch.zeros(4, 16, 2, 136, dtype=torch.uint8)
    table = torch.zeros(2, 2, dtype=torch.int32)
    c = fb.PagedCache(k, fb.FA_Q8_0, k.clone(), fb.FA_Q8_0, table, D=128, Dv=128)
    x, i2 = torch.zeros(2, 2, 128), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 128)
    raises = lambda f, *a, **kw: pytest.raises(fb.FaBackError, f, *a, **kw)  # noqa: E731
    raises(fb.PagedCache, k, fb.FA_F16, k, fb.FA_Q8_0, table, D=128, Dv=128)  # row size of another type
    raises(fb.PagedCache, k, fb.FA_Q8_0, k[:3], fb.FA_Q8_0, table, D=128, Dv=128)
    raises(fb.PagedCache, k[:, ::2], fb.FA_Q8_0, k[:, ::2], fb.FA_Q8_0, table, D=128, Dv=128)
    raises(fb.PagedCache, k, fb.FA_Q8_0, k, fb.FA_Q8_0, table.long(), D=128, Dv=128)
    raises(fb.cache_append, x.double(), x.double(), c, i2, i2)
    raises(fb.cache_append, x, x.half(), c, i2, i2)
    raises(fb.cache_append, x, x, c, i2.long(), i2)
    raises(fb.cache_append, x, x[:1], c, i2, i2)
    raises(fb.cache_append, x[:, :1], x, c, i2, i2)
    raises(fb.cache_append, x, x, c, i2[:1], i2)
    raises(fb.cache_append, x, x, c, i2, i2, k_norm=torch.zeros(64))
    raises(fb.cache_append, x, x, c, i2, i2, rope=torch.zeros(64))
    raises(fb.cache_append, x.transpose(1, 2).contiguous().transpose(1, 2), x, c, i2, i2)  # components not contiguous
    raises(fb.cache_read, c, i2, i2, dtype=torch.float64)
    raises(fb.cache_read, c, i2, i2[:1])
    raises(fb.paged_decode, q, c, i2.long(), scale=1.0)
    raises(fb.paged_decode, q[:1], c, i2, scale=1.0)
    raises(fb.paged_decode, q[..., :64], c, i2, scale=1.0)
    raises(fb.paged_decode, q, c, i2, scale=1.0, sinks=torch.zeros(3))
    raises(fb.qk_norm_rope, q, x, i2, wq=torch.zeros(4))
    raises(fb.qk_norm_rope, q, x.half(), i2)
    raises(fb.qk_norm_rope, q, x, i2.long(), rope=torch.zeros(64, dtype=torch.int64))
    raises(fb.qk_norm_rope, q, x, i2, dtype=torch.int32)
    raises(fb.qk_norm_rope, q, x, None, rope=torch.zeros(64, dtype=torch.int64))
    raises(fb.qk_norm_rope, q[:1, :1].expand(2 ** 32 + 2, 1, 128), None, i2)  # more rows than 31 bits hold
    raises(fb.qk_norm_rope_backward, q, None, q, x, i2)
    raises(fb.qk_norm_rope_backward, q[:1], x, q, x, i2)
    # tensors that are in order but live on the CPU: there is no fallback
    raises(fb.cache_append, x, x, c, i2, i2)
    raises(fb.paged_decode, q, c, i2, scale=1.0)
    raises(fb.qk_norm_rope, q, x, i2)


def test_kernels_that_start_early_read_with_ordinary_loads():
    """A kernel that may begin before the one before it on the stream has ended reads what that one writes:
    non-coherent loads are for data that nobody writes while the kernel runs."""
    folder = os.path.join(ROOT, "flash_attention_backward_gb300", "csrc")
    files = [f for f in sorted(os.listdir(folder)) if re.match(r"fa_(paged|decode|cache|norm_rope)", f)]
    assert {"fa_paged.cuh", "fa_decode.cuh", "fa_cache.cu", "fa_norm_rope.cuh"} <= set(files)
    for f in files:
        code = re.sub(r"//.*", "", open(os.path.join(folder, f)).read())
        assert not re.search(r"__ldg|ld\.global\.nc|__restrict__|__ldcv?a?\b", code), f
