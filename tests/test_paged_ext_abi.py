"""Host side of fa_paged_ext.h: exports, argument checks before any launch, and the refusals of the Python wrappers."""
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

import flash_attention_backward_gb300 as fb  # noqa: E402
import paged_ext_ref as E  # noqa: E402
from flash_attention_backward_gb300 import build, paged  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fa_paged_ext.h")


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return fb.lib()


def test_declared_functions_are_exported_and_bound(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(["fa_qk_norm_rope_axes", "fa_qk_norm_rope_axes_backward", "fa_cache_append_axes", "fa_pages_extend",
                            "fa_pages_trim", "fa_page_bounds", "fa_page_select_workspace_size", "fa_page_select",
                            "fa_paged_decode_pages"])
    for n in names:
        assert hasattr(L, n) and hasattr(fb, n), n


def test_structures_have_the_headers_layout(tmp_path):
    """Sizes and the last members' offsets, as a C compiler lays them out."""
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fa_paged_ext.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %zu\\n", sizeof(fa_rope_axes), offsetof(fa_rope_axes, n_axes), sizeof(fa_page_lists), '
                   'offsetof(fa_page_lists, max_pages), sizeof(fa_page_bounds_pool));\nreturn 0;\n}\n')
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], stdout=subprocess.PIPE, text=True, check=True).stdout.split()]
    import ctypes
    assert got == [ctypes.sizeof(fb.fa_rope_axes), fb.fa_rope_axes.n_axes.offset, ctypes.sizeof(fb.fa_page_lists),
                   fb.fa_page_lists.max_pages.offset, ctypes.sizeof(fb.fa_page_bounds_pool)]


def cache(**kw):
    c = dict(k=0x10000, v=0x20000, page_table=0x30000, k_type=2, v_type=2, num_pages=8, page_size=16, B=2, max_pages=4,
             Hkv=2, D=128, Dv=128)
    c.update({f: kw.pop(f) for f in list(kw) if f in dict(fb.fa_paged_cache._fields_)})
    return fb.fa_paged_cache(**c), kw


CACHE_ERRORS = [
    (dict(k_type=4), "FA_ERR_TYPE"),
    (dict(num_pages=-1), "FA_ERR_SHAPE"),
    (dict(page_size=0), "FA_ERR_SHAPE"),
    (dict(Hkv=0), "FA_ERR_SHAPE"),
    (dict(D=96), "FA_ERR_UNSUPPORTED"),
    (dict(max_pages=1 << 27), "FA_ERR_UNSUPPORTED"),
    (dict(page_size=1, Hkv=1), "FA_ERR_ALIGN"),
    (dict(k=None), "FA_ERR_NULL"),
    (dict(page_table=None), "FA_ERR_NULL"),
    (dict(cache=None), "FA_ERR_NULL"),
]


def axes(freqs=0x80000, axis=0x81000, pos_stride=5, n_rot=64, style=1, n_axes=3):
    return fb.fa_rope_axes(freqs, axis, pos_stride, n_rot, style, n_axes)


AXES_ERRORS = [
    (axes(n_axes=0), "FA_ERR_SHAPE"),
    (axes(n_axes=9), "FA_ERR_SHAPE"),
    (axes(pos_stride=-1), "FA_ERR_SHAPE"),
    (axes(style=2), "FA_ERR_SHAPE"),
    (axes(n_rot=7, style=0), "FA_ERR_SHAPE"),
    (axes(n_rot=258), "FA_ERR_SHAPE"),
    (axes(n_rot=24), "FA_ERR_UNSUPPORTED"),
    (axes(axis=None), "FA_ERR_NULL"),
    (axes(freqs=0x80004), "FA_ERR_ALIGN"),
]


@pytest.mark.parametrize("kw,code", [(dict(rope=r), e) for r, e in AXES_ERRORS] + [
    (dict(pos=None), "FA_ERR_NULL"), (dict(pos=0x32001), "FA_ERR_ALIGN"), (dict(x_type=3), "FA_ERR_TYPE"), (dict(D=80), "FA_ERR_UNSUPPORTED")])
@pytest.mark.parametrize("back", [False, True])
def test_norm_axes_argument_errors(kw, code, back):
    a = dict(q=0x10000, k=0x20000, x_type=0, views=None, wq=0x30000, wk=0x31000, eps=1e-6, pos=0x32000, rope=axes(), N=5, H=4, Hkv=2,
             D=128, y_type=0, stream=None)
    a.update(dict(gq=0x40000, gk=0x50000, dq=0x60000, dk=0x70000, dwq=0x82000, dwk=0x83000, workspace=0x90000,
                  workspace_bytes=1 << 24) if back else dict(q_out=0x40000, k_out=0x50000))
    a.update(kw)
    assert fb.STATUS[(fb.fa_qk_norm_rope_axes_backward if back else fb.fa_qk_norm_rope_axes)(**a)] == code


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + [(dict(rope=r), e) for r, e in AXES_ERRORS] + [
    (dict(rope_pos=None), "FA_ERR_NULL"), (dict(rope_pos=0x90002), "FA_ERR_ALIGN"), (dict(pos=None), "FA_ERR_NULL"),
    (dict(T=-1), "FA_ERR_SHAPE"), (dict(xk=None), "FA_ERR_NULL")])
def test_append_axes_argument_errors(kw, code):
    c, kw = cache(**dict(kw))
    a = dict(k=0x40000, v=0x50000, x_type=0, views=None, cache=c, seq=0x60000, pos=0x70000, T=5, k_norm=None, eps=1e-6, rope_pos=0x90000,
             rope=axes(), stream=None)
    a.update({("k" if f == "xk" else f): x for f, x in kw.items()})
    assert fb.STATUS[fb.fa_cache_append_axes(**a)] == code


def page_lists(**kw):
    a = dict(page_table=0x10000, seq_lens=0x20000, free_pages=0x30000, num_free=0x40000, num_pages=9, page_size=16, B=3, max_pages=4)
    a.update({f: kw.pop(f) for f in list(kw) if f in a})
    return fb.fa_page_lists(**a), kw


LIST_ERRORS = [
    (dict(num_pages=-1), "FA_ERR_SHAPE"),
    (dict(page_size=0), "FA_ERR_SHAPE"),
    (dict(B=-1), "FA_ERR_SHAPE"),
    (dict(max_pages=-1), "FA_ERR_SHAPE"),
    (dict(B=(1 << 20) + 1), "FA_ERR_UNSUPPORTED"),
    (dict(max_pages=1 << 27), "FA_ERR_UNSUPPORTED"),
    (dict(num_pages=1 << 27), "FA_ERR_UNSUPPORTED"),
    (dict(page_table=None), "FA_ERR_NULL"),
    (dict(seq_lens=None), "FA_ERR_NULL"),
    (dict(free_pages=None), "FA_ERR_NULL"),
    (dict(num_free=None), "FA_ERR_NULL"),
    (dict(seq_lens=0x20002), "FA_ERR_ALIGN"),
    (dict(num_free=0x40001), "FA_ERR_ALIGN"),
    (dict(lists=None), "FA_ERR_NULL"),
]


@pytest.mark.parametrize("kw,code", LIST_ERRORS + [
    (dict(T=-1), "FA_ERR_SHAPE"), (dict(T=(1 << 30) + 1), "FA_ERR_UNSUPPORTED"), (dict(new_tokens=None), "FA_ERR_NULL"),
    (dict(starts=None), "FA_ERR_NULL"), (dict(first=None), "FA_ERR_NULL"), (dict(row=None), "FA_ERR_NULL"), (dict(seq=0x70002), "FA_ERR_ALIGN")])
def test_extend_argument_errors(kw, code):
    lists, kw = page_lists(**dict(kw))
    a = dict(lists=lists, new_tokens=0x50000, T=5, starts=0x60000, first=0x61000, seq=0x70000, pos=0x71000, row=0x72000, stream=None)
    a.update(kw)
    assert fb.STATUS[fb.fa_pages_extend(**a)] == code


@pytest.mark.parametrize("kw,code", LIST_ERRORS + [(dict(keep=None), "FA_ERR_NULL"), (dict(keep=0x50001), "FA_ERR_ALIGN")])
def test_trim_argument_errors(kw, code):
    lists, kw = page_lists(**dict(kw))
    a = dict(lists=lists, keep=0x50000, stream=None)
    a.update(kw)
    assert fb.STATUS[fb.fa_pages_trim(**a)] == code


def pool(codes=0x100000, scales=0x200000):
    return fb.fa_page_bounds_pool(codes, scales)


BOUND_ERRORS = CACHE_ERRORS + [
    (dict(bounds=None), "FA_ERR_NULL"),
    (dict(bounds=pool(codes=None)), "FA_ERR_NULL"),
    (dict(bounds=pool(scales=0x200008)), "FA_ERR_ALIGN"),
    (dict(seq_lens=None), "FA_ERR_NULL"),
    (dict(seq_lens=0x50002), "FA_ERR_ALIGN"),
]


@pytest.mark.parametrize("kw,code", BOUND_ERRORS + [(dict(first=0x60001), "FA_ERR_ALIGN")])
def test_bounds_argument_errors(kw, code):
    c, kw = cache(**dict(kw))
    a = dict(cache=c, bounds=pool(), first=None, seq_lens=0x50000, stream=None)
    a.update(kw)
    assert fb.STATUS[fb.fa_page_bounds(**a)] == code


@pytest.mark.parametrize("kw,code", BOUND_ERRORS + [
    (dict(act=3), "FA_ERR_TYPE"),
    (dict(H=7), "FA_ERR_SHAPE"),
    (dict(H=0), "FA_ERR_SHAPE"),
    (dict(q_head=-1), "FA_ERR_SHAPE"),
    (dict(K=0), "FA_ERR_SHAPE"),
    (dict(first=-1), "FA_ERR_SHAPE"),
    (dict(last=-1), "FA_ERR_SHAPE"),
    (dict(first=2, last=2, K=3), "FA_ERR_SHAPE"),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1, K=2 ** 31 - 1), "FA_ERR_SHAPE"),
    (dict(H=65536), "FA_ERR_UNSUPPORTED"),
    (dict(max_pages=(1 << 22) + 1), "FA_ERR_UNSUPPORTED"),
    (dict(B=1 << 21), "FA_ERR_UNSUPPORTED"),
    (dict(q=None), "FA_ERR_NULL"),
    (dict(pages=None), "FA_ERR_NULL"),
    (dict(q=0x40002), "FA_ERR_ALIGN"),
    (dict(pages=0x300002), "FA_ERR_ALIGN"),
    (dict(alibi_slopes=0x1), "FA_ERR_ALIGN"),
])
def test_select_argument_errors(kw, code):
    c, kw = cache(**dict(kw))
    a = dict(q=0x40000, act=0, q_row=1024, q_head=128, cache=c, bounds=pool(), seq_lens=0x50000, H=8, scale=0.1, alibi_slopes=None, K=3,
             first=1, last=1, pages=0x300000, workspace=0x400000, workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    assert fb.STATUS[fb.fa_page_select(**a)] == code


def test_select_workspace_size():
    c, _ = cache()
    assert fb.fa_page_select_workspace_size(c, 8, 3) >= 256
    for bad in ((c, 7, 3), (c, 8, 0), (cache(D=96)[0], 8, 3), (cache(max_pages=(1 << 22) + 1)[0], 8, 3), (c, 0, 1)):
        assert fb.fa_page_select_workspace_size(*bad) == 0
    long, _ = cache(max_pages=1 << 20)  # a key for each page
    assert fb.fa_page_select_workspace_size(long, 8, 3) == 2 * 2 * 4 << 20


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + [
    (dict(K=0), "FA_ERR_SHAPE"),
    (dict(pages=None), "FA_ERR_NULL"),
    (dict(pages=0x80002), "FA_ERR_ALIGN"),
    (dict(act=3), "FA_ERR_TYPE"),
    (dict(H=7), "FA_ERR_SHAPE"),
    (dict(softcap=-1.0), "FA_ERR_SHAPE"),
    (dict(q=None), "FA_ERR_NULL"),
    (dict(O=0x60008), "FA_ERR_ALIGN"),
])
def test_decode_pages_argument_errors(kw, code):
    c, kw = cache(**dict(kw))
    a = dict(q=0x40000, act=0, q_row=1024, q_head=128, cache=c, seq_lens=0x50000, pages=0x80000, K=3, H=8, scale=0.1, alibi_slopes=None,
             softcap=0.0, sinks=None, O=0x60000, lse=0x70000, workspace=0x100000, workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    assert fb.STATUS[fb.fa_paged_decode_pages(**a)] == code


# ------------------------------------------------------------------------------------------------
# wrappers

def test_rope_sections():
    assert fb.rope_sections([2, 1, 1], device="cpu").tolist() == [0, 0, 1, 2]
    assert fb.rope_sections([3, 1, 2], interleaved=True, device="cpu").tolist() == [0, 1, 2, 0, 2, 0]
    assert fb.rope_sections([0, 2], interleaved=True, device="cpu").tolist() == [1, 1]
    assert fb.rope_sections([4], device="cpu").dtype is torch.uint8
    for bad in ([], [1] * 9, [2, -1]):
        with pytest.raises(fb.FaBackError, match="sections"):
            fb.rope_sections(bad, device="cpu")


def paged_cache(D=128):
    k = torch.zeros(4, 16, 2, fb.fa_row_bytes(fb.FA_Q8_0, D), dtype=torch.uint8)
    return fb.PagedCache(k, fb.FA_Q8_0, k.clone(), fb.FA_Q8_0, torch.zeros(2, 2, dtype=torch.int32), D=D, Dv=D)


def test_objects_keep_what_they_were_made_with():
    lists, bounds = fb.PageLists.empty(3, 2, 8, 16, device="cpu"), fb.PageBounds.of(paged_cache())
    for o, names in ((lists, ("page_table", "seq_lens", "free", "num_free", "page_size", "c")), (bounds, ("codes", "scales", "c"))):
        for n in names:
            with pytest.raises(fb.FaBackError, match=n):
                setattr(o, n, getattr(o, n))
    lists.seq_lens.fill_(0)  # in place
    assert lists.seq_lens.tolist() == [0, 0, 0] and lists.free.tolist() == list(range(7, -1, -1)) and bounds.codes.shape == (4, 2, 2, 128)


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("make", [
    lambda: fb.PageLists(ints(3), ints(3), ints(8), ints(1), page_size=16),
    lambda: fb.PageLists(ints(3, 2), ints(4), ints(8), ints(1), page_size=16),
    lambda: fb.PageLists(ints(3, 2), ints(3).long(), ints(8), ints(1), page_size=16),
    lambda: fb.PageLists(ints(3, 2), ints(3), ints(2, 8), ints(1), page_size=16),
    lambda: fb.PageLists(ints(3, 2), ints(3), ints(8), ints(2), page_size=16),
    lambda: fb.PageLists(ints(2, 3).t(), ints(3), ints(8), ints(1), page_size=16),
    lambda: fb.PageBounds(torch.zeros(4, 2, 2, 100, dtype=torch.int8), torch.zeros(4, 2, 3)),
    lambda: fb.PageBounds(torch.zeros(4, 2, 2, 128), torch.zeros(4, 2, 4)),
    lambda: fb.PageBounds(torch.zeros(4, 2, 2, 128, dtype=torch.int8), torch.zeros(4, 2, 8)),
    lambda: fb.PageBounds(torch.zeros(4, 2, 128, dtype=torch.int8), torch.zeros(4, 2, 4)),
])
def test_objects_of_other_tensors_are_refused(make):
    with pytest.raises(fb.FaBackError):
        make()


def test_calls_with_other_tensors_are_refused():
    c, lists = paged_cache(), fb.PageLists.empty(3, 2, 8, 16, device="cpu")
    b, other = fb.PageBounds.of(c), fb.PageBounds.of(paged_cache(64))
    q, lens = torch.zeros(2, 4, 128), ints(2)
    x, rope = torch.zeros(5, 2, 128), fb.rope_frequencies(64, device="cpu")
    ax = fb.rope_sections([16, 16], device="cpu")
    for match, call in (
            ("bounds", lambda: fb.page_bounds(c, other, lens)),
            ("bounds", lambda: fb.page_select(q, c, other, lens, 2, scale=1.0)),
            ("seq_lens", lambda: fb.page_bounds(c, b, ints(3))),
            ("first", lambda: fb.page_bounds(c, b, lens, first=lens.float())),
            ("q", lambda: fb.page_select(q[:, :, :64], c, b, lens, 2, scale=1.0)),
            ("alibi_slopes", lambda: fb.page_select(q, c, b, lens, 2, scale=1.0, alibi_slopes=torch.zeros(3))),
            ("new_tokens", lambda: fb.pages_extend(lists, ints(2), 5)),
            ("T", lambda: fb.pages_extend(lists, ints(3), -1)),
            ("keep", lambda: fb.pages_trim(lists, ints(3).short())),
            ("pages", lambda: fb.paged_decode(q, c, lens, scale=1.0, pages=ints(2, 2))),
            ("pages", lambda: fb.paged_decode(q, c, lens, scale=1.0, pages=ints(2, 3, 4))),
            ("pages", lambda: fb.paged_decode(q, c, lens, scale=1.0, pages=ints(2, 2, 4).long())),
            ("rope_axes", lambda: fb.qk_norm_rope(x, None, ints(2, 5), rope=rope, rope_axes=ax[:5])),
            ("rope_axes", lambda: fb.qk_norm_rope(x, None, ints(2, 5), rope=rope, rope_axes=ax.int())),
            ("rope_axes", lambda: fb.qk_norm_rope(x, None, ints(2, 5), rope_axes=ax)),
            ("pos", lambda: fb.qk_norm_rope(x, None, ints(5), rope=rope, rope_axes=ax)),
            ("pos", lambda: fb.qk_norm_rope(x, None, ints(5, 2).t(), rope=rope, rope_axes=ax)),
            ("pos", lambda: fb.qk_norm_rope_backward(x, None, x, None, ints(2, 4), rope=rope, rope_axes=ax)),
            ("rope_pos", lambda: fb.cache_append(x, x, c, ints(5), ints(5), rope=rope, rope_axes=ax)),
            ("rope_pos", lambda: fb.cache_append(x, x, c, ints(5), ints(5), rope=rope, rope_pos=ints(2, 5))),
            ("CUDA", lambda: fb.pages_extend(lists, ints(3), 5)),
            ("CUDA", lambda: fb.pages_trim(lists, ints(3))),
            ("CUDA", lambda: fb.page_bounds(c, b, lens)),
            ("CUDA", lambda: fb.page_select(q, c, b, lens, 2, scale=1.0))):
        with pytest.raises(fb.FaBackError, match=match):
            call()


def test_the_reference_lists_take_and_give_back():
    """The lists that the kernels are held to, on a case worked by hand: pages of 4, the second request finds no room in its
    row and asks for none, the third finds too few pages, and the fourth needs none."""
    import numpy as np
    table = np.array([[5, -1, -1], [0, 1, 2], [-1, -1, -1], [3, -1, -1]])
    r = E.Lists(table, [3, 11, 0, 1], [7, 6, 4], 8, 4)
    got = r.extend([6, 2, 8, 2], 18)
    assert got["starts"] == [0, 6, 8, 16, 18] and got["first"] == [3, -1, -1, 1]
    assert r.table == [[5, 4, 6], [0, 1, 2], [-1, -1, -1], [3, -1, -1]] and r.stack == [7] and r.lens == [9, 11, 0, 3]
    assert got["row"] == [23, 16, 17, 18, 19, 24] + [-1] * 10 + [13, 14]
    r.trim([3, -1, 0, 99])
    assert r.stack == [7, 6, 4] and r.lens == [3, 11, 0, 3] and r.table[0] == [5, -1, -1]
