"""Page tables on the CPU: the oracle against itself run as a whole (a step of
many tokens is many steps of one), and the refusals."""

import os

import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from attention_sm_flashattention_gb300 import _native
from attention_sm_flashattention_gb300.paging import _apart
from oracle import paging as orc

FAKE = 1 << 20  # an aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        from attention_sm_flashattention_gb300 import build
        build.build()
    return _native.lib()


def test_steps_of_one_are_a_step_of_many():
    stack, table = list(range(19, -1, -1)), [[-1] * 6, [-1] * 6]
    lens, count, t1 = [3, 0], 20, [list(r) for r in table]
    t1[0][0] = 7  # a page that is there
    whole = orc.step(stack, count, t1, lens, [5, 0], 5, 4)
    t, now, n, slots = [list(r) for r in t1], lens, count, []
    for i in range(5):
        s, _, now, n, t = orc.step(stack, n, t, now, [1, 0], 1, 4)
        slots.append(s[0][0])
    assert (slots, now, n, t) == (whole[0][0], whole[2], whole[3], whole[4])
    assert whole[0][0] == [7 * 4 + 3, 0, 1, 2, 3] and whole[0][1] == [-1] * 5 and whole[3] == 19


def test_release_gives_back_what_steps_took():
    stack, table = [4, 3, 2, 1, 0], [[-1] * 3, [-1] * 3]
    _, _, lens, count, table = orc.step(stack, 5, table, [0, 0], [5, 3], 5, 2)
    assert count == 0 and table == [[0, 1, 2], [3, 4, -1]] and lens == [5, 3]
    lens, count, stack = orc.release(stack, count, table, lens, [True, False], 2)
    assert lens == [0, 3] and count == 3 and stack[:3] == [0, 1, 2]


def test_too_few_pages():
    slots, _, lens, count, table = orc.step([1, 0], 2, [[-1] * 4], [0], [7], 8, 2)
    assert count == -2 and table == [[0, 1, -1, -1]] and slots == [[0, 1, 2, 3, -1, -1, -1, -1]] and lens == [7]


def step(lib, B=4, N=8, pages=64, page=16, row=8, **kw):
    a = dict(zip("stack count table lens q slots pos out_lens out_count".split(), [FAKE] * 9), **kw)
    return lib.fa_cache_step(a["stack"], a["count"], a["table"], a["lens"], a["q"], a["slots"], a["pos"], a["out_lens"],
                             a["out_count"], B, N, pages, page, row, None)


def release(lib, B=4, pages=64, page=16, row=8, ws=FAKE, ws_bytes=20, **kw):
    a = dict(zip("stack count table lens done out_lens out_count".split(), [FAKE] * 7), **kw)
    return lib.fa_cache_release(a["stack"], a["count"], a["table"], a["lens"], a["done"], a["out_lens"], a["out_count"],
                                ws, ws_bytes, B, pages, page, row, None)


BAD, BIG = _native.FA_ERR_INVALID_ARG, _native.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [(dict(stack=None), BAD), (dict(count=None), BAD), (dict(table=None), BAD),
                                     (dict(lens=None), BAD), (dict(out_lens=None), BAD), (dict(out_count=None), BAD),
                                     (dict(lens=FAKE + 2), BAD), (dict(B=0), BAD), (dict(pages=0), BAD),
                                     (dict(page=-1), BAD), (dict(row=0), BAD), (dict(B=1 << 20, row=1 << 11), BIG),
                                     (dict(pages=0x7fffffff), BIG)])
def test_refusals(lib, kw, code):
    assert step(lib, **kw) == code
    assert release(lib, **({"ws_bytes": 1 << 40} | kw)) == code


def test_more_refusals(lib):
    for kw in (dict(slots=None), dict(pos=None), dict(N=0), dict(slots=FAKE + 4), dict(pos=FAKE + 4), dict(q=FAKE + 1)):
        assert step(lib, **kw) == BAD, kw
    assert release(lib, done=None) == BAD
    for kw in (dict(ws=None), dict(ws=FAKE + 2), dict(ws_bytes=19)):
        assert release(lib, **kw) == _native.FA_ERR_WORKSPACE, kw
    assert lib.fa_cache_release_workspace_size(4) == 20 and lib.fa_cache_release_workspace_size(0) == 0


def test_python_refusals():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(free_pages=i32(8), free_count=i32(1), block_table=i32(2, 3), cached_lens=i32(2), q_lens=None, N=1,
                page_size=16)
    for name, x in good.items():
        if isinstance(x, torch.Tensor):
            with pytest.raises(ValueError):  # (also as they are: not on a GPU)
                fa.cache_step(**(good | {name: x.reshape(-1)[None, None]}))
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_step(**good)
    with pytest.raises(ValueError):
        fa.page_pool(0)
    stack, count = fa.page_pool(3, device="cpu")
    assert stack.tolist() == [2, 1, 0] and count.tolist() == [3]


def test_outputs_that_overlap():
    x = torch.zeros(16, dtype=torch.int32)
    _apart((("a", x[:4], "in"), ("b", x[4:8], None)), (("in", x[:4]), ("other", x[8:])))
    for out, taken in (((("a", x[:4], None),), (("in", x[:4]),)), ((("a", x[1:5], "in"),), (("in", x[:4]),)),
                       ((("a", x[:4], None), ("b", x[3:6], None)), ())):
        with pytest.raises(ValueError, match="overlaps"):
            _apart(out, taken)


def test_rotary_axes_of_sections():
    assert fa.rotary_axes([4, 2, 2], device="cpu").tolist() == [0, 0, 0, 0, 1, 1, 2, 2]
    assert fa.rotary_axes([4, 2, 2], dealt=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert fa.rotary_axes([0, 3], dealt=True, device="cpu").tolist() == [1, 1, 1]
    for bad in ([], [0, 0], [2, -1]):
        with pytest.raises(ValueError):
            fa.rotary_axes(bad, device="cpu")


def test_rotary_axes_refusals(lib):
    import ctypes
    st = (ctypes.c_longlong * 3)(0, 64, 64)

    def turn(axes=FAKE, n=3, rot=64, pos=FAKE, Z=1):
        return lib.fa_rotary_axes(FAKE, st, FAKE, st, None, None, None, None, pos, 4, 4, axes, n, FAKE, Z, 1, 0, 4, 64, rot,
                                  0, 0, 1.0, 0, None)
    assert turn(axes=None) == BAD and turn(axes=FAKE + 2) == BAD and turn(n=0) == BAD and turn(pos=None) == BAD
    assert turn(rot=63) == BIG and turn(rot=128) == BIG
    assert turn(Z=0) == _native.FA_OK
