"""Whole numbers beyond the 32 bits of the ABI's ints: a window or a number of first
tokens of any size is all tokens, anything else is refused.  None becomes another
number (ctypes keeps the low 32 bits without an error)."""

import numpy as np
import pytest

import bit_mla_kv_lowbit_gb300 as pkg

BIG = [1 << 31, 1 << 32, (1 << 32) + 64, 1 << 40, -(1 << 32) + 64, -(1 << 40)]


@pytest.mark.parametrize("cb", [4, 16])
@pytest.mark.parametrize("window,sinks", [(1 << 40, 0), (2 ** 32 + 100, 0), (64, 1 << 40), (64, 2 ** 32 + 4), (1 << 31, 1 << 31)])
def test_a_huge_window_is_all_tokens(cb, window, sinks):
    lay = pkg.layout(cb, 4 if cb != 16 else 16)
    most = 512 * 64
    assert pkg.window_plan(lay, 2, 16, 1, window, sinks, 512, num_sms=152) == \
        pkg.window_plan(lay, 2, 16, 1, min(window, most), min(sinks, most), 512, num_sms=152)


def test_numbers_that_do_not_fit_are_refused():
    lay = pkg.layout(4, 4)
    plan = dict(num_seqs=2, heads=16, queries=1, window=64, sinks=0, max_pages=8, num_sms=152)
    assert pkg.window_plan(lay, **plan)[0] >= 1
    for v in BIG:
        for name in ("num_seqs", "heads", "queries", "max_pages", "num_sms"):
            with pytest.raises(ValueError, match=name):
                pkg.window_plan(lay, **{**plan, name: v})
        with pytest.raises(ValueError):
            pkg.decode_plan(lay, v, [100])
        with pytest.raises(ValueError):
            pkg.decode_plan(lay, 16, [100], num_sms=v)
        with pytest.raises(ValueError):
            pkg.rope_table(v)
        with pytest.raises(ValueError):
            pkg.rope_table(64, scaling="yarn", factor=2.0, original_len=v)
        with pytest.raises(ValueError):
            pkg.layout(v, 4)
        with pytest.raises(ValueError):
            pkg.layout(4, v)
        with pytest.raises(ValueError):
            pkg.set_fault_injection(v)
    with pytest.raises(pkg.LibraryError):
        pkg.window_plan(lay, **{**plan, "window": -(1 << 32) + 64})
    with pytest.raises(pkg.LibraryError):
        pkg.window_plan(lay, **{**plan, "sinks": -(1 << 32)})
    with pytest.raises(pkg.LibraryError):
        pkg.set_fault_injection(0, -(1 << 64) + 5)


def test_parts_of_numbers_are_not_cut_off():
    lay = pkg.layout(4, 4)
    plan = dict(num_seqs=2, heads=16, queries=1, window=64, sinks=0, max_pages=8, num_sms=152)
    for name in plan:
        with pytest.raises(ValueError, match=name):
            pkg.window_plan(lay, **{**plan, name: plan[name] + 0.5})
        assert pkg.window_plan(lay, **{**plan, name: float(plan[name])}) == pkg.window_plan(lay, **plan)
    for v in (64.5, float("nan")):
        with pytest.raises(ValueError):
            pkg.rope_table(v)


def test_sizes_of_a_call_are_not_cut():
    # the Python way to a launch: nothing is called when a size does not fit
    b = pkg.binding
    fn = pkg.load().mla_lowbit_assign

    def call(*args):
        raise AssertionError("called")
    call.argtypes = fn.argtypes
    for k in range(4):
        args = [4, 8, 32, 16] + [None] * 13
        args[k] = (1 << 32) + 4
        with pytest.raises(pkg.LibraryError, match="size"):
            b._launch(call, "mla_lowbit_assign", 0, args, None)
    with pytest.raises(pkg.LibraryError, match="size"):
        b._check_sizes("mla_lowbit_write", 4, (1 << 32) + 4)
    b._check_sizes("mla_lowbit_write", 4, (1 << 31) - 1)


@pytest.mark.gpu
@pytest.mark.parametrize("native", [True, False])
def test_calls_with_numbers_beyond_32_bits(native, monkeypatch):
    import torch
    if not native:
        monkeypatch.setattr(pkg.binding, "_NATIVE", None)
    torch.manual_seed(3)
    c = pkg.PagedCache.empty(4, 4, 2, 8, 16, 700)
    c.assign(torch.tensor([300, 400], dtype=torch.int32, device="cuda"))
    c.append(torch.randn(700, 576, device="cuda").bfloat16(), None, pkg.Rope(64))
    q = torch.randn(2, 16, 576, device="cuda").bfloat16()
    # (512 tokens are the whole table: the same plan, so the same bits)
    for kw, same in ((dict(window=2 ** 32 + 100), dict(window=512)), (dict(window=1 << 40), dict(window=512)),
                     (dict(window=7, sinks=1 << 40), dict(window=7, sinks=512)),
                     (dict(window=7, sinks=2 ** 32), dict(window=7, sinks=512))):
        assert torch.equal(c.decode_window(q, c.seq_lens, 0.07, **kw), c.decode_window(q, c.seq_lens, 0.07, **same)), kw
    for kw in (dict(window=-(1 << 32) + 100), dict(window=7, sinks=-(1 << 40))):
        with pytest.raises(pkg.LibraryError):
            c.decode_window(q, c.seq_lens, 0.07, **kw)
    x = torch.randn(5, 2, 128, device="cuda")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    for offset in (1 << 32, -(1 << 32), 1 << 40):
        with pytest.raises(pkg.LibraryError):
            pkg.rope(x, pos, pkg.Rope(64), offset=offset)
    with pytest.raises(ValueError, match="offset"):
        pkg.rope(x, pos, pkg.Rope(64), offset=2.5)
    for kw in (dict(window=7.5), dict(window=7, sinks=0.5)):
        with pytest.raises(ValueError, match="whole"):
            c.decode_window(q, c.seq_lens, 0.07, **kw)
    # more rows than an int counts, all of them one element
    rows = torch.zeros(1, 1, 1, dtype=torch.bfloat16, device="cuda").expand((1 << 32) + 5, 1, 1)
    with pytest.raises(pkg.LibraryError):
        pkg.norm_rope(rows, out=rows)
    assert c.error() == 0
