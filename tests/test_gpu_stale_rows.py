"""Rows that no query sees, full of NaN: what an earlier sequence left behind the end in
a page that was given out again, and drafted tokens behind a query's own.  A weight of 0
does not undo a NaN, so they must not be read into a product: results are the same bit
for bit, whatever the rows hold."""

import pytest

pytestmark = pytest.mark.gpu

LENS = [1, 5, 64, 131, 300, 517]


def _cache(torch, pkg, cb, rotate=False):
    c = pkg.PagedCache.empty(cb, 4 if cb != 16 else 16, len(LENS), 9, 9 * len(LENS), sum(LENS), rotate=rotate)
    c.assign(torch.tensor(LENS, dtype=torch.int32, device="cuda"))
    c.append(torch.randn(sum(LENS), 576, device="cuda").bfloat16(), None, pkg.Rope(64))
    return c


def _spoil_behind(torch, c, cb):
    for s, L in enumerate(LENS):
        page = int(c.block_table[s, (L - 1) // 64])
        first = (L - 1) % 64 + 1
        if cb == 16:
            c.pool[page].view(torch.bfloat16).view(64, 576)[first:] = float("nan")
        else:
            off = 64 * (64 * cb + 32)
            c.pool[page, off + 36 * first:off + 36 * 64] = 0xFF
            for k in range(128):  # ring entries of no token of the sequence
                if k >= L:
                    c.recent[s, k] = float("nan")
            if L < 4:
                c.sink[s, L:] = float("nan")


@pytest.mark.parametrize("heads", [16, 48, 128])
@pytest.mark.parametrize("cb,rotate", [(4, False), (2, False), (4, True), (16, False)])
def test_rows_behind_the_end(cb, rotate, heads):
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    torch.manual_seed(cb + heads)
    c = _cache(torch, pkg, cb, rotate)
    q = torch.randn(len(LENS), heads, 576, device="cuda").bfloat16()
    want, want_w = c.decode(q, c.seq_lens, LENS, 0.07).clone(), c.decode_window(q, c.seq_lens, 0.07, 200, sinks=3).clone()
    _spoil_behind(torch, c, cb)
    assert bool(torch.isfinite(want).all())
    assert torch.equal(c.decode(q, c.seq_lens, LENS, 0.07), want)
    assert torch.equal(c.decode_window(q, c.seq_lens, 0.07, 200, sinks=3), want_w)
    assert c.error() == 0


@pytest.mark.parametrize("n", [2, 5])
@pytest.mark.parametrize("cb,rotate", [(4, False), (2, False), (4, True), (16, False)])
def test_drafted_tokens_behind_a_query(cb, rotate, n):
    # (16 n rows: the 16-row kernel)
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    torch.manual_seed(cb + n)
    c = _cache(torch, pkg, cb, rotate)
    lens = LENS[1:]
    c.block_table, c.num_seqs = c.block_table[1:].contiguous(), len(lens)
    if cb != 16:
        c.sink, c.recent = c.sink[1:].contiguous(), c.recent[1:].contiguous()
    dev = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(len(lens), n, 16, 576, device="cuda").bfloat16()
    want = c.decode_multi(q, dev, lens, 0.07).clone()
    for s, L in enumerate(lens):
        p = L - 1
        if cb == 16:
            c.pool[int(c.block_table[s, p // 64])].view(torch.bfloat16).view(64, 576)[p % 64] = float("nan")
        elif p < 4:
            c.sink[s, p] = float("nan")
        else:
            c.recent[s, p % 128] = float("nan")
    got = c.decode_multi(q, dev, lens, 0.07)
    assert torch.equal(got[:, :n - 1], want[:, :n - 1]) and bool(torch.isnan(got[:, n - 1]).all())
    assert c.error() == 0
