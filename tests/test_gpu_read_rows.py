"""What mla_lowbit_read leaves in the rows of tokens that it skips (padding, errors):
what was there, or zeros where the caller asks for them, as PagedCache.read does for
an output of its own."""

import pytest

pytestmark = pytest.mark.gpu


def _cache(torch, pkg, cb, rotate, n):
    c = pkg.PagedCache.empty(cb, 4 if cb != 16 else 16, 3, n // 64 + 2, n // 64 + 6, n + 96, rotate=rotate)
    c.assign(torch.tensor([n, 0, 70], dtype=torch.int32, device="cuda"))
    c.append(torch.randn(n + 96, 576, device="cuda").bfloat16(), None, pkg.Rope(64))
    assert c.error() == 0
    return c


# (a token a warp, and eight: more than 64 tokens an SM)
@pytest.mark.parametrize("n", [1, 131, 12000])
@pytest.mark.parametrize("cb,rotate", [(4, False), (2, True), (16, False)])
def test_an_output_of_its_own_has_no_row_that_nobody_wrote(cb, rotate, n):
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    torch.manual_seed(n + cb)
    c = _cache(torch, pkg, cb, rotate, n)
    tokens = n + 70
    for lens in (None, c.seq_lens):
        # memory that the next allocation of its size gets, full of NaN
        junk = torch.full((n + 96, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        at = junk.data_ptr()
        del junk
        got = c.read(c.seq_idx, c.pos, seq_lens=lens)
        assert got.data_ptr() == at  # (else the test shows nothing)
        assert not bool(got[tokens:].any()) and bool(torch.isfinite(got).all()) and bool(got[:tokens].any(1).all())
    assert c.error() == 0


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("cb,rotate", [(4, True), (2, False), (16, False)])
@pytest.mark.parametrize("n", [40, 12000])
def test_skipped_rows(cb, rotate, dtype, n, native, monkeypatch):
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    if not native:
        monkeypatch.setattr(pkg.binding, "_NATIVE", None)
    torch.manual_seed(9)
    c = _cache(torch, pkg, cb, rotate, n)
    idx, pos = c.seq_idx[:n].clone(), c.pos[:n].clone()
    idx[3], idx[4], pos[5], pos[6] = -1, 3, -1, c.max_pages * 64
    idx[n - 1] = -7
    skipped = torch.zeros(n, dtype=torch.bool, device="cuda")
    skipped[[3, 4, 5, 6, n - 1]] = True
    dt = getattr(torch, dtype)

    def read(clear):
        out = torch.full((n + 1, 576), float("nan"), dtype=dt, device="cuda")
        pkg.read(c.layout, idx, pos, c.block_table, c.pool, c.sink, c.recent, out[:n], c.err, seq_lens=c.seq_lens,
                 clear_skipped=clear)
        assert c.error() == 1 | 2
        c.clear_error()
        assert bool(torch.isnan(out[n]).all())  # the row behind the last token
        return out[:n]

    kept, cleared = read(False), read(True)
    assert bool(torch.isnan(kept[skipped]).all()) and not bool(cleared[skipped].any())
    assert torch.equal(kept[~skipped], cleared[~skipped]) and bool(torch.isfinite(kept[~skipped]).all())
    # a bad page: its tokens too
    c.block_table[0, 0] = c.pool.shape[0]
    out = torch.full((n, 576), float("nan"), dtype=dt, device="cuda")
    pkg.read(c.layout, idx, pos, c.block_table, c.pool, c.sink, c.recent, out, c.err, clear_skipped=True)
    assert c.error() == 1 | 2 | 4 and not bool(out[:min(n, 64)].any())
    c.clear_error()
