"""The windowed decode over many splits: the combine beyond 32 of them, splits of 64
and 128 units (the most that the kernels take), a shorter last split on the cluster
kernel, a bad page's tokens left out.  The plans of these shapes are named in
tests/test_window_cut.py.

The pages of a long sequence are one page, named again and again, so that its tokens
are 64 and the protected ones, with the numbers of times that a query sees them: the
reference is a softmax with weights, in 64 bits over the library's own values of those
tokens (mla_lowbit_read as float32: s code + m to 2^-24).  Tolerance as for every
decode: max-abs 2e-3, rel-L2 1e-3, lse 1e-4; on the cluster kernel's packed pages the
lse has room for its additions, derived in tests/test_gpu_window.py."""

import numpy as np
import pytest

from tests.gpu_util import MAX_ABS, REL_L2

pytestmark = pytest.mark.gpu


class Repeated:
    """B sequences of length L whose pages are all page 0 (n new tokens at the end)."""

    def __init__(self, cb, rotate, B, L, seed, num_pages=1):
        import torch
        import bit_mla_kv_lowbit_gb300 as pkg
        self.torch, self.pkg, self.cb, self.L, self.B = torch, pkg, cb, L, B
        torch.manual_seed(seed)
        mp = -(-L // 64)
        c = self.cache = pkg.PagedCache(cb, 4 if cb != 16 else 16, np.zeros((B, mp), np.int32), num_pages, rotate=rotate)
        idx, pos = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.arange(64, dtype=torch.int32, device="cuda")
        c.append(torch.randn(64, 576, device="cuda").bfloat16(), None, pkg.Rope(64), pos=pos, seq_idx=idx)
        if cb != 16:
            c.sink.normal_()
            c.recent.normal_()
        self.lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
        # the tokens that differ, of sequence b: the page's rows, then sink and recent
        self.page = self._read(idx, pos, None)
        self.packed = cb != 16

    def _read(self, idx, pos, lens):
        torch, c = self.torch, self.cache
        out = torch.empty(len(pos), 576, device="cuda")
        self.pkg.read(c.layout, idx, pos, c.block_table, c.pool, c.sink, c.recent, out, c.err, seq_lens=lens)
        return out.double().cpu().numpy()

    def reference(self, q, b, scale, W, K, left_out=lambda t: np.zeros(len(t), bool)):
        """q [n][H][576] of sequence b -> out [n][H][512], lse [n][H], room [n][H]."""
        L, t = self.L, np.arange(self.L)
        kept = np.flatnonzero((t < 4) | (t >= L - 128)) if self.packed else np.zeros(0, int)
        own = np.zeros(0)
        if len(kept):
            torch = self.torch
            own = self._read(torch.full((len(kept),), b, dtype=torch.int32, device="cuda"),
                             torch.tensor(kept, dtype=torch.int32, device="cuda"), self.lens)
        keys = np.concatenate([self.page, own]) if len(kept) else self.page
        from_page = np.ones(L, bool)
        from_page[kept] = False
        from_page &= ~left_out(t)
        outs, lses, rooms = [], [], []
        for i, qi in enumerate(q):
            p = L - len(q) + i
            sees = (t <= p) & ((t < K) | (t > p - W))
            count = np.concatenate([np.bincount(t[sees & from_page] % 64, minlength=64), sees[kept].astype(int)])
            z = scale * (qi @ keys.T)
            m = z[:, count > 0].max(1, keepdims=True)
            w = np.where(count > 0, np.exp(np.minimum(z - m, 0)), 0) * count
            outs.append(w @ keys[:, :512] / w.sum(1, keepdims=True))
            lses.append(m[:, 0] + np.log(w.sum(1)))
            parts = np.zeros((len(qi), 64))
            for g in range(9):
                x, qg = self.page[:, 64 * g:64 * g + 64], qi[:, 64 * g:64 * g + 64]
                part = (2 / 3 if self.cb == 2 and g < 8 else 8 / 15) * (x.max(1) - x.min(1))
                parts += np.abs(qg).sum(1)[:, None] * part + np.abs(qg.sum(1))[:, None] * np.abs(x).max(1)
            largest = parts.max(1)
            if len(kept):
                largest = np.maximum(largest, (np.abs(qi) @ np.abs(own).T).max(1))
            rooms.append(scale * 38 * 2.0 ** -23 * largest)
        return np.stack(outs), np.stack(lses), np.stack(rooms)


def compare(run, q, out, lse, scale, W, K, clusters, seqs, rows=slice(None), left_out=None):
    bf16 = out.dtype != run.torch.float32
    for b in seqs:
        qb = q[b].double().cpu().numpy()[:, rows]
        kw = {} if left_out is None else dict(left_out=left_out)
        ref, ref_lse, room = run.reference(qb, b, scale, W, K, **kw)
        got = out[b].double().cpu().numpy()[:, rows]
        assert np.all(np.isfinite(got))
        step = 2.0 ** -8 * np.abs(ref) if bf16 else 0.0
        assert np.all(np.abs(got - ref) <= MAX_ABS + step), f"max-abs {np.abs(got - ref).max():.3g}"
        assert np.linalg.norm(got - ref) <= (REL_L2 + (2.0 ** -8 if bf16 else 0)) * np.linalg.norm(ref)
        off = np.abs(lse[b].double().cpu().numpy()[:, rows] - ref_lse)
        assert np.all(off <= 1e-4 + (room if clusters and run.packed else 0)), f"lse {off.max():.3g}"


def on_clusters(run, q, scale, W, K):
    try:
        run.pkg.set_fault_injection(1, 200_000)
        run.cache.decode_window(q, run.lens, scale, W, sinks=K)
        code = run.cache.error()
    finally:
        run.pkg.set_fault_injection(0, 0)
    run.cache.clear_error()
    return bool(code & 32)


# content bits, rotated, sequences, queries, heads, length, window, first tokens, pages of
# a table, splits, on clusters
CASES = {
    "130 splits": (4, False, 1, 1, 16, 19000, 8192, 0, 300, 130, False),
    "130 splits, rotated": (4, True, 1, 1, 16, 19137, 8192, 0, 300, 130, False),
    "129 splits of bf16 pages": (16, False, 1, 1, 16, 19199, 8192, 0, 300, 129, False),
    "unequal cuts on clusters": (4, False, 32, 1, 128, 16380, 4096, 64, 256, 3, True),
    "whole rows, 33 splits of 128 units, bf16 pages": (16, False, 1, 16, 128, 4200 * 64 - 1, 1 << 30, 0, 4200, 33, True),
    "whole rows, 33 splits of 128 units": (4, False, 1, 16, 128, 4200 * 64, 1 << 30, 0, 4200, 33, True),
    "152 splits of 64 units, bf16 pages": (16, False, 1, 1, 16, 9720 * 64, 1 << 30, 0, 9720, 152, False),
    "152 splits of 64 units, INT2": (2, False, 1, 1, 16, 9720 * 64 - 5, 1 << 30, 0, 9720, 152, False),
    "152 splits of 64 units, rotated": (4, True, 1, 1, 16, 9720 * 64, 1 << 30, 0, 9720, 152, False),
}


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_many_splits(name, bf16):
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    cb, rotate, B, n, H, L, W, K, mp, splits, clusters = CASES[name]
    run = Repeated(cb, rotate, B, L, seed=900 + len(name))
    c = run.cache
    c.block_table = torch.zeros(B, mp, dtype=torch.int32, device="cuda")
    c.max_pages = mp
    assert pkg.window_plan(c.layout, B, H, n, W, K, mp, num_sms=152)[0] == splits
    scale = 192 ** -0.5
    q = torch.randn(B, n, H, 576, device="cuda").bfloat16()
    assert on_clusters(run, q, scale, W, K) == clusters
    lse = torch.empty(B, n, H, device="cuda")
    out = torch.full((B, n, H, 512), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    c.decode_window(q, run.lens, scale, W, sinks=K, out=out, lse=lse)
    assert c.error() == 0
    compare(run, q, out, lse, scale, W, K, clusters, {0, B // 2, B - 1}, rows=slice(None, None, 5))
    again = torch.empty_like(out)
    c.decode_window(q, run.lens, scale, W, sinks=K, out=again)
    assert torch.equal(out, again)  # the order of additions does not depend on timing


@pytest.mark.parametrize("cb,rotate,heads,clusters", [(4, False, 16, False), (2, False, 16, False), (4, True, 16, False),
                                                      (16, False, 16, False), (4, False, 128, True), (2, False, 128, True),
                                                      (16, False, 128, True)])
@pytest.mark.parametrize("bad", [-1, 1, 1 << 30])
def test_a_bad_pages_tokens_are_left_out(cb, rotate, heads, clusters, bad):
    import torch
    L, W, K = 1000, 700, 70
    B = 40 if clusters else 2
    run = Repeated(cb, rotate, B, L, seed=77)
    c = run.cache
    # (a first page, one in the window, the last one: on packed pages its tokens are protected)
    pages = [0, 8, (L - 1) // 64]
    for p in pages:
        c.block_table[:, p] = bad
    scale = 192 ** -0.5
    q = torch.randn(B, 1, heads, 576, device="cuda").bfloat16()
    lse = torch.empty(B, 1, heads, device="cuda")
    out = c.decode_window(q, run.lens, scale, W, sinks=K, lse=lse)
    assert c.error() == 4
    c.clear_error()
    left_out = lambda t: np.isin(t // 64, pages)  # noqa: E731
    # (values of the protected tokens do not need their page)
    table = c.block_table.clone()
    c.block_table.zero_()
    if clusters:
        assert on_clusters(run, q, scale, W, K)
    compare(run, q, out, lse, scale, W, K, clusters, {0, B - 1}, left_out=left_out)
    c.block_table.copy_(table)


@pytest.mark.parametrize("cb,heads,n,W,K", [(4, 48, 1, 700, 0), (4, 128, 1, 500, 64), (4, 16, 8, 260, 6), (2, 112, 1, 260, 3),
                                            (2, 64, 2, 150, 0)])
def test_lse_of_the_16_row_kernel(cb, heads, n, W, K):
    # small batches of many rows run there, whose logits are not in one accumulator
    # each: 1e-4, without room for additions
    import torch
    run = Repeated(cb, False, 4, 2050, seed=78)
    q = torch.randn(4, n, heads, 576, device="cuda").bfloat16()
    scale = 192 ** -0.5
    assert not on_clusters(run, q, scale, W, K)
    lse = torch.empty(4, n, heads, device="cuda")
    out = run.cache.decode_window(q, run.lens, scale, W, sinks=K, lse=lse)
    assert run.cache.error() == 0
    compare(run, q, out, lse, scale, W, K, False, {0, 3})
