"""Windowed decode of several queries a sequence: a token that is not finite reaches
the queries that see it and no other, also where queries of several positions share
a block of 128 rows (the cluster kernel) and the other query's weight for it is 0.

A query that does not see the token has the same additions with and without it (a
weight of 0 times a finite value or times 0), so its output is the same bit for bit."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def ran_on_clusters(pkg, cache, *args, **kw):
    """Whether the call runs on the cluster kernel: its withheld hand-off runs out."""
    try:
        pkg.set_fault_injection(1, 200_000)
        cache.decode_window(*args, **kw)
        code = cache.error()
    finally:
        pkg.set_fault_injection(0, 0)
    cache.clear_error()
    return bool(code & 32)


# content bits, heads, queries, window, first tokens, cluster kernel
CASES = [(4, 32, 3, 200, 3, True), (4, 64, 2, 130, 0, True), (4, 16, 8, 1, 0, True), (4, 48, 5, 90, 70, True),
         (2, 64, 3, 150, 2, True), (2, 32, 4, 600, 0, True), (16, 64, 2, 200, 3, True), (16, 32, 3, 65, 0, True),
         (16, 16, 16, 40, 5, True), (16, 48, 5, 600, 0, True),
         (4, 32, 3, 200, 3, False), (2, 16, 5, 90, 0, False), (16, 16, 4, 150, 2, False), (4, 128, 2, 200, 3, True)]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("one_split", [False, True])
def test_values_that_are_not_finite_reach_only_who_sees_them(case, one_split):
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    cb, H, n, W, K, clusters = CASES[case]
    if one_split and not clusters:
        pytest.skip("so many sequences run on the cluster kernel")
    torch.manual_seed(800 + case)
    lens = [n, 20, 131, 300, 517]
    # idle rows of the batch: with that many sequences the plan takes the cluster kernel
    idle = 0 if not clusters else 300 if one_split else 40
    B = len(lens) + idle
    c = pkg.PagedCache.empty(cb, 4 if cb != 16 else 16, B, 9, 9 * len(lens), sum(lens))
    c.assign(torch.tensor(lens + [0] * idle, dtype=torch.int32, device="cuda"))
    c.append(torch.randn(sum(lens), 576, device="cuda").bfloat16(), None, pkg.Rope(64))
    q = torch.randn(B, n, H, 576, device="cuda").bfloat16()
    if clusters != ran_on_clusters(pkg, c, q, c.seq_lens, 0.07, W, sinks=K):
        assert H == 128 or one_split or clusters, "the case is meant for the other kernel"
        pytest.skip("the plan takes the other kernel")
    clean = c.decode_window(q, c.seq_lens, 0.07, W, sinks=K)
    assert bool(torch.isfinite(clean).all())

    def row(s, p):  # the bf16 values of a token
        if cb == 16:
            return c.pool[int(c.block_table[s, p // 64])].view(torch.bfloat16).view(64, 576)[p % 64]
        return c.sink[s, p] if p < 4 else c.recent[s, p % 128]

    rng = np.random.default_rng(case)
    for value in (float("nan"), float("inf"), -float("inf")) + ((70000.0,) if cb != 16 else ()):
        # the newest token; one of the newest n; the oldest that the first query sees
        for pick in (lambda L: L - 1, lambda L: L - 1 - int(rng.integers(0, n)), lambda L: max(0, L - n - W + 1)):
            for ch in (slice(0, 576), slice(300, 301), slice(70, 71), slice(520, 521), slice(560, 561)):
                kept, at = [], []
                for s, L in enumerate(lens):
                    p = pick(L)
                    if cb != 16 and 4 <= p < L - 128:
                        continue  # packed: its values are always finite
                    kept.append((s, p, row(s, p).clone()))
                    row(s, p)[ch] = value
                    at.append((s, p))
                got = c.decode_window(q, c.seq_lens, 0.07, W, sinks=K)
                for s, p in at:
                    for i in range(n):
                        pos = lens[s] - n + i
                        if p <= pos and (p < K or p > pos - W):
                            bad = ~torch.isfinite(got[s, i])
                            assert bool(bad.any()), (s, p, i)
                            if value != value:
                                assert bool(bad.all()), (s, p, i)
                        else:
                            assert torch.equal(got[s, i], clean[s, i]), (s, p, i, value, ch)
                for s, p, v in kept:
                    row(s, p).copy_(v)
    assert torch.equal(c.decode_window(q, c.seq_lens, 0.07, W, sinks=K), clean)
    assert c.error() == 0


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("one_split", [False, True])
def test_lse_of_who_sees_a_nan(case, one_split):
    # not a number, as the sum that it is the logarithm of; the others' stays
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    cb, H, n, W, K, clusters = CASES[case]
    torch.manual_seed(850 + case)
    lens = [n, 20, 131, 300, 517]
    B = len(lens) + (300 if one_split else 40 if clusters else 0)
    c = pkg.PagedCache.empty(cb, 4 if cb != 16 else 16, B, 9, 9 * len(lens), sum(lens))
    c.assign(torch.tensor(lens + [0] * (B - len(lens)), dtype=torch.int32, device="cuda"))
    c.append(torch.randn(sum(lens), 576, device="cuda").bfloat16(), None, pkg.Rope(64))
    q = torch.randn(B, n, H, 576, device="cuda").bfloat16()
    lse = [torch.zeros(B, n, H, device="cuda") for _ in range(2)]
    c.decode_window(q, c.seq_lens, 0.07, W, sinks=K, lse=lse[0])
    for s, L in enumerate(lens):
        if cb == 16:
            c.pool[int(c.block_table[s, (L - 1) // 64])].view(torch.bfloat16).view(64, 576)[(L - 1) % 64, 5] = float("nan")
        else:
            (c.sink[s, L - 1] if L <= 4 else c.recent[s, (L - 1) % 128])[5] = float("nan")
    c.decode_window(q, c.seq_lens, 0.07, W, sinks=K, lse=lse[1])
    assert bool(torch.isnan(lse[1][:len(lens), n - 1]).all())
    assert torch.equal(lse[1][:, :n - 1], lse[0][:, :n - 1]) and torch.equal(lse[1][len(lens):], lse[0][len(lens):])
    assert bool(torch.isneginf(lse[0][len(lens):]).all()) and not bool(torch.isnan(lse[0]).any())
