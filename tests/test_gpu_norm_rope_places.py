"""norm_rope between two parts of one buffer: every pair of parts that do not meet, in
the ways in which a fused projection's output has them, and refusals of those that do."""

import pytest

pytestmark = pytest.mark.gpu

N, H, D = 37, 5, 24


def _run(torch, pkg, x, y, weight=None, rot=True):
    pos = torch.arange(x.shape[0], dtype=torch.int32, device="cuda") * 77
    rope = pkg.Rope(8, interleaved=False) if rot else None
    kept = x.clone()
    want = pkg.norm_rope(kept, pos, rope, weight, offset=3, out=torch.empty_like(kept)) if rot else \
        pkg.norm_rope(kept, weight=weight, out=torch.empty_like(kept))
    pkg.norm_rope(x, pos if rot else None, rope, weight, offset=3 if rot else 0, out=y)
    # sums of another alignment are in another order: a few steps of the type
    tol = 16 * torch.finfo(x.dtype).eps
    assert float((y.float() - want.float()).abs().max()) <= tol * float(want.float().abs().max() + 1)
    return kept


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("swap", [False, True])
@pytest.mark.parametrize("gap", [0, 1, 8])
def test_beside_each_other(dtype, swap, gap):
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    torch.manual_seed(gap)
    dt = getattr(torch, dtype)
    w = torch.rand(D, device="cuda").to(dt)
    wide = H * D
    # [token][q heads | gap | k heads with channels between them]
    buf = torch.randn(N, wide + gap + 2 * wide, device="cuda").to(dt)
    a = buf[:, :wide].view(N, H, D)
    b = buf[:, wide + gap:].unflatten(1, (H, 2 * D))[..., D - 5:2 * D - 5]
    # [head][tokens | tokens]
    heads = torch.randn(H, 2 * N + gap, D, device="cuda").to(dt)
    c, d = heads[:, :N].transpose(0, 1), heads[:, N + gap:].transpose(0, 1)
    # one head each
    one = torch.randn(N, 3 * D + gap, device="cuda").to(dt)
    e, f = one[:, :D].unsqueeze(1), one[:, D + gap:2 * D + gap].unsqueeze(1)
    # one token's heads
    g, h = buf[:1, :wide].view(1, H, D), buf[:1, wide + gap:].unflatten(1, (H, 2 * D))[..., :D]
    for whole, x, y in ((buf, a, b), (heads, c, d), (one, e, f), (buf, g, h)):
        if swap:
            x, y = y, x
        before = whole.clone()
        y.fill_(7)
        mark = whole.clone()  # x and everything that is not y
        kept = _run(torch, pkg, x, y, w)
        assert torch.equal(x, kept)
        got = y.clone()
        y.fill_(7)
        assert torch.equal(whole, mark)  # nothing but y was written
        whole.copy_(before)
        del got
    _run(torch, pkg, a, b, None, rot=False)


def test_parts_that_meet_are_refused():
    import torch
    import bit_mla_kv_lowbit_gb300 as pkg
    buf = torch.randn(N, 4 * H * D, device="cuda")
    x = buf[:, :H * D].view(N, H, D)
    for y in (buf[:, H * D - 1:2 * H * D - 1].view(N, H, D),             # the last channel of the last head
              buf[:, 4:4 + H * D].view(N, H, D),
              buf[:, D:].unflatten(1, (4 * H - 1, D))[:, :H],             # from the second head on
              buf.view(-1)[H * D:H * D + N * H * D].view(N, H, D),       # other strides, through x's tokens
              buf[:, 3 * H * D + 1:].as_strided((N - 1, H, D), (4 * H * D, D, 1), 3 * H * D + 1)):  # into the next token's x
        xx = x[:y.shape[0]]
        with pytest.raises(pkg.LibraryError):
            pkg.norm_rope(xx, out=y)
        with pytest.raises(pkg.LibraryError):
            pkg.norm_rope(y, out=xx)
    torch.cuda.synchronize()
