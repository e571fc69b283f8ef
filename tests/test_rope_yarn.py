"""YaRN's sharpening of attention: in the rotation where whole heads are rotated, in the
rotation and the softmax scale by the checkpoint's mscale and mscale_all_dim where
only a decoupled key is."""

import math

import numpy as np
import pytest

import bit_mla_kv_lowbit_gb300 as pkg


def t(factor, m):
    return 0.1 * m * math.log(factor) + 1


@pytest.mark.parametrize("factor", [1.0, 2.0, 8.0, 40.0])
@pytest.mark.parametrize("mscale,all_dim", [(1.0, 1.0), (0.707, 0.707), (1.0, 0.0), (0.707, 1.0), (2.0, 0.5), (0.0, 0.0)])
def test_the_rotation_and_the_softmax_share_the_factor(factor, mscale, all_dim):
    r = pkg.Rope(64, scaling="yarn", factor=factor, device="cpu", mscale=mscale, mscale_all_dim=all_dim)
    # (held as a float32 at most: half a step of 2^-23)
    assert abs(r.mscale - t(factor, mscale) / t(factor, all_dim)) <= 2.0 ** -24 * r.mscale
    assert r.softmax_factor == t(factor, all_dim) ** 2
    if mscale == all_dim:
        assert r.mscale == 1.0
    # a logit's rotated part has mscale of the query and of the key, all of it the
    # softmax's factor: together t(mscale)^2, the unrotated part t(mscale_all_dim)^2
    whole = r.mscale ** 2 * r.softmax_factor
    assert abs(whole - t(factor, mscale) ** 2) <= 2.0 ** -22 * whole


def test_the_default_is_that_of_whole_heads():
    r = pkg.Rope(64, scaling="yarn", factor=40.0, device="cpu")
    assert r.mscale == pkg.rope_table(64, scaling="yarn", factor=40.0)[1] and r.softmax_factor == 1.0
    for scaling in ("none", "linear", "ntk"):
        r = pkg.Rope(64, scaling=scaling, factor=2.0, device="cpu")
        assert r.mscale == 1.0 and r.softmax_factor == 1.0


def test_the_frequencies_do_not_depend_on_it():
    a = pkg.Rope(64, scaling="yarn", factor=40.0, device="cpu").phase.numpy()
    b = pkg.Rope(64, scaling="yarn", factor=40.0, device="cpu", mscale=0.7, mscale_all_dim=0.7).phase.numpy()
    assert np.array_equal(a, b)


@pytest.mark.parametrize("kw", [dict(mscale=-1.0), dict(mscale_all_dim=-0.1), dict(mscale=float("nan")),
                                dict(mscale_all_dim=float("inf"))])
def test_refusals(kw):
    with pytest.raises(ValueError):
        pkg.Rope(64, scaling="yarn", factor=4.0, device="cpu", **kw)
    for scaling in ("none", "linear", "ntk"):
        with pytest.raises(ValueError):
            pkg.Rope(64, scaling=scaling, factor=4.0, device="cpu", mscale=0.7, mscale_all_dim=0.7)


@pytest.mark.gpu
@pytest.mark.parametrize("native", [True, False])
def test_logits_of_a_decoupled_key(native, monkeypatch):
    # one cached token and one query: the lse is its logit.  Content and rotated part
    # are scaled alike with equal parameters
    import torch
    if not native:
        monkeypatch.setattr(pkg.binding, "_NATIVE", None)
    torch.manual_seed(2)
    factor, scale = 40.0, 0.07
    rope = pkg.Rope(64, scaling="yarn", factor=factor, mscale=1.0, mscale_all_dim=1.0)
    c = pkg.PagedCache.empty(16, 16, 1, 1, 1, 1)
    c.assign(torch.tensor([1], dtype=torch.int32, device="cuda"))
    kv = torch.randn(1, 576, device="cuda").bfloat16()
    c.append(kv, None, rope)
    q = torch.randn(1, 16, 576, device="cuda").bfloat16()
    rot = torch.empty_like(q)
    rot[..., :512] = q[..., :512]
    pkg.rope(q[..., 512:], torch.zeros(1, dtype=torch.int32, device="cuda"), rope, out=rot[..., 512:])
    lse = torch.empty(1, 16, device="cuda")
    c.decode_window(rot, c.seq_lens, scale * rope.softmax_factor, 8, lse=lse)
    k = kv[0].double()
    ckv = k[:512] / torch.sqrt((k[:512] ** 2).mean() + 1e-6)
    logit = scale * t(factor, 1.0) ** 2 * (q[0].double() @ torch.cat([ckv.bfloat16().double(), k[512:]]))
    # (position 0: the rotation is the identity, values are bf16 as they are; the latent
    # is rounded once from exact arithmetic and differs only where float64's sum would)
    assert float((lse[0].double() - logit).abs().max()) <= 1e-4
