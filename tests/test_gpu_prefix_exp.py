"""The exponentials of hyb_prefix_attn_fwd, seen through the fp32 lse: their error
where few keys with small scores leave nothing else, and values that are not
finite, at every place of a key among its tile's."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hb():
    import compressed_sparse_sliding_b200 as hb
    return hb


@pytest.mark.parametrize("B,Hq", [(1, 4), (4, 64)])     # alternating key tiles; two query tiles
@pytest.mark.parametrize("part", ["shared", "own", "window"])
def test_a_score_that_is_not_finite_shows_in_lse(hb, B, Hq, part):
    d, n = 64, 32
    g = torch.Generator().manual_seed(B)
    q = torch.rand((B, 1, Hq, d), generator=g).add(0.5).bfloat16().cuda()
    k0 = torch.randn((n, 1, d), generator=g).bfloat16().cuda()
    v = torch.randn((n, 1, d), generator=g).bfloat16().cuda()
    q_pos = torch.full((B, 1), n - 1, dtype=torch.int32, device="cuda")
    kv0 = torch.zeros((B,), dtype=torch.int32, device="cuda")
    each = lambda x: x.expand(B, n, 1, d).contiguous()
    for bad in (float("nan"), float("inf")):
        for at in range(n):
            k = k0.clone()
            k[at, :, 5] = bad                            # q[5] > 0: the score is NaN or +infinity
            lse = torch.zeros((B, Hq, 1), device="cuda")
            if part == "shared":
                p = hb.problem(B=B, Lq=1, Lkv=0, Hq=Hq, Hkv=1, d=d, m=1, W=0, Nc=0, q_pos=q_pos)
                hb.hyb_prefix_attn_fwd(p, q, k, v, lse=lse)
            elif part == "own":
                p = hb.problem(B=B, Lq=1, Lkv=0, Hq=Hq, Hkv=1, d=d, m=1, W=0, Nc=n, q_pos=q_pos)
                hb.hyb_prefix_attn_fwd(p, q, None, None, each(k), each(v), lse=lse)
            else:
                p = hb.problem(B=B, Lq=1, Lkv=n, Hq=Hq, Hkv=1, d=d, m=1, W=n, Nc=0, q_pos=q_pos, kv_pos0=kv0)
                hb.hyb_prefix_attn_fwd(p, q, None, None, None, None, each(k), each(v), lse=lse)
            assert torch.all(torch.isnan(lse)), (bad, at)
    assert hb.hyb_get_device_status() == hb.HYB_OK


@pytest.mark.parametrize("Hq", [100, 176])              # one query tile; two
@pytest.mark.parametrize("n", [4, 16, 77])
def test_exponentials_are_as_good_as_the_hardwares(hb, Hq, n):
    # key 0 has score 0 and all others -s_h, exact in fp32: lse = log(1 + (n - 1) exp(-s_h)).
    # Error of a weight w = 2^-x, x = s log2(e): 2^-22 for 2^x, and x rounds twice (log2(e)
    # and the product), 2^-24 x each, which moves w by ln 2 as much; n fp32 terms, 2^-24 of
    # the sum each; log2 to 2^-23 of itself or of 1 (its units in the last place), and
    # twice 2^-24 for its product with ln 2.
    d = 64
    q = torch.zeros((1, 1, Hq, d))
    q[0, 0, :, 7] = torch.arange(Hq) / 16                # bf16 holds these
    k = torch.zeros((n, 1, d))
    k[1:, 0, 7] = -1
    q_pos = torch.full((1, 1), n - 1, dtype=torch.int32, device="cuda")
    p = hb.problem(B=1, Lq=1, Lkv=0, Hq=Hq, Hkv=1, d=d, m=1, W=0, Nc=0, q_pos=q_pos)
    lse = torch.zeros((1, Hq, 1), device="cuda")
    hb.hyb_prefix_attn_fwd(p, q.bfloat16().cuda(), k.bfloat16().cuda(), torch.zeros_like(k).bfloat16().cuda(), lse=lse)
    s = np.arange(Hq) / 16 / 8                           # the scale is 1 / sqrt(64)
    w = (n - 1) * np.exp(-s)
    want, share, x = np.log1p(w), w / (1 + w), s / np.log(2)
    tol = share * (2.0 ** -22 + np.log(2) * 2 * 2.0 ** -24 * x) + n * 2.0 ** -24
    tol += np.log(2) * 2.0 ** -23 * np.maximum(want / np.log(2), 1) + 2 * 2.0 ** -24 * want
    err = np.abs(lse[0, :, 0].double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err / tol).max())
