"""The exponentials of hyb_prefix_attn_fwd, seen through the fp32 lse: values that
are not finite, at every place of a key among its tile's."""
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
