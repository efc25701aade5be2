"""hyb_prefix_attn_fwd where a CTA works through several items one after another:
what the warps hand over between items.  Against the fp64 definition, with the
tolerances of test_gpu_prefix, and with equal bits from equal calls."""
import pytest
import torch

from tests.test_gpu_prefix import _case, _check, _ref, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hb():
    import compressed_sparse_sliding_b200 as hb
    return hb


def _check_case(hb, B, Lq, Hq, Hkv, d, m, W, Np, Nc, repeats=10):
    c, q_pos, kv0, Lkv = _case(B, Lq, Hq, Hkv, d, m, W, Np, Nc)
    o, lse = _run(hb, c, q_pos, kv0, Lkv, m, W)
    _check(o, lse, _ref(c, q_pos, kv0, m, W), d)
    for _ in range(repeats):
        o2, lse2 = _run(hb, c, q_pos, kv0, Lkv, m, W)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


# One query tile a sequence and KV head, o written by the items themselves, three to
# ten items a CTA (own entry counts from none to all, so items of no tile to several):
# warps without rows in the tile must not free an O for those that still read it.
@pytest.mark.parametrize("B,Lq,Hq,Hkv,d,m,W,Np,Nc", [
    (64, 1, 64, 8, 64, 4, 0, 0, 64),         # 512 items of one tile or none, eight rows
    (64, 1, 64, 8, 128, 1, 0, 0, 300),       # up to three tiles
    (48, 1, 320, 8, 64, 4, 0, 0, 140),       # 40 rows: two row quads
    (100, 1, 384, 4, 64, 2, 100, 0, 60),     # 96 rows: three; entries and a window
    (90, 2, 80, 16, 128, 128, 130, 0, 3),    # five heads x two tokens
    (64, 1, 96, 8, 64, 4, 128, 130, 130),    # through the shared entries as well
    (40, 1, 96, 16, 128, 4, 60, 60, 60),
])
def test_single_query_tiles(hb, B, Lq, Hq, Hkv, d, m, W, Np, Nc):
    _check_case(hb, B, Lq, Hq, Hkv, d, m, W, Np, Nc)


# Two query tiles an item, whose exponentials go in turns: several such items a CTA,
# beside items of one query tile and items whose key tiles alternate.  The turns of one
# item follow those of the item before it.
@pytest.mark.parametrize("B,Lq,Hq,Hkv,d,m,W,Np,Nc", [
    (40, 130, 8, 8, 64, 4, 16, 30, 200),     # three a CTA, o written by the items themselves
    (16, 260, 8, 8, 64, 4, 16, 100, 150),    # a pair, then the sequence's third query tile alone
    (12, 70, 80, 16, 128, 4, 30, 260, 200),  # five heads a tile, three tiles a sequence
    (100, 1, 512, 16, 64, 4, 0, 1000, 150),  # up to two over the shared entries, then alternating items
    (64, 1, 256, 16, 128, 4, 128, 2000, 300),
])
def test_query_tiles_in_turns(hb, B, Lq, Hq, Hkv, d, m, W, Np, Nc):
    _check_case(hb, B, Lq, Hq, Hkv, d, m, W, Np, Nc)
