"""hyb_attn_weights on the GPU against the fp64 definition.

Tolerance.  A score is an fp32 sum of d exact products (off by at most d 2^-24
of e = scale sum |q||k|); scaling to log2 units and subtracting lse round by
2^-23 of e and |lse| more, so exp of it is off by (d + 4) 2^-23 (e + |lse|)
relative, and by 2^-21 for the hardware exp2.  The fp32 sum over R query rows
adds at most R 2^-24.  serving.attention_weights returns sum P (e + |lse|):
  |acc - ref| <= (d + 4) 2^-23 tol + (2^-21 + R 2^-24) ref + 2^-24 |acc before + ref|
"""
import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hb():
    import compressed_sparse_sliding_b200 as hb
    return hb


def _f64(t):
    return t.double().cpu().numpy()


def _case(B, Lq, Hq, Hkv, d, m, W, Nc, K=0, e0=0, seed=0, q_pos=None):
    g = torch.Generator().manual_seed(seed + 31 * Nc + B)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
    if q_pos is None:
        own = [(b * 53 + Nc) % (Nc + 1) for b in range(B)]
        q_pos = np.array([[(e0 + n) * m + W - 1 + b % m + t for t in range(Lq)] for b, n in enumerate(own)], np.int32)
    q, kc = bf(B, Lq, Hq, d), bf(B, Nc, Hkv, d)
    idx = None
    if K:
        rng = np.random.default_rng(seed + K)
        idx = np.full((B, 1, K), -1, np.int32)
        for b in range(B):
            nv = min(max(serving._visible(int(q_pos[b, 0]), m, W) - e0, 0), Nc)
            n = min(K - K // 8, nv)
            idx[b, 0, rng.permutation(K)[:n]] = rng.choice(nv, size=n, replace=False) if n else []
    # log-sum-exp rows near those of these scores (N(0, 1)), as an attention over
    # these keys and a window would leave them
    lse = torch.randn((B, Hq, Lq), generator=g) * 0.1 + float(np.log(max(Nc, 1)) + 0.5)
    return q, kc, lse, idx, q_pos


def _call(hb, q, kc, lse, idx, q_pos, m, W, acc=None, e0=0, **kw):
    B, Lq, Hq, d = q.shape
    p = hb.problem(B=B, Lq=Lq, Lkv=0, Hq=Hq, Hkv=kc.shape[2], d=d, m=m, W=W, Nc=kc.shape[1],
                   topk=0 if idx is None else idx.shape[2], q_pos=torch.from_numpy(q_pos).cuda())
    out = hb.hyb_attn_weights(p, q.cuda(), kc.cuda(), lse.cuda(), idx=None if idx is None else torch.from_numpy(idx).cuda(),
                              acc=acc, e0=e0, **kw)
    torch.cuda.synchronize()
    return out


def _check(got, q, kc, lse, idx, q_pos, m, W, before=None, e0=0):
    ref, tol = serving.attention_weights(_f64(q), _f64(kc), _f64(lse), m, W, q_pos, idx=idx, e0=e0)
    d, R = q.shape[3], q.shape[1] * q.shape[2]
    b0 = 0.0 if before is None else before
    bound = (d + 4) * 2.0 ** -23 * tol + (2.0 ** -21 + R * 2.0 ** -24) * ref + 2.0 ** -24 * np.abs(b0 + ref)
    err = np.abs(_f64(got) - (b0 + ref))
    assert np.all(err <= bound), f"{float((err - bound).max()):.3e} over the bound"


SHAPES = [
    (3, 1, 64, 1, 128, 4, 128, 700, 0),      # decode, one KV head: resident queries
    (2, 1, 64, 8, 128, 128, 128, 300, 0),    # eight KV heads of eight
    (2, 1, 5, 5, 64, 4, 16, 513, 0),         # one head a group: one-row blocks
    (2, 3, 20, 4, 128, 7, 61, 260, 0),       # five heads a group, odd sizes
    (1, 32, 32, 4, 128, 4, 128, 400, 0),     # a prompt's last tokens: streamed queries
    (1, 90, 4, 4, 64, 2, 5, 135, 0),         # 90 tokens of one head
    (1, 2, 144, 1, 128, 4, 128, 140, 0),     # a group wider than a block
    (2, 1, 3, 1, 64, 1, 0, 1, 0),            # one entry
    (3, 1, 64, 1, 128, 4, 128, 900, 256),    # a selection
    (2, 1, 8, 2, 64, 4, 128, 500, 77),       # ... of an odd size, two KV heads
    (2, 1, 4, 1, 128, 4, 128, 64, 1),        # ... of one
    (2, 1, 384, 6, 128, 4, 128, 600, 200),   # ... with more query rows than stay resident
    (2, 14, 48, 1, 128, 4, 128, 300, 0),     # five slots of 96 rows for seven blocks
    (2, 40, 64, 2, 64, 3, 9, 400, 0),        # d = 64, streamed
]


@pytest.mark.parametrize("B,Lq,Hq,Hkv,d,m,W,Nc,K", SHAPES)
def test_matches_definition(hb, B, Lq, Hq, Hkv, d, m, W, Nc, K):
    q, kc, lse, idx, q_pos = _case(B, Lq, Hq, Hkv, d, m, W, Nc, K)
    got = _call(hb, q, kc, lse, idx, q_pos, m, W)
    assert hb.hyb_get_device_status() == hb.HYB_OK
    _check(got, q, kc, lse, idx, q_pos, m, W)
    # once more, added to what is there; entries without a weight keep their bits
    before = torch.rand((B, Nc), generator=torch.Generator().manual_seed(1))
    acc = before.cuda()
    again = _call(hb, q, kc, lse, idx, q_pos, m, W, acc=acc)
    assert again.data_ptr() == acc.data_ptr()
    _check(again, q, kc, lse, idx, q_pos, m, W, before=_f64(before))
    ref, _ = serving.attention_weights(_f64(q), _f64(kc), _f64(lse), m, W, q_pos, idx=idx)
    assert torch.equal(again.cpu()[torch.from_numpy(ref == 0)], before[torch.from_numpy(ref == 0)])


def test_entries_behind_a_shared_prefix(hb):
    # row j of the cache is entry e0 + j
    for K in (0, 40):
        q, kc, lse, idx, q_pos = _case(3, 1, 16, 2, 128, 4, 128, 200, K, e0=1000)
        got = _call(hb, q, kc, lse, idx, q_pos, 4, 128, e0=1000)
        _check(got, q, kc, lse, idx, q_pos, 4, 128, e0=1000)


def test_unseen_rows_may_hold_anything(hb):
    # early positions: some sequences see nothing, some query rows see less than others
    q_pos = np.array([[0, 100, 131], [500, 300, 20], [3, 2, 1]], np.int32)
    q, kc, lse, _, _ = _case(3, 3, 8, 2, 64, 4, 128, 150, q_pos=q_pos)
    clean = kc.clone()
    for b in range(3):
        n = max(serving._visible(int(t), 4, 128) for t in q_pos[b])
        kc[b, n:] = float("nan")
        clean[b, n:] = 0
    lse[2] = float("-inf")            # the rows of an empty key set
    lse[0, :, 0] = float("-inf")
    acc = torch.full((3, 150), float("nan"), device="cuda")
    got = _call(hb, q, kc, lse, None, q_pos, 4, 128, acc=acc, accumulate=False)
    _check(got, q, clean, torch.where(torch.isinf(lse), 0.0, lse), None, q_pos, 4, 128)
    assert torch.all(got[2] == 0)
    keep = torch.full((3, 150), 5.0, device="cuda")
    got = _call(hb, q, kc, lse, None, q_pos, 4, 128, acc=keep)
    assert torch.all(got[2] == 5)


def test_repeated_and_bad_selection_entries(hb):
    q, kc, lse, idx, q_pos = _case(2, 1, 8, 1, 128, 4, 128, 300, 64, q_pos=np.full((2, 1), 300 * 4 + 127, np.int32))
    idx[0, 0, :4] = [7, 7, 7, 7]
    idx[0, 0, 4:] = -1
    got = _call(hb, q, kc, lse, idx, q_pos, 4, 128)
    assert hb.hyb_get_device_status() == hb.HYB_OK
    one = idx.copy()
    one[0, 0, 1:] = -1
    single = _call(hb, q, kc, lse, one, q_pos, 4, 128)
    assert float(got[0, 7]) == pytest.approx(4 * float(single[0, 7]), rel=2.0 ** -22)
    idx[1, 0, 5] = 300                # behind the cache: skipped and flagged
    good = idx.copy()
    good[1, 0, 5] = -1
    got = _call(hb, q, kc, lse, idx, q_pos, 4, 128)
    assert hb.hyb_get_device_status() == hb.HYB_ERR_DEVICE_BOUNDS
    assert torch.equal(got, _call(hb, q, kc, lse, good, q_pos, 4, 128))


@pytest.mark.parametrize("K", [0, 200])
def test_streams_and_capture(hb, K):
    q, kc, lse, idx, q_pos = _case(5, 1, 64, 1, 128, 4, 128, 1500, K)
    p = hb.problem(B=5, Lq=1, Lkv=0, Hq=64, Hkv=1, d=128, m=4, W=128, Nc=1500, topk=K,
                   q_pos=torch.from_numpy(q_pos).cuda())
    x = [q.cuda(), kc.cuda(), lse.cuda()]
    sel = None if idx is None else torch.from_numpy(idx).cuda()
    want = hb.hyb_attn_weights(p, *x, idx=sel)
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [hb.hyb_attn_weights(p, *x, idx=sel, stream=t) for t in s]
        torch.cuda.synchronize()
        assert all(torch.equal(want, y) for y in got)
    acc = torch.zeros((5, 1500), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hb.hyb_attn_weights(p, *x, idx=sel, acc=acc, accumulate=False)
        hb.hyb_attn_weights(p, *x, idx=sel, acc=acc)
    for _ in range(2):
        acc.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(acc, 2 * want)
    assert hb.hyb_get_device_status() == hb.HYB_OK


def test_many_sequences_and_many_positions(hb):
    # more sequences, or more query positions, than a CTA counts at its start
    for B, Lq, Nc in ((1100, 1, 140), (9, 1000, 150)):
        q, kc, lse, _, q_pos = _case(B, Lq, 2, 1, 64, 4, 16, Nc)
        if Lq > 1:
            q_pos = np.array([[(b * 67 + t) % 700 for t in range(Lq)] for b in range(B)], np.int32)
        acc = torch.full((B, Nc), float("nan"), device="cuda")
        got = _call(hb, q, kc, lse, None, q_pos, 4, 16, acc=acc, accumulate=False)
        _check(got, q, kc, lse, None, q_pos, 4, 16)


def test_wait_timeout_is_reported_and_the_device_recovers(hb):
    q, kc, lse, _, q_pos = _case(4, 1, 64, 1, 128, 4, 128, 3000)
    ref = _call(hb, q, kc, lse, None, q_pos, 4, 128)
    assert hb.hyb_get_device_status() == hb.HYB_OK
    hb.hyb_set_wait_limit_ns(1)
    try:
        _call(hb, q, kc, lse, None, q_pos, 4, 128)
    finally:
        hb.hyb_set_wait_limit_ns(0)
    assert hb.hyb_get_device_status() == hb.HYB_ERR_DEVICE_TIMEOUT
    again = _call(hb, q, kc, lse, None, q_pos, 4, 128)
    assert hb.hyb_get_device_status() == hb.HYB_OK and torch.equal(ref, again)
