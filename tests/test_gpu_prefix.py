"""hyb_prefix_attn_fwd on the GPU against the fp64 definition.

Tolerances.  P is rounded to bf16 as the MMA operand (at most 2^-8 of each
term) and o to bf16 (2^-8 of it); the fp32 row sums and the hardware exp2
(2^-22) are far below.  Scores are fp32 sums of d exact products: off by at most
d 2^-24 of sum |q||k| scale = e, which moves P and lse by that much, twice for P
(numerator and sum); log2-scaling and the subtraction of the maximum round by
2^-23 of |s| <= e more each.  So, with A = sum P |v| and r = (d + 4) 2^-23 e:
  |o - ref|   <= 2^-8 (|ref| + A) (1 + 2^-8) + 2 r A + 2^-20 A
  |lse - ref| <= r + n 2^-24 + 2^-20 (1 + |ref|)     (n terms in the fp32 sum)
A quarter of the exponentials come from a polynomial that is off by at most 2.8e-6
< 2^-18 of the value, which the bounds above hold without a term of their own:
with u = 2^-8 / (1 + 2^-8) (half a bf16 step, relative to the value) o is off by at most
u (|ref| + A) + u^2 A + 2 * 2^-18 A < 2^-8 (|ref| + A) - 2^-16 |ref| + 2^-17 A + 2^-23 A,
less than the first term of its bound; and lse moves by less than 2^-18, while r
counts the d 2^-24 e of a score twice: the half that is over, (d + 4) 2^-24 e, is more
than 2^-18 from e = 0.94 on (d = 64; 0.49 at d = 128), and e is above 2 in these inputs.
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


def _check(o, lse, ref, d):
    A = ref["a"]
    r = (d + 4) * 2.0 ** -23 * ref["e"]                                 # [B, Hq, Lq]
    ro = np.moveaxis(r, 1, 2)[..., None]
    bound = 2.0 ** -8 * (np.abs(ref["o"]) + A) * (1 + 2.0 ** -8) + 2 * ro * A + 2.0 ** -20 * A
    err = np.abs(_f64(o) - ref["o"])
    assert np.all(err <= bound), f"o: {float((err - bound).max()):.3e} over its bound"
    got, want = _f64(lse), ref["lse"]
    empty = np.isneginf(want)
    assert np.array_equal(empty, np.isneginf(got))
    n = np.broadcast_to(ref["n"][:, None], want.shape)
    got, want = np.where(empty, 0.0, got), np.where(empty, 0.0, want)
    assert np.all(np.abs(got - want) <= r + n * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(want)))


def _case(B, Lq, Hq, Hkv, d, m, W, Np, Nc, q_pos=None, garbage=False, seed=0, Lkv=None):
    """Inputs on the CPU.  Positions: every own entry count between 0 and Nc, the
    raw rows the last W + Lq - 1 positions."""
    g = torch.Generator().manual_seed(seed + B + 7 * Np + Nc)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
    if q_pos is None:
        own = [(b * 5 + 3) % (Nc + 1) for b in range(B)]
        first = [(Np + n) * m + W - 1 + b % m for b, n in enumerate(own)]
        q_pos = np.array([[f + t for t in range(Lq)] for f in first], np.int32)
    q_pos = np.asarray(q_pos, np.int32)
    Lkv = (W + Lq - 1 if W else 0) if Lkv is None else Lkv
    kv0 = np.maximum(q_pos.min(1) - W + 1, 0).astype(np.int32)
    c = dict(q=bf(B, Lq, Hq, d), kp=bf(Np, Hkv, d), vp=bf(Np, Hkv, d), kc=bf(B, Nc, Hkv, d),
             vc=bf(B, Nc, Hkv, d), k_raw=bf(B, Lkv, Hkv, d), v_raw=bf(B, Lkv, Hkv, d))
    if garbage:      # what no query sees holds NaN and infinities
        seen = [[serving._visible(int(t), m, W) for t in row] for row in q_pos]
        top = max(max(r) for r in seen)
        for x, bad in (("kp", float("nan")), ("vp", float("inf"))):
            c[x][min(top, Np):] = bad
        for b in range(B):
            n = min(max(max(seen[b]) - Np, 0), Nc)
            c["kc"][b, n:], c["vc"][b, n:] = float("-inf"), float("nan")
            hi = int(q_pos[b].max() - kv0[b])
            c["k_raw"][b, hi + 1:], c["v_raw"][b, hi + 1:] = float("nan"), float("nan")
    return c, q_pos, kv0, Lkv


def _run(hb, c, q_pos, kv0, Lkv, m, W, **kw):
    B, Lq, Hq, d = c["q"].shape
    Np, Hkv = c["kp"].shape[:2]
    Nc = c["kc"].shape[1]
    p = hb.problem(B=B, Lq=Lq, Lkv=Lkv, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc,
                   q_pos=torch.from_numpy(q_pos).cuda(), kv_pos0=torch.from_numpy(kv0).cuda())
    lse = torch.full((B, Hq, Lq), 7.0, device="cuda")
    x = {n: t.cuda() if t.numel() else None for n, t in c.items()}
    o = hb.hyb_prefix_attn_fwd(p, x["q"], x["kp"], x["vp"], x["kc"], x["vc"], x["k_raw"], x["v_raw"], lse=lse, **kw)
    torch.cuda.synchronize()
    assert hb.hyb_get_device_status() == hb.HYB_OK
    return o, lse


def _ref(c, q_pos, kv0, m, W):
    f = {n: _f64(t) for n, t in c.items()}
    return serving.prefix_attention(f["q"], f["kp"], f["vp"], f["kc"], f["vc"], f["k_raw"], f["v_raw"], m, W,
                                    q_pos, kv0)


@pytest.mark.parametrize("B,Lq,Hq,Hkv,d,m,W,Np,Nc", [
    (4, 1, 4, 1, 64, 4, 128, 256, 64),       # one query tile: its key tiles alternate
    (3, 1, 64, 1, 128, 4, 128, 300, 70),     # two query tiles over the prefix
    (5, 1, 64, 1, 128, 4, 128, 1000, 130),   # an odd number of query tiles
    (2, 1, 16, 8, 128, 128, 128, 33, 5),     # few rows per KV head
    (6, 5, 20, 4, 128, 7, 61, 203, 41),      # five heads a group, sizes on no grid
    (2, 3, 6, 6, 64, 1, 0, 400, 150),        # one head a group, no window
    (2, 40, 8, 1, 128, 4, 16, 140, 30),      # several query tiles per sequence
    (1, 70, 5, 5, 64, 3, 40, 90, 20),        # one head, 70 tokens
    (1, 2, 144, 1, 128, 2, 8, 200, 10),      # a group wider than a query tile
    (2, 1, 130, 1, 64, 4, 128, 129, 0),      # ... and no own entries
    (3, 1, 32, 2, 128, 4, 128, 0, 150),      # no shared entries
    (2, 2, 8, 2, 64, 4, 0, 0, 9),            # own entries alone
    (2, 2, 8, 2, 64, 4, 33, 0, 0),           # window alone
    (1, 1, 1, 1, 64, 1, 1, 1, 1),            # one of everything
    (1, 1, 8, 1, 128, 4, 128, 20000, 0),     # a long prefix for one token: many splits
    (4, 3, 32, 1, 128, 4, 128, 900, 700),    # 96 rows a sequence: three lane quadrants
    (3, 1, 40, 1, 64, 4, 16, 500, 1200),     # 40 rows: two lane quadrants, one partly filled
    (70, 1, 33, 1, 128, 4, 128, 40, 300),    # 33 rows
    (60, 1, 8, 1, 128, 4, 0, 0, 513),        # eight rows over own entries alone
    (2, 130, 2, 1, 128, 4, 128, 1500, 300),  # a chunk: one stream a sequence, whole
    (1, 300, 8, 8, 64, 4, 30, 5000, 64),     # ... and cut
])
def test_matches_definition(hb, B, Lq, Hq, Hkv, d, m, W, Np, Nc):
    c, q_pos, kv0, Lkv = _case(B, Lq, Hq, Hkv, d, m, W, Np, Nc)
    o, lse = _run(hb, c, q_pos, kv0, Lkv, m, W)
    _check(o, lse, _ref(c, q_pos, kv0, m, W), d)


def test_early_positions_without_q_pos(hb):
    # q_pos and kv_pos0 NULL: token t sits at position t; the first rows see no
    # entry, some of the shared ones, then all; W = 0 leaves rows without any key
    for W in (0, 8):
        c, _, _, _ = _case(2, 60, 6, 2, 64, 4, W, 9, 4, Lkv=60)
        q_pos = np.tile(np.arange(60, dtype=np.int32), (2, 1))
        kv0 = np.zeros(2, np.int32)
        p = hb.problem(B=2, Lq=60, Lkv=60, Hq=6, Hkv=2, d=64, m=4, W=W, Nc=4)
        lse = torch.empty((2, 6, 60), device="cuda")
        o = hb.hyb_prefix_attn_fwd(p, *(c[n].cuda() for n in ("q", "kp", "vp", "kc", "vc", "k_raw", "v_raw")),
                                   lse=lse)
        torch.cuda.synchronize()
        ref = _ref(c, q_pos, kv0, 4, W)
        assert (ref["n"] == 0).any() == (W == 0)
        _check(o, lse, ref, 64)
        if W == 0:
            assert torch.all(o[:, :3] == 0) and torch.all(torch.isneginf(lse[:, :, :3]))


def test_no_key_at_all(hb):
    p = hb.problem(B=2, Lq=1, Lkv=0, Hq=4, Hkv=1, d=64, m=4, W=0, Nc=0)
    lse = torch.zeros((2, 4, 1), device="cuda")
    o = hb.hyb_prefix_attn_fwd(p, torch.randn((2, 1, 4, 64), device="cuda").bfloat16(), None, None, lse=lse)
    torch.cuda.synchronize()
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("B,Lq,Hq,Hkv,d,m,W,Np,Nc", [
    (5, 1, 8, 1, 128, 4, 128, 300, 200), (2, 3, 64, 1, 128, 4, 30, 200, 140), (3, 1, 4, 4, 64, 2, 0, 130, 129),
])
def test_unseen_rows_may_hold_anything(hb, B, Lq, Hq, Hkv, d, m, W, Np, Nc):
    # sequences that see part of the prefix only, and part of their own cache
    first = [min(Np, 100 + 150 * b) * m + W - 1 + (m * (b * 37 % Nc) if 100 + 150 * b >= Np else 0) for b in range(B)]
    q_pos = np.array([[f + t for t in range(Lq)] for f in first], np.int32)
    if first[-1] >= Np * m:     # leave the last shared entry unseen, so that its garbage is there
        q_pos = np.minimum(q_pos, (Np - 1) * m + W - 1 + np.arange(Lq, dtype=np.int32)) if B == 3 else q_pos
    c, q_pos, kv0, Lkv = _case(B, Lq, Hq, Hkv, d, m, W, Np, Nc, q_pos=q_pos, garbage=True, Lkv=2 * W + 3 if W else 0)
    o, lse = _run(hb, c, q_pos, kv0, Lkv, m, W)
    clean = {n: torch.nan_to_num(t, nan=0.0, posinf=0.0, neginf=0.0) for n, t in c.items()}
    assert any(not torch.equal(clean[n], c[n]) for n in c)
    _check(o, lse, _ref(clean, q_pos, kv0, m, W), d)


def test_order_of_positions_and_ring_rows(hb):
    # q_pos in any order, a window row range that starts before raw row 0 and
    # ends behind the last one
    q_pos = np.array([[900, 40, 333], [5, 4, 910]], np.int32)
    c, q_pos, _, _ = _case(2, 3, 8, 2, 128, 4, 128, 150, 60, q_pos=q_pos, Lkv=901)
    kv0 = np.array([3, 0], np.int32)
    o, lse = _run(hb, c, q_pos, kv0, 901, 4, 128)
    _check(o, lse, _ref(c, q_pos, kv0, 4, 128), 128)


def test_equals_dense_attention_over_joined_caches(hb):
    # the same entries in one cache per sequence, through hyb_attn_fwd
    B, Hq, Hkv, d, m, W, Np, Nc = 3, 16, 2, 128, 4, 128, 200, 90
    c, q_pos, kv0, Lkv = _case(B, 1, Hq, Hkv, d, m, W, Np, Nc)
    o, lse = _run(hb, c, q_pos, kv0, Lkv, m, W)
    x = {n: t.cuda() for n, t in c.items()}
    kc, vc = (torch.cat([x[s + "p"].expand(B, Np, Hkv, d), x[s + "c"]], 1).contiguous() for s in "kv")
    p = hb.problem(B=B, Lq=1, Lkv=Lkv, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, Nc=Np + Nc,
                   q_pos=torch.from_numpy(q_pos).cuda(), kv_pos0=torch.from_numpy(kv0).cuda())
    lse2 = torch.empty_like(lse)
    o2 = hb.hyb_attn_fwd(p, x["q"], kc, vc, None, x["k_raw"], x["v_raw"], lse=lse2)
    torch.cuda.synchronize()
    # each is within 2^-8 (|o| + A) of the definition, A <= max |v| of a row's average
    assert torch.allclose(lse, lse2, rtol=0, atol=1e-4)
    ref = _ref(c, q_pos, kv0, m, W)
    assert np.all(np.abs(_f64(o) - _f64(o2)) <= 2 * (2.0 ** -8 * (np.abs(ref["o"]) + ref["a"]) * 1.01 + 1e-3 * ref["a"]))


def test_streams_capture_and_repeat(hb):
    # equal calls give equal bits: eager, on another stream, captured and replayed
    # with new inputs in the same buffers, two at once with a workspace each
    m, W = 4, 128
    c, q_pos, kv0, Lkv = _case(9, 1, 64, 1, 128, m, W, 700, 90)
    d, _, _, _ = _case(9, 1, 64, 1, 128, m, W, 700, 90, seed=50)
    x = {n: t.cuda() for n, t in c.items()}
    y = {n: t.cuda() for n, t in d.items()}
    names = ("q", "kp", "vp", "kc", "vc", "k_raw", "v_raw")
    p = hb.problem(B=9, Lq=1, Lkv=Lkv, Hq=64, Hkv=1, d=128, m=m, W=W, Nc=90,
                   q_pos=torch.from_numpy(q_pos).cuda(), kv_pos0=torch.from_numpy(kv0).cuda())
    call = lambda z, **kw: hb.hyb_prefix_attn_fwd(p, *(z[n] for n in names), **kw)
    ox, oy = call(x), call(y)
    assert torch.equal(ox, call(x))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a, b = call(x, stream=s1), call(y, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a, ox) and torch.equal(b, oy)
    buf = {n: x[n].clone() for n in names}
    ws = torch.empty(hb.hyb_prefix_workspace_size(p, 700), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(ox)
    call(buf, o=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(buf, o=out, ws=ws)
    for z, want in ((y, oy), (x, ox)):
        for n in names:
            buf[n].copy_(z[n])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert hb.hyb_get_device_status() == hb.HYB_OK


def test_wait_timeout_is_reported_and_the_device_recovers(hb):
    # every wait inside the kernel is bounded: with a bound of 1 ns the first one
    # that is not already satisfied runs out, and the call still returns
    for shape in ((9, 1, 64, 1, 128, 4, 128, 700, 90), (3, 1, 4, 1, 64, 4, 128, 700, 90)):
        c, q_pos, kv0, Lkv = _case(*shape)
        ref, _ = _run(hb, c, q_pos, kv0, Lkv, 4, 128)
        x = {n: t.cuda() for n, t in c.items()}
        B, _, Hq, Hkv, d = shape[:5]
        p = hb.problem(B=B, Lq=1, Lkv=Lkv, Hq=Hq, Hkv=Hkv, d=d, m=4, W=128, Nc=90,
                       q_pos=torch.from_numpy(q_pos).cuda(), kv_pos0=torch.from_numpy(kv0).cuda())
        hb.hyb_set_wait_limit_ns(1)
        try:
            hb.hyb_prefix_attn_fwd(p, *(x[n] for n in ("q", "kp", "vp", "kc", "vc", "k_raw", "v_raw")))
            torch.cuda.synchronize()
        finally:
            hb.hyb_set_wait_limit_ns(0)
        assert hb.hyb_get_device_status() == hb.HYB_ERR_DEVICE_TIMEOUT
        again, _ = _run(hb, c, q_pos, kv0, Lkv, 4, 128)
        assert torch.equal(ref, again)
