"""hyb_evict_select and hyb_cache_compact(_fp4) on the GPU: selections and moved
rows equal the definition exactly; and a decode loop whose full caches are cut."""
import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hb():
    import compressed_sparse_sliding_b200 as hb
    return hb


def _select(hb, acc, n_keep, n_first=0, n_last=0, n_valid=None):
    nv = None if n_valid is None else torch.tensor(n_valid, dtype=torch.int32, device="cuda")
    keep = hb.hyb_evict_select(torch.from_numpy(acc).cuda(), n_keep, n_first, n_last, nv)
    torch.cuda.synchronize()
    return keep.cpu().numpy()


@pytest.mark.parametrize("B,Nc,n_keep,n_first,n_last", [
    (1, 1, 1, 0, 0), (2, 2, 1, 0, 1), (3, 1000, 333, 1, 7), (2, 4099, 4098, 0, 0), (1, 9001, 100, 50, 50),
    (1, 70001, 20000, 4, 64), (150, 300, 128, 2, 2), (2, 33000, 16384, 0, 100), (1, 300001, 150000, 10, 10),
    (5, 64, 100, 3, 3), (1, 5000, 1, 0, 0), (2, 20000, 19990, 9, 0), (40, 9000, 1000, 0, 30), (1, 600001, 250000, 3, 9),
])
@pytest.mark.parametrize("kind", ["heavy", "ties"])
def test_selection_matches_definition(hb, B, Nc, n_keep, n_first, n_last, kind):
    rng = np.random.default_rng(Nc + n_keep)
    if kind == "heavy":
        acc = np.exp(2 * rng.standard_normal((B, Nc))).astype(np.float32)
        acc[rng.random((B, Nc)) < 0.1] = 0
    else:            # a handful of values, signed zeros, infinities, NaN, negative weights
        pool = np.array([0.0, -0.0, 1.0, 1.0 + 2.0 ** -23, -1.0, np.inf, -np.inf, np.nan, 1e-42, -1e-42], np.float32)
        acc = pool[rng.integers(0, len(pool), (B, Nc))]
    n_valid = None if Nc < 64 else [Nc if b % 3 == 0 else max(0, Nc - b * 97) for b in range(B)]
    got = _select(hb, acc, n_keep, n_first, n_last, n_valid)
    assert hb.hyb_get_device_status() == hb.HYB_OK
    np.testing.assert_array_equal(got, serving.evict_select(acc, n_keep, n_first, n_last, n_valid))


def test_one_value_everywhere_and_counts_out_of_range(hb):
    acc = np.zeros((3, 20000), np.float32)
    np.testing.assert_array_equal(_select(hb, acc, 7000, 10, 10), serving.evict_select(acc, 7000, 10, 10))
    got = _select(hb, np.ascontiguousarray(acc[:, :50]), 20, n_valid=[-5, 51, 30])
    assert hb.hyb_get_device_status() == hb.HYB_ERR_DEVICE_BOUNDS
    np.testing.assert_array_equal(got, serving.evict_select(acc[:, :50], 20, n_valid=[0, 50, 30]))


@pytest.mark.parametrize("B,Nc,n_keep,No,Hkv,d,di", [
    (3, 100, 33, 33, 2, 64, 0), (2, 700, 300, 700, 1, 128, 64), (1, 257, 256, 300, 8, 128, 32), (4, 5, 1, 2, 1, 64, 64),
])
def test_compaction_moves_rows(hb, B, Nc, n_keep, No, Hkv, d, di):
    g = torch.Generator().manual_seed(Nc)
    rng = np.random.default_rng(Nc)
    keep = np.full((B, n_keep), -1, np.int32)
    for b in range(B):
        n = n_keep if b == 0 else max(1, n_keep - 3 * b)
        keep[b, :n] = np.sort(rng.choice(Nc, size=n, replace=False))
    rnd = lambda *s: torch.randint(-2 ** 15, 2 ** 15, s, generator=g).to(torch.int16).view(torch.bfloat16)
    x = dict(kc=rnd(B, Nc, Hkv, d), vc=rnd(B, Nc, Hkv, d), acc=torch.rand((B, Nc), generator=g))
    if di:
        x["kic"] = rnd(B, Nc, di)
    old = {n: rnd(B, No, *t.shape[2:]) if t.dtype == torch.bfloat16 else torch.rand((B, No), generator=g)
           for n, t in x.items()}
    p = hb.problem(B=B, Lq=1, Lkv=0, Hq=Hkv, Hkv=Hkv, d=d, m=4, W=0, di=di, Nc=Nc)
    dev = {n: t.cuda() for n, t in x.items()}
    out = {n + "_out": t.cuda() for n, t in old.items()}
    got = hb.hyb_cache_compact(p, torch.from_numpy(keep).cuda(), **dev, **out)
    torch.cuda.synchronize()
    assert hb.hyb_get_device_status() == hb.HYB_OK
    bits = lambda t: t.view(torch.int16).cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
    for n in x:
        np.testing.assert_array_equal(bits(got[n]), serving.compact(bits(x[n]), keep, bits(old[n])))
    # without outputs: tensors of n_keep rows; a bad index is skipped and flagged
    keep[0, -1] = Nc
    got = hb.hyb_cache_compact(p, torch.from_numpy(keep).cuda(), kc=dev["kc"])
    torch.cuda.synchronize()
    assert hb.hyb_get_device_status() == hb.HYB_ERR_DEVICE_BOUNDS
    assert got["kc"].shape == (B, n_keep, Hkv, d) and got["vc"] is None
    for b in range(B):
        for i in np.flatnonzero((keep[b] >= 0) & (keep[b] < Nc)):
            assert torch.equal(got["kc"][b, i].view(torch.int16).cpu(), x["kc"][b, keep[b, i]].view(torch.int16))


@pytest.mark.parametrize("B,Nc,n_keep,Hkv,d,di", [(2, 300, 111, 1, 128, 64), (1, 65, 64, 3, 64, 32)])
def test_compaction_of_4bit_caches(hb, B, Nc, n_keep, Hkv, d, di):
    g = torch.Generator().manual_seed(Nc)
    rng = np.random.default_rng(Nc)
    keep = np.stack([np.sort(rng.choice(Nc, size=n_keep, replace=False)) for _ in range(B)]).astype(np.int32)
    x = {n: hb.hyb_fp4_quantize(torch.randn(s, generator=g).bfloat16().cuda())
         for n, s in (("kc", (B, Nc, Hkv, d)), ("vc", (B, Nc, Hkv, d)))}
    kic = torch.randn((B, Nc, di), generator=g).bfloat16().cuda()
    x["kic"] = hb.Fp4Cache(torch.randint(0, 256, (B, Nc, di // 2), generator=g, dtype=torch.uint8).cuda(),
                           kic[..., :2].float().contiguous())
    acc = torch.rand((B, Nc), generator=g).cuda()
    p = hb.problem(B=B, Lq=1, Lkv=0, Hq=Hkv, Hkv=Hkv, d=d, m=4, W=0, di=di, Nc=Nc)
    got = hb.hyb_cache_compact_fp4(p, torch.from_numpy(keep).cuda(), **x, acc=acc)
    torch.cuda.synchronize()
    assert hb.hyb_get_device_status() == hb.HYB_OK
    for n, c in x.items():
        for have, was in ((got[n].codes, c.codes), (got[n].qp, c.qp)):
            was = was.cpu().numpy()
            np.testing.assert_array_equal(have.cpu().numpy(), serving.compact(was, keep, np.zeros_like(was[:, :n_keep])))
    np.testing.assert_array_equal(got["acc"].cpu().numpy(), serving.compact(acc.cpu().numpy(), keep, np.zeros((B, n_keep), np.float32)))


def test_decode_goes_on_after_an_eviction(hb):
    # append -> attention over prefix, own entries and window -> weights, until the
    # caches are full; select + compact; then on with shifted positions.  Every
    # step's output against the definition over the caches as the library holds them.
    B, Hq, Hkv, d, m, W, Np, Nc, n_keep = 3, 8, 2, 64, 4, 16, 30, 40, 24
    E = Nc - n_keep                                   # m * E is a multiple of W
    assert m * E % W == 0
    g = torch.Generator().manual_seed(9)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    kp, vp = bf(Np, Hkv, d), bf(Np, Hkv, d)
    caches = [dict(kc=torch.zeros((B, Nc, Hkv, d), dtype=torch.bfloat16, device="cuda"),
                   vc=torch.zeros((B, Nc, Hkv, d), dtype=torch.bfloat16, device="cuda"),
                   acc=torch.zeros((B, Nc), device="cuda")) for _ in range(2)]
    ring = [torch.zeros((B, 2 * W, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wk, wv = (torch.randn((m, d), generator=g).cuda() for _ in range(2))
    now, pos = 0, [0, 1, 7]                           # tokens each sequence has of its own
    evicted = 0
    f64 = lambda t: t.double().cpu().numpy()
    for step in range(2 * m * Nc // 2):
        c = caches[now]
        if max(pos) + 1 >= m * Nc:                    # the next block might not fit: evict
            n_valid = torch.tensor([t // m for t in pos], dtype=torch.int32, device="cuda")
            p = hb.problem(B=B, Lq=1, Lkv=0, Hq=Hkv, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc)
            # every sequence gives up the same E entries, so that its ring stays aligned
            keep = torch.full((B, n_keep), -1, dtype=torch.int32, device="cuda")
            for b in range(B):
                n = int(n_valid[b]) - E
                keep[b, :n] = hb.hyb_evict_select(c["acc"][b:b + 1], n, n_first=1, n_last=W // m + 1,
                                                  n_valid=n_valid[b:b + 1])[0]
            o = caches[1 - now]
            hb.hyb_cache_compact(p, keep, c["kc"], c["vc"], acc=c["acc"], kc_out=o["kc"], vc_out=o["vc"],
                                 acc_out=o["acc"])
            for b in range(B):
                rows = [j for j in keep[b].tolist() if j >= 0]
                assert rows == sorted(rows) and rows[0] == 0 and rows[-(W // m + 1):] == list(
                    range(int(n_valid[b]) - W // m - 1, int(n_valid[b])))
                assert torch.equal(o["kc"][b, :len(rows)], c["kc"][b, rows])
                o["acc"][b, len(rows):] = 0
            now, c = 1 - now, o
            pos = [t - m * E for t in pos]
            evicted += 1
        t_new = torch.tensor(pos, dtype=torch.int32, device="cuda")
        pa = hb.problem(B=B, Lq=1, Lkv=2 * W, Hq=Hkv, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc)
        kv0 = hb.hyb_decode_append(pa, t_new, bf(B, Hkv, d), bf(B, Hkv, d), ring[0], ring[1], c["kc"], c["vc"], wk, wv)
        # behind the prefix: positions and the ring's first row Np * m further on
        q_pos = (t_new + Np * m).view(B, 1).contiguous()
        kv_pos0 = (kv0 + Np * m).contiguous()
        # positions of the window: own tokens only (the prefix holds no raw rows)
        p = hb.problem(B=B, Lq=1, Lkv=2 * W, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc, q_pos=q_pos, kv_pos0=kv_pos0)
        q, lse = bf(B, 1, Hq, d), torch.empty((B, Hq, 1), device="cuda")
        o = hb.hyb_prefix_attn_fwd(p, q, kp, vp, c["kc"], c["vc"], ring[0], ring[1], lse=lse)
        hb.hyb_attn_weights(p, q, c["kc"], lse, acc=c["acc"], e0=Np)
        if step % 13 == 0 or evicted:
            ref = serving.prefix_attention(f64(q), f64(kp), f64(vp), f64(c["kc"]), f64(c["vc"]), f64(ring[0]),
                                           f64(ring[1]), m, W, q_pos.cpu().numpy(), kv_pos0.cpu().numpy())
            # 2^-8 for the rounding of P and of o each (see test_gpu_prefix)
            bound = 2.0 ** -8 * (np.abs(ref["o"]) + ref["a"]) * 1.01 + 1e-4 * ref["a"]
            assert np.all(np.abs(f64(o) - ref["o"]) <= bound)
            assert np.all(np.abs(f64(lse) - ref["lse"]) <= 1e-4)
        pos = [t + 1 for t in pos]
    torch.cuda.synchronize()
    assert evicted >= 1 and hb.hyb_get_device_status() == hb.HYB_OK
