"""Shared and bounded caches at the ends of their ranges: scales other than the
default, padded batches, a captured eviction, and tensors of more than 2^31 elements."""
import numpy as np
import pytest
import torch

from oracle import serving
from tests import test_gpu_prefix as prefix
from tests import test_gpu_weights as weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hb():
    import compressed_sparse_sliding_b200 as hb
    return hb


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("scale", [1e-3, 0.03, 0.7])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (64, 1), (16, 8)])
def test_scales(hb, scale, Hq, Hkv):
    B, d, m, W, Np, Nc = 3, 128, 4, 128, 300, 70
    c, q_pos, kv0, Lkv = prefix._case(B, 1, Hq, Hkv, d, m, W, Np, Nc)
    p = hb.problem(B=B, Lq=1, Lkv=Lkv, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc, scale=scale,
                   q_pos=torch.from_numpy(q_pos).cuda(), kv_pos0=torch.from_numpy(kv0).cuda())
    scale = float(np.float32(scale))
    x = {n: t.cuda() for n, t in c.items()}
    lse = torch.empty((B, Hq, 1), device="cuda")
    o = hb.hyb_prefix_attn_fwd(p, *(x[n] for n in ("q", "kp", "vp", "kc", "vc", "k_raw", "v_raw")), lse=lse)
    f = {n: _f64(t) for n, t in c.items()}
    ref = serving.prefix_attention(f["q"], f["kp"], f["vp"], f["kc"], f["vc"], f["k_raw"], f["v_raw"], m, W, q_pos,
                                   kv0, scale=scale)
    # The bounds of test_gpu_prefix, whose score terms go with the scale; for the lse at any
    # scale the polynomial's 1.7e-7 and the unit's 2^-22 lie inside its 2^-20.
    prefix._check(o, lse, ref, d)
    acc = hb.hyb_attn_weights(p, x["q"], x["kc"], lse, e0=Np)
    want, tol = serving.attention_weights(f["q"], f["kc"], _f64(lse), m, W, q_pos, e0=Np, scale=scale)
    bound = (d + 4) * 2.0 ** -23 * tol + (2.0 ** -21 + Hq * 2.0 ** -24) * want + 2.0 ** -24 * want
    assert np.all(np.abs(_f64(acc) - want) <= bound)
    assert hb.hyb_get_device_status() == hb.HYB_OK


@pytest.mark.parametrize("Hq,Hkv,Lq", [(4, 1, 3), (64, 1, 2), (8, 8, 130)])
def test_padded_tokens_see_nothing(hb, Hq, Hkv, Lq):
    # position -1: o = 0, lse = -infinity, and no weight
    B, d, m, W, Np, Nc = 4, 64, 4, 16, 60, 50
    q_pos = np.array([[(Np + 7 * b) * m + W + t for t in range(Lq)] for b in range(B)], np.int32)
    q_pos[1, 1:], q_pos[3] = -1, -1
    c, _, _, _ = prefix._case(B, Lq, Hq, Hkv, d, m, W, Np, Nc, q_pos=q_pos)
    kv0 = np.array([max(int(r.max()) - W - Lq + 2, 0) for r in q_pos], np.int32)
    o, lse = prefix._run(hb, c, q_pos, kv0, W + Lq - 1, m, W)
    prefix._check(o, lse, prefix._ref(c, q_pos, kv0, m, W), d)
    assert torch.all(o[3] == 0) and torch.all(torch.isneginf(lse[1, :, 1:])) and torch.all(torch.isneginf(lse[3]))
    acc = torch.full((B, Nc), 2.0, device="cuda")
    weights._call(hb, c["q"], c["kc"], lse, None, q_pos, m, W, acc=acc, e0=Np)
    assert torch.all(acc[3] == 2)
    real = torch.where(torch.isinf(lse), 0.0, lse)
    weights._check(acc, c["q"], c["kc"], real, None, q_pos, m, W, before=2.0, e0=Np)


def test_an_eviction_is_captured_and_replayed(hb):
    # weights, selection and compaction in one graph, replayed with other inputs
    B, Hq, Hkv, d, m, W, Nc, n_keep = 3, 16, 2, 64, 4, 16, 500, 200
    g = torch.Generator().manual_seed(5)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    q_pos = torch.full((B, 1), Nc * m + W, dtype=torch.int32, device="cuda")
    p = hb.problem(B=B, Lq=1, Lkv=0, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc, q_pos=q_pos)
    bufs = dict(q=bf(B, 1, Hq, d), kc=bf(B, Nc, Hkv, d), vc=bf(B, Nc, Hkv, d), lse=torch.full((B, Hq, 1), 6.0, device="cuda"),
                acc=torch.rand((B, Nc), generator=g).cuda(), n=torch.tensor([500, 350, 120], dtype=torch.int32, device="cuda"))
    other = dict(q=bf(B, 1, Hq, d), kc=bf(B, Nc, Hkv, d), vc=bf(B, Nc, Hkv, d), lse=torch.full((B, Hq, 1), 5.5, device="cuda"),
                 acc=torch.rand((B, Nc), generator=g).cuda(), n=torch.tensor([90, 500, 201], dtype=torch.int32, device="cuda"))
    first = {k: v.clone() for k, v in bufs.items()}
    out = dict(kc_out=torch.zeros((B, n_keep, Hkv, d), dtype=torch.bfloat16, device="cuda"),
               vc_out=torch.zeros((B, n_keep, Hkv, d), dtype=torch.bfloat16, device="cuda"),
               acc_out=torch.zeros((B, n_keep), device="cuda"))
    keep = torch.empty((B, n_keep), dtype=torch.int32, device="cuda")

    def run(x, keep, out):
        hb.hyb_attn_weights(p, x["q"], x["kc"], x["lse"], acc=x["acc"])
        hb.hyb_evict_select(x["acc"], n_keep, 1, 5, n_valid=x["n"], keep=keep)
        hb.hyb_cache_compact(p, keep, x["kc"], x["vc"], acc=x["acc"], **out)

    run({k: v.clone() for k, v in bufs.items()}, keep, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(bufs, keep, out)
    for x in (other, first):
        want_x = {k: v.clone() for k, v in x.items()}
        want_keep = torch.empty_like(keep)
        want = {k: torch.zeros_like(v) for k, v in out.items()}
        run(want_x, want_keep, want)
        for k in bufs:
            bufs[k].copy_(x[k])
        for v in out.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(keep, want_keep) and all(torch.equal(out[k], want[k]) for k in out)
        assert np.array_equal(keep.cpu().numpy(), serving.evict_select(bufs["acc"].cpu().numpy(), n_keep, 1, 5,
                                                                       x["n"].cpu().numpy()))
    assert hb.hyb_get_device_status() == hb.HYB_OK


def test_caches_of_more_than_2_31_elements(hb):
    # the last sequence and the last KV heads lie behind the 32-bit range
    B, Hkv, d, m, W, Nc = 2, 64, 128, 1, 0, 140_001
    assert B * Nc * Hkv * d > 2 ** 31 and Nc * Hkv * d < 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(8)
    big = lambda: torch.randn((B, Nc, Hkv, d), generator=g, device="cuda", dtype=torch.bfloat16)
    kc, vc = big(), big()
    q = torch.randn((B, 1, Hkv, d), generator=g, device="cuda", dtype=torch.bfloat16)
    q_pos = torch.full((B, 1), Nc - 1, dtype=torch.int32, device="cuda")
    p = hb.problem(B=B, Lq=1, Lkv=0, Hq=Hkv, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc, q_pos=q_pos)
    lse = torch.empty((B, Hkv, 1), device="cuda")
    o = hb.hyb_prefix_attn_fwd(p, q, None, None, kc, vc, lse=lse)
    acc = hb.hyb_attn_weights(p, q, kc, lse)
    # the bounds of test_gpu_prefix and test_gpu_weights
    want, tol = (torch.zeros((Nc,), dtype=torch.float64, device="cuda") for _ in range(2))
    for h in range(Hkv):
        k, v, qh = kc[1, :, h].double(), vc[1, :, h].double(), q[1, 0, h].double()
        s, e, got = (k @ qh) / np.sqrt(d), (k.abs() @ qh.abs()) / np.sqrt(d), float(lse[1, h, 0])
        top, r = float(torch.logsumexp(s, 0)), float((d + 4) * 2.0 ** -23 * e.max())
        assert abs(got - top) <= r + Nc * 2.0 ** -24 + 2.0 ** -20 * (1 + abs(top))
        w = torch.exp(s - top)
        ref, A = w @ v, w @ v.abs()
        bound = 2.0 ** -8 * (ref.abs() + A) * (1 + 2.0 ** -8) + 2 * r * A + 2.0 ** -20 * A
        assert torch.all((o[1, 0, h].double() - ref).abs() <= bound)
        w = torch.exp(s - got)
        want += w
        tol += w * (e + abs(got))
    bound = (d + 4) * 2.0 ** -23 * tol + (2.0 ** -21 + Hkv * 2.0 ** -24) * want
    assert torch.all((acc[1].double() - want).abs() <= bound)
    # compaction: rows of the last sequence from the end of the cache
    n_keep = Nc - 100
    keep = torch.arange(100, Nc, dtype=torch.int32, device="cuda").expand(B, n_keep).contiguous()
    out = hb.hyb_cache_compact(p, keep, kc=kc, acc=acc)
    assert torch.equal(out["kc"], kc[:, 100:]) and torch.equal(out["acc"], acc[:, 100:])
    assert hb.hyb_get_device_status() == hb.HYB_OK


def test_weights_of_more_than_2_31_entries_are_selected(hb):
    B, Nc, n_keep = 65_535, 33_000, 40
    assert B * Nc > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(9)
    acc = torch.rand((B, Nc), generator=g, device="cuda")
    keep = hb.hyb_evict_select(acc, n_keep, 2, 3)
    rows = [0, 1, 65_074, 65_075, 65_076, B - 1]             # around element 2^31, and the last
    got = keep[rows].cpu().numpy()
    np.testing.assert_array_equal(got, serving.evict_select(acc[rows].cpu().numpy(), n_keep, 2, 3))
    assert hb.hyb_get_device_status() == hb.HYB_OK
