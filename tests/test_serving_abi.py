"""Host-side checks of the operators around shared and bounded caches: refused
calls launch nothing, so they need no GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def hb():
    from compressed_sparse_sliding_b200 import build
    build.build()
    import compressed_sparse_sliding_b200 as hb
    return hb


def _prefix(hb, Np=8, ws_bytes=1 << 30, swap=None, **kw):
    """Status of a call whose pointers are aligned addresses that are never read;
    swap = (argument, address) replaces one of them."""
    args = dict(B=2, Lq=1, Lkv=16, Hq=4, Hkv=2, d=64, m=4, W=8, Nc=4)
    args.update(kw)
    p = hb.problem(**args)
    names = ["q", "kp", "vp", "kc", "vc", "k_raw", "v_raw", "o", "lse", "ws"]
    ptr = {n: ctypes.c_void_p(4096) for n in names}
    if swap:
        ptr[swap[0]] = None if swap[1] is None else ctypes.c_void_p(swap[1])
    return hb._lib.hyb_prefix_attn_fwd(ctypes.byref(p), Np, *(ptr[n] for n in names), ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(Np=-1), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"),
    (dict(Hkv=3), "INVALID_ARG"), (dict(Lkv=0), "INVALID_ARG"), (dict(B=0), "INVALID_ARG"),
    (dict(Lq=0), "INVALID_ARG"), (dict(m=0), "INVALID_ARG"), (dict(W=-1), "INVALID_ARG"),
    (dict(Nc=-1), "INVALID_ARG"), (dict(d=96), "UNSUPPORTED"), (dict(topk=4), "UNSUPPORTED"),
    (dict(Np=1 << 29, Nc=1 << 29), "UNSUPPORTED"), (dict(B=1 << 20, Lq=1 << 12), "UNSUPPORTED"),
    (dict(W=1 << 30), "UNSUPPORTED"), (dict(B=1 << 20, Nc=1 << 16), "UNSUPPORTED"),
])
def test_prefix_refusals(hb, change, status):
    assert _prefix(hb, **change) == getattr(hb, "HYB_ERR_" + status)


def test_prefix_refuses_misaligned_fp32_and_int32(hb):
    assert _prefix(hb, swap=("lse", 4096 + 2)) == hb.HYB_ERR_INVALID_ARG
    p = hb.problem(B=2, Lq=1, Lkv=16, Hq=4, Hkv=2, d=64, m=4, W=8, Nc=4)
    p.q_pos = 4096 + 2
    a = [ctypes.c_void_p(4096)] * 10
    assert hb._lib.hyb_prefix_attn_fwd(ctypes.byref(p), 8, *a, 1 << 30, None) == hb.HYB_ERR_INVALID_ARG


def test_prefix_refuses_a_missing_short_or_misaligned_workspace(hb):
    big = dict(B=2, Lq=1, Lkv=16, Hq=4, Hkv=2, d=64, m=4, W=8, Nc=4)
    need = hb.hyb_prefix_workspace_size(hb.problem(**big), 100000)
    assert need > 0
    for bad in (dict(ws_bytes=need - 1), dict(swap=("ws", None)), dict(swap=("ws", 4096 + 16))):
        assert _prefix(hb, Np=100000, **bad) == hb.HYB_ERR_WORKSPACE


@pytest.mark.parametrize("name", ["q", "kp", "vp", "kc", "vc", "k_raw", "v_raw", "o"])
def test_prefix_refuses_missing_and_misaligned_tensors(hb, name):
    for address in (None, 4096 + 8):
        assert _prefix(hb, swap=(name, address)) == hb.HYB_ERR_INVALID_ARG


def test_prefix_workspace(hb):
    # partial results of every row: (maximum, sum) pairs and fp32 rows of d; none
    # where the sequences' streams are short enough to stay whole
    p = hb.problem(B=2, Lq=1, Lkv=16, Hq=4, Hkv=2, d=64, m=4, W=8, Nc=4)
    one = 2 * 4 * (8 + 64 * 4)
    size = hb.hyb_prefix_workspace_size(p, 100000)
    assert size >= 2 * one and size % 256 == 0 and hb.hyb_prefix_workspace_size(p, 8) == 0
    # nothing to attend to: nothing to keep
    p = hb.problem(B=2, Lq=1, Lkv=0, Hq=4, Hkv=2, d=64, m=4, W=0, Nc=0)
    assert hb.hyb_prefix_workspace_size(p, 0) == 0
    # a refused problem needs none
    p.topk = 4
    assert hb.hyb_prefix_workspace_size(p, 8) == 0


def test_python_calls_check_shapes_and_types(hb):
    p = hb.problem(B=2, Lq=1, Lkv=0, Hq=4, Hkv=2, d=64, m=4, W=0, Nc=4)
    bf = dict(dtype=torch.bfloat16)
    q, kp, kc = torch.zeros((2, 1, 4, 64), **bf), torch.zeros((8, 2, 64), **bf), torch.zeros((2, 4, 2, 64), **bf)
    for bad in (dict(q=q[..., :32]), dict(q=q.float()), dict(kp=kp[:, :1]), dict(vp=kp[:4]), dict(kc=None),
                dict(vc=kc[:1]), dict(kc=kc.transpose(1, 2).contiguous().transpose(1, 2))):
        x = dict(q=q, kp=kp, vp=kp, kc=kc, vc=kc)
        x.update(bad)
        with pytest.raises(ValueError):
            hb.hyb_prefix_attn_fwd(p, **x)
    with pytest.raises(ValueError, match="CUDA"):
        hb.hyb_prefix_attn_fwd(p, q, kp, kp, kc, kc)


def _weights(hb, e0=0, swap=None, idx=False, **kw):
    args = dict(B=2, Lq=1, Lkv=0, Hq=4, Hkv=2, d=64, m=4, W=8, Nc=4, topk=3 if idx else 0)
    args.update(kw)
    p = hb.problem(**args)
    names = ["q", "kc", "lse", "idx", "acc"]
    ptr = {n: ctypes.c_void_p(4096) for n in names}
    if not idx:
        ptr["idx"] = None
    if swap:
        ptr[swap[0]] = None if swap[1] is None else ctypes.c_void_p(swap[1])
    return hb._lib.hyb_attn_weights(ctypes.byref(p), ptr["q"], ptr["kc"], ptr["lse"], ptr["idx"], e0, ptr["acc"], 1,
                                    None)


@pytest.mark.parametrize("change,status", [
    (dict(e0=-1), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"), (dict(Nc=0), "INVALID_ARG"),
    (dict(Hkv=3), "INVALID_ARG"), (dict(topk=3), "INVALID_ARG"), (dict(idx=True, topk=0), "INVALID_ARG"),
    (dict(swap=("q", None)), "INVALID_ARG"), (dict(swap=("kc", None)), "INVALID_ARG"),
    (dict(swap=("lse", None)), "INVALID_ARG"), (dict(swap=("acc", None)), "INVALID_ARG"),
    (dict(swap=("q", 4096 + 8)), "INVALID_ARG"), (dict(swap=("kc", 4096 + 2)), "INVALID_ARG"),
    (dict(swap=("lse", 4096 + 2)), "INVALID_ARG"), (dict(swap=("acc", 4096 + 1)), "INVALID_ARG"),
    (dict(idx=True, swap=("idx", 4096 + 2)), "INVALID_ARG"),
    (dict(idx=True, Lq=2), "UNSUPPORTED"), (dict(idx=True, topk=2049), "UNSUPPORTED"), (dict(d=32), "UNSUPPORTED"),
    (dict(idx=True, B=2, Hq=320, Hkv=1, d=128, Nc=600, topk=200), "UNSUPPORTED"),
    (dict(e0=1 << 30), "UNSUPPORTED"), (dict(B=1 << 20, Lq=1 << 12), "UNSUPPORTED"),
])
def test_weights_refusals(hb, change, status):
    assert _weights(hb, **change) == getattr(hb, "HYB_ERR_" + status)


@pytest.mark.parametrize("args,status", [
    ((None, 1, 8, 4, 0, 0, True), "INVALID_ARG"), ((True, 1, 8, 4, 0, 0, None), "INVALID_ARG"),
    ((True, 0, 8, 4, 0, 0, True), "INVALID_ARG"), ((True, 1, 0, 4, 0, 0, True), "INVALID_ARG"),
    ((True, 1, 8, 0, 0, 0, True), "INVALID_ARG"), ((True, 1, 8, 4, -1, 0, True), "INVALID_ARG"),
    ((True, 1, 8, 4, 0, -1, True), "INVALID_ARG"), ((True, 1, 8, 4, 3, 2, True), "INVALID_ARG"),
    ((True, 1, 8, 1 << 30, 1 << 30, 1 << 30, True), "INVALID_ARG"),
    ((True, 65536, 8, 4, 0, 0, True), "UNSUPPORTED"), ((True, 1, 1 << 30, 4, 0, 0, True), "UNSUPPORTED"),
    ((True, 1, 8, 1 << 30, 0, 0, True), "UNSUPPORTED"),
])
def test_select_refusals(hb, args, status):
    acc, B, Nc, n_keep, first, last, keep = args
    at = ctypes.c_void_p(4096)
    assert hb._lib.hyb_evict_select(at if acc else None, B, Nc, None, n_keep, first, last, at if keep else None,
                                    None) == getattr(hb, "HYB_ERR_" + status)


def test_compact_refusals(hb):
    p = hb.problem(B=2, Lq=1, Lkv=0, Hq=2, Hkv=2, d=64, m=4, W=8, Nc=16, di=64)
    v = ctypes.c_void_p
    kv, ki, ac = 2 * 16 * 2 * 64 * 2, 2 * 16 * 64 * 2, 2 * 16 * 4          # bytes of each input
    base, out = 1 << 20, 1 << 24                                           # far apart, never read
    good = dict(keep=1 << 16, n_keep=8, No=8, kc=base, vc=base + kv, kic=base + 2 * kv, acc=base + 2 * kv + ki,
                kc_out=out, vc_out=out + kv, kic_out=out + 2 * kv, acc_out=out + 2 * kv + ki)

    def call(**kw):
        a = dict(good, **kw)
        ptr = [v(a[n]) if a[n] else None for n in ("kc", "vc", "kic", "acc", "kc_out", "vc_out", "kic_out", "acc_out")]
        return hb._lib.hyb_cache_compact(ctypes.byref(p), v(a["keep"]) if a["keep"] else None, a["n_keep"], a["No"],
                                         *ptr, None)

    none = dict(kc=None, vc=None, kic=None, acc=None, kc_out=None, vc_out=None, kic_out=None, acc_out=None)
    for bad in (dict(keep=None), dict(n_keep=0), dict(No=7), dict(kc_out=None), dict(acc=None), none,
                dict(kc_out=base), dict(kc_out=base + kv - 4),             # on its input, or on the end of it
                dict(vc_out=base),                                         # on another cache's input
                dict(kc_out=out + kv), dict(acc_out=out + 4),              # on another output
                dict(kc_out=1 << 16), dict(acc_out=(1 << 16) + 60),        # on the list of kept entries
                dict(kc=base + 2), dict(acc_out=out + 2 * kv + ki + 2)):
        assert call(**bad) == hb.HYB_ERR_INVALID_ARG, bad
    assert call(No=1 << 30) == hb.HYB_ERR_UNSUPPORTED
    p.Nc = 0
    assert call() == hb.HYB_ERR_INVALID_ARG
    p.Nc = 16
    # 4-bit caches: codes and pairs come together
    a = [v(base + i * (1 << 16)) for i in range(7)] + [v(out + i * (1 << 16)) for i in range(7)]
    for i in (0, 1, 7, 8):
        b = list(a)
        b[i] = None
        assert hb._lib.hyb_cache_compact_fp4(ctypes.byref(p), v(1 << 16), 8, 8, *b, None) == hb.HYB_ERR_INVALID_ARG


def test_python_calls_of_the_eviction_check_shapes(hb):
    p = hb.problem(B=2, Lq=1, Lkv=0, Hq=4, Hkv=2, d=64, m=4, W=0, Nc=4, di=64)
    bf = dict(dtype=torch.bfloat16)
    q, kc, lse = torch.zeros((2, 1, 4, 64), **bf), torch.zeros((2, 4, 2, 64), **bf), torch.zeros((2, 4, 1))
    for bad in (dict(q=q[:1]), dict(kc=kc[:, :2]), dict(lse=lse.double()), dict(acc=torch.zeros((2, 5))),
                dict(idx=torch.zeros((2, 1, 4), dtype=torch.int32))):
        with pytest.raises(ValueError):
            hb.hyb_attn_weights(p, **{**dict(q=q, kc=kc, lse=lse), **bad})
    with pytest.raises(ValueError):
        hb.hyb_evict_select(torch.zeros((2, 4), dtype=torch.float64), 2)
    with pytest.raises(ValueError):
        hb.hyb_evict_select(torch.zeros((2, 4)), 2, n_valid=torch.zeros(2))
    keep = torch.zeros((2, 3), dtype=torch.int32)
    for bad in (dict(keep=keep.long()), dict(keep=keep[:1]), dict(kc=kc[..., :32]), dict(kc=None, kc_out=kc),
                dict(kc=kc.transpose(0, 1))):
        with pytest.raises(ValueError):
            hb.hyb_cache_compact(p, **{**dict(keep=keep, kc=kc), **bad})
