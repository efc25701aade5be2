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
    (dict(W=1 << 30), "UNSUPPORTED"), (dict(ws_bytes=16), "WORKSPACE"), (dict(swap=("ws", None)), "WORKSPACE"),
    (dict(swap=("ws", 4096 + 16)), "WORKSPACE"),
])
def test_prefix_refusals(hb, change, status):
    assert _prefix(hb, **change) == getattr(hb, "HYB_ERR_" + status)


@pytest.mark.parametrize("name", ["q", "kp", "vp", "kc", "vc", "k_raw", "v_raw", "o"])
def test_prefix_refuses_missing_and_misaligned_tensors(hb, name):
    for address in (None, 4096 + 8):
        assert _prefix(hb, swap=(name, address)) == hb.HYB_ERR_INVALID_ARG


def test_prefix_workspace(hb):
    # partial results of every row: (maximum, sum) pairs and fp32 rows of d
    p = hb.problem(B=2, Lq=1, Lkv=16, Hq=4, Hkv=2, d=64, m=4, W=8, Nc=4)
    one = 2 * 4 * (8 + 64 * 4)
    assert hb.hyb_prefix_workspace_size(p, 8) >= one and hb.hyb_prefix_workspace_size(p, 8) % 256 == 0
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
