"""Memory and streams of the entry points around shared and bounded caches: what a
call allocates when it is given a stream belongs to that stream."""
import contextlib

import pytest
import torch

import compressed_sparse_sliding_b200 as hb


def test_allocations_come_from_the_given_streams_pool(monkeypatch):
    # without a GPU: which stream is current when a call's tensor is made, and which
    # streams the allocator is told of
    log, current = [], ["caller"]

    class Tensor:
        def record_stream(self, s):
            log.append(("used on", s))

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch, "empty", lambda *a, **k: log.append(("made on", current[-1])) or Tensor())
    for given, want in ((None, [("made on", "caller")]), ("side", [("made on", "side"), ("used on", "caller")])):
        on = object.__new__(hb._On)
        on.device, on.stream = "cuda:0", given
        log.clear()
        on.new((4,), torch.float32)
        assert log == want


def _calls():
    """name, a function (stream) -> outputs; inputs on the current stream."""
    B, Hq, Hkv, d, m, W, Np, Nc = 8, 64, 1, 128, 4, 128, 700, 90
    g = torch.Generator().manual_seed(3)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    q, kp, vp, kc, vc = bf(B, 1, Hq, d), bf(Np, Hkv, d), bf(Np, Hkv, d), bf(B, Nc, Hkv, d), bf(B, Nc, Hkv, d)
    kr, vr = bf(B, W, Hkv, d), bf(B, W, Hkv, d)
    t = (Np + Nc) * m + W - 1
    q_pos = torch.full((B, 1), t, dtype=torch.int32, device="cuda")
    kv0 = torch.full((B,), t - W + 1, dtype=torch.int32, device="cuda")
    p = hb.problem(B=B, Lq=1, Lkv=W, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc, q_pos=q_pos, kv_pos0=kv0)
    lse = torch.full((B, Hq, 1), 5.0, device="cuda")
    acc = torch.rand((B, Nc), generator=g).cuda()
    keep = hb.hyb_evict_select(acc, 50, 1, 7)
    return [("prefix", lambda s: hb.hyb_prefix_attn_fwd(p, q, kp, vp, kc, vc, kr, vr, stream=s)),
            ("weights", lambda s: hb.hyb_attn_weights(p, q, kc, lse, e0=Np, stream=s)),
            ("select", lambda s: hb.hyb_evict_select(acc, 50, 1, 7, stream=s)),
            ("compact", lambda s: hb.hyb_cache_compact(p, keep, kc, vc, acc=acc, stream=s))]


@pytest.mark.gpu
def test_blocks_freed_on_the_callers_stream_are_left_alone(monkeypatch):
    # work is pending on the current stream in blocks that have been freed there: a call
    # on another stream takes none of them, and both sides' results are right
    made = []
    new = hb._On.new
    monkeypatch.setattr(hb._On, "new", lambda self, *a: made.append(new(self, *a)) or made[-1])
    flat = lambda r: [t for t in (r.values() if isinstance(r, dict) else [r]) if t is not None]
    side = torch.cuda.Stream()
    for name, call in _calls():
        made.clear()
        want = [t.clone() for t in flat(call(None))]
        sizes = [t.numel() * t.element_size() for t in made]
        made.clear()
        torch.cuda.synchronize()
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in blocks]
        sums = []
        torch.cuda._sleep(20_000_000)
        for t in blocks:
            t.fill_(3)
            sums.append(t.sum(dtype=torch.int64))
        lens = [t.numel() for t in blocks]
        del blocks, t
        got = flat(call(side))
        for t in made:
            lo, hi = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
            assert not any(lo < e and s < hi for s, e in spans), name
        del t
        torch.cuda.synchronize()
        assert [int(s) for s in sums] == [3 * n for n in lens], name
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    assert hb.hyb_get_device_status() == hb.HYB_OK
