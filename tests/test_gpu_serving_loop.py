"""Decode loops over shared and bounded caches as the header describes them: a batch
behind a prompt that it shares, and a ragged batch that goes on after one eviction.
The raw tokens are kept beside the rings, and every step is held against the
definition over them."""
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


def _check(o, lse, ref):
    # 2^-8 for the rounding of P and of o each (see test_gpu_prefix)
    bound = 2.0 ** -8 * (np.abs(ref["o"]) + ref["a"]) * 1.01 + 1e-4 * ref["a"]
    assert np.all(np.abs(_f64(o) - ref["o"]) <= bound)
    assert np.all(np.abs(_f64(lse) - ref["lse"]) <= 1e-4)


@pytest.mark.parametrize("P,m,W", [(203, 4, 16), (150, 7, 33), (40, 1, 9), (20, 4, 32)])
def test_tokens_behind_a_shared_prompt(hb, P, m, W):
    # the entries that end before the window of the first new token are shared; the
    # prompt's other tokens go through the append into every sequence's ring and caches
    B, Hq, Hkv, d, steps = 3, 8, 2, 64, 2 * W + 3
    g = torch.Generator().manual_seed(P)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    wk, wv = (torch.randn((m, d), generator=g).cuda() for _ in range(2))
    prompt = [bf(P, Hkv, d) for _ in range(2)]
    own = [bf(B, steps, Hkv, d) for _ in range(2)]
    raw = [torch.cat([x.expand(B, P, Hkv, d), y], 1).contiguous() for x, y in zip(prompt, own)]
    Np = max(P - W + 1, 0) // m
    Nc = (P - Np * m + steps) // m
    shared = [hb.hyb_hca_compress(x[None, :Np * m].contiguous(), w, m)[0] if Np else None
              for x, w in zip(prompt, (wk, wv))]
    kc, vc = (torch.full((B, Nc, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ring = [torch.zeros((B, 2 * W, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    entries = [hb.hyb_hca_compress(x, w, m) for x, w in zip(raw, (wk, wv))]
    none = np.zeros((0, Hkv, d))
    for t in range(Np * m, P + steps):
        t_new = torch.full((B,), t - Np * m, dtype=torch.int32, device="cuda")
        p = hb.problem(B=B, Lq=1, Lkv=2 * W, Hq=Hkv, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc)
        kv0 = hb.hyb_decode_append(p, t_new, raw[0][:, t].contiguous(), raw[1][:, t].contiguous(), *ring, kc, vc, wk, wv)
        if t < P:
            continue
        q_pos = (t_new + Np * m).view(B, 1).contiguous()
        p = hb.problem(B=B, Lq=1, Lkv=2 * W, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc, q_pos=q_pos,
                       kv_pos0=(kv0 + Np * m).contiguous())
        q, lse = bf(B, 1, Hq, d), torch.empty((B, Hq, 1), device="cuda")
        o = hb.hyb_prefix_attn_fwd(p, q, *shared, kc, vc, *ring, lse=lse)
        ref = serving.prefix_attention(_f64(q), none, none, _f64(entries[0]), _f64(entries[1]), _f64(raw[0]),
                                       _f64(raw[1]), m, W, q_pos.cpu().numpy(), np.zeros(B, np.int64))
        assert (ref["n"] == min(t + 1, W) + serving._visible(t, m, W)).all()
        _check(o, lse, ref)
    assert hb.hyb_get_device_status() == hb.HYB_OK


@pytest.mark.parametrize("m,W", [(3, 16), (4, 16), (5, 5)])
def test_a_ragged_batch_goes_on_after_one_eviction(hb, m, W):
    # one selection and one compaction for sequences of different lengths: each loses
    # its own number E of entries, and its ring rows move by m E with its positions
    B, Hq, Hkv, d, Nc, n_keep = 5, 8, 2, 64, 40, 24
    n_last = -(-W // m) + 1
    g = torch.Generator().manual_seed(m * 100 + W)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    wk, wv = (torch.randn((m, d), generator=g).cuda() for _ in range(2))
    ring = [torch.zeros((B, 2 * W, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kc, vc = (torch.full((B, Nc, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    acc = torch.zeros((B, Nc), device="cuda")
    length = [m * Nc, m * Nc - 1, m * 31 + 2, m * n_keep, m * 7 + 1]      # tokens before the eviction
    raw = [[[] for _ in range(B)] for _ in range(2)]                      # K and V rows of every token
    entries = [[None] * B, [None] * B]                                    # K and V entries each sequence holds
    pos = [0] * B

    def append(active):
        # one more token of the active sequences (the others repeat their last one)
        rows = [bf(B, Hkv, d) for _ in range(2)]
        t = list(pos)
        for b in range(B):
            if active[b]:
                for i in range(2):
                    raw[i][b].append(rows[i][b])
                pos[b] += 1
            else:
                t[b] -= 1
                for i in range(2):
                    rows[i][b] = raw[i][b][-1]
        t_new = torch.tensor(t, dtype=torch.int32, device="cuda")
        p = hb.problem(B=B, Lq=1, Lkv=2 * W, Hq=Hkv, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc)
        return t_new, hb.hyb_decode_append(p, t_new, *rows, *ring, kc, vc, wk, wv)

    def decode(active):
        t_new, kv0 = append(active)
        p = hb.problem(B=B, Lq=1, Lkv=2 * W, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc, q_pos=t_new.view(B, 1), kv_pos0=kv0)
        q, lse = bf(B, 1, Hq, d), torch.empty((B, Hq, 1), device="cuda")
        o = hb.hyb_prefix_attn_fwd(p, q, None, None, kc, vc, *ring, lse=lse)
        hb.hyb_attn_weights(p, q, kc, lse, acc=acc)
        return t_new, q, o, lse

    while any(p < n for p, n in zip(pos, length)):
        decode([p < n for p, n in zip(pos, length)])
    n_valid = torch.tensor([p // m for p in pos], dtype=torch.int32, device="cuda")
    p = hb.problem(B=B, Lq=1, Lkv=0, Hq=Hkv, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc)
    keep = hb.hyb_evict_select(acc, n_keep, n_first=1, n_last=n_last, n_valid=n_valid)
    out = [torch.full_like(kc, float("nan")), torch.full_like(vc, float("nan")), torch.zeros_like(acc)]
    hb.hyb_cache_compact(p, keep, kc, vc, acc=acc, kc_out=out[0], vc_out=out[1], acc_out=out[2])
    lost = [max(n - n_keep, 0) for n in n_valid.tolist()]
    assert len(set(lost)) > 2 and (m % W == 0 or any(m * e % W for e in lost))
    for b in range(B):
        rows = [j for j in keep[b].tolist() if j >= 0]
        for i, c in enumerate((kc, vc)):
            entries[i][b] = c[b, rows].clone()
        for r in ring:          # row r goes to (r - m E) mod W, in both halves
            r[b] = torch.cat([torch.roll(h, -(m * lost[b]) % W, 0) for h in (r[b, :W], r[b, W:])])
        pos[b] -= m * lost[b]
    kc, vc, acc = out
    for _ in range(3 * W):
        if max(pos) + 1 > m * Nc:
            break
        before = list(pos)
        t_new, q, o, lse = decode([True] * B)
        for b in range(B):
            if (before[b] + 1) % m == 0:             # a block closed: the last m tokens
                for i, (c, w) in enumerate(((kc, wk), (vc, wv))):
                    block = torch.stack(raw[i][b][-m:])
                    have, new = c[b, before[b] // m], hb.hyb_hca_compress(block[None].contiguous(), w, m)[0, 0]
                    # two fp32 sums of m terms (each term's weight 2^-22 off, sums and quotients
                    # 2^-24 a step, of sum P |x| <= max |x|), each rounded to bf16 (half a
                    # step is 2^-8 of the value, so the two are a step apart at most)
                    fp32 = 2 * (2.0 ** -22 + (2 * m + 2) * 2.0 ** -24) * float(block.abs().max())
                    step = 2 * 2.0 ** -8 * torch.maximum(have.abs(), new.abs()).double()
                    assert torch.all((have.double() - new.double()).abs() <= step + fp32)
                    entries[i][b] = torch.cat([entries[i][b], have[None]])
            # the definition over the entries held and the last W tokens
            t = before[b]
            assert len(entries[0][b]) == (t + 1) // m
            win = [torch.stack(raw[i][b][-W:]) for i in range(2)]
            ref = serving.prefix_attention(
                _f64(q[b:b + 1]), *(np.zeros((0, Hkv, d)),) * 2, *(_f64(e[b][None]) for e in entries),
                *(_f64(x[None]) for x in win), m, W, np.array([[t]]), np.array([t + 1 - len(win[0])]))
            _check(o[b:b + 1], lse[b:b + 1], ref)
    assert hb.hyb_get_device_status() == hb.HYB_OK
