"""Operators of a serving loop over bounded and shared caches: what is measured.

Four calls of the package, and the same mathematics in plain torch:

  prefix   hyb_prefix_attn_fwd: one softmax over compressed entries that every
           sequence of the batch shares, the sequence's own entries and its raw
           window
  weights  hyb_attn_weights: the attention weight each cached entry received,
           summed over heads and query tokens (dense or over a selection)
  evict    hyb_evict_select + hyb_cache_compact(_fp4): the entries a full cache
           keeps by that weight, and the caches rewritten with them (4-bit rows
           are moved, not computed: their codes are compared as they are)

Visibility everywhere: entry e (raw positions e*m .. e*m+m-1) is visible to a
query at position t iff (e + 1) * m - 1 < t - W + 1.
"""
import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a few chat turns over a short shared system prompt: latency counts
        dict(name="prefix_small", op="prefix", B=4, Lq=1, Hq=4, Hkv=1, d=64, m=4, W=128, Np=256, Nc=64),
        # heavily compressed decode: 64 continuations of one 131072-token document
        dict(name="prefix_hca_decode", op="prefix", B=64, Lq=1, Hq=64, Hkv=8, d=128, m=128, W=128, Np=1024,
             Nc=64),
        # lightly compressed decode: 64 sequences over a 65536-token prefix, 8192 tokens of their own
        dict(name="prefix_mqa_decode", op="prefix", B=64, Lq=1, Hq=64, Hkv=1, d=128, m=4, W=128, Np=16384,
             Nc=2048),
        # drafted tokens verified five at a time; sizes on no grid
        dict(name="prefix_draft_ragged", op="prefix", B=13, Lq=5, Hq=20, Hkv=4, d=128, m=7, W=61, Np=5003,
             Nc=611),
        # chunks of user prompts prefilled behind a shared prefix
        dict(name="prefix_chunk", op="prefix", B=8, Lq=256, Hq=16, Hkv=16, d=128, m=4, W=128, Np=2048, Nc=256),
        # uncompressed entries (m = 1, no window): many samples of one long prompt
        dict(name="prefix_samples", op="prefix", B=128, Lq=1, Hq=32, Hkv=8, d=128, m=1, W=0, Np=65536, Nc=1024),
        # every entry of 64 decode caches, the weights of one step
        dict(name="weights_decode", op="weights", B=64, Lq=1, Hq=64, Hkv=1, d=128, m=4, W=128, Nc=16384, K=0,
             more=False),
        # only the selected entries, added to the weights of earlier steps
        dict(name="weights_selected", op="weights", B=64, Lq=1, Hq=64, Hkv=1, d=128, m=4, W=128, Nc=16384,
             K=1024, more=True),
        # the last 32 tokens of a prompt score its cache before the first eviction
        dict(name="weights_prompt", op="weights", B=2, Lq=32, Hq=32, Hkv=4, d=128, m=4, W=128, Nc=8192, K=0,
             more=False),
        # 64 full decode caches cut to half
        dict(name="evict_decode", op="evict", B=64, Nc=16384, keep=8192, first=4, last=64, Hkv=1, d=128, di=64,
             bits=16),
        # one million-token sequence over 4-bit caches
        dict(name="evict_fp4_long", op="evict", B=1, Nc=262144, keep=65536, first=16, last=32, Hkv=1, d=128,
             di=64, bits=4),
        # a small odd batch, some sequences with fewer entries than are kept
        dict(name="evict_small", op="evict", B=3, Nc=1000, keep=333, first=1, last=7, Hkv=2, d=64, di=0, bits=16),
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prefix", "weights", "evict"])
    d = rng.choice([64, 128, 128])
    if op == "evict":
        B, bits = _log(rng, 1, 64), rng.choice([16, 16, 4])
        Nc = _log(rng, 64, max(64, min(262144, (1 << 20) // B)))
        keep = max(2, int(Nc * rng.uniform(0.1, 0.95)))
        first = rng.randint(0, keep // 8)
        return dict(op=op, B=B, Nc=Nc, keep=keep, first=first, last=rng.randint(0, keep // 8),
                    Hkv=rng.choice([1, 1, 2, 4] if Nc * B <= 1 << 18 else [1]), d=d,
                    di=rng.choice([0, 64]) if bits == 16 else 64, bits=bits)
    Hkv, g = rng.choice([(1, 64), (1, 32), (1, 4), (8, 8), (8, 4), (4, 5), (2, 7), (16, 1)])
    m, W = rng.choice([(4, 128), (4, 128), (128, 128), (1, 0), (7, 61), (16, 200)])
    B = _log(rng, 1, 96)
    Lq = rng.choice([1, 1, 1, 2, 5, 33])
    if op == "prefix":
        Np = _log(rng, 1, 32768)
        Nc = _log(rng, 1, max(1, min(4096, (1 << 20) // (B * Hkv * 2))))
        while Hkv * g * B * Lq * (Np + Nc) > 1 << 27:
            B, Lq = max(1, B // 2), max(1, Lq // 2)
            if B == Lq == 1:
                break
        return dict(op=op, B=B, Lq=Lq, Hq=Hkv * g, Hkv=Hkv, d=d, m=m, W=W, Np=Np, Nc=Nc)
    K = 0
    if rng.random() < 0.4:
        Lq, K = 1, _log(rng, 1, 2048)
    Nc = _log(rng, max(1, K), max(K, 1, min(65536, (1 << 20) // (B * Hkv))))
    while Hkv * g * B * Lq * Nc > 1 << 26 and B * Lq > 1:
        B, Lq = max(1, B // 2), max(1, Lq // 2)
    return dict(op=op, B=B, Lq=Lq, Hq=Hkv * g, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc, K=K, more=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _own_counts(case):
    """Own entries of each sequence: between half of the capacity and all of it."""
    Nc = case["Nc"]
    return [Nc - (b * 7919) % (Nc // 2 + 1) for b in range(case["B"])]


def _positions(case, entries):
    """Position of each sequence's first query token: just past `entries` visible ones."""
    return [e * case["m"] + case["W"] - 1 + (b % case["m"]) for b, e in enumerate(entries)]


def _bf16(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    B, d, Hkv = case["B"], case["d"], case["Hkv"]
    if case["op"] == "evict":
        Nc, n = case["Nc"], case["keep"]
        # heavy-tailed weights; entries that were never attended to are exactly 0
        acc = torch.exp(2 * torch.randn((B, Nc), generator=gen, device=dev))
        acc *= torch.rand((B, Nc), generator=gen, device=dev) > 0.1
        counts = [Nc - (b * 7919) % (Nc // 4 + 1) if b % 3 else Nc for b in range(B)]
        if B > 2:
            counts[2] = max(1, n // 2)        # a sequence that has nothing to evict yet
        s = dict(case=case, acc=acc, n_valid=torch.tensor(counts, dtype=torch.int32, device=dev))
        zeros = lambda t: torch.zeros((B, n, *t.shape[2:]), dtype=t.dtype, device=dev)
        if case["bits"] == 4:
            for name, lead, dx in (("kc", (B, Nc, Hkv), d), ("vc", (B, Nc, Hkv), d), ("kic", (B, Nc), case["di"])):
                s[name] = (torch.randint(0, 256, (*lead, dx // 2), generator=gen, device=dev, dtype=torch.uint8),
                           torch.randn((*lead, 2), generator=gen, device=dev))
                s[name + "_out"] = tuple(zeros(t) for t in s[name])
        else:
            s["kc"], s["vc"] = _bf16(gen, B, Nc, Hkv, d), _bf16(gen, B, Nc, Hkv, d)
            s["kic"] = _bf16(gen, B, Nc, case["di"]) if case["di"] else None
            for name in ("kc", "vc", "kic"):
                s[name + "_out"] = None if s[name] is None else zeros(s[name])
        s["acc_out"] = zeros(acc)
        if own:
            import compressed_sparse_sliding_b200 as hb
            s["p"] = hb.problem(B=B, Lq=1, Lkv=0, Hq=Hkv, Hkv=Hkv, d=d, m=1, W=0, di=case["di"], Nc=Nc)
            if case["bits"] == 4:
                for name in ("kc", "vc", "kic"):
                    s[name + "_fp4"] = hb.Fp4Cache(*s[name])
                    s[name + "_out_fp4"] = hb.Fp4Cache(*s[name + "_out"])
        return s

    Lq, Hq, m, W, Nc = case["Lq"], case["Hq"], case["m"], case["W"], case["Nc"]
    Np = case.get("Np", 0)
    first = _positions(case, [Np + n for n in _own_counts(case)])
    first = torch.tensor(first, dtype=torch.int32, device=dev)
    q_pos = (first[:, None] + torch.arange(Lq, dtype=torch.int32, device=dev)).contiguous()
    s = dict(case=case, q=_bf16(gen, B, Lq, Hq, d), kc=_bf16(gen, B, Nc, Hkv, d), q_pos=q_pos)
    if case["op"] == "prefix":
        s.update(vc=_bf16(gen, B, Nc, Hkv, d), kp=_bf16(gen, Np, Hkv, d), vp=_bf16(gen, Np, Hkv, d),
                 k_raw=None, v_raw=None, kv_pos0=None)
        if W:
            # the raw rows positions first - W + 1 .. first + Lq - 1
            s["k_raw"], s["v_raw"] = _bf16(gen, B, W + Lq - 1, Hkv, d), _bf16(gen, B, W + Lq - 1, Hkv, d)
            s["kv_pos0"] = (first - (W - 1)).contiguous()
        if own:
            import compressed_sparse_sliding_b200 as hb
            s["p"] = hb.problem(B=B, Lq=Lq, Lkv=W + Lq - 1 if W else 0, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, Nc=Nc,
                                q_pos=q_pos, kv_pos0=s["kv_pos0"])
            s["ws"] = torch.empty(max(256, hb.hyb_prefix_workspace_size(s["p"], Np)), dtype=torch.uint8, device=dev)
        return s

    # weights: the log-sum-exp rows of the attention that ran before
    K = case["K"]
    vis = _visible(q_pos, m, W, Nc)                                        # [B, Lq]
    s["idx"] = None
    if K:
        pick = torch.rand((B, Nc), generator=gen, device=dev)
        pick.masked_fill_(torch.arange(Nc, device=dev) >= vis, -1.0)
        top = pick.topk(K, dim=1)
        idx = torch.where(top.values >= 0, top.indices, Nc).sort(dim=1).values
        s["idx"] = torch.where(idx < Nc, idx, -1).to(torch.int32).view(B, 1, K).contiguous()
    s["acc"] = torch.rand((B, Nc), generator=gen, device=dev)
    s["lse"] = torch.full((B, Hq, Lq), float("-inf"), device=dev)
    for b in range(B):
        k = s["kc"][b].float()
        if K:
            k = k[s["idx"][b, 0].clamp(min=0).long()]
            seen = (s["idx"][b] >= 0).view(1, 1, 1, K)
        else:
            seen = (torch.arange(Nc, device=dev) < vis[b, :, None]).view(1, 1, Lq, Nc)
        z = torch.einsum("thgd,khd->hgtk", s["q"][b].float().view(Lq, Hkv, Hq // Hkv, d), k) * d ** -0.5
        s["lse"][b] = torch.logsumexp(z.masked_fill(~seen, float("-inf")), -1).view(Hq, Lq)
    if own:
        import compressed_sparse_sliding_b200 as hb
        s["p"] = hb.problem(B=B, Lq=Lq, Lkv=0, Hq=Hq, Hkv=Hkv, d=d, m=m, W=W, topk=K, Nc=Nc, q_pos=q_pos)
    return s


def _visible(pos, m, W, n):
    """Entries of a cache of n that a query at `pos` sees."""
    return torch.div(pos - W + 1, m, rounding_mode="floor").clamp(0, n)


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    return dict(prefix=_run_prefix, weights=_run_weights, evict=_run_evict)[case["op"]](s, case)


def _run_prefix(s, case):
    B, Lq, Hq, Hkv, d = (case[n] for n in ("B", "Lq", "Hq", "Hkv", "d"))
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=s["q"].device)
    if own:
        import compressed_sparse_sliding_b200 as hb
        o = hb.hyb_prefix_attn_fwd(s["p"], s["q"], s["kp"], s["vp"], s["kc"], s["vc"], s["k_raw"], s["v_raw"],
                                   lse=lse, ws=s["ws"])
        return dict(o=o, lse=lse)
    m, W, Np, Nc = case["m"], case["W"], case["Np"], case["Nc"]
    dev = s["q"].device
    q = s["q"].float().view(B, Lq, Hkv, Hq // Hkv, d) * d ** -0.5
    vis = _visible(s["q_pos"], m, W, Np + Nc)                              # [B, Lq]
    scores = [torch.einsum("bthgd,khd->bhgtk", q, s["kp"].float()),
              torch.einsum("bthgd,bkhd->bhgtk", q, s["kc"].float())]
    seen = [torch.arange(Np + Nc, device=dev) < vis[..., None]]            # [B, Lq, keys]
    if W:
        raw = s["kv_pos0"][:, None, None] + torch.arange(s["k_raw"].shape[1], device=dev)
        t = s["q_pos"][..., None]
        seen.append((raw >= (t - W + 1).clamp(min=0)) & (raw <= t))
        scores.append(torch.einsum("bthgd,bkhd->bhgtk", q, s["k_raw"].float()))
    scores, seen = torch.cat(scores, -1), torch.cat(seen, -1)[:, None, None]
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top.isfinite(), top, 0.0)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    e = e / torch.where(total > 0, total, 1.0)
    o = torch.einsum("bhgtk,khd->bthgd", e[..., :Np], s["vp"].float())
    o = o + torch.einsum("bhgtk,bkhd->bthgd", e[..., Np:Np + Nc], s["vc"].float())
    if W:
        o = o + torch.einsum("bhgtk,bkhd->bthgd", e[..., Np + Nc:], s["v_raw"].float())
    lse.copy_((top + torch.log(total)).view(B, Hq, Lq))
    return dict(o=o.reshape(B, Lq, Hq, d).to(torch.bfloat16), lse=lse)


def _run_weights(s, case):
    B, Lq, Hq, Hkv, d, K, Nc = (case[n] for n in ("B", "Lq", "Hq", "Hkv", "d", "K", "Nc"))
    if own:
        import compressed_sparse_sliding_b200 as hb
        acc = s["acc"].clone() if case["more"] else None
        return hb.hyb_attn_weights(s["p"], s["q"], s["kc"], s["lse"], idx=s["idx"], acc=acc)
    q = s["q"].float().view(B, Lq, Hkv, Hq // Hkv, d) * d ** -0.5
    lse = s["lse"].view(B, Hkv, Hq // Hkv, Lq, 1)
    if K:
        at = s["idx"][:, 0].clamp(min=0).long()                            # [B, K]
        k = torch.gather(s["kc"], 1, at[:, :, None, None].expand(B, K, Hkv, d)).float()
        w = torch.exp(torch.einsum("bthgd,bkhd->bhgtk", q, k) - lse).sum((1, 2, 3))
        w = torch.where(s["idx"][:, 0] >= 0, w, 0.0)
        sums = torch.zeros((B, Nc), device=w.device).scatter_add_(1, at, w)
    else:
        vis = _visible(s["q_pos"], case["m"], case["W"], Nc)
        seen = (torch.arange(Nc, device=q.device) < vis[..., None])[:, None, None]
        z = torch.einsum("bthgd,bkhd->bhgtk", q, s["kc"].float()) - lse
        sums = torch.exp(z.masked_fill(~seen, float("-inf"))).sum((1, 2, 3))
    return s["acc"] + sums if case["more"] else sums


def _run_evict(s, case):
    n, names = case["keep"], ("kc", "vc", "kic")
    if own:
        import compressed_sparse_sliding_b200 as hb
        keep = hb.hyb_evict_select(s["acc"], n, n_first=case["first"], n_last=case["last"], n_valid=s["n_valid"])
        if case["bits"] == 4:
            hb.hyb_cache_compact_fp4(s["p"], keep, *(s[x + "_fp4"] for x in names), acc=s["acc"],
                                     acc_out=s["acc_out"], **{x + "_out": s[x + "_out_fp4"] for x in names})
        else:
            hb.hyb_cache_compact(s["p"], keep, *(s[x] for x in names), acc=s["acc"], acc_out=s["acc_out"],
                                 **{x + "_out": s[x + "_out"] for x in names})
    else:
        Nc = case["Nc"]
        j = torch.arange(Nc, device="cuda")
        count = s["n_valid"][:, None]
        rank = torch.where((j < case["first"]) | (j >= count - case["last"]), float("inf"), s["acc"])
        rank = torch.where(j < count, rank, -1.0)                          # weights are never negative
        order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :n]
        order = torch.where(torch.arange(n, device="cuda") < count, order, Nc).sort(dim=1).values
        keep = torch.where(order < Nc, order, -1).to(torch.int32)
        at = keep.clamp(min=0).long()

        def rows(x, out):
            got = torch.gather(x, 1, at.view(*at.shape, *[1] * (x.dim() - 2)).expand(*at.shape, *x.shape[2:]))
            return torch.where((keep >= 0).view(*at.shape, *[1] * (x.dim() - 2)), got, out)

        s = dict(s, acc_out=rows(s["acc"], s["acc_out"]))
        for x in names:
            if s[x] is not None:
                s[x + "_out"] = (tuple(map(rows, s[x], s[x + "_out"])) if case["bits"] == 4
                                 else rows(s[x], s[x + "_out"]))
    got = {x: s[x + "_out"] for x in names if s[x] is not None}
    return dict(keep=keep, acc=s["acc_out"], **got)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    B, d, Hkv = case["B"], case["d"], case["Hkv"]
    if case["op"] == "evict":
        per = 2 * Hkv * (d * 2 if case["bits"] == 16 else d // 2 + 8) + 4
        if case["di"]:
            per += case["di"] * 2 if case["bits"] == 16 else case["di"] // 2 + 8
        return dict(bytes=B * (case["Nc"] * 4 + case["keep"] * (2 * per + 4)), flops=0)
    Lq, Hq, Nc = case["Lq"], case["Hq"], case["Nc"]
    counts = _own_counts(case)
    rows = B * Lq * Hq
    if case["op"] == "weights":
        K = case["K"]
        seen = sum(min(K, n) if K else n for n in counts)
        return dict(bytes=rows * (d * 2 + 4) + seen * Hkv * d * 2 + B * K * 4 + (B * Nc + seen if case["more"] else B * Nc) * 4,
                    flops=2 * d * Hq * Lq * seen)
    Np, W = case["Np"], case["W"]
    keys = sum(counts) + B * (Np + W)
    own_rows = sum(counts) + (B * (W + Lq - 1) if W else 0)
    return dict(bytes=rows * (d * 4 + 4) + (Np + own_rows) * Hkv * d * 4, flops=4 * d * Hq * Lq * keys)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s, case)
    B, Lq, Hq, Hkv, d, m, W, Nc = (case[n] for n in ("B", "Lq", "Hq", "Hkv", "d", "m", "W", "Nc"))
    g, Np = Hq // Hkv, case.get("Np", 0)
    pos = s["q_pos"].tolist()
    f64 = dict(dtype=torch.float64, device="cuda")
    if case["op"] == "weights":
        out = s["acc"].double() if case["more"] else torch.zeros((B, Nc), **f64)
        for b in range(B):
            for t in range(Lq):
                n = min(max((pos[b][t] - W + 1) // m, 0), Nc)
                rows = torch.arange(n, device="cuda")
                if case["K"]:
                    rows = s["idx"][b, t].long()
                    rows = rows[rows >= 0]
                for h in range(Hkv):
                    z = s["kc"][b, rows, h].double() @ s["q"][b, t, h * g:(h + 1) * g].double().T / d ** 0.5
                    out[b, rows] += torch.exp(z - s["lse"][b, h * g:(h + 1) * g, t].double()).sum(1)
        return out
    o, lse = torch.zeros((B, Lq, Hq, d), **f64), torch.full((B, Hq, Lq), float("-inf"), **f64)
    for b in range(B):
        keys, vals = [torch.cat([s[x + "p"], s[x + "c"][b]]).double().transpose(0, 1) for x in "kv"]
        raw = [s[x + "_raw"][b].double().transpose(0, 1) for x in "kv"] if W else None
        first = s["kv_pos0"][b].item() if W else 0
        for t in range(Lq):
            n = min(max((pos[b][t] - W + 1) // m, 0), Np + Nc)
            k, v = keys[:, :n], vals[:, :n]
            if W:
                lo, hi = max(pos[b][t] - W + 1, 0) - first, pos[b][t] - first + 1
                k, v = torch.cat([k, raw[0][:, lo:hi]], 1), torch.cat([v, raw[1][:, lo:hi]], 1)
            if not k.shape[1]:
                continue
            z = s["q"][b, t].double().view(Hkv, g, d) @ k.transpose(1, 2) / d ** 0.5
            lse[b, :, t] = torch.logsumexp(z, -1).view(Hq)
            o[b, t] = (torch.softmax(z, -1) @ v).view(Hq, d)
    return dict(o=o, lse=lse)


def _exact_evict(s, case):
    n, names = case["keep"], ("kc", "vc", "kic")
    acc, counts = s["acc"].double().cpu(), s["n_valid"].tolist()
    kept = []
    for b, count in enumerate(counts):
        held = set(range(min(case["first"], count))) | set(range(max(0, count - case["last"]), count))
        w = acc[b].tolist()
        rest = sorted((j for j in range(count) if j not in held), key=lambda j: (-w[j], j))
        kept.append(sorted((list(held) + rest)[:n] if count > n else range(count)))

    def rows(x, out):
        if not x.is_floating_point():
            return None
        out = out.double()
        for b, ids in enumerate(kept):
            out[b, :len(ids)] = x[b, torch.tensor(ids, device="cuda")].double()
        return out

    got = dict(keep=None, acc=rows(s["acc"], s["acc_out"]))
    for x in names:
        if s[x] is not None:
            got[x] = tuple(map(rows, s[x], s[x + "_out"])) if case["bits"] == 4 else rows(s[x], s[x + "_out"])
    return got
