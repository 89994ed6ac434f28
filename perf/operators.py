"""Decode-side operators around the quantised products: what a 7B-shaped decoder needs between its projections
once the prompt is in the cache.  Cases, inputs, a plain torch form, the library's calls and 64-bit values.

  rope     rotary positions on the q and k projections' f32 rows; k and v go into the paged cache
  attn     attention of the newest token(s) of every sequence over the paged cache, optionally adding each
           entry's attention weight to the cache's running total
  evict    eviction down to a budget: the newest entries and those of the largest accumulated weight stay
  verify   drafted tokens against the target's probabilities, from given uniform numbers
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    """Head layouts: 32 heads of 128 are the repository's 7B shape (4096 wide); 32 over 8 is the same with shared key heads."""
    return [
        # one token of one sequence, the smallest launch of a decode step
        dict(name="rope_token", op="rope", seqs=1, new=1, ragged=False, q_heads=32, kv_heads=32, dim=128, rot=128,
             interleaved=False, scaling="none", dtype="f16", page=16, length=513, layout="hnd"),
        # a prompt chunk with shared key heads, half of each head rotated, frequencies stretched for a long context
        dict(name="rope_chunk_shared", op="rope", seqs=1, new=512, ragged=False, q_heads=32, kv_heads=8, dim=128, rot=64,
             interleaved=True, scaling="by_parts", dtype="bf16", page=64, length=33000, layout="nhd"),
        # a long prompt of the 7B shape
        dict(name="rope_prompt", op="rope", seqs=1, new=4096, ragged=False, q_heads=32, kv_heads=32, dim=128, rot=128,
             interleaved=False, scaling="linear", dtype="f16", page=16, length=4096, layout="hnd"),
        # one sequence at an odd short length: latency counts
        dict(name="attn_token", op="attn", seqs=1, new=1, ragged=False, q_heads=32, kv_heads=32, dim=128, dtype="f16",
             page=16, length=513, layout="hnd", accumulate=False),
        # the ordinary batch of the 7B shape, lengths of all sizes, with the weights that eviction goes by
        dict(name="attn_batch_weights", op="attn", seqs=8, new=1, ragged=True, q_heads=32, kv_heads=32, dim=128,
             dtype="f16", page=16, length=4096, layout="hnd", accumulate=True),
        # a serving batch with shared key heads and long contexts, ragged
        dict(name="attn_serving", op="attn", seqs=16, new=1, ragged=True, q_heads=32, kv_heads=8, dim=128, dtype="bf16",
             page=64, length=32768, layout="hnd", accumulate=False),
        # one very long context: work has to be split over its length
        dict(name="attn_long", op="attn", seqs=1, new=1, ragged=False, q_heads=32, kv_heads=8, dim=128, dtype="f16",
             page=64, length=131071, layout="nhd", accumulate=False),
        # drafted tokens scored together: five new tokens a sequence, causal among themselves, heads of 64
        dict(name="attn_drafts", op="attn", seqs=8, new=5, ragged=True, q_heads=32, kv_heads=8, dim=64, dtype="bf16",
             page=24, length=4099, layout="hnd", accumulate=False),
        # a single sequence that has run a little past its budget
        dict(name="evict_one", op="evict", seqs=1, kv_heads=32, dim=128, dtype="f16", page=16, length=1100, ragged=False,
             budget=1024, recent=256, layout="hnd"),
        # a batch cut down to an eighth after long prompts
        dict(name="evict_batch", op="evict", seqs=16, kv_heads=8, dim=128, dtype="bf16", page=64, length=32768, ragged=True,
             budget=4096, recent=1024, layout="hnd"),
        # three drafted tokens of one sequence
        dict(name="verify_one", op="verify", seqs=1, drafts=3, vocab=32000, dtype="f32", ragged=False),
        # a batch with a wide odd vocabulary and half-size probabilities
        dict(name="verify_batch", op="verify", seqs=64, drafts=7, vocab=128001, dtype="bf16", ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "evict", "verify"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 32])
    share = dict(kv_heads=kv_heads, dim=rng.choice([64, 80, 128, 128, 192, 256]), dtype=rng.choice(["f16", "bf16"]),
                 page=rng.choice([16, 24, 32, 64, 100, 128]), layout=rng.choice(["hnd", "nhd"]))
    per_entry = kv_heads * share["dim"]
    if op == "rope":
        new = _log(rng, 1, 4096)
        seqs = _log(rng, 1, max(1, min(64, 4096 // new)))
        q_heads = kv_heads * rng.choice([1, 2, 4] if kv_heads < 32 else [1])
        while seqs * new * (q_heads + 2 * kv_heads) * share["dim"] > 4096 * 96 * 128:
            new = max(1, new // 2)
        rot = rng.choice([share["dim"], share["dim"] // 2])
        return dict(op=op, seqs=seqs, new=new, ragged=rng.random() < 0.5, q_heads=q_heads, rot=rot,
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "by_parts"]),
                    length=new + _log(rng, 1, 8192), **share)
    if op == "verify":
        return dict(op=op, seqs=_log(rng, 1, 64), drafts=rng.randint(1, 7), vocab=_log(rng, 300, 128001),
                    dtype=rng.choice(["f32", "f16", "bf16"]), ragged=rng.random() < 0.5)
    length = _log(rng, 1, 131072) if op == "attn" else _log(rng, 64, 65536)
    seqs = _log(rng, 1, 64)
    while seqs > 1 and seqs * length * per_entry > 16 * 32768 * 8 * 128:
        seqs = max(1, seqs // 2)
    while seqs * length * per_entry > 16 * 32768 * 8 * 128:
        length = length // 2 + 1
    if op == "attn":
        group = rng.choice([1, 2, 3, 4, 8])
        new = rng.choice([1, 1, 1, 2, 4, 6])
        return dict(op=op, seqs=seqs, new=min(new, length), ragged=rng.random() < 0.7, q_heads=kv_heads * group, length=length,
                    accumulate=rng.random() < 0.4, **share)
    budget = _log(rng, 16, length)
    return dict(op=op, seqs=seqs, length=length, ragged=rng.random() < 0.7, budget=budget, recent=rng.randint(0, budget // 2), **share)


def _frequencies(rot, scaling):
    """Radians per position of every rotated pair, in 64 bits: base 10000; "linear" divides positions by 4;
    "by_parts" stretches by 8 the pairs that turn less than once over 4096 positions, keeps those that turn more
    than 32 times, blends between, and scales the rotated part by 0.1 ln 8 + 1."""
    inv = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [f / 4.0 for f in inv], 1.0
    if scaling == "by_parts":
        out = []
        for f in inv:
            keep = min(1.0, max(0.0, (4096 * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)))
            out.append(f * keep + f / 8.0 * (1 - keep))
        return out, 0.1 * math.log(8.0) + 1.0
    return inv, 1.0


def _fixed(inv):
    """Turns per position as 64-bit fractions, so that position x frequency wraps exactly."""
    return torch.tensor([((int(f / (2 * math.pi) * 2.0 ** 64) + (1 << 63)) % (1 << 64)) - (1 << 63) for f in inv], dtype=torch.int64)


def _pool(case, g, dev):
    """k, v [pages][heads][page][dim] (a view of the other order for "nhd"), a shuffled page table, lengths."""
    B, H, ps, D = case["seqs"], case["kv_heads"], case["page"], case["dim"]
    new = case.get("new", 0)
    cols = -(-(case["length"] + new) // ps)
    pages = B * cols
    dt = DTYPES[case["dtype"]]
    shape = (pages, H, ps, D) if case["layout"] == "hnd" else (pages, ps, H, D)
    k, v = (torch.randn(shape, generator=g, device=dev, dtype=dt) for _ in range(2))
    if case["layout"] == "nhd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(B, cols)
    lens = torch.full((B,), case["length"], dtype=torch.int32, device=dev)
    if case["ragged"] and B > 1:
        lo = max(1, new, case["length"] // 8)
        r = torch.randint(lo, case["length"] + 1, (B - 1,), generator=g, device=dev, dtype=torch.int32)
        lens[1:] = r
    return k, v, table.contiguous(), lens


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case=case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def counts(B, N):
        """How many of its N new tokens each sequence has: the first all of them, another perhaps none."""
        n = torch.randint(0, N + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        n[0] = N
        return n

    if case["op"] == "verify":
        B, N, V = case["seqs"], case["drafts"], case["vocab"]
        logits = normal(B, N + 1, V) * 2.5
        s["target"] = torch.softmax(logits, -1).to(DTYPES[case["dtype"]])
        draft = torch.softmax(logits[:, :N] + 0.7 * normal(B, N, V), -1)
        s["tokens"] = torch.multinomial(draft.view(B * N, V), 1, generator=g).view(B, N).to(torch.int32)
        s["draft"] = draft.to(DTYPES[case["dtype"]])
        s["uniform"] = torch.rand((B, N + 1), generator=g, device=dev)
        s["count"] = counts(B, N) if case["ragged"] else None
        return s

    B, H, D = case["seqs"], case["kv_heads"], case["dim"]
    s["k"], s["v"], s["table"], s["lens"] = _pool(case, g, dev)
    pages, ps = s["k"].shape[0], case["page"]
    s["weight"] = s["pos"] = None
    if case["op"] in ("rope", "attn"):
        N, Hq = case["new"], case["q_heads"]
        s["new"] = counts(B, N) if case["ragged"] and N > 1 else None
    if case["op"] == "rope":
        # one row of the q, k and v projections side by side, as a product over their concatenated rows leaves it
        row = normal(B * N, (Hq + 2 * H) * D)
        s["q"] = row[:, :Hq * D].view(B * N, Hq, D)
        s["k_new"] = row[:, Hq * D:(Hq + H) * D].view(B * N, H, D)
        s["v_new"] = row[:, (Hq + H) * D:].view(B * N, H, D)
        n = s["new"] if s["new"] is not None else N
        s["at"] = ((s["lens"] - n)[:, None] + torch.arange(N, device=dev, dtype=torch.int32)).reshape(-1).to(torch.int32)
        s["weight"] = normal(pages, H, ps).abs()
        s["pos"] = torch.zeros((pages, H, ps), dtype=torch.int32, device=dev)
        inv, s["magnitude"] = _frequencies(case["rot"], case["scaling"])
        s["freq"] = _fixed(inv).to(dev)
    elif case["op"] == "attn":
        s["q"] = 1.5 * normal(B * N, Hq, D)
        if case["accumulate"]:
            s["weight"] = torch.zeros((pages, H, ps), device=dev)
    else:
        # accumulated attention is heavy-tailed; positions count up along the cache
        s["weight"] = torch.exp(1.5 * normal(pages, H, ps))
        slot = torch.arange(s["table"].shape[1] * ps, device=dev, dtype=torch.int32)
        s["pos"] = torch.zeros((pages, H, ps), dtype=torch.int32, device=dev)
        s["pos"][s["table"].long()] = slot.view(-1, 1, ps).expand(-1, H, ps)
        s["keep_from"] = s["lens"] - case["recent"]
        s["weight_out"] = torch.zeros_like(s["weight"])
        s["pos_out"] = torch.zeros_like(s["pos"])
    if own:
        from quantized_prefill_gemm_mmq_gb300 import ops
        s["cache"] = ops.KVCache(s["k"], s["v"], s["table"], s["lens"], weight=s["weight"], pos=s["pos"])
        if case["op"] == "rope":
            s["rope"] = ops.rope_table(case["rot"], base=10000.0, scaling=case["scaling"], device=dev,
                                       factor={"none": 1.0, "linear": 4.0, "by_parts": 8.0}[case["scaling"]], context=4096)
        elif case["op"] == "attn":
            s["workspace"] = ops.attn_workspace(s["cache"], case["q_heads"], case["new"], accumulate=case["accumulate"])
        else:
            s["workspace"] = ops.evict_workspace(s["cache"], case["budget"])
    return s


# ------------------------------------------------------------------ one pass ---

def run(s):
    return (_run_own if own else _PLAIN[s["case"]["op"]])(s)


def _run_own(s):
    from quantized_prefill_gemm_mmq_gb300 import ops
    case = s["case"]
    if case["op"] == "verify":
        tokens, accepted = ops.spec_verify(s["target"], s["draft"], s["tokens"], s["uniform"], count=s["count"])
        return {"tokens": tokens, "accepted": accepted}
    cache = s["cache"]
    if case["op"] == "rope":
        q = ops.rope_append(cache, s["rope"], s["q"], s["k_new"], s["v_new"], s["at"], interleaved=case["interleaved"], new=s["new"])
        return {"q": q, "k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"]}
    if case["op"] == "attn":
        out = ops.attn_decode(cache, s["q"], new=s["new"], accumulate=case["accumulate"], workspace=s["workspace"])
        return {"out": out, "weight": s["weight"]} if case["accumulate"] else {"out": out}
    ops.kv_evict(cache, case["budget"], s["keep_from"], s["weight_out"], s["pos_out"], workspace=s["workspace"])
    return {"k": s["k"], "v": s["v"], "weight": s["weight_out"], "pos": s["pos_out"]}


def _places(s, slots):
    """Page and offset of slots [B][n] of every sequence."""
    ps = s["case"]["page"]
    return torch.gather(s["table"].long(), 1, slots // ps), slots % ps


def _rotate(x, c, sn, rot, interleaved):
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * c - b * sn, a * sn + b * c), -1)
    return torch.cat((r, rest), -1)


def _plain_rope(s):
    case = s["case"]
    B, N, H, D = case["seqs"], case["new"], case["kv_heads"], case["dim"]
    dev, dt = s["q"].device, s["k"].dtype
    turns = ((s["at"].long()[:, None] * s["freq"][None]) >> 32).float() * 2.0 ** -32
    c = (torch.cos(turns * (2 * math.pi)) * s["magnitude"])[:, None]
    sn = (torch.sin(turns * (2 * math.pi)) * s["magnitude"])[:, None]
    n = torch.full((B,), N, device=dev) if s["new"] is None else s["new"].long()
    live = torch.arange(N, device=dev)[None] < n[:, None]
    q = _rotate(s["q"], c, sn, case["rot"], case["interleaved"])
    q = torch.where(live.view(-1, 1, 1), q, torch.zeros((), device=dev))
    k = _rotate(s["k_new"], c, sn, case["rot"], case["interleaved"]).to(dt).view(B, N, H, D)
    v = s["v_new"].to(dt).view(B, N, H, D)
    page, off = _places(s, (s["lens"].long() - n)[:, None] + torch.arange(N, device=dev))
    keep = live[..., None, None]
    s["k"][page, :, off] = torch.where(keep, k, s["k"][page, :, off])
    s["v"][page, :, off] = torch.where(keep, v, s["v"][page, :, off])
    s["weight"][page, :, off] = torch.where(live[..., None], torch.zeros((), device=dev), s["weight"][page, :, off])
    s["pos"][page, :, off] = torch.where(live[..., None], s["at"].view(B, N, 1), s["pos"][page, :, off])
    return {"q": q, "k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"]}


def _plain_attn(s):
    case = s["case"]
    B, N, H, D, L = case["seqs"], case["new"], case["kv_heads"], case["dim"], case["length"]
    G, dev = case["q_heads"] // H, s["q"].device
    slots = torch.arange(L, device=dev)[None].expand(B, L)
    page, off = _places(s, slots)
    lens = s["lens"].long()
    n = torch.full((B,), N, device=dev) if s["new"] is None else s["new"].long()
    t = torch.arange(N, device=dev)[None]
    limit = torch.where(t < n[:, None], lens[:, None] - n[:, None] + t + 1, torch.zeros((), dtype=torch.int64, device=dev))
    seen = (slots[:, None, :] < limit[:, :, None])[:, None, None]                       # [B][1][1][N][L]
    k = s["k"][page, :, off].permute(0, 2, 3, 1).float()                                # [B][H][D][L]
    q = s["q"].view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    sc = (torch.matmul(q, k) * D ** -0.5).view(B, H, G, N, L)
    sc = torch.where(seen, sc, torch.full((), -math.inf, device=dev))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros((), device=dev))
    p = torch.exp(sc - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros((), device=dev))
    v = s["v"][page, :, off].permute(0, 2, 1, 3).float()                                # [B][H][L][D]
    out = torch.matmul(p.view(B, H, G * N, L), v)
    out = out.view(B, H, G, N, D).permute(0, 3, 1, 2, 4).reshape(B * N, H * G, D)
    if not case["accumulate"]:
        return {"out": out}
    s["weight"][page, :, off] = s["weight"][page, :, off] + p.sum((2, 3)).permute(0, 2, 1)
    return {"out": out, "weight": s["weight"]}


def _plain_evict(s):
    case = s["case"]
    B, H, L, budget = case["seqs"], case["kv_heads"], case["length"], case["budget"]
    dev = s["k"].device
    slots = torch.arange(L, device=dev)[None].expand(B, L)
    page, off = _places(s, slots)
    lens = s["lens"].long()[:, None, None]
    w, pos = s["weight"][page, :, off].permute(0, 2, 1), s["pos"][page, :, off].permute(0, 2, 1)  # [B][H][L]
    at = slots[:, None]
    key = torch.where(pos >= s["keep_from"][:, None, None], torch.full((), math.inf, device=dev), w)
    key = torch.where(at < lens, key, torch.full((), -math.inf, device=dev))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, at.expand(B, H, L))
    keep = (rank < budget) & (at < lens)
    hole, mover = ~keep & (at < budget) & (at < lens), keep & (at >= budget)
    nth = torch.where(mover, mover.long().cumsum(-1) - 1, torch.full((), L, device=dev))
    source = torch.zeros((B, H, L + 1), dtype=torch.int64, device=dev).scatter_(2, nth, at.expand(B, H, L))
    source = torch.where(hole, torch.gather(source, 2, (hole.long().cumsum(-1) - 1).clamp(min=0)), at)
    M = min(budget, L)
    source = source[..., :M]                                                           # [B][H][M]: where slot m comes from
    head = torch.arange(H, device=dev)[None, :, None]
    src_page = torch.gather(page[:, None].expand(B, H, L), 2, source)
    src_off = torch.gather(off[:, None].expand(B, H, L), 2, source)
    dst_page, dst_off = page[:, None, :M], off[:, None, :M]
    k, v = s["k"][src_page, head, src_off], s["v"][src_page, head, src_off]
    s["k"][dst_page, head, dst_off] = k
    s["v"][dst_page, head, dst_off] = v
    there = at[..., :M] < lens
    s["weight_out"][dst_page, head, dst_off] = torch.where(there, s["weight"][src_page, head, src_off], s["weight_out"][dst_page, head, dst_off])
    s["pos_out"][dst_page, head, dst_off] = torch.where(there, s["pos"][src_page, head, src_off], s["pos_out"][dst_page, head, dst_off])
    return {"k": s["k"], "v": s["v"], "weight": s["weight_out"], "pos": s["pos_out"]}


def _plain_verify(s):
    case = s["case"]
    B, N, V = case["seqs"], case["drafts"], case["vocab"]
    dev = s["target"].device
    n = torch.full((B,), N, device=dev) if s["count"] is None else s["count"].long()
    i = torch.arange(N, device=dev)[None]
    tok = s["tokens"].long()
    p = torch.gather(s["target"][:, :N], 2, tok[..., None])[..., 0].float()
    q = torch.gather(s["draft"], 2, tok[..., None])[..., 0].float()
    ok = (s["uniform"][:, :N] * q < p) & (i < n[:, None])
    accepted = ok.long().cumprod(1).sum(1)
    row = s["target"][torch.arange(B, device=dev), accepted].float()
    minus = s["draft"][torch.arange(B, device=dev), accepted.clamp(max=N - 1)].float()
    rest = torch.where((accepted < n)[:, None], (row - minus).clamp(min=0), row)
    fixed = torch.round(rest * 2.0 ** 40).long()
    # where rounding leaves nothing of the difference, the target itself
    fixed = torch.where(fixed.sum(1, keepdim=True) > 0, fixed, torch.round(row * 2.0 ** 40).long())
    cum = fixed.cumsum(1)
    u = (s["uniform"][:, N] * 2.0 ** 24).long()
    total = cum[:, -1]
    r = (total >> 24) * u + (((total & 0xFFFFFF) * u) >> 24)
    last = (cum > r[:, None]).long().argmax(1)
    out = torch.where(i < accepted[:, None], tok, torch.full((), -1, device=dev))
    out = torch.cat((out, torch.full((B, 1), -1, device=dev)), 1)
    out = out.scatter(1, accepted[:, None], last[:, None])
    return {"tokens": out.to(torch.int32), "accepted": accepted.to(torch.int32)}


_PLAIN = {"rope": _plain_rope, "attn": _plain_attn, "evict": _plain_evict, "verify": _plain_verify}


# ---------------------------------------------------------------------- work ---

def _entries(case):
    """Expected entries over all sequences: the first has `length`, the others lie evenly between an eighth of it and all of it."""
    return case["length"] * (1 + (case["seqs"] - 1) * ((1 + 1 / 8) / 2 if case["ragged"] else 1))


def work(case):
    op = case["op"]
    if op == "verify":
        size = 4 if case["dtype"] == "f32" else 2
        rows = case["seqs"] * 1.75            # the target's row, and the draft's where a token was turned down
        return {"bytes": rows * case["vocab"] * size, "flops": 3 * case["seqs"] * case["vocab"]}
    H, D = case["kv_heads"], case["dim"]
    if op == "rope":
        T = case["seqs"] * case["new"] * (0.5 if case["ragged"] and case["new"] > 1 else 1)
        return {"bytes": T * D * (8 * case["q_heads"] + 12 * H), "flops": 3 * T * case["rot"] * (case["q_heads"] + H)}
    e = _entries(case)
    if op == "attn":
        rows = case["q_heads"] // H * case["new"] * (0.5 if case["ragged"] and case["new"] > 1 else 1)
        return {"bytes": e * H * (4 * D + (8 if case["accumulate"] else 0)) + case["seqs"] * case["new"] * case["q_heads"] * D * 8,
                "flops": 4 * e * H * rows * D}
    L, b, r = case["length"], min(case["budget"], case["length"]), case["recent"]
    moved = 0.0
    if L > b:                                  # newest entries past the budget, and the heavy ones among the rest there
        past = min(r, L - b)
        moved = past + max(0, b - r) / max(1, L - r) * (L - b - past)
    return {"bytes": e * H * 8 + case["seqs"] * H * (b * 8 + moved * 8 * D), "flops": e * H}


# --------------------------------------------------------------- in 64 bits ---

def exact(case, seed):
    if case["op"] == "verify":
        return None                            # whole numbers, the same whatever the order of sums
    s = prepare(case, seed)
    B, H, D, ps = case["seqs"], case["kv_heads"], case["dim"], case["page"]
    table, lens = s["table"].tolist(), s["lens"].tolist()
    if case["op"] == "evict":
        if s["k"].numel() > 1 << 26:
            return None
        k, v = s["k"].double(), s["v"].double()
        w, pos = s["weight"].double(), s["pos"]
        w_out = torch.zeros_like(w)
        pos_all, keep_from = pos.cpu(), s["keep_from"].tolist()
        for b in range(B):
            pages = torch.tensor(table[b])
            for h in range(H):
                n = lens[b]
                keys = w[pages, h].reshape(-1)[:n].tolist()
                where = pos_all[pages, h].reshape(-1)[:n].tolist()
                first = sorted(range(n), key=lambda j: (-(math.inf if where[j] >= keep_from[b] else keys[j]), j))[:case["budget"]]
                stay = set(first)
                m = min(n, case["budget"])
                holes = [j for j in range(m) if j not in stay]
                movers = [j for j in sorted(stay) if j >= m]
                src = list(range(m))
                for d, j in zip(holes, movers):
                    src[d] = j
                sp, so = [table[b][j // ps] for j in src], [j % ps for j in src]
                dp, do = [table[b][j // ps] for j in range(m)], [j % ps for j in range(m)]
                k[dp, h, do], v[dp, h, do] = k[sp, h, so], v[sp, h, so]
                w_out[dp, h, do] = w[sp, h, so]
        return {"k": k, "v": v, "weight": w_out, "pos": None}
    N, Hq = case["new"], case["q_heads"]
    new = [N] * B if s["new"] is None else s["new"].tolist()
    if case["op"] == "rope":
        inv, magnitude = _frequencies(case["rot"], case["scaling"])
        angle = s["at"].double()[:, None] * torch.tensor(inv, dtype=torch.float64, device="cuda")
        unit = torch.polar(torch.full_like(angle, magnitude), angle)[:, None]

        def turn(x):
            x = x.double().clone()
            half = case["rot"] // 2
            i = torch.arange(half, device="cuda")
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            z = torch.complex(x[..., a], x[..., b]) * unit
            x[..., a], x[..., b] = z.real, z.imag
            return x

        q, kr, k, v, w = turn(s["q"]), turn(s["k_new"]), s["k"].double(), s["v"].double(), s["weight"].double()
        for b in range(B):
            q[b * N + new[b]:(b + 1) * N] = 0
            j = list(range(lens[b] - new[b], lens[b]))
            pg, of = [table[b][x // ps] for x in j], [x % ps for x in j]
            rows = slice(b * N, b * N + new[b])
            if j:
                k[pg, :, of], v[pg, :, of], w[pg, :, of] = kr[rows], s["v_new"][rows].double(), 0.0
        return {"q": q, "k": k, "v": v, "weight": w, "pos": None}
    G = Hq // H
    out = torch.zeros((B * N, Hq, D), dtype=torch.float64, device="cuda")
    w = s["weight"].double() if case["accumulate"] else None
    for b in range(B):
        pages = torch.tensor(table[b][:-(-lens[b] // ps)], device="cuda")
        for h in range(H):
            k = s["k"][pages, h].reshape(-1, D)[:lens[b]].double()
            v = s["v"][pages, h].reshape(-1, D)[:lens[b]].double()
            total = torch.zeros(lens[b], dtype=torch.float64, device="cuda")
            for t in range(new[b]):
                m = lens[b] - new[b] + t + 1
                if m < 1:
                    continue
                rows = s["q"][b * N + t, h * G:(h + 1) * G].double()
                p = torch.softmax(rows @ k[:m].T / math.sqrt(D), -1)
                out[b * N + t, h * G:(h + 1) * G] = p @ v[:m]
                total[:m] += p.sum(0)
            if w is not None:
                flat = torch.zeros(len(pages) * ps, dtype=torch.float64, device="cuda")
                flat[:lens[b]] = total
                w[pages, h] += flat.view(-1, ps)
    return {"out": out, "weight": w} if w is not None else {"out": out}
