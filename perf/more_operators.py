"""Operators around the paged cache that prompts and trees of drafts need: cases, inputs, a plain torch form, the library's
calls and 64-bit values.

  norm     per-head norms of the q and k projections' f32 rows with rotary positions (one or several axes) in the same
           pass; k and v go into the paged cache, q comes out in f32 or the cache's type
  prefill  attention of any number of new tokens per sequence over the paged cache, with scores capped by a tanh, a bias
           that grows with the distance, a window, a prefix that sees itself whole, packed documents
  tree     attention of a tree of drafted tokens: every node sees the context and its own ancestors
  keep     the accepted path of a tree moves to the front of the tree's entries
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    """Head layouts: 32 heads of 128 are the repository's 7B shape (4096 wide); 32 over 8 is the same with shared key heads."""
    return [
        # one token of one sequence, the smallest launch of a decode step; f32 q for the decode attention
        dict(name="norm_token", op="norm", seqs=1, new=1, ragged=False, q_heads=32, kv_heads=8, dim=128, rot=128, axes=1,
             interleaved=False, q_out="f32", dtype="f16", page=16, length=513, layout="hnd"),
        # a prompt with an image in it: time, height and width positions, shared key heads
        dict(name="norm_image", op="norm", seqs=1, new=1000, ragged=False, q_heads=32, kv_heads=8, dim=128, rot=128, axes=3,
             interleaved=False, q_out="bf16", dtype="bf16", page=64, length=5000, layout="nhd"),
        # a long prompt of the 7B shape
        dict(name="norm_prompt", op="norm", seqs=1, new=4096, ragged=False, q_heads=32, kv_heads=32, dim=128, rot=128, axes=1,
             interleaved=False, q_out="f16", dtype="f16", page=16, length=4096, layout="hnd"),
        # one token with capped scores at an odd short length: latency counts
        dict(name="prefill_token_cap", op="prefill", seqs=1, new=1, ragged=False, q_heads=32, kv_heads=32, dim=128, dtype="f16",
             page=16, length=513, layout="hnd", cap=30.0, slopes=False, window=0, prefix=False, docs=0, out="f16"),
        # a small ragged batch of heads of 80 with distance bias, pages that end inside every tile
        dict(name="prefill_ragged_bias", op="prefill", seqs=8, new=300, ragged=True, q_heads=32, kv_heads=32, dim=80, dtype="f16",
             page=24, length=1100, layout="hnd", cap=0.0, slopes=True, window=0, prefix=False, docs=0, out="f16"),
        # the ordinary prompt of the 7B shape; what stands before the answer sees itself whole
        dict(name="prefill_prompt_prefix", op="prefill", seqs=1, new=4096, ragged=False, q_heads=32, kv_heads=32, dim=128,
             dtype="f16", page=16, length=4096, layout="hnd", cap=0.0, slopes=False, window=0, prefix=True, docs=0, out="f16"),
        # a chunk of a long prompt in a layer with a sliding window
        dict(name="prefill_chunk_window", op="prefill", seqs=1, new=2048, ragged=False, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", page=64, length=32768, layout="nhd", cap=0.0, slopes=False, window=8192, prefix=False, docs=0, out="bf16"),
        # packed documents of a scoring run, capped scores: the largest call
        dict(name="prefill_documents_cap", op="prefill", seqs=1, new=8192, ragged=False, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", page=64, length=8192, layout="hnd", cap=30.0, slopes=False, window=0, prefix=False, docs=3, out="bf16"),
        # a tree of sixteen drafts of one sequence
        dict(name="tree_one", op="tree", seqs=1, new=16, ragged=False, q_heads=32, kv_heads=32, dim=128, dtype="f16", page=16,
             length=4099, layout="hnd", cap=0.0, out="f16"),
        # a serving batch with shared key heads: trees of up to 48 nodes over long ragged contexts
        dict(name="tree_batch", op="tree", seqs=16, new=48, ragged=True, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=64,
             length=16384, layout="hnd", cap=0.0, out="bf16"),
        # the path that one sequence's tree leaves
        dict(name="keep_one", op="keep", seqs=1, new=16, q_heads=32, kv_heads=32, dim=128, dtype="f16", page=16, length=1100,
             layout="hnd"),
        # the paths of a batch, key heads shared
        dict(name="keep_batch", op="keep", seqs=64, new=48, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=64, length=1100,
             layout="nhd"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


PAIRS = 8192 * 8192 * 32 * 128           # query row x entry x head value of the largest listed attention
POOL = 1 << 27                           # values of k in a drawn cache


def draw(rng):
    op = rng.choice(["norm", "prefill", "prefill", "prefill", "tree", "tree", "keep"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 32])
    group = rng.choice([1, 2, 3, 4, 8]) if kv_heads < 32 else 1
    c = dict(op=op, q_heads=kv_heads * group, kv_heads=kv_heads, dim=rng.choice([64, 72, 80, 96, 128, 128, 128, 192, 256]),
             dtype=rng.choice(["f16", "bf16"]), page=rng.choice([7, 16, 24, 32, 64, 100, 128]), layout=rng.choice(["hnd", "nhd"]))
    ragged = rng.random() < 0.6
    if op == "norm":
        new = _log(rng, 1, 4096)
        seqs = _log(rng, 1, max(1, min(64, 4096 // new)))
        while seqs * new * (c["q_heads"] + 2 * kv_heads) * c["dim"] > 4096 * 96 * 128:
            new = max(1, new // 2)
        return dict(seqs=seqs, new=new, ragged=ragged, rot=rng.choice([c["dim"], c["dim"] // 2]), axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.4, q_out=rng.choice(["f32", c["dtype"]]), length=new + _log(rng, 1, 4096), **c)
    if op == "keep":
        seqs, length = _log(rng, 1, 64), _log(rng, 64, 4000)
        while seqs > 1 and seqs * length * kv_heads * c["dim"] > POOL // 2:
            seqs = seqs // 2
        return dict(seqs=seqs, new=rng.randint(1, 64), length=length, **c)
    c["cap"] = rng.choice([0.0, 0.0, 30.0])
    c["out"] = c["dtype"]
    seqs = _log(rng, 1, 32)
    if op == "tree":
        new, length = rng.randint(1, 64), _log(rng, 64, 65536)
    else:
        new = rng.choice([1, _log(rng, 1, 8192), _log(rng, 1, 8192)])
        length = new + rng.choice([0, _log(rng, 1, 32768)])
    while seqs > 1 and (seqs * length * kv_heads * c["dim"] > POOL or seqs * new * length * c["q_heads"] * 128 > PAIRS // 2):
        seqs = seqs // 2
    while seqs * length * kv_heads * c["dim"] > POOL or seqs * new * length * c["q_heads"] * max(128, c["dim"]) > PAIRS // 2:
        length = max(new, length // 2)
        if length == new and op == "prefill":
            new = length = max(1, new * 3 // 4)
    if op == "tree":
        return dict(seqs=seqs, new=new, ragged=ragged, length=max(length, new), **c)
    return dict(seqs=seqs, new=new, ragged=ragged, length=length, slopes=rng.random() < 0.3, prefix=rng.random() < 0.3,
                window=rng.choice([0, 0, _log(rng, 1, length)]), docs=rng.choice([0, 0, rng.randint(2, 9)]), **c)


# -------------------------------------------------------------------- inputs ---

def _pool(case, g, dev, lens):
    """k, v [pages][heads][page][dim] (a view of the other order for "nhd") and a shuffled page table."""
    B, H, ps, D = case["seqs"], case["kv_heads"], case["page"], case["dim"]
    cols = -(-case["length"] // ps)
    pages = B * cols
    dt = DTYPES[case["dtype"]]
    shape = (pages, H, ps, D) if case["layout"] == "hnd" else (pages, ps, H, D)
    k, v = (torch.randn(shape, generator=g, device=dev, dtype=dt) for _ in range(2))
    if case["layout"] == "nhd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return k, v, torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(B, cols).contiguous()


def _inverse(rot):
    """Radians per position of every rotated pair, base 10000."""
    return [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]


def _fixed(inv):
    """Turns per position as 64-bit fractions, so that position x frequency wraps exactly."""
    return torch.tensor([((int(f / (2 * math.pi) * 2.0 ** 64) + (1 << 63)) % (1 << 64)) - (1 << 63) for f in inv], dtype=torch.int64)


def _sections(rot, axes):
    """How many pairs turn by each axis, one block of pairs after the other: a quarter for time, the rest shared."""
    n = rot // 2
    if axes == 1:
        return [n]
    first = max(1, n // 4) if axes == 3 else n // 2
    rest = (n - first) // (axes - 1)
    return [first] + [rest] * (axes - 2) + [n - first - rest * (axes - 2)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case=case)
    op, B, N, H, D, Hq, L = (case[n] for n in ("op", "seqs", "new", "kv_heads", "dim", "q_heads", "length"))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev, dtype=torch.int32)

    def ancestors(parent):
        """Words [B][N]: bit j of word t says that node t sees node j; a node's parent is an earlier one (or none, -1)."""
        words = torch.zeros((B, N), dtype=torch.int64, device=dev)
        for t in range(N):
            p = parent[:, t]
            up = torch.gather(words, 1, p.clamp(min=0)[:, None])[:, 0]
            words[:, t] = torch.where(p >= 0, up, torch.zeros_like(up)) | ((1 << t) if t < 63 else -(1 << 63))
        return words

    # the first sequence has all of the length and of the new tokens, another perhaps none of these
    lens = torch.full((B,), L, dtype=torch.int32, device=dev)
    s["new"] = None
    if case.get("ragged") and N > 1:
        s["new"] = whole(0, N + 1, B)
        s["new"][0] = N
    if case.get("ragged") and B > 1:
        lens[1:] = torch.maximum(whole(max(1, L // 8), L + 1, B - 1), s["new"][1:] if s["new"] is not None else torch.full_like(lens[1:], N))
    s["lens"] = lens
    s["k"], s["v"], s["table"] = _pool(case, g, dev, lens)
    pages, ps = s["k"].shape[0], case["page"]
    s["weight"] = s["pos"] = None
    n = s["new"] if s["new"] is not None else torch.full_like(lens, N)
    at = ((lens - n)[:, None] + torch.arange(N, device=dev, dtype=torch.int32)).to(torch.int32)     # [B][N] slots of the new tokens
    if op == "norm":
        # one row of the q, k and v projections side by side, as a product over their concatenated rows leaves it
        row = normal(B * N, (Hq + 2 * H) * D) * torch.exp(0.5 * normal(B * N, 1))
        s["q"] = row[:, :Hq * D].view(B * N, Hq, D)
        s["k_new"] = row[:, Hq * D:(Hq + H) * D].view(B * N, H, D)
        s["v_new"] = row[:, (Hq + H) * D:].view(B * N, H, D)
        s["q_norm"], s["k_norm"] = 1.0 + 0.3 * normal(D), 1.0 + 0.3 * normal(D)
        s["at"] = torch.stack([at.reshape(-1)] + [whole(0, 200, B * N) for _ in range(case["axes"] - 1)]).contiguous()
        s["weight"] = normal(pages, H, ps).abs()
        s["pos"] = torch.zeros((pages, H, ps), dtype=torch.int32, device=dev)
        s["freq"] = _fixed(_inverse(case["rot"])).to(dev)
        s["axis"] = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(_sections(case["rot"], case["axes"]))).to(torch.int32).to(dev)
    elif op == "prefill":
        s["q"] = ((3.0 if case["cap"] else 1.5) * normal(B * N, Hq, D)).to(DTYPES[case["dtype"]])
        # eight heads' worth of halving slopes, repeated down to 2^-8
        s["slopes"] = torch.exp2(-8.0 * (torch.arange(Hq, device=dev) + 1) / Hq) if case["slopes"] else None
        # the prefix ends somewhere in the new tokens of most sequences
        s["prefix"] = (lens - n + (torch.rand((B,), generator=g, device=dev) * 0.5 * n).to(torch.int32)).to(torch.int32) if case["prefix"] else None
        s["first"] = None
        if case["docs"]:
            cuts = (torch.rand((B, case["docs"] - 1), generator=g, device=dev) * lens[:, None]).to(torch.int32)
            below = torch.where(cuts[:, None] <= at[:, :, None], cuts[:, None], torch.zeros_like(cuts[:, None]))
            s["first"] = below.amax(-1).reshape(-1).contiguous()
    elif op == "tree":
        s["q"] = ((3.0 if case["cap"] else 1.5) * normal(B * N, Hq, D)).to(DTYPES[case["dtype"]])
        # drafts hang on one of the four nodes before them
        t = torch.arange(N, device=dev)
        parent = torch.where(t[None] > 0, (t[None] - 1 - whole(0, 4, B, N)).clamp(min=0), torch.full((), -1, device=dev))
        s["tree"] = ancestors(parent.long())
    else:
        s["weight"] = normal(pages, H, ps).abs()
        s["pos"] = whole(0, 40000, pages, H, ps)
        # a path: a few of the nodes, in order; its length differs from sequence to sequence
        order = torch.sort(torch.rand((B, N), generator=g, device=dev), dim=1).indices
        most = max(1, min(N, 8))
        s["keep"] = torch.sort(order[:, :most], dim=1).values.to(torch.int32).contiguous()
        s["kept"] = whole(0, most + 1, B)
        s["kept"][0] = most
    if own:
        from quantized_prefill_gemm_mmq_gb300 import ops
        s["cache"] = ops.KVCache(s["k"], s["v"], s["table"], s["lens"], weight=s["weight"], pos=s["pos"])
        if op == "norm":
            s["rope"] = ops.rope_table(case["rot"], base=10000.0, device=dev, sections=_sections(case["rot"], case["axes"]))
        elif op != "keep":
            s["workspace"] = ops.prefill_workspace(s["cache"], Hq, N)
    return s


# ------------------------------------------------------------------ one pass ---

def run(s):
    return (_run_own if own else _PLAIN[s["case"]["op"]])(s)


def _run_own(s):
    from quantized_prefill_gemm_mmq_gb300 import ops
    case, cache = s["case"], s["cache"]
    if case["op"] == "norm":
        q = ops.norm_rope_append(cache, s["rope"], s["q"], s["k_new"], s["v_new"], s["at"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                                 eps=1e-6, interleaved=case["interleaved"], new=s["new"], out_dtype=DTYPES[case["q_out"]])
        return {"q": q, "k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"]}
    if case["op"] == "prefill":
        return {"out": ops.attn_prefill(cache, s["q"], cap=case["cap"], slopes=s["slopes"], window=case["window"], prefix=s["prefix"],
                                        first=s["first"], new=s["new"], out_dtype=DTYPES[case["out"]], workspace=s["workspace"])}
    if case["op"] == "tree":
        return {"out": ops.attn_tree(cache, s["q"], s["tree"], cap=case["cap"], new=s["new"], out_dtype=DTYPES[case["out"]],
                                     workspace=s["workspace"])}
    ops.kv_keep(cache, s["keep"], s["kept"], case["new"])
    return {"k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"]}


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


def _counts(s):
    B, N = s["case"]["seqs"], s["case"]["new"]
    return torch.full((B,), N, device=s["lens"].device) if s["new"] is None else s["new"].long()


def _plain_norm(s):
    case = s["case"]
    B, N, H, D = case["seqs"], case["new"], case["kv_heads"], case["dim"]
    dev, dt = s["q"].device, s["k"].dtype
    pos = s["at"][s["axis"].long()].t().long()                                          # [rows][pairs]
    turns = ((pos * s["freq"][None]) >> 32).float() * 2.0 ** -32
    c, sn = torch.cos(turns * (2 * math.pi))[:, None], torch.sin(turns * (2 * math.pi))[:, None]
    q = s["q"] * torch.rsqrt((s["q"] * s["q"]).mean(-1, keepdim=True) + 1e-6) * s["q_norm"]
    k = s["k_new"] * torch.rsqrt((s["k_new"] * s["k_new"]).mean(-1, keepdim=True) + 1e-6) * s["k_norm"]
    n = _counts(s)
    live = torch.arange(N, device=dev)[None] < n[:, None]
    q = _rotate(q, c, sn, case["rot"], case["interleaved"])
    q = torch.where(live.view(-1, 1, 1), q, torch.zeros((), device=dev)).to(DTYPES[case["q_out"]])
    k = _rotate(k, c, sn, case["rot"], case["interleaved"]).to(dt).view(B, N, H, D)
    v = s["v_new"].to(dt).view(B, N, H, D)
    page, off = _places(s, ((s["lens"].long() - n)[:, None] + torch.arange(N, device=dev)).clamp(max=s["table"].shape[1] * case["page"] - 1))
    b, t = live.nonzero(as_tuple=True)
    page, off = page[b, t], off[b, t]
    s["k"][page, :, off] = k[b, t]
    s["v"][page, :, off] = v[b, t]
    s["weight"][page, :, off] = 0.0
    s["pos"][page, :, off] = s["at"][0].view(B, N)[b, t][:, None].expand(-1, H)
    return {"q": q, "k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"]}


def _attend(s, seen, bias):
    """softmax over the entries that each row sees ([B][N][L]; a row that sees none gives 0), times v."""
    case = s["case"]
    B, N, H, D, L = case["seqs"], case["new"], case["kv_heads"], case["dim"], case["length"]
    G, dev = case["q_heads"] // H, s["q"].device
    page, off = _places(s, torch.arange(L, device=dev)[None].expand(B, L))
    k = s["k"][page, :, off].permute(0, 2, 3, 1).float()                                # [B][H][D][L]
    q = s["q"].float().view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    sc = torch.matmul(q, k) * D ** -0.5
    if case["cap"]:
        sc = torch.tanh(sc / case["cap"]) * case["cap"]
    sc = sc.view(B, H, G, N, L)
    if bias is not None:
        sc = sc + bias
    sc = torch.where(seen[:, None, None], sc, torch.full((), -math.inf, device=dev))
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(torch.isfinite(top), top, torch.zeros((), device=dev)))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros((), device=dev))
    v = s["v"][page, :, off].permute(0, 2, 1, 3).float()                                # [B][H][L][D]
    out = torch.matmul(p.view(B, H, G * N, L), v)
    out = out.view(B, H, G, N, D).permute(0, 3, 1, 2, 4).reshape(B * N, H * G, D)
    return {"out": out.to(DTYPES[case["out"]])}


def _plain_prefill(s):
    case = s["case"]
    B, N, H, L = case["seqs"], case["new"], case["kv_heads"], case["length"]
    dev, n = s["q"].device, _counts(s)
    t, j = torch.arange(N, device=dev)[None], torch.arange(L, device=dev)
    i = (s["lens"].long() - n)[:, None] + t                                             # [B][N]
    hi = i + 1 if s["prefix"] is None else torch.maximum(i + 1, torch.minimum(s["prefix"].long(), s["lens"].long())[:, None])
    lo = torch.zeros_like(i) if not case["window"] else i - case["window"] + 1
    if s["first"] is not None:
        lo = torch.maximum(lo, s["first"].view(B, N).long())
    hi = torch.where(t < n[:, None], hi, torch.zeros_like(hi))
    seen = (j >= lo[..., None]) & (j < hi[..., None])
    if s["slopes"] is None:
        return _attend(s, seen, None)
    away = (j[None, None] - i[..., None]).float()                                       # [B][N][L]
    return _attend(s, seen, s["slopes"].view(1, H, -1, 1, 1) * away[:, None, None])


def _plain_tree(s):
    case = s["case"]
    N, L = case["new"], case["length"]
    dev, n = s["q"].device, _counts(s)
    j = torch.arange(L, device=dev)
    start = s["lens"].long() - n
    node = j[None] - start[:, None]                                                     # [B][L]
    bit = (s["tree"][:, :, None] >> node[:, None].clamp(min=0, max=63)) & 1
    inside = (node >= 0) & (node < n[:, None])
    seen = (node < 0)[:, None] | (inside[:, None] & (bit != 0))
    seen = seen & (torch.arange(N, device=dev)[None] < n[:, None])[..., None]
    return _attend(s, seen, None)


def _plain_keep(s):
    case = s["case"]
    M = s["keep"].shape[1]
    start = (s["lens"] - case["new"]).long()[:, None]
    i = torch.arange(M, device=s["lens"].device)[None]
    b, m = (i < s["kept"][:, None]).nonzero(as_tuple=True)
    sp, so = _places(s, start + s["keep"].long())
    dp, do = _places(s, start + i)
    sp, so, dp, do = (x[b, m] for x in (sp, so, dp, do))
    for x in (s["k"], s["v"], s["weight"], s["pos"]):
        x[dp, :, do] = x[sp, :, so]
    return {"k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"]}


_PLAIN = {"norm": _plain_norm, "prefill": _plain_prefill, "tree": _plain_tree, "keep": _plain_keep}


# ---------------------------------------------------------------------- work ---

def work(case):
    op, B, N, H, D, Hq, L = (case[n] for n in ("op", "seqs", "new", "kv_heads", "dim", "q_heads", "length"))
    size = {"f16": 2, "bf16": 2, "f32": 4}
    part = 0.5 if case.get("ragged") and N > 1 else 1.0                  # of the rows; the first sequence has all of them
    rows = N * (1 + (B - 1) * part)
    if op == "norm":
        return {"bytes": rows * D * (4 * Hq + size[case["q_out"]] * Hq + 12 * H), "flops": rows * D * (Hq + H) * 8}
    if op == "keep":
        moved = min(N, 8) * (1 + (B - 1) / 2)
        return {"bytes": moved * H * (8 * D + 16), "flops": 0}
    mean = L if not case.get("ragged") or B == 1 else L * (1 + (B - 1) * (1 + 1 / 8) / 2) / B
    if op == "tree":
        pairs = rows * mean
        entries = B * mean
    else:
        n = rows / B
        each = max(0.0, mean - n / 2)                                    # entries a row sees under the causal mask
        if case["prefix"]:
            each += n / 24                                               # x^2 / 2 of n with x uniform in 0 .. 1/2
        if case["window"]:
            w = min(case["window"], mean)
            each = min(each, w if mean - n >= w else w - (w - (mean - n)) ** 2 / (2 * n))
        if case["docs"]:
            each = min(each, each * 2 / (case["docs"] + 1))
        pairs = rows * each
        entries = B * min(mean, (case["window"] + n) if case["window"] else mean)
    return {"bytes": entries * H * 4 * D + B * N * Hq * D * (2 + size[case["out"]]), "flops": 4 * pairs * Hq * D}


# --------------------------------------------------------------- in 64 bits ---

def exact(case, seed):
    s = prepare(case, seed)
    op, B, N, H, D, Hq, L = (case[n] for n in ("op", "seqs", "new", "kv_heads", "dim", "q_heads", "length"))
    ps, table, lens = case["page"], s["table"].tolist(), s["lens"].tolist()
    new = [N] * B if s["new"] is None else s["new"].tolist()
    if op == "keep":
        k, v, w = s["k"].double(), s["v"].double(), s["weight"].double()
        keep, kept = s["keep"].tolist(), s["kept"].tolist()
        for b in range(B):
            for m in range(kept[b]):                                     # ascending: a source is never a place written before
                src, dst = lens[b] - N + keep[b][m], lens[b] - N + m
                for x in (k, v, w):
                    x[table[b][dst // ps], :, dst % ps] = x[table[b][src // ps], :, src % ps].clone()
        return {"k": k, "v": v, "weight": w, "pos": None}
    if op == "norm":
        inv = torch.tensor(_inverse(case["rot"]), dtype=torch.float64, device="cuda")
        where = torch.cat([s["at"][a].double()[:, None].expand(-1, n) for a, n in enumerate(_sections(case["rot"], case["axes"]))], 1)
        unit = torch.polar(torch.ones_like(where), where * inv)[:, None]

        def turn(x, gain):
            x = x.double()
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + 1e-6) * gain.double()
            i = torch.arange(case["rot"] // 2, device="cuda")
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
            z = torch.complex(x[..., a], x[..., b]) * unit
            x[..., a], x[..., b] = z.real, z.imag
            return x

        q, kr, k, v, w = turn(s["q"], s["q_norm"]), turn(s["k_new"], s["k_norm"]), s["k"].double(), s["v"].double(), s["weight"].double()
        for b in range(B):
            q[b * N + new[b]:(b + 1) * N] = 0
            j = list(range(lens[b] - new[b], lens[b]))
            pg, of = [table[b][x // ps] for x in j], [x % ps for x in j]
            rows = slice(b * N, b * N + new[b])
            if j:
                k[pg, :, of], v[pg, :, of], w[pg, :, of] = kr[rows], s["v_new"][rows].double(), 0.0
        return {"q": q, "k": k, "v": v, "weight": w, "pos": None}
    if B * N * L * Hq * D > PAIRS:
        return None
    out = torch.zeros((B * N, Hq, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        n, ln = new[b], lens[b]
        if n == 0:
            continue
        pages = torch.tensor(table[b][:-(-ln // ps)], device="cuda")
        i = torch.arange(ln - n, ln, device="cuda")[:, None]
        j = torch.arange(ln, device="cuda")[None]
        if op == "tree":
            words = [int(x) & ((1 << 64) - 1) for x in s["tree"][b, :n].tolist()]
            own_nodes = torch.tensor([[(x >> c) & 1 for c in range(n)] for x in words], dtype=torch.bool, device="cuda")
            hide = torch.cat((torch.zeros((n, ln - n), dtype=torch.bool, device="cuda"), ~own_nodes), 1)
        else:
            end = i if s["prefix"] is None else torch.clamp(i, min=min(int(s["prefix"][b]), ln) - 1)
            hide = j > end
            if case["window"]:
                hide = hide | (i - j >= case["window"])
            if s["first"] is not None:
                hide = hide | (j < s["first"][b * N:b * N + n, None])
        empty = hide.all(1)
        for h in range(Hq):
            k = s["k"][pages, h // (Hq // H)].reshape(-1, D)[:ln].double()
            v = s["v"][pages, h // (Hq // H)].reshape(-1, D)[:ln].double()
            sc = s["q"][b * N:b * N + n, h].double() @ k.T / math.sqrt(D)
            if case["cap"]:
                sc = case["cap"] * torch.tanh(sc / case["cap"])
            if op == "prefill" and s["slopes"] is not None:
                sc = sc - s["slopes"][h].double() * (i - j)
            p = torch.softmax(sc.masked_fill(hide, -math.inf), -1).masked_fill(empty[:, None], 0.0)
            out[b * N:b * N + n, h] = p @ v
    return {"out": out}
