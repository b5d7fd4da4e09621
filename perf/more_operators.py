"""Cases of the full-attention layer's operators around a cache held in 8 bits,
and their plain forms.

Five paths, as a hybrid model's full-attention layer takes them: the per-head
norm and rotation by positions with several axes (time, height, width: "rope");
a prompt's chunk going into the cache and the sequences' keys and values coming
back packed for its attention ("append"); a decode step, one new token into the
cache and its attention ("step"); the attention alone, with or without the
weights that each cached token received ("decode"); and the eviction of the
tokens that received least ("evict").

The cache holds e4m3 numbers and a scale for every 16 tokens and head, a power
of two: the smallest, of 2^-40 to 2^40, with which the largest of the block's
values so far is at most 448.

`run` computes the plain form with elementary torch operations, or, where
`own` is true, calls the framework's operators on the same state.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8 = torch.float8_e4m3fn
EPS = 1e-6
THETA = 1e6
BLOCK = 16            # tokens that share a scale


def listed():
    return [
        # one new token behind a long context with images: a launch's latency
        dict(name="rope one token", op="rope", n=1, hq=16, hkv=4, d=256, rot=64, layout="half",
             io="bf16", text=100_000, side=0, mixed=True, split=1),
        # a prompt of text and images, whole head rotated
        dict(name="rope images", op="rope", n=16411, hq=32, hkv=8, d=128, rot=128,
             layout="half", io="bf16", text=300, side=32, mixed=False, split=2),
        # a chunk of one prompt behind what its earlier chunks left in the cache
        dict(name="append chunk", op="append", n=1000, seqs=1, hq=16, hkv=4, d=256, rot=64,
             layout="half", io="bf16", page=64, start=3001, split=3),
        # packed prompts of the benchmark's batch, small pages
        dict(name="append prompts", op="append", n=16384, seqs=7, hq=16, hkv=4, d=256, rot=64,
             layout="half", io="bf16", page=16, start=0, split=4),
        # one token of one short sequence: latency
        dict(name="step one", op="step", n=1, hq=16, hkv=4, d=256, rot=64, layout="half", io="bf16",
             page=64, most=700, gate=True, split=5),
        # the benchmark's 64 sequences, lengths anywhere up to 8192
        dict(name="step batch", op="step", n=64, hq=16, hkv=4, d=256, rot=64, layout="half",
             io="bf16", page=64, most=8192, gate=True, split=6),
        # two long documents
        dict(name="decode long", op="decode", n=2, hq=16, hkv=2, d=256, io="bf16", page=128,
             most=131_072, gate=True, weights=False, split=7),
        # many rows of smaller heads, small pages
        dict(name="decode rows", op="decode", n=200, hq=32, hkv=8, d=128, io="fp16", page=16,
             most=3000, gate=False, weights=False, split=8),
        # a batch that collects what its cached tokens receive
        dict(name="decode weights", op="decode", n=32, hq=16, hkv=4, d=256, io="bf16", page=64,
             most=16_384, gate=True, weights=True, split=9),
        # one sequence that has outgrown its share by a quarter
        dict(name="evict one", op="evict", n=1, hkv=4, d=256, io="bf16", page=64, most=5120,
             keep=4096, first=4, last=256, split=10),
        # a batch cut down to a quarter of its longest sequence
        dict(name="evict batch", op="evict", n=32, hkv=4, d=256, io="bf16", page=64, most=16_384,
             keep=4096, first=16, last=1024, split=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "step", "decode", "decode", "evict"])
    hq, hkv, d = rng.choice([(16, 4, 256), (16, 2, 256), (32, 8, 128), (12, 4, 128), (8, 8, 128),
                             (24, 2, 256), (16, 16, 64), (32, 4, 64)])
    c = dict(op=op, hkv=hkv, d=d, io=rng.choice(["bf16", "bf16", "fp16"]),
             split=rng.randrange(1 << 20))
    if op != "evict":
        c.update(hq=hq)
    if op != "rope":
        c.update(page=rng.choice([16, 32, 64, 128]))
    if op in ("rope", "append", "step"):
        c.update(rot=rng.choice([d // 4, d // 2, d]), layout=rng.choice(["half", "interleaved"]))
    if op == "rope":
        c.update(n=_log(rng, 1, 16384), text=rng.choice([20, 300, 100_000]),
                 side=rng.choice([0, 5, 16, 32]), mixed=rng.random() < 0.5)
    elif op == "append":
        n = _log(rng, 1, 8192)
        c.update(n=n, seqs=min(n, _log(rng, 1, 16)), start=rng.choice([0, 16, rng.randint(1, 3000)]))
    elif op == "step":
        c.update(n=_log(rng, 1, 64), most=_log(rng, 2, 8192), gate=rng.random() < 0.5)
    elif op == "decode":
        c.update(n=_log(rng, 1, 64), most=_log(rng, 1, 8192), gate=rng.random() < 0.5,
                 weights=rng.random() < 0.4)
    else:
        most = _log(rng, 64, 8192)
        keep = rng.randint(most // 8 + 1, most)
        c.update(n=_log(rng, 1, 32), most=most, keep=keep, first=rng.randint(0, min(16, keep // 4)),
                 last=rng.randint(0, keep // 2))
    return c


def _lengths(case):
    """Host lengths of the case's sequences: fixed by the case, not by the seed."""
    r = random.Random(case["split"])
    if case["op"] == "append":
        cuts = sorted(r.sample(range(1, case["n"]), case["seqs"] - 1))
        return [b - a for a, b in zip([0] + cuts, cuts + [case["n"]])]
    lens = [r.randint(1, case["most"]) for _ in range(case["n"])]
    lens[r.randrange(len(lens))] = case["most"]
    return lens


def _axis_of_pair(rot, mixed):
    """Which of time, height and width turns each pair of channels: a half, a
    quarter and a quarter of them, in a row or (mixed) taking turns."""
    half = rot // 2
    if mixed:
        return [(0, 1, 0, 2)[i % 4] for i in range(half)]
    return [0 if i < half - half // 2 else 1 if i < half - half // 4 else 2 for i in range(half)]


def _positions(case, host):
    """[3][n] of text runs with square images between them: along a run all
    three advance, an image has one time and its own rows and columns."""
    n, side, text = case["n"], case["side"], case["text"]
    at = host.randrange(64) + (text if n == 1 else 0)
    parts, left = [], n
    while left > 0:
        run = torch.arange(min(left, text), device="cuda") + at
        parts.append(run.expand(3, -1))
        at, left = at + len(run), left - len(run)
        if left > 0 and side > 0:
            i = torch.arange(min(left, side * side), device="cuda")
            row = torch.div(i, side, rounding_mode="floor")
            parts.append(torch.stack([torch.zeros_like(i), row, i - row * side]) + at)
            at, left = at + side, left - len(i)
    return torch.cat(parts, 1).to(torch.int32)


def _frequencies(rot):
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    return THETA ** (-2.0 * i / rot)


def _pool(g, case, lens):
    """Codes, scales and block table of a cache that holds these sequences, their
    pages anywhere in a pool with a few to spare."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    used = [(v + page - 1) // page for v in lens]
    pool = sum(used) + 3
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(used), dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u

    def half():
        # after norm and rotation a key channel is of order one, a value alike; tokens differ in size
        x = torch.randn(pool, hkv, page // BLOCK, BLOCK, d, generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(pool, hkv, page // BLOCK, BLOCK, 1, generator=g, device="cuda"))
        s = _scale(x.abs().amax((-1, -2)))
        return _codes(x / s[..., None, None]).view(pool, hkv, page, d), s
    (k, ks), (v, vs) = half(), half()
    return dict(kc=k, vc=v, ks=ks, vs=vs, table=table)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    io = DTYPES[case["io"]]
    n, hkv, d = case["n"], case["hkv"], case["d"]
    host = random.Random(seed)

    def normal(*shape, dtype=io):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    s = dict(case=dict(case))
    if case["op"] in ("rope", "append", "step"):
        # the projections' outputs: q next to its gate, k next to v, as one matmul leaves them
        hq = case["hq"]
        qg, kv = normal(n, hq, 2 * d), normal(n, 2 * hkv, d)
        s.update(q=qg[:, :, :d], k=kv[:, :hkv], v=kv[:, hkv:], freq=_frequencies(case["rot"]),
                 wq=1 + 0.1 * normal(d, dtype=torch.float32),
                 wk=1 + 0.1 * normal(d, dtype=torch.float32))
        if case["op"] == "step":
            s["gate"] = qg[:, :, d:] if case["gate"] else None
    if case["op"] == "rope":
        axis = _axis_of_pair(case["rot"], case["mixed"])
        s.update(pos=_positions(case, host), axis=axis, axis_at=torch.tensor(axis, device="cuda"))
    elif case["op"] == "append":
        lens, start = _lengths(case), case["start"]
        cu, all_cu = [0], [0]
        for v in lens:
            cu.append(cu[-1] + v)
            all_cu.append(all_cu[-1] + start + v)
        at = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), ints(lens))
        i = torch.arange(n, device="cuda") - ints(cu)[at]
        s.update(_pool(g, case, [start + v for v in lens]), cu=ints(cu), all_cu=ints(all_cu),
                 total=all_cu[-1], starts=ints([start] * len(lens)),
                 pos=(i + start).to(torch.int32).view(1, n))
    elif case["op"] == "step":
        lens = _lengths(case)
        before = ints([v - 1 for v in lens])
        s.update(_pool(g, case, lens), starts=before, lens=ints(lens), pos=before.view(1, n))
    elif case["op"] == "decode":
        lens = _lengths(case)
        s.update(_pool(g, case, lens), q=normal(n, case["hq"], d), lens=ints(lens),
                 gate=normal(n, case["hq"], 2 * d)[:, :, d:] if case["gate"] else None)
        if case["weights"]:
            shape = (n, hkv, s["table"].shape[1] * case["page"])
            s["weights"] = torch.rand(shape, generator=g, device="cuda") * 0.01
    else:
        lens, page = _lengths(case), case["page"]
        s.update(_pool(g, case, lens), lens=ints(lens))
        # most tokens receive little; some the same
        w = torch.rand(n, hkv, s["table"].shape[1] * page, generator=g, device="cuda")
        s["weights"] = torch.where(w < 0.05, 0.25, w ** 8)
        width = (case["keep"] + page - 1) // page
        new = dict(case, most=width * page)
        s["new"] = _pool(g, new, [width * page] * n)
        s["weights_new"] = torch.zeros(n, hkv, width * page, device="cuda")
    return s


# ---- the plain forms -------------------------------------------------------


def _scale(amax):
    """The smallest 2^e, e in [-40, 40], with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax.float())
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax == 0, torch.full_like(e, -40), e).clamp(-40, 40)
    return torch.ldexp(torch.ones((), device=amax.device), e)


def _codes(x):
    return x.clamp(-448, 448).to(F8)


def _norm_rope(x, w, angle, layout):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    half = angle.shape[1]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if layout == "half":
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([rot, rest], -1)


def _append(codes, scales, x, blk, row, starts, first_blk):
    """x [n][h][d] into the pool's blocks blk at rows `row`; a sequence's first
    block keeps what it held below starts % 16, at the new scale."""
    pool, h, page, d = codes.shape
    nb = page // BLOCK
    c = codes.view(torch.uint8).view(pool, h, nb, BLOCK, d)
    page_of, in_page = torch.div(blk, nb, rounding_mode="floor"), blk % nb
    most = torch.zeros(pool * nb, h, device=x.device).index_reduce_(
        0, blk, x.abs().amax(-1), "amax")
    fp, fi = torch.div(first_blk, nb, rounding_mode="floor"), first_blk % nb
    held = torch.arange(BLOCK, device=x.device) < (starts % BLOCK)[:, None]
    old = torch.where(held[:, :1], scales[fp, :, fi], torch.zeros((), device=x.device))
    new = _scale(most)
    new[first_blk] = torch.maximum(new[first_blk], old)
    before = c[fp, :, fi].view(F8).float() * (old / new[first_blk])[..., None, None]
    c[fp, :, fi] = torch.where(held[:, None, :, None], _codes(before).view(torch.uint8),
                               c[fp, :, fi])
    c[page_of, :, in_page, row] = _codes(x / new[blk][..., None]).view(torch.uint8)
    scales[page_of, :, in_page] = new[blk]


def _places(s, seq, place):
    page = s["case"]["page"]
    nb = page // BLOCK
    pages = s["table"][seq, torch.div(place, page, rounding_mode="floor")].long()
    return pages * nb + torch.div(place % page, BLOCK, rounding_mode="floor"), place % BLOCK


def _fill(s, seq, place):
    """The new rows' q, and their keys and values into the cache."""
    case, io = s["case"], DTYPES[s["case"]["io"]]
    angle = s["pos"][0].double()[:, None] * s["freq"]
    q = _norm_rope(s["q"], s["wq"], angle, case["layout"]).to(io)
    k = _norm_rope(s["k"], s["wk"], angle, case["layout"])
    blk, row = _places(s, seq, place)
    starts = s["starts"].long()
    first, _ = _places(s, torch.arange(len(starts), device="cuda"), starts)
    _append(s["kc"], s["ks"], k, blk, row, starts, first)
    _append(s["vc"], s["vs"], s["v"].float(), blk, row, starts, first)
    return q


def _values(codes, scales):
    return codes.float() * scales.repeat_interleave(BLOCK, -1)[..., None]


def _softmax(scores, mask):
    scores = scores.masked_fill(~mask, -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _attend(s, q):
    case = s["case"]
    n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
    table, g = s["table"].long(), hq // hkv
    k = _values(s["kc"][table], s["ks"][table]).transpose(1, 2).reshape(n, hkv, -1, d)
    v = _values(s["vc"][table], s["vs"][table]).transpose(1, 2).reshape(n, hkv, -1, d)
    seen = torch.arange(k.shape[2], device="cuda") < s["lens"][:, None]
    q = q.float().view(n, hkv, g, d)
    p = _softmax(q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d)), seen[:, None, None, :])
    o = (p @ v).view(n, hq, d)
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    return o.to(DTYPES[case["io"]]), p.sum(2)


def _keep(s):
    """Places kept per sequence and head, in order, -1 behind the last."""
    case, lens = s["case"], s["lens"].long()[:, None, None]
    keep, first, last = case["keep"], case["first"], case["last"]
    w = s["weights"]
    at = torch.arange(w.shape[2], device="cuda")
    always = (at < first) | (at >= lens - last)
    w = torch.where(always, math.inf, w).masked_fill(at >= lens, -math.inf)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.sort(torch.where(best < lens, best, w.shape[2]), dim=-1).values
    return torch.where(kept < w.shape[2], kept, -1)


def _move(codes, scales, kept, table, to_codes, to_scales, to_table):
    """The kept rows into the other pages, every 16 with the largest of their scales."""
    n, h, keep = kept.shape
    page, d = codes.shape[2], codes.shape[3]
    there = kept >= 0
    src = kept.clamp(min=0)
    seq = torch.arange(n, device="cuda")[:, None, None]
    head = torch.arange(h, device="cuda")[None, :, None]
    pages = table.long()[seq, torch.div(src, page, rounding_mode="floor")]
    rows = codes.view(torch.uint8)[pages, head, src % page].view(F8).float()
    old = scales[pages, head, torch.div(src % page, BLOCK, rounding_mode="floor")]
    old = torch.where(there, old, torch.zeros((), device="cuda"))
    pad = -keep % BLOCK
    new = torch.nn.functional.pad(old, (0, pad)).view(n, h, -1, BLOCK).amax(-1)
    rows = _codes(rows * (old / new.repeat_interleave(BLOCK, -1)[..., :keep])[..., None])
    to = torch.arange(keep, device="cuda")
    b, j, i = torch.nonzero(there, as_tuple=True)
    to_page = to_table.long()[b, torch.div(to[i], page, rounding_mode="floor")]
    to_codes.view(torch.uint8)[to_page, j, to[i] % page] = rows.view(torch.uint8)[b, j, i]
    b, j, i = torch.nonzero(new > 0, as_tuple=True)
    per = page // BLOCK
    to_page = to_table.long()[b, torch.div(i, per, rounding_mode="floor")]
    to_scales[to_page, j, i % per] = new[b, j, i]


def _plain(s):
    case = s["case"]
    io, n = DTYPES[case["io"]], case["n"]
    if case["op"] == "rope":
        # angles of far positions in 64 bits
        angle = (s["pos"][s["axis_at"]].double() * s["freq"][:, None]).T
        return {"q": _norm_rope(s["q"], s["wq"], angle, case["layout"]).to(io),
                "k": _norm_rope(s["k"], s["wk"], angle, case["layout"]).to(io)}
    if case["op"] == "append":
        t = torch.arange(n, device="cuda")
        seq = torch.searchsorted(s["cu"].long(), t, right=True) - 1
        q = _fill(s, seq, t - s["cu"].long()[seq] + s["starts"].long()[seq])
        t = torch.arange(s["total"], device="cuda")
        seq = torch.searchsorted(s["all_cu"].long(), t, right=True) - 1
        blk, row = _places(s, seq, t - s["all_cu"].long()[seq])
        nb = case["page"] // BLOCK
        page, b = torch.div(blk, nb, rounding_mode="floor"), blk % nb

        def packed(codes, scales):
            rows = codes.view(torch.uint8)[page, :, b * BLOCK + row].view(F8).float()
            return (rows * scales[page, :, b][..., None]).to(io)
        return {"q": q, "k": packed(s["kc"], s["ks"]), "v": packed(s["vc"], s["vs"])}
    if case["op"] == "step":
        q = _fill(s, torch.arange(n, device="cuda"), s["starts"].long())
        return {"q": q, "o": _attend(s, q)[0], "k_cache": s["kc"], "v_cache": s["vc"]}
    if case["op"] == "decode":
        o, p = _attend(s, s["q"])
        if not case["weights"]:
            return o
        s["weights"] += p
        return {"o": o, "weights": s["weights"]}
    kept, new = _keep(s), s["new"]
    for x, sc in (("kc", "ks"), ("vc", "vs")):
        _move(s[x], s[sc], kept, s["table"], new[x], new[sc], new["table"])
    w = s["weights"].gather(2, kept.clamp(min=0))
    s["weights_new"].zero_()
    s["weights_new"][..., :case["keep"]] = torch.where(kept >= 0, w, 0.0)
    return {"lens": s["lens"].clamp(max=case["keep"]), "kept": kept.to(torch.int32),
            "weights": s["weights_new"], "k_cache": new["kc"], "v_cache": new["vc"],
            "k_scale": new["ks"], "v_scale": new["vs"]}


# ---- the framework's operators -----------------------------------------------


def _own(s):
    import gated_deltanet_linear_07_gb300 as gdn
    case = s["case"]
    dims = s.get("dims")
    if dims is None:   # what a program makes once
        dims = s["dims"] = gdn.make_attn_dims(
            case.get("hq", case["hkv"]), case["hkv"], case["d"], io=case["io"],
            rot_dim=case.get("rot", 0), rope=case.get("layout", "half"),
            page_size=case.get("page", 64), norm_eps=EPS)
        if case["op"] == "rope":
            s["axes"] = gdn.make_rope_axes(s["axis"])
        else:
            s["cache"] = gdn.Kv8Cache(s["kc"], s["vc"], s["ks"], s["vs"], s["table"])
        if case["op"] in ("step", "decode"):
            width = s["weights"].shape[2] if case.get("weights") else 0
            size = gdn.gdn_attn_decode_kv8_workspace_size(dims, case["n"], width)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        if case["op"] == "evict":
            new = s["new"]
            s["cache_new"] = gdn.Kv8Cache(new["kc"], new["vc"], new["ks"], new["vs"], new["table"])
    if case["op"] == "rope":
        q, k = gdn.gdn_qk_norm_rope_axes(dims, s["q"], s["k"], s["wq"], s["wk"], s["freq"], s["pos"],
                                         s["axes"])
        return {"q": q, "k": k}
    if case["op"] == "append":
        q = gdn.gdn_kv8_append(dims, s["q"], s["k"], s["v"], s["wq"], s["wk"], s["freq"], s["pos"],
                               s["cache"], s["starts"], cu_seqlens=s["cu"])
        k, v = gdn.gdn_kv8_gather(dims, s["cache"], s["all_cu"], s["total"])
        return {"q": q, "k": k, "v": v}
    if case["op"] == "step":
        q = gdn.gdn_kv8_append(dims, s["q"], s["k"], s["v"], s["wq"], s["wk"], s["freq"], s["pos"],
                               s["cache"], s["starts"])
        o = gdn.gdn_attn_decode_kv8(dims, q, s["cache"], s["lens"], s["workspace"], gate=s["gate"])
        return {"q": q, "o": o, "k_cache": s["kc"], "v_cache": s["vc"]}
    if case["op"] == "decode":
        o = gdn.gdn_attn_decode_kv8(dims, s["q"], s["cache"], s["lens"], s["workspace"],
                                    gate=s["gate"], weights=s.get("weights"))
        return {"o": o, "weights": s["weights"]} if case["weights"] else o
    new = s["new"]
    lens, kept = gdn.gdn_kv8_evict(dims, s["cache"], s["weights"], s["lens"], case["keep"],
                                   s["cache_new"], s["weights_new"], first=case["first"],
                                   last=case["last"])
    return {"lens": lens, "kept": kept, "weights": s["weights_new"], "k_cache": new["kc"],
            "v_cache": new["vc"], "k_scale": new["ks"], "v_scale": new["vs"]}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    n, hkv, d = case["n"], case["hkv"], case["d"]
    token = 2 * hkv * d                # a cached token's bytes
    if case["op"] == "rope":
        return {"bytes": 2 * 2 * n * (case["hq"] + hkv) * d, "flops": 0}
    if case["op"] == "append":
        old = case["seqs"] * case["start"]
        rows = 2 * n * (2 * case["hq"] + 2 * hkv) * d + n * token
        return {"bytes": rows + old * token + 2 * (old + n) * token, "flops": 0}
    lens = _lengths(case)
    if case["op"] == "evict":
        kept = sum(min(v, case["keep"]) for v in lens)
        return {"bytes": 4 * hkv * sum(lens) + 2 * kept * token + 8 * hkv * kept, "flops": 0}
    ends = 2 * (3 if case["gate"] else 2) * n * case["hq"] * d    # q, gate read; o written
    if case["op"] == "step":
        ends += 2 * n * (case["hq"] + 2 * hkv) * d + n * token
    if case["op"] == "decode" and case["weights"]:
        ends += 8 * hkv * sum(lens)
    return {"bytes": ends + sum(lens) * token, "flops": 4 * d * case["hq"] * sum(lens)}


# ---- from the definitions, in 64 bits --------------------------------------------


def _exact_rotated(x, w, angle, layout):
    """x [n][h][d] normed and rotated as complex numbers."""
    x = x.to(torch.float64)
    d, half = x.shape[-1], angle.shape[1]
    x = w.to(torch.float64) * x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt()
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    even = slice(0, half) if layout == "half" else slice(0, 2 * half, 2)
    odd = slice(half, 2 * half) if layout == "half" else slice(1, 2 * half, 2)
    z = torch.complex(x[..., even], x[..., odd]) * turn
    y = x.clone()
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _exact_round(x):
    """To the nearest number with four significant bits, of steps of 2^-9 at least, ties to even."""
    size = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(size - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_scale(top):
    e = torch.ceil(torch.log2(top / 448)).clamp(-40, 40)
    # a logarithm may be off at the border itself
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((top <= 448 * torch.exp2(e - 1)) & (e > -40), e - 1, e)
    return torch.exp2(e.clamp(-40, 40))


def _exact_sequence(codes, scales, pages, length):
    """Codes and scales per token of one sequence, [h][length][d] and [h][length]."""
    h, d = codes.shape[1], codes.shape[3]
    c = codes[pages.long()].double().transpose(0, 1).reshape(h, -1, d)[:, :length]
    per = scales[pages.long()].double().transpose(0, 1).reshape(h, -1)
    return c, per.unsqueeze(-1).expand(-1, -1, BLOCK).reshape(h, -1)[:, :length]


def _exact_filled(c, per, x, start):
    """The same of a sequence whose tokens from `start` on become x [h][m][d]."""
    h, m, d = x.shape
    end = start + m
    c, per = c[:, :end].clone(), per[:, :end].clone()
    for at in range(start // BLOCK * BLOCK, end, BLOCK):
        a, b = max(at, start), min(at + BLOCK, end)
        new = _exact_scale(x[:, a - start:b - start].abs().amax((1, 2)))
        if a > at:
            old = per[:, at]
            new = torch.maximum(new, old)
            c[:, at:a] = _exact_round(c[:, at:a] * (old / new)[:, None, None])
        per[:, at:b] = new[:, None]
        c[:, a:b] = _exact_round(x[:, a - start:b - start] / new[:, None, None])
    return c, per


def _exact_attention(q, gate, k, v):
    """q [hq][d] over k, v [h][s][d]: (o, weights [h][s])."""
    h, s, d = k.shape
    e = torch.einsum("hgd,hsd->hgs", q.double().view(h, -1, d), k) / math.sqrt(d)
    p = torch.softmax(e, dim=-1)
    o = torch.einsum("hgs,hsd->hgd", p, v).reshape(-1, d)
    if gate is not None:
        o = o / (1 + torch.exp(-gate.double()))
    return o, p.sum(1)


def exact(case, seed):
    s = prepare(case, seed)
    n, hkv, d, op = case["n"], case["hkv"], case["d"], case["op"]
    if op == "rope":
        angle = torch.stack([s["pos"][a].double() * f for a, f in zip(s["axis"], s["freq"])], 1)
        return {x: _exact_rotated(s[x], s["w" + x], angle, case["layout"]) for x in ("q", "k")}
    lens = s["lens"].tolist() if "lens" in s else [case["start"] + v for v in _lengths(case)]
    if op in ("append", "step"):
        angle = s["pos"][0].double().outer(s["freq"])
        q, k = (_exact_rotated(s[x], s["w" + x], angle, case["layout"]) for x in ("q", "k"))
        new, at = {"k": k.transpose(0, 1), "v": s["v"].double().transpose(0, 1)}, 0
        out = {"k": [], "v": []}
        o = []
        codes = {"k": s["kc"].double(), "v": s["vc"].double()} if op == "step" else {}
        for b, length in enumerate(lens):
            start = case["start"] if op == "append" else length - 1
            m, now = length - start, {}
            for x in ("k", "v"):
                c, per = _exact_sequence(s[x + "c"], s[x + "s"], s["table"][b], length)
                c, per = _exact_filled(c, per, new[x][:, at:at + m], start)
                now[x] = c * per[..., None]
                if op == "append":
                    out[x].append(now[x].transpose(0, 1))
                else:
                    i = (length - 1) // BLOCK * BLOCK
                    page, row = s["table"][b, i // case["page"]].long(), i % case["page"]
                    codes[x][page, :, row:row + length - i] = c[:, i:]
            if op == "step":
                # the step's query is what the norm and rotation leave in the model's type
                rounded = q[b].to(DTYPES[case["io"]])
                o.append(_exact_attention(rounded, None if s["gate"] is None else s["gate"][b],
                                          now["k"], now["v"])[0])
            at += m
        if op == "append":
            return {"q": q, "k": torch.cat(out["k"]), "v": torch.cat(out["v"])}
        return {"q": q, "o": torch.stack(o), "k_cache": codes["k"], "v_cache": codes["v"]}
    if op == "decode":
        o = []
        total = s["weights"].double() if case["weights"] else None
        for b, length in enumerate(lens):
            k, v = (c * per[..., None] for c, per in
                    (_exact_sequence(s[x + "c"], s[x + "s"], s["table"][b], length) for x in "kv"))
            y, p = _exact_attention(s["q"][b], None if s["gate"] is None else s["gate"][b], k, v)
            o.append(y)
            if total is not None:
                total[b, :, :length] += p
        return torch.stack(o) if total is None else {"o": torch.stack(o), "weights": total}
    keep, page, t = case["keep"], case["page"], s["new"]
    kept = torch.full((n, hkv, keep), -1, dtype=torch.int32, device="cuda")
    weights = torch.zeros_like(s["weights_new"], dtype=torch.float64)
    codes = {x: t[x + "c"].double() for x in "kv"}
    scales = {x: t[x + "s"].double() for x in "kv"}
    for b, length in enumerate(lens):
        here = {x: _exact_sequence(s[x + "c"], s[x + "s"], s["table"][b], length) for x in "kv"}
        m = min(length, keep)
        middle = range(case["first"], length - case["last"])
        for j in range(hkv):
            if length <= keep:
                places = list(range(length))
            else:
                w = s["weights"][b, j].tolist()
                best = sorted(middle, key=lambda i: (-w[i], i))[:keep - case["first"] - case["last"]]
                places = sorted([*range(case["first"]), *best,
                                 *range(length - case["last"], length)])
            at = torch.tensor(places, device="cuda")
            kept[b, j, :m] = at.int()
            weights[b, j, :m] = s["weights"][b, j, at].double()
            for x in "kv":
                c, per = here[x][0][j, at], here[x][1][j, at]
                pad = -m % BLOCK
                top = torch.nn.functional.pad(per, (0, pad)).view(-1, BLOCK).amax(1)
                ratio = per / top.repeat_interleave(BLOCK)[:m]
                c = _exact_round(c * ratio[:, None])
                to = t["table"][b].long()
                i = torch.arange(m, device="cuda")
                codes[x][to[i // page], j, i % page] = c
                i = torch.arange(len(top), device="cuda")
                per_page = page // BLOCK
                scales[x][to[i // per_page], j, i % per_page] = top
    return {"lens": s["lens"].clamp(max=keep), "kept": kept, "weights": weights,
            "k_cache": codes["k"], "v_cache": codes["v"], "k_scale": scales["k"],
            "v_scale": scales["v"]}
