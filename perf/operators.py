"""Cases of the full-attention layer's operators and their plain forms.

Four operators, in the order in which a hybrid model's full-attention layer
calls them: the per-head norm and rotation of queries and keys ("rope"), the
same with the keys and values going into a paged cache ("append"), causal
attention over packed prompts ("prefill") and one-token attention over the
paged cache, with or without a prefix that the whole batch shares ("decode").

`run` computes the plain form with elementary torch operations, or, where
`own` is true, calls the framework's operators on the same state.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
THETA = 1e6


def listed():
    return [
        # one new token of one sequence, far into its context: a launch's latency
        dict(name="rope one token", op="rope", n=1, hq=16, hkv=4, d=256, rot=64, layout="half",
             io="bf16", start=100_000),
        # a prompt of the benchmark's length
        dict(name="rope 4096", op="rope", n=4096, hq=16, hkv=4, d=256, rot=64, layout="half",
             io="bf16", start=0),
        # a long packed batch, whole head rotated, interleaved pairs, far positions
        dict(name="rope long", op="rope", n=30011, hq=32, hkv=8, d=128, rot=128,
             layout="interleaved", io="fp16", start=900_000),
        # a decode step of the benchmark's 64 rows: each writes one cache row
        dict(name="append step", op="append", n=64, seqs=64, hq=16, hkv=4, d=256, rot=64,
             layout="half", io="bf16", page=64, start=3000, split=1),
        # packed prompts going into a cache with small pages
        dict(name="append prompts", op="append", n=16384, seqs=7, hq=16, hkv=4, d=256, rot=64,
             layout="half", io="bf16", page=16, start=0, split=2),
        # many short prompts in one call
        dict(name="prefill short", op="prefill", n=1000, seqs=24, hq=16, hkv=2, d=128, io="fp16",
             gate=False, split=3),
        # the benchmark's prompt length, gated output
        dict(name="prefill 4096", op="prefill", n=4096, seqs=1, hq=16, hkv=4, d=256, io="bf16",
             gate=True, split=4),
        # a ragged batch of prompts
        dict(name="prefill packed", op="prefill", n=24001, seqs=16, hq=32, hkv=8, d=128, io="bf16",
             gate=False, split=5),
        # one long prompt
        dict(name="prefill long", op="prefill", n=16384, seqs=1, hq=16, hkv=4, d=256, io="bf16",
             gate=True, split=6),
        # one token of one short sequence: latency
        dict(name="decode one", op="decode", n=1, hq=16, hkv=4, d=256, io="bf16", page=64, shared=0,
             most=700, gate=True, split=7),
        # the benchmark's 64 sequences, lengths anywhere up to 8192
        dict(name="decode batch", op="decode", n=64, hq=16, hkv=4, d=256, io="bf16", page=64,
             shared=0, most=8192, gate=True, split=8),
        # the same batch behind a long common prompt
        dict(name="decode shared", op="decode", n=64, hq=16, hkv=4, d=256, io="bf16", page=64,
             shared=32768, most=1024, gate=True, split=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "prefill", "decode", "prefill", "decode"])
    hq, hkv, d = rng.choice([(16, 4, 256), (16, 2, 256), (32, 8, 128), (12, 4, 128), (8, 8, 128),
                             (24, 2, 256), (16, 16, 64), (32, 4, 64)])
    c = dict(op=op, hq=hq, hkv=hkv, d=d, io=rng.choice(["bf16", "bf16", "fp16"]),
             split=rng.randrange(1 << 20))
    if op in ("rope", "append"):
        n = _log(rng, 1, 16384)
        c.update(n=n, rot=rng.choice([d // 4, d // 2, d]),
                 layout=rng.choice(["half", "interleaved"]), start=rng.choice([0, 4000, 200_000]))
        if op == "append":
            c.update(start=min(c["start"], 4000), seqs=min(n, _log(rng, 1, 64)),
                     page=rng.choice([16, 32, 64, 128]))
    elif op == "prefill":
        n = _log(rng, 1, 8192)
        c.update(n=n, seqs=min(n, _log(rng, 1, 16)), gate=rng.random() < 0.5)
    else:
        page = rng.choice([16, 32, 64, 128])
        n = _log(rng, 1, 64)
        shared = rng.choice([0, 0, _log(rng, 256, 32768) // page * page])
        c.update(n=n, page=page, shared=shared, most=_log(rng, 1, 8192 if shared == 0 else 1024),
                 gate=rng.random() < 0.5)
    return c


def _lengths(case):
    """Host lengths of the case's sequences: fixed by the case, not by the seed."""
    r = random.Random(case["split"])
    if case["op"] == "decode":
        lens = [r.randint(1, case["most"]) for _ in range(case["n"])]
        lens[r.randrange(len(lens))] = case["most"]
        return [case["shared"] + v for v in lens]
    cuts = sorted(r.sample(range(1, case["n"]), case["seqs"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["n"]])]


def _frequencies(rot):
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    return THETA ** (-2.0 * i / rot)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    io = DTYPES[case["io"]]
    n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
    host = random.Random(seed)

    def normal(*shape, dtype=io, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    s = dict(case=dict(case))
    if case["op"] in ("rope", "append"):
        # the projections' outputs: q next to its gate, k next to v, as one matmul leaves them
        qg, kv = normal(n, hq, 2 * d), normal(n, 2 * hkv, d)
        s.update(q=qg[:, :, :d], k=kv[:, :hkv], v=kv[:, hkv:], freq=_frequencies(case["rot"]),
                 wq=1 + 0.1 * normal(d, dtype=torch.float32),
                 wk=1 + 0.1 * normal(d, dtype=torch.float32))
    if case["op"] == "rope":
        s["pos"] = (torch.arange(n, device="cuda") + case["start"] + host.randrange(64)).to(torch.int32)
    elif case["op"] == "append":
        lens, page = _lengths(case), case["page"]
        pos, seq = [], []
        for b, length in enumerate(lens):
            pos.extend(range(case["start"], case["start"] + length))
            seq.extend([b] * length)
        # the sequences' pages lie anywhere in a pool that has some to spare
        width = (case["start"] + max(lens) + page - 1) // page
        used = [(case["start"] + v + page - 1) // page for v in lens]
        pool = sum(used) + 5
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = ids[at:at + u]
            at += u
        s.update(pos=ints(pos), seq=ints(seq), table=table,
                 kc=normal(pool, hkv, page, d), vc=normal(pool, hkv, page, d))
    elif case["op"] == "prefill":
        lens = _lengths(case)
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
        # after norm and rotation a query or key channel is of order one
        s.update(q=normal(n, hq, d), k=normal(n, hkv, d), v=normal(n, hkv, d), cu=ints(cu),
                 most=max(lens), gate=normal(n, hq, 2 * d)[:, :, d:] if case["gate"] else None)
    elif case["op"] == "decode":
        lens, page = _lengths(case), case["page"]
        sp = case["shared"] // page
        width = (max(lens) + page - 1) // page
        used = [(v + page - 1) // page - sp for v in lens]
        pool = sp + sum(used) + 3
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(n, width, dtype=torch.int32, device="cuda")
        table[:, :sp] = ids[:sp]
        at = sp
        for b, u in enumerate(used):
            table[b, sp:sp + u] = ids[at:at + u]
            at += u
        s.update(q=normal(n, hq, d), kc=normal(pool, hkv, page, d), vc=normal(pool, hkv, page, d),
                 table=table, lens=ints(lens), most=max(lens),
                 gate=normal(n, hq, 2 * d)[:, :, d:] if case["gate"] else None)
    return s


# ---- the plain forms -------------------------------------------------------


def _norm_rope(x, w, pos, freq, layout):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    # angles of far positions in 64 bits
    angle = pos.double()[:, None] * freq[None, :]
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    half = freq.numel()
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if layout == "half":
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([rot, rest], -1)


def _softmax(scores, mask):
    scores = scores.masked_fill(~mask, -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _gated(o, gate):
    return o if gate is None else o * torch.sigmoid(gate.float())


def _plain(s):
    case = s["case"]
    io, hq, hkv, d = DTYPES[case["io"]], case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        return {"q": _norm_rope(s["q"], s["wq"], s["pos"], s["freq"], case["layout"]).to(io),
                "k": _norm_rope(s["k"], s["wk"], s["pos"], s["freq"], case["layout"]).to(io)}
    if case["op"] == "append":
        q = _norm_rope(s["q"], s["wq"], s["pos"], s["freq"], case["layout"]).to(io)
        k = _norm_rope(s["k"], s["wk"], s["pos"], s["freq"], case["layout"]).to(io)
        pos = s["pos"].long()
        page, off = s["table"][s["seq"].long(), pos // case["page"]].long(), pos % case["page"]
        s["kc"][page, :, off] = k
        s["vc"][page, :, off] = s["v"]
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    scale, g = 1.0 / math.sqrt(d), hq // hkv
    if case["op"] == "prefill":
        # every sequence padded to the longest
        cu, n, most = s["cu"].long(), case["n"], s["most"]
        i = torch.arange(most, device="cuda")
        row = (cu[:-1, None] + i).clamp(max=n - 1)
        q = s["q"].float()[row].view(-1, most, hkv, g, d).permute(0, 2, 3, 1, 4)
        k = s["k"].float()[row].transpose(1, 2)
        v = s["v"].float()[row].transpose(1, 2)
        scores = q.reshape(-1, hkv, g * most, d) @ k.transpose(-1, -2) * scale
        p = _softmax(scores.view(-1, hkv, g, most, most), i[:, None] >= i[None, :])
        o = (p.view(-1, hkv, g * most, most) @ v).view(-1, hq, most, d)
        t = torch.arange(n, device="cuda")
        b = torch.searchsorted(cu, t, right=True) - 1
        return _gated(o[b, :, t - cu[b]], s["gate"]).to(io)
    # decode: every sequence's pages gathered and padded to the longest
    n, most = case["n"], s["most"]
    table = s["table"].long()
    k = s["kc"][table].float().transpose(1, 2).reshape(n, hkv, -1, d)
    v = s["vc"][table].float().transpose(1, 2).reshape(n, hkv, -1, d)
    q = s["q"].float().view(n, hkv, g, d)
    seen = torch.arange(k.shape[2], device="cuda") < s["lens"][:, None]
    p = _softmax(q @ k.transpose(-1, -2) * scale, seen[:, None, None, :])
    return _gated((p @ v).view(n, hq, d), s["gate"]).to(io)


# ---- the framework's operators -----------------------------------------------


def _own(s):
    import gated_deltanet_linear_07_gb300 as gdn
    case = s["case"]
    dims = s.get("dims")
    if dims is None:   # what a program makes once
        dims = s["dims"] = gdn.make_attn_dims(
            case["hq"], case["hkv"], case["d"], io=case["io"], rot_dim=case.get("rot", 0),
            rope=case.get("layout", "half"), page_size=case.get("page", 64), norm_eps=EPS)
        if case["op"] == "decode":
            size = gdn.gdn_attn_decode_workspace_size(dims, case["n"], case["shared"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if case["op"] == "rope":
        q, k = gdn.gdn_qk_norm_rope(dims, s["q"], s["k"], s["wq"], s["wk"], s["freq"], s["pos"])
        return {"q": q, "k": k}
    if case["op"] == "append":
        q = gdn.gdn_kv_append(dims, s["q"], s["k"], s["v"], s["wq"], s["wk"], s["freq"], s["pos"],
                              s["kc"], s["vc"], s["table"], row_seq=s["seq"])
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    if case["op"] == "prefill":
        return gdn.gdn_attn_prefill(dims, s["q"], s["k"], s["v"], s["cu"], gate=s["gate"])
    return gdn.gdn_attn_decode(dims, s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                               s["workspace"], shared_len=case["shared"], gate=s["gate"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        return {"bytes": 2 * 2 * n * (hq + hkv) * d, "flops": 0}
    if case["op"] == "append":
        return {"bytes": 2 * 2 * n * (hq + 2 * hkv) * d, "flops": 0}
    ends = (3 if case["gate"] else 2) * n * hq * d       # q, gate read; o written
    if case["op"] == "prefill":
        pairs = sum(v * (v + 1) // 2 for v in _lengths(case))
        return {"bytes": 2 * (ends + 2 * n * hkv * d), "flops": 4 * d * hq * pairs}
    lens = _lengths(case)
    rows = case["shared"] + sum(v - case["shared"] for v in lens)
    return {"bytes": 2 * (ends + 2 * rows * hkv * d), "flops": 4 * d * hq * sum(lens)}


# ---- from the definitions, in 64 bits --------------------------------------------


def _exact_rotated(x, w, pos, freq, layout):
    """x [n][h][d] normed and rotated as complex numbers."""
    x = x.to(torch.float64)
    d, half = x.shape[-1], freq.numel()
    x = w.to(torch.float64) * x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       pos.to(torch.float64).outer(freq)).unsqueeze(1)
    even = slice(0, half) if layout == "half" else slice(0, 2 * half, 2)
    odd = slice(half, 2 * half) if layout == "half" else slice(1, 2 * half, 2)
    z = torch.complex(x[..., even], x[..., odd]) * turn
    y = x.clone()
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _exact_rows(q, k, v, limit):
    """Attention of rows q [r][d] over keys k [s][d], row i seeing the first limit[i]."""
    e = (q @ k.T) / math.sqrt(q.shape[1])
    e.masked_fill_(torch.arange(len(k), device=q.device) >= limit[:, None], -math.inf)
    return torch.softmax(e, dim=1) @ v


def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    if case["op"] in ("rope", "append"):
        q = _exact_rotated(s["q"], s["wq"], s["pos"], s["freq"], case["layout"])
        k = _exact_rotated(s["k"], s["wk"], s["pos"], s["freq"], case["layout"])
        if case["op"] == "rope":
            return {"q": q, "k": k}
        kc, vc = s["kc"].double(), s["vc"].double()
        slot = s["pos"].long()
        page = s["table"].long()[s["seq"].long(), torch.div(slot, case["page"], rounding_mode="floor")]
        slot = torch.remainder(slot, case["page"])
        for h in range(hkv):
            kc[page, h, slot] = k[:, h]
            vc[page, h, slot] = s["v"][:, h].double()
        return {"q": q, "k_cache": kc, "v_cache": vc}
    o = torch.zeros(case["n"], hq, d, dtype=torch.float64, device="cuda")
    lens = _lengths(case)
    at = 0
    for b, length in enumerate(lens):
        if case["op"] == "prefill":
            k64, v64 = (s[x][at:at + length].double() for x in ("k", "v"))
            for t in range(0, length, 2048):
                u = min(length, t + 2048)
                limit = torch.arange(t, u, device="cuda") + 1
                for h in range(hq):
                    o[at + t:at + u, h] = _exact_rows(s["q"][at + t:at + u, h].double(),
                                                      k64[:u, h // g], v64[:u, h // g], limit)
            at += length
        else:
            pages = s["table"][b, :-(-length // case["page"])].long()
            for h in range(hkv):
                k64, v64 = (s[x][pages, h].double().reshape(-1, d)[:length] for x in ("kc", "vc"))
                limit = torch.full((g,), length, device="cuda")
                o[b, h * g:(h + 1) * g] = _exact_rows(s["q"][b, h * g:(h + 1) * g].double(), k64,
                                                      v64, limit)
    return o if s["gate"] is None else o / (1 + torch.exp(-s["gate"].double()))
