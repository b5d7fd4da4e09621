"""gdn_qk_norm_rope and gdn_kv_append against 64-bit forms (tests/_attn.py has
the bounds): every I/O type, head dim and rotation layout, partial and whole
rotation, one token to several CTAs of tokens, far positions, strided views,
in place, missing weights, padding rows, rows without a place in the cache."""
import pytest
import torch

import gated_deltanet_linear_07_gb300 as gdn
from tests import _attn
from tests._attn import IO, normal

pytestmark = pytest.mark.gpu


def _inputs(seed, n, hq, hkv, d, rot, io, start=0, theta=1e6):
    g = torch.Generator().manual_seed(seed)
    dt = IO[io]
    qg, kv = normal(g, n, hq, 2 * d, dtype=dt), normal(g, n, 2 * hkv, d, dtype=dt)
    wq, wk = 1 + 0.1 * normal(g, d, dtype=torch.float32), 1 + 0.1 * normal(g, d, dtype=torch.float32)
    pos = (start + torch.randint(0, 1000, (n,), generator=g)).to(torch.int32)
    freq = gdn.rope_frequencies(rot, theta)[0] if rot else None
    return dict(qg=qg.cuda(), kv=kv.cuda(), wq=wq.cuda(), wk=wk.cuda(), pos=pos.cuda(),
                freq=None if freq is None else freq.cuda(), cpu=(qg, kv, wq, wk, pos, freq))


def _check(got, x, w, pos, freq, layout, dt, what, eps=1e-6, scale=1.0):
    ref, slack = _attn.norm_rope(x, w, eps, pos, freq if freq is not None else torch.zeros(0), layout,
                                 scale)
    _attn.check(got, ref, slack, dt, what)


CASES = [   # n, hq, hkv, d, rot, layout, io, start
    (1, 16, 4, 256, 64, "half", "bf16", 100_000),
    (1, 3, 1, 64, 64, "interleaved", "fp32", 0),
    (5, 6, 2, 128, 96, "half", "fp16", 1_000_000),      # rot / 2 = 48: not a power of two
    (7, 6, 2, 128, 48, "interleaved", "bf16", 2_000_000_000),
    (33, 4, 4, 64, 16, "half", "bf16", 0),
    (130, 16, 4, 256, 256, "half", "fp32", 262_144),
    (64, 2, 1, 256, 0, "half", "bf16", 0),              # norms alone
    (2049, 8, 2, 64, 32, "interleaved", "fp16", 5),     # four tokens per CTA, a ragged last one
    (2050, 5, 1, 128, 128, "half", "bf16", 0),
    (1024, 16, 4, 256, 64, "half", "bf16", 500_000),
    (1100, 40, 8, 256, 256, "half", "fp32", 3),         # a token's rows in several parts
    (1500, 96, 2, 128, 32, "interleaved", "bf16", 9),
]


@pytest.mark.parametrize("n,hq,hkv,d,rot,layout,io,start", CASES)
def test_norm_rope(gpu_lib, n, hq, hkv, d, rot, layout, io, start):
    i = _inputs(11 + n, n, hq, hkv, d, rot, io, start)
    qg, kv, wq, wk, pos, freq = i["cpu"]
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, rot_dim=rot, rope=layout)
    # strided views: q beside its gate, k beside v
    q, k = gdn.gdn_qk_norm_rope(dims, i["qg"][:, :, :d], i["kv"][:, :hkv], i["wq"], i["wk"],
                                i["freq"], i["pos"])
    _check(q, qg[:, :, :d], wq, pos, freq, layout, IO[io], "q")
    _check(k, kv[:, :hkv], wk, pos, freq, layout, IO[io], "k")


def test_norm_rope_in_place_without_weights_one_side_and_scale(gpu_lib):
    n, hq, hkv, d = 19, 4, 2, 128
    i = _inputs(5, n, hq, hkv, d, 64, "bf16", 77)
    qg, kv, wq, wk, pos, freq = i["cpu"]
    dims = gdn.make_attn_dims(hq, hkv, d, rot_dim=64, norm_eps=0.5)
    q = i["qg"][:, :, :d].contiguous()
    out, none = gdn.gdn_qk_norm_rope(dims, q, None, i["wq"], None, i["freq"], i["pos"], q_out=q,
                                     rope_scale=1.25)
    assert none is None and out is q
    _check(q, qg[:, :, :d], wq, pos, freq, "half", torch.bfloat16, "q", eps=0.5, scale=1.25)
    none, k = gdn.gdn_qk_norm_rope(dims, None, i["kv"][:, :hkv], None, None, i["freq"], i["pos"])
    assert none is None
    _check(k, kv[:, :hkv], None, pos, freq, "half", torch.bfloat16, "k")
    empty = torch.empty(0, hq, d, dtype=torch.bfloat16, device="cuda")
    eq, _ = gdn.gdn_qk_norm_rope(dims, empty, None, None, None, i["freq"], i["pos"][:0])
    assert eq.shape == (0, hq, d)


def test_norm_of_zero_and_large_rows(gpu_lib):
    """A row of zeros stays zero (eps keeps the root away from it); a row whose
    squares pass the fp16 range does not overflow."""
    d = 256
    x = torch.zeros(2, 1, d, dtype=torch.float16)
    x[1] = 60000.0
    dims = gdn.make_attn_dims(1, 1, d, io="fp16")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    w = torch.ones(d, device="cuda")
    q, _ = gdn.gdn_qk_norm_rope(dims, x.cuda(), None, w, None, None, pos)
    assert (q[0] == 0).all() and (q[1] == 1).all()


def test_append_of_many_rows_repeats_the_few(gpu_lib):
    """The kernels for many and for few tokens give the same bits: a prompt
    appended at once and the same prompt in pieces."""
    n, hq, hkv, d, page = 1303, 4, 2, 256, 64
    i = _inputs(31, n, hq, hkv, d, 64, "bf16", 0)
    dims = gdn.make_attn_dims(hq, hkv, d, rot_dim=64, page_size=page)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    pos[700] = -1
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    table = torch.arange(21, dtype=torch.int32, device="cuda").flip(0).view(1, 21).contiguous()
    made = []
    for cuts in ([0, n], [0, 1, 130, 1000, n]):
        kc = torch.zeros(21, hkv, page, d, dtype=torch.bfloat16, device="cuda")
        vc, qs = torch.zeros_like(kc), []
        for a, b in zip(cuts, cuts[1:]):
            qs.append(gdn.gdn_kv_append(dims, i["qg"][a:b, :, :d], i["kv"][a:b, :hkv],
                                        i["kv"][a:b, hkv:], i["wq"], i["wk"], i["freq"], pos[a:b], kc,
                                        vc, table, row_seq=seq[a:b]))
        made.append((torch.cat(qs), kc, vc))
    for one, many in zip(*made):
        assert torch.equal(one, many)
    qg, kv, wq, wk, _, freq = i["cpu"]
    live = torch.arange(n) != 700
    p = pos.cpu()[live]
    _check(made[0][0][live.cuda()], qg[live][:, :, :d], wq, p, freq, "half", torch.bfloat16, "q")
    assert (made[0][0][700] == 0).all()
    pg, off = 20 - p.long() // page, p.long() % page
    _check(made[0][1].cpu()[pg, :, off], kv[live][:, :hkv], wk, p, freq, "half", torch.bfloat16, "k")
    assert torch.equal(made[0][2].cpu()[pg, :, off], kv[live][:, hkv:])


@pytest.mark.parametrize("io,d,page,layout", [("bf16", 256, 64, "half"), ("fp16", 128, 16, "half"),
                                              ("fp32", 64, 32, "interleaved"),
                                              ("bf16", 64, 128, "half")])
def test_append(gpu_lib, io, d, page, layout):
    n, hq, hkv, seqs, per = 57, 4, 2, 3, 5
    dt = IO[io]
    i = _inputs(21, n, hq, hkv, d, 32, io)
    qg, kv, wq, wk, _, freq = i["cpu"]
    g = torch.Generator().manual_seed(3)
    pool = seqs * per + 2
    table = torch.randperm(pool, generator=g)[:seqs * per].view(seqs, per).to(torch.int32)
    kc, vc = normal(g, pool, hkv, page, d, dtype=dt), normal(g, pool, hkv, page, d, dtype=dt)
    seq = torch.arange(n) % seqs
    pos = (torch.arange(n) // seqs) * 3 + 1          # distinct places, pages crossed
    pos[7] = pos[30] = -1                            # padding rows
    pos = pos.clamp(max=per * page - 1).to(torch.int32)
    seq = seq.to(torch.int32)
    dims = gdn.make_attn_dims(hq, hkv, d, io=io, rot_dim=32, rope=layout, page_size=page)
    kcd, vcd = kc.cuda(), vc.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = gdn.gdn_kv_append(dims, i["qg"][:, :, :d], i["kv"][:, :hkv], i["kv"][:, hkv:], i["wq"],
                          i["wk"], i["freq"], pos.cuda(), kcd, vcd, table.cuda(), row_seq=seq.cuda(),
                          d_status=status)
    assert status.item() == 0
    live = pos >= 0
    _check(q[live.cuda()], qg[live][:, :, :d], wq, pos[live], freq, layout, dt, "q")
    assert (q[7] == 0).all() and (q[30] == 0).all()
    touched = torch.zeros(pool, page, dtype=torch.bool)
    pg = table[seq[live].long(), pos[live].long() // page].long()
    off = pos[live].long() % page
    assert len(set(zip(pg.tolist(), off.tolist()))) == int(live.sum())
    touched[pg, off] = True
    _check(kcd.cpu()[pg, :, off], kv[live][:, :hkv], wk, pos[live], freq, layout, dt, "k")
    assert torch.equal(vcd.cpu()[pg, :, off], kv[live][:, hkv:])
    rest = ~touched[:, None, :, None].expand_as(kc)
    assert torch.equal(kcd.cpu()[rest], kc[rest]) and torch.equal(vcd.cpu()[rest], vc[rest])


def test_append_rows_without_a_place_are_reported_and_left_out(gpu_lib):
    hq, hkv, d, page = 2, 1, 64, 16
    dims = gdn.make_attn_dims(hq, hkv, d, page_size=page)
    g = torch.Generator().manual_seed(1)
    q, k, v = (normal(g, 4, h, d).cuda() for h in (hq, hkv, hkv))
    w = torch.ones(d, device="cuda")
    table = torch.tensor([[0, 1], [2, 99], [3, -1]], dtype=torch.int32, device="cuda")

    def call(pos, seq):
        kc = torch.zeros(4, hkv, page, d, dtype=torch.bfloat16, device="cuda")
        vc, status = torch.zeros_like(kc), torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_kv_append(dims, q, k, v, w, w, None,
                          torch.tensor(pos, dtype=torch.int32, device="cuda"), kc, vc, table,
                          row_seq=torch.tensor(seq, dtype=torch.int32, device="cuda"),
                          d_status=status)
        return status.item(), int((vc != 0).any(-1).sum())
    assert call([0, 1, 2, 31], [0, 0, 0, 0]) == (0, 4)
    assert call([0, 1, 2, 32], [0, 0, 0, 0]) == (gdn.GDN_DEV_BAD_LENGTH, 3)
    assert call([0, 1, 2, 3], [0, 0, 3, -1]) == (gdn.GDN_DEV_BAD_LENGTH, 2)
    assert call([0, 1, 16, 17], [0, 0, 1, 2]) == (gdn.GDN_DEV_BAD_PAGE, 2)


def test_append_without_queries_and_one_row_per_sequence(gpu_lib):
    hq, hkv, d, page, n = 8, 4, 128, 32, 6
    i = _inputs(9, n, hq, hkv, d, 128, "bf16", 0)
    _, kv, _, wk, _, freq = i["cpu"]
    pos = torch.tensor([0, 31, 32, 63, 5, 40], dtype=torch.int32)
    table = torch.arange(2 * n, dtype=torch.int32).flip(0).view(n, 2).contiguous()
    kc = torch.zeros(2 * n, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    dims = gdn.make_attn_dims(hq, hkv, d, rot_dim=128, page_size=page)
    assert gdn.gdn_kv_append(dims, None, i["kv"][:, :hkv], i["kv"][:, hkv:], None, i["wk"],
                             i["freq"], pos.cuda(), kc, vc, table.cuda()) is None
    pg = table[torch.arange(n), pos.long() // page].long()
    _check(kc.cpu()[pg, :, pos.long() % page], kv[:, :hkv], wk, pos, freq, "half", torch.bfloat16, "k")
    assert torch.equal(vc.cpu()[pg, :, pos.long() % page], kv[:, hkv:])


@pytest.mark.parametrize("n", [50, 700])
def test_append_with_packed_keys_is_the_norm_and_rotation_and_the_append(gpu_lib, n):
    hq, hkv, d, page = 4, 2, 128, 16
    i = _inputs(41, n, hq, hkv, d, 128, "bf16", 0)
    dims = gdn.make_attn_dims(hq, hkv, d, rot_dim=128, page_size=page)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    pos[9] = -1
    q, k, v = i["qg"][:, :, :d], i["kv"][:, :hkv], i["kv"][:, hkv:]
    w = (i["wq"], i["wk"], i["freq"], pos)
    qn, kn = gdn.gdn_qk_norm_rope(dims, q, k, *w)
    pages = (n + page - 1) // page
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    kc = torch.zeros(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc, packed = torch.zeros_like(kc), torch.full((n, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    qa = gdn.gdn_kv_append(dims, q, k, v, *w, kc, vc, table, row_seq=seq, k_out=packed)
    live = torch.arange(n, device="cuda") != 9
    assert torch.equal(qa[live], qn[live]) and torch.equal(packed[live], kn[live])
    assert (qa[9] == 0).all() and (packed[9] == 0).all()
    rows = kc.transpose(1, 2).reshape(-1, hkv, d)[:n]
    assert torch.equal(rows[live], kn[live]) and (rows[9] == 0).all()
    assert torch.equal(vc.transpose(1, 2).reshape(-1, hkv, d)[:n][live], v[live])
