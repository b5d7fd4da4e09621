"""The gated full-attention layer of a hybrid model, served from a paged cache.

A batch of requests that share a long prompt (a system prompt, say): the common
part is prefilled once, every request's own part behind it, then tokens are
decoded one by one.  Per layer and step the calls are

  prompt   gdn_kv_append     norm and rotate q and k, fill the cache's pages
           gdn_attn_prefill  causal attention over the packed prompts
  token    gdn_kv_append     the new token's q, k, v
           gdn_attn_decode   against the cache, the common part once for all

between the layer's projections (plain matmuls here) and with the output gate.
The request's own part attends to the common part too: its keys are those of the
common prompt and its own, packed one after the other (cu_seqlens_kv).

  python examples/full_attention_layer.py [--requests 64] [--common 2048]
         [--own 200] [--steps 16] [--check]

--check compares the last decoded outputs with a plain fp32 attention over the
whole sequences.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_07_gb300 as gdn  # noqa: E402

H_Q, H_KV, D, ROT, PAGE, WIDTH = 16, 4, 256, 64, 64, 2560


class Layer:
    """Random weights of one layer: fused q|gate and k|v projections and norms."""

    def __init__(self, gen):
        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device="cuda") * cols ** -0.5).bfloat16()
        self.w_qg, self.w_kv = weight(H_Q * 2 * D, WIDTH), weight(2 * H_KV * D, WIDTH)
        self.w_o = weight(WIDTH, H_Q * D)
        self.q_norm = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        self.k_norm = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        self.freq, self.rope_scale = gdn.rope_frequencies(ROT, 1e7, device="cuda")
        self.dims = gdn.make_attn_dims(H_Q, H_KV, D, rot_dim=ROT, page_size=PAGE)

    def project(self, x):
        """hidden [n, WIDTH] -> q, gate, k, v as views of the two projections."""
        qg = (x @ self.w_qg.T).view(-1, H_Q, 2 * D)
        kv = (x @ self.w_kv.T).view(-1, 2 * H_KV, D)
        return qg[..., :D], qg[..., D:], kv[:, :H_KV], kv[:, H_KV:]


class Cache:
    """A page pool and the sequences' block tables; the common pages come first."""

    def __init__(self, requests, common, longest):
        pages = -(-(common + longest) // PAGE)
        shared = common // PAGE
        pool = shared + requests * (pages - shared)
        self.k = torch.zeros(pool, H_KV, PAGE, D, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        table = torch.arange(pool, dtype=torch.int32)
        self.table = torch.cat([table[:shared].expand(requests, shared),
                                table[shared:].view(requests, -1)], 1).contiguous().cuda()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def append(layer, cache, q, k, v, positions, seq, **kw):
    return gdn.gdn_kv_append(layer.dims, q, k, v, layer.q_norm, layer.k_norm, layer.freq, positions,
                             cache.k, cache.v, cache.table, row_seq=seq,
                             rope_scale=layer.rope_scale, **kw)


def run(requests=64, common=2048, own=200, steps=16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = Layer(gen)
    common = common // PAGE * PAGE                       # whole pages are shared
    cache = Cache(requests, common, own + steps)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = requests * own

    # the common prompt, once; it goes to the pages of every request's table
    x0 = torch.randn(common, WIDTH, generator=gen, device="cuda").bfloat16()
    q, gate, k, v = layer.project(x0)
    k0 = torch.empty(common, H_KV, D, dtype=torch.bfloat16, device="cuda")
    q = append(layer, cache, q, k, v, torch.arange(common, dtype=torch.int32, device="cuda"),
               torch.zeros(common, dtype=torch.int32, device="cuda"), k_out=k0, d_status=status)
    out0 = gdn.gdn_attn_prefill(layer.dims, q, k0, v, ints([0, common]), gate=gate)
    v0 = v

    # every request's own part behind it
    x1 = torch.randn(rows, WIDTH, generator=gen, device="cuda").bfloat16()
    q, gate, k, v = layer.project(x1)
    pos = (common + torch.arange(own, dtype=torch.int32, device="cuda")).repeat(requests)
    seq = torch.arange(requests, dtype=torch.int32, device="cuda").repeat_interleave(own)
    k1 = torch.empty(rows, H_KV, D, dtype=torch.bfloat16, device="cuda")
    q = append(layer, cache, q, k, v, pos, seq, k_out=k1, d_status=status)

    def packed(a, b):   # [common | own] of every request
        return torch.cat([a.expand(requests, common, H_KV, D), b.reshape(requests, own, H_KV, D)],
                         1).view(-1, H_KV, D)
    out1 = gdn.gdn_attn_prefill(layer.dims, q, packed(k0, k1), packed(v0, v),
                                ints([i * own for i in range(requests + 1)]),
                                ints([i * (common + own) for i in range(requests + 1)]), gate=gate)

    # token by token
    workspace = torch.empty(gdn.gdn_attn_decode_workspace_size(layer.dims, requests, common),
                            dtype=torch.uint8, device="cuda")
    hidden = out1.view(requests, own, -1)[:, -1] @ layer.w_o.T
    lens = torch.full((requests,), common + own, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        q, gate, k, v = layer.project(hidden)
        q = append(layer, cache, q, k, v, lens, None, d_status=status)
        lens = lens + 1
        o = gdn.gdn_attn_decode(layer.dims, q, cache.k, cache.v, cache.table, lens, workspace,
                                shared_len=common, gate=gate, d_status=status)
        hidden = o.view(requests, -1) @ layer.w_o.T
    assert status.item() == 0
    return dict(layer=layer, cache=cache, lens=lens, q=q, gate=gate, o=o, prompt=out0, own=out1)


def plain(r):
    """The last step's outputs by a plain fp32 attention over the cached sequences."""
    cache, n = r["cache"], int(r["lens"][0])
    out = []
    for b in range(len(r["lens"])):
        k, v = (c[cache.table[b].long()].transpose(0, 1).reshape(H_KV, -1, D)[:, :n].float()
                for c in (cache.k, cache.v))
        s = r["q"][b].float().view(H_KV, -1, D) @ k.transpose(1, 2) / D ** 0.5
        out.append((torch.softmax(s, -1) @ v).view(H_Q, D))
    return torch.stack(out) * torch.sigmoid(r["gate"].float())


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("requests", 64), ("common", 2048), ("own", 200), ("steps", 16)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    r = run(a.requests, a.common, a.own, a.steps)
    print(f"{a.requests} requests, {a.common} common and {a.own} own tokens each, "
          f"{a.steps} decoded: lengths {int(r['lens'][0])}")
    if a.check:
        ref = plain(r)
        print(f"relative difference from plain attention: "
              f"{float((r['o'].float() - ref).norm() / ref.norm()):.2e}")


if __name__ == "__main__":
    main()
