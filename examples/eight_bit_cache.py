"""The gated full-attention layer of a model that sees images, served from a paged cache
held in 8 bits and cut down by what its tokens' attention is worth.

Every request is a prompt of text around one image, whose tokens have a position in
time, height and width; then tokens are decoded one by one.  Per layer the calls are

  prompt   gdn_kv8_append       norm and rotate q and k, fill the cache's pages
           gdn_attn_prefill     causal attention over the packed prompts
  token    gdn_kv8_append       the new token's q, k, v
           gdn_attn_decode_kv8  against the cache, adding up what each cached token
                                receives
  full     gdn_kv8_evict        the first and last tokens and those that received most
                                go to new pages, the old ones are free

between the layer's projections (plain matmuls here) and with the output gate.  A token
keeps the positions that it was rotated by wherever it comes to lie in the cache.

  python examples/eight_bit_cache.py [--requests 64] [--text 200] [--image 24]
         [--steps 48] [--keep 512] [--check]

--check compares the last decoded outputs with a plain fp32 attention over the
cache's numbers.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_07_gb300 as gdn  # noqa: E402
from full_attention_layer import D, H_KV, H_Q, PAGE, ROT, Layer, ints  # noqa: E402

FIRST, LAST = 4, 32          # places that stay in any case


def prompt_positions(text, side):
    """[3][text + side * side + text]: before, an image of side x side tokens, after."""
    t = torch.arange(text, dtype=torch.int32)
    rows = torch.arange(side, dtype=torch.int32).repeat_interleave(side)
    cols = torch.arange(side, dtype=torch.int32).repeat(side)
    image = torch.stack([torch.zeros_like(rows), rows, cols]) + text
    return torch.cat([t.expand(3, text), image, (t + text + side).expand(3, text)], 1)


def new_cache(dims, requests, places):
    pages = -(-places // PAGE)
    table = torch.arange(requests * pages, dtype=torch.int32, device="cuda").view(requests, pages)
    return gdn.make_kv8_cache(dims, requests * pages, table)


def run(requests=64, text=200, side=24, steps=48, keep=512, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = Layer(gen)
    axes = gdn.make_rope_axes(gdn.rope_sections([ROT // 2 - 2 * (ROT // 8), ROT // 8, ROT // 8],
                                                interleaved=True))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    width = layer.w_qg.shape[1]
    one = prompt_positions(text, side)
    prompt, last = one.shape[1], int(one.max())
    cache = new_cache(layer.dims, requests, prompt + steps)

    def append(q, k, v, positions, starts, cu=None, k_out=None):
        return gdn.gdn_kv8_append(layer.dims, q, k, v, layer.q_norm, layer.k_norm, layer.freq, positions,
                                  cache, starts, cu_seqlens=cu, axes=axes, k_out=k_out,
                                  rope_scale=layer.rope_scale, d_status=status)

    # the prompts; their attention reads the keys as they went in
    x = torch.randn(requests * prompt, width, generator=gen, device="cuda").bfloat16()
    q, gate, k, v = layer.project(x)
    cu = ints([i * prompt for i in range(requests + 1)])
    keys = torch.empty(requests * prompt, H_KV, D, dtype=torch.bfloat16, device="cuda")
    q = append(q, k, v, one.repeat(1, requests).cuda(), ints([0] * requests), cu, keys)
    out = gdn.gdn_attn_prefill(layer.dims, q, keys, v, cu, gate=gate, d_status=status)

    # token by token
    def buffers():
        places = cache.block_table.shape[1] * PAGE
        size = gdn.gdn_attn_decode_kv8_workspace_size(layer.dims, requests, places)
        return (torch.zeros(requests, H_KV, places, device="cuda"),
                torch.empty(size, dtype=torch.uint8, device="cuda"))
    weights, workspace = buffers()
    hidden = out.view(requests, prompt, -1)[:, -1] @ layer.w_o.T
    length, evictions, limit = prompt, 0, max(prompt, keep) + steps // 3
    for step in range(steps):
        if length >= limit:
            to = new_cache(layer.dims, requests, keep + steps)
            kept = torch.empty(requests, H_KV, to.block_table.shape[1] * PAGE, device="cuda")
            gdn.gdn_kv8_evict(layer.dims, cache, weights, ints([length] * requests), keep, to,
                              weights_out=kept, first=FIRST, last=LAST, d_status=status)
            cache, length, evictions, limit = to, keep, evictions + 1, keep + steps // 3
            _, workspace = buffers()
            weights = kept
        q, gate, k, v = layer.project(hidden)
        q = append(q, k, v, ints([last + 1 + step] * (3 * requests)).view(3, requests),
                   ints([length] * requests))
        length += 1
        o = gdn.gdn_attn_decode_kv8(layer.dims, q, cache, ints([length] * requests), workspace, gate=gate,
                                    weights=weights, d_status=status)
        hidden = o.view(requests, -1) @ layer.w_o.T
    assert status.item() == 0
    return dict(layer=layer, cache=cache, length=length, q=q, gate=gate, o=o, weights=weights,
                evictions=evictions, prompt=prompt)


def plain(r):
    """The last step's outputs by a plain fp32 attention over the cache's numbers."""
    c, n = r["cache"], r["length"]
    out = []
    for b in range(len(r["q"])):
        pages = c.block_table[b].long()
        k, v = ((x.view(torch.uint8)[pages].view(x.dtype).float() *
                 s[pages].repeat_interleave(gdn.GDN_KV8_BLOCK, 2)[..., None]
                 ).transpose(0, 1).reshape(H_KV, -1, D)[:, :n]
                for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
        s = r["q"][b].float().view(H_KV, -1, D) @ k.transpose(1, 2) / D ** 0.5
        out.append((torch.softmax(s, -1) @ v).view(H_Q, D))
    return torch.stack(out) * torch.sigmoid(r["gate"].float())


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("requests", 64), ("text", 200), ("image", 24), ("steps", 48), ("keep", 512)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    r = run(a.requests, a.text, a.image, a.steps, a.keep)
    print(f"{a.requests} prompts of {r['prompt']} tokens, {a.steps} decoded, cut to {a.keep} "
          f"{r['evictions']} times: lengths {r['length']}")
    if a.check:
        ref = plain(r)
        print(f"relative difference from plain attention: "
              f"{float((r['o'].float() - ref).norm() / ref.norm()):.2e}")


if __name__ == "__main__":
    main()
