"""A KV cache's whole way through the library, on one MI355X:

    received     the coded cache is decoded to fp16 (kvc_decode)
    resident     its tokens are written into a paged 4-bit pool (kvc_kv4_append)
    served       every new token is written and attended with all before it
                 (kvc_kv4_append + kvc_kv4_attention), one captured HIP graph a step
    sent on      the tokens are read back (kvc_kv4_read) and coded again

    python examples/resident_cache.py [--tokens 4096] [--steps 64]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import entropy_coding_02_amd as kvc  # noqa: E402
import kvgen  # noqa: E402

H, D, R, PAGE = 8, 128, 4, 64  # kv heads, channels a head, query heads a kv head, tokens a page


def main(n_tokens: int = 4096, n_steps: int = 64) -> dict:
    cfg = kvgen.CONFIGS["c3"].scaled(n_layers=2, n_tokens=n_tokens, layer_bins=((0, 2, 32),))
    L, T = cfg.n_layers, n_tokens
    kv = torch.from_numpy(kvgen.generate(cfg)[0].view(np.int16)).cuda()

    # received: here coded and decoded in one process
    desc = kvc.Desc(L, H * D, T, cfg.bins(), cfg.chunk_tokens)
    buf = kvc.alloc(desc)
    kvc.encode(buf, kv)
    kvc.decode(buf)
    dec = buf.out[: kv.numel()].view(L, 2, T, H, D)

    # resident: one pool a layer, the same page table for all
    n_pages = -(-(T + n_steps) // PAGE)
    table = torch.randperm(n_pages, device="cuda").to(torch.int32).view(1, n_pages)
    pos = torch.arange(T, device="cuda")
    slots = table[0].long()[pos // PAGE] * PAGE + pos % PAGE
    pools = [kvc.Kv4Cache(H, D, n_pages, page_tokens=PAGE) for _ in range(L)]
    for layer, pool in enumerate(pools):
        kvc.kv4_append(pool, dec[layer, 0], dec[layer, 1], slots)

    # served: the step's inputs live at fixed addresses, the graph is captured once
    q = torch.zeros((L, 1, H * R, D), dtype=torch.bfloat16, device="cuda")
    new = torch.zeros((L, 2, 1, H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    slot = torch.full((1,), -1, dtype=torch.int64, device="cuda")  # none: the warm-up call writes nothing
    length = torch.tensor([T], dtype=torch.int32, device="cuda")
    work = torch.empty(kvc.kv4_work_bytes(pools[0], 1, H * R, 1, n_pages, 1), dtype=torch.uint8, device="cuda")

    def step():
        for layer, pool in enumerate(pools):
            kvc.kv4_append(pool, new[layer, 0], new[layer, 1], slot)
            kvc.kv4_attention(pool, q[layer], table, length, out=out[layer], work=work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    gen = torch.Generator(device="cuda").manual_seed(0)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for i in range(n_steps):
        t = T + i
        slot.copy_(table[0, t // PAGE].long().view(1) * PAGE + t % PAGE)
        length.fill_(t + 1)
        q.normal_(generator=gen)
        new.normal_(generator=gen)
        graph.replay()
    end.record()
    torch.cuda.synchronize()

    # sent on: what was received, as the pool holds it
    back = torch.empty_like(dec)
    for layer, pool in enumerate(pools):
        kvc.kv4_read(pool, slots, k=back[layer, 0], v=back[layer, 1])
    kvc.encode(buf, back)
    kvc.decode(buf)
    torch.cuda.synchronize()
    status = int(buf.dev_status.item()) | sum(int(p.dev_status.item()) for p in pools)
    err = (back.float() - dec.float()).square().mean().sqrt() / dec.float().square().mean().sqrt()
    coded = int(buf.slab_off[desc.n_slabs].item())
    return {"status": status, "out": out, "rms_error": float(err), "us_per_step": begin.elapsed_time(end) * 1e3 / n_steps,
            "bytes_fp16": kv.numel() * 2, "bytes_resident": sum(p.codes.numel() + 2 * p.params.numel() for p in pools),
            "bytes_coded": coded}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    r = main(a.tokens, a.steps)
    r.pop("out")
    print(r)
