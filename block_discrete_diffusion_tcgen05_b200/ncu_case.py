"""Runs one attention call of a named workload a few times, for profiler captures (ncu).

    python -m block_discrete_diffusion_tcgen05_b200.ncu_case \
        {encoder|decoder_train|encoder_backward|decoder_backward|decoder_sample|kv_append|
         paged_token|paged_block|paged_wide|paged_d64|append_paged|weigh|evict|evict_prompt} [repeats]

Shapes are the benchmark's: E2D2 train pass (B8 L1024 S16 H16 d64) for the two train calls and
their backward (one forward call, then `repeats` backward calls),
E2D2 sampling step (B32 P2048 S16 Hq16 Hkv8 d128) for the sampling call and the append, and the same over
pages of 64 rows for the paged calls (paged_token: S1; evict: to half of the rows; paged_wide and evict_prompt:
B4 P32768 Hq32 Hkv8, to a quarter of the rows; paged_d64: B4 P6000 Hq32 Hkv8 d64).
Inputs are seeded normals drawn on the device (the values do not change the work)."""
from __future__ import annotations

import sys

import torch

from . import attn, workloads


def main(argv):
    which = argv[1] if len(argv) > 1 else "encoder"
    reps = int(argv[2]) if len(argv) > 2 else 3
    dev = torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(1234)

    def rnd(*shape, sigma=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * sigma).to(torch.bfloat16)

    tw, sw = workloads.TRAIN, workloads.SAMPLE
    if which in ("encoder", "decoder_train"):
        shp = (tw.batch, tw.q_heads, tw.L, tw.head_dim)
        q, k, v, ke, ve = (rnd(*shp, sigma=tw.sigma) for _ in range(5))
        for _ in range(reps):
            if which == "encoder":
                attn.encoder_blockcausal(q, k, v, tw.S)
            else:
                attn.decoder_train(q, ke, ve, k, v, tw.S)
    elif which in ("encoder_backward", "decoder_backward"):
        shp = (tw.batch, tw.q_heads, tw.L, tw.head_dim)
        q, k, v, ke, ve = (rnd(*shp, sigma=tw.sigma) for _ in range(5))
        go = rnd(*shp)
        ws = torch.empty(attn.train_backward_workspace_bytes(tw.batch, tw.q_heads, tw.kv_heads, tw.head_dim, tw.L),
                         dtype=torch.uint8, device=dev)
        if which == "encoder_backward":
            o, lse = attn.encoder_blockcausal(q, k, v, tw.S)
            for _ in range(reps):
                attn.encoder_backward(q, k, v, o, lse, go, tw.S, workspace=ws)
        else:
            o, lse = attn.decoder_train(q, ke, ve, k, v, tw.S)
            for _ in range(reps):
                attn.decoder_train_backward(q, ke, ve, k, v, o, lse, go, tw.S, workspace=ws)
    elif which in ("decoder_sample", "kv_append"):
        cap = sw.P + sw.S
        q = rnd(sw.batch, sw.q_heads, sw.S, sw.head_dim)
        kc, vc = (rnd(sw.batch, sw.kv_heads, cap, sw.head_dim) for _ in range(2))
        kb, vb = (rnd(sw.batch, sw.kv_heads, sw.S, sw.head_dim) for _ in range(2))
        ws = attn.sample_workspace(q, kc)
        for _ in range(reps):
            if which == "decoder_sample":
                attn.decoder_sample(q, kc, vc, sw.P, kb, vb, workspace=ws)
            else:
                attn.kv_cache_append(kc, vc, sw.P, kb, vb)
    elif which in ("paged_token", "paged_block", "paged_wide", "paged_d64", "append_paged", "weigh", "evict", "evict_prompt"):
        long = {"paged_wide": (4, 32, 8, 128, 32768), "paged_d64": (4, 32, 8, 64, 6000), "evict_prompt": (4, 8, 8, 128, 32768)}
        B, Hq, Hkv, d, rows = long.get(which, (sw.batch, sw.q_heads, sw.kv_heads, sw.head_dim, sw.P))
        S, page = 1 if which == "paged_token" else sw.S, 64
        keep = rows // (4 if which == "evict_prompt" else 2)
        each = -(-(rows + S) // page)
        kp, vp = (rnd(B * each, Hkv, page, d) for _ in range(2))
        table = torch.randperm(B * each, generator=g, device=dev).view(B, each).to(torch.int32)
        P = torch.full((B,), rows, dtype=torch.int32, device=dev)
        q = rnd(B, Hq, S, d)
        kb, vb = (rnd(B, Hkv, S, d) for _ in range(2))
        w = torch.rand(B, Hkv, each * page, generator=g, device=dev)
        pos = torch.arange(each * page, dtype=torch.int32, device=dev).expand(B, Hkv, -1).contiguous()
        ws, ews = attn.sample_paged_workspace(q, kp), attn.evict_workspace(w)
        w_out, pos_out, P_out = torch.zeros_like(w), torch.zeros_like(pos), torch.zeros_like(P)
        lse = attn.decoder_sample_paged(q, kp, vp, table, P, workspace=ws)[1]
        for _ in range(reps):
            if which.startswith("paged_"):
                attn.decoder_sample_paged(q, kp, vp, table, P, kb, vb, workspace=ws)
            elif which == "append_paged":
                attn.kv_cache_append_paged(kp, vp, table, P, kb, vb)
            elif which == "weigh":
                attn.kv_cache_weigh(q, kp, table, P, lse, w, out=w_out)
            else:
                attn.kv_cache_evict(kp, vp, table, P, w, pos, P, keep, recent=64, weight_out=w_out, pos_out=pos_out,
                                    P_out=P_out, workspace=ews)
    else:
        raise SystemExit(f"unknown call {which}")
    torch.cuda.synchronize()
    assert attn.last_device_error() == 0
    print(f"{which}: {reps} calls ok")


if __name__ == "__main__":
    main(sys.argv)
