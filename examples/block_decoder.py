"""A block-diffusion decoder whose layers have both halves: attention over a paged cache of the
prefix and the masked block (bidirectional in the block, [AIT 四]), and the MoE step.

Per layer:  x -> Wqkv -> kv_cache_write, block_attention -> Wo -> block_residual_norm -> router,
coreset, experts -> block_residual_norm -> the next layer's x.  The last norm feeds the LM head and
the LowConfidence commit.  While a block is being resolved its keys and values are written anew every
round, at the same positions; a resolved block is passed once more, so that the cache holds the
committed tokens', and the next block follows it.

    python examples/block_decoder.py [--fp8-cache] [--requests 2] [--prefix 100] [--blocks 2]
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_step_gb300 as ms  # noqa: E402


@dataclass
class Layer:
    Wqkv: torch.Tensor     # [(Hq + 2 Hkv) * D, H]
    Wo: torch.Tensor       # [H, Hq * D]
    attn_in: torch.Tensor  # norm weights [H]: before and after the attention, before and after the experts
    attn_out: torch.Tensor
    moe_in: torch.Tensor
    moe_out: torch.Tensor
    moe: object            # ms.Layer
    Wr: torch.Tensor
    cache: object          # ms.KvCache
    pools: tuple


class BlockDecoder:
    """R requests, blocks of d.P positions; random weights."""

    def __init__(self, d: ms.ModelDims, kd: ms.KvDims, R: int, n_layers: int, seed: int = 0, top_p: float = 0.9):
        self.d, self.kd, self.R, self.T = d, kd, R, R * d.P
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = torch.bfloat16
        w = lambda *s, std=0.02: (std * torch.randn(s, generator=g, device="cuda")).to(bf)  # noqa: E731
        norm = lambda: (1 + 0.1 * torch.randn(d.H, generator=g, device="cuda")).to(bf)  # noqa: E731
        store = torch.float8_e4m3fn if kd.dtype == ms.FP8 else bf
        # each request's pages, dealt out in turn
        self.table = torch.arange(R * kd.max_pages, dtype=torch.int32, device="cuda").view(kd.max_pages, R).t().contiguous()
        self.layers = []
        for _ in range(n_layers):
            pools = [torch.zeros((kd.n_pages, kd.Hkv, kd.page, kd.D), device="cuda").to(store) for _ in "kv"]
            exps = [torch.zeros((kd.n_pages, kd.Hkv, kd.page), dtype=torch.uint8, device="cuda")
                    if kd.dtype == ms.FP8 else None for _ in "kv"]
            Wr = w(d.E, d.H)
            moe = ms.layer(Wr, w(d.E, d.I, 2, d.H), w(d.E, d.H, d.I), w(d.Is, 2, d.H), w(d.H, d.Is))
            self.layers.append(Layer(w((kd.Hq + 2 * kd.Hkv) * kd.D, d.H), w(d.H, kd.Hq * kd.D), norm(), norm(), norm(),
                                     norm(), moe, Wr, ms.kv_cache(*pools, self.table, *exps), (*pools, *exps)))
        self.final = norm()
        self.gate = 0.5 + 0.1 * torch.randn((R, d.H), generator=g, device="cuda")  # of each request's residual updates
        self.emb, self.pos_emb, self.Wlm = w(d.V, d.H, std=1.0), torch.randn((d.P, d.H), generator=g, device="cuda"), w(d.V, d.H)
        self.mask_id = d.V - 1
        self.top_p = torch.full((R,), top_p, device="cuda")
        self.ws, self.kv_ws = ms.workspace(d, R), ms.kv_workspace(kd, R, d.P)
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda")  # noqa: E731
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        T = self.T
        self.h, self.x = f32(T, d.H), torch.empty((T, d.H), dtype=bf, device="cuda")
        self.att = torch.empty((T, kd.Hq, kd.D), dtype=bf, device="cuda")
        self.idx, self.mass, self.gates, self.gate_rr = i32(T, d.k), f32(T, d.k), f32(T, d.k), f32(T, d.k)
        self.n_sel, self.sel, self.out = i32(R), i32(R, d.E), f32(T, d.H)
        self.survive = torch.empty((T, d.k), dtype=torch.uint8, device="cuda")
        self.tokens, self.masked = i32(T), torch.ones(T, dtype=torch.uint8, device="cuda")
        self.choice, self.conf = i32(T), f32(T)
        self.accept, self.n_committed = torch.zeros(T, dtype=torch.uint8, device="cuda"), i32(R)
        self.kv_len = i32(R)

    def forward(self, record=None) -> None:
        """One pass of the block through the layers; its positions are kv_len .. kv_len + P - 1."""
        d, kd, R = self.d, self.kd, self.R
        pos = self.kv_len[:, None] + torch.arange(d.P, dtype=torch.int32, device="cuda")
        seen = self.kv_len + d.P
        ids = torch.where(self.masked.bool(), self.mask_id, self.tokens)
        ms.block_residual_norm(d, self.emb[ids.long()], self.pos_emb.repeat(R, 1), self.h, self.x,
                               w_pre=self.layers[0].attn_in)
        for i, L in enumerate(self.layers):
            if record is not None:
                record.append(dict(h=self.h.clone(), x=self.x.clone()))
            qkv = (self.x @ L.Wqkv.t()).view(self.T, kd.Hq + 2 * kd.Hkv, kd.D)
            q, k, v = qkv[:, :kd.Hq], qkv[:, kd.Hq:kd.Hq + kd.Hkv], qkv[:, kd.Hq + kd.Hkv:]
            ms.kv_cache_write(kd, R, k, v, pos, L.cache, self.kv_ws)
            ms.block_attention(kd, R, q, seen, L.cache, self.att, self.kv_ws, kd.D ** -0.5)
            ms.block_residual_norm(d, self.att.view(self.T, -1) @ L.Wo.t(), self.h, self.h, self.x, w_pre=L.moe_in,
                                   w_post=L.attn_out, gate=self.gate)
            if record is not None:
                record[-1] |= dict(h_mid=self.h.clone(), x_mid=self.x.clone())
            ms.moe_block_route(d, self.x, L.Wr, self.idx, self.mass, self.gates, self.ws)
            ms.coreset_select(d, R, self.top_p, self.idx, self.mass, self.n_sel, self.sel, self.survive, self.gate_rr,
                              self.ws)
            ms.moe_block_ffn(d, R, self.x, L.moe, self.gate_rr, self.out, self.ws)
            after = self.layers[i + 1].attn_in if i + 1 < len(self.layers) else self.final
            ms.block_residual_norm(d, self.out, self.h, self.h, self.x, w_pre=after, w_post=L.moe_out, gate=self.gate)

    def decode_block(self, threshold: float = 0.95, logit_scale: float = 1.0) -> int:
        """Resolve one block; returns the rounds it took.  The tokens are in self.tokens."""
        self.masked.fill_(1)
        rounds = 0
        while rounds < self.d.P and bool(self.masked.any()):
            self.forward()
            ms.lm_head_commit(self.d, self.R, self.x, self.Wlm, threshold, self.tokens, self.masked, self.choice,
                              self.conf, self.accept, self.n_committed, self.ws, logit_scale=logit_scale)
            rounds += 1
        self.forward()  # the committed tokens' keys and values stay
        self.kv_len += self.d.P
        return rounds

    def check(self) -> None:
        for ws in (self.ws, self.kv_ws):
            word = ms.read_device_error(ws)
            if word != ms.OK:
                raise ms.MoeStepError(word, "device error word")


def small(R: int, prefix: int, blocks: int, fp8: bool, P: int = 32, seed: int = 0, layers: int = 2) -> BlockDecoder:
    d = ms.ModelDims(H=512, E=32, k=4, I=128, Is=128, V=4096, P=P)
    pages = -(-(prefix + (blocks + 1) * P) // 16)
    kd = ms.KvDims(Hq=8, Hkv=2, D=64, page=16, n_pages=R * pages, max_pages=pages, dtype=ms.FP8 if fp8 else ms.BF16)
    m = BlockDecoder(d, kd, R, layers, seed)
    # a prefix as if it had been decoded: its keys and values, written in one call
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    if prefix:
        pos = torch.arange(prefix, dtype=torch.int32, device="cuda").repeat(R, 1)
        for L in m.layers:
            kv = torch.randn((R * prefix, 2 * kd.Hkv, kd.D), generator=g, device="cuda").bfloat16()
            ms.kv_cache_write(kd, R, kv[:, :kd.Hkv], kv[:, kd.Hkv:], pos, L.cache, m.kv_ws)
    m.kv_len.fill_(prefix)
    return m


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--fp8-cache", action="store_true")
    ap.add_argument("--requests", type=int, default=2)
    ap.add_argument("--prefix", type=int, default=100)
    ap.add_argument("--blocks", type=int, default=2)
    a = ap.parse_args()
    m = small(a.requests, a.prefix, a.blocks, a.fp8_cache)
    for b in range(a.blocks):
        rounds = m.decode_block(logit_scale=8.0)
        m.check()
        print(f"block {b}: {rounds} rounds, cached positions {m.kv_len.tolist()}, "
              f"tokens of request 0 {m.tokens[:m.d.P].tolist()}")


if __name__ == "__main__":
    main()
