"""A block-diffusion decoder whose layers have both halves: attention over a paged cache of the
prefix and the masked block (bidirectional in the block, [AIT 四]), and the MoE step.

Per layer:  x -> Wqkv -> kv_cache_write, block_attention -> Wo -> block_residual_norm -> router,
coreset, experts -> block_residual_norm -> the next layer's x.  The last norm feeds the LM head and
the LowConfidence commit.  While a block is being resolved its keys and values are written anew every
round, at the same positions; a resolved block is passed once more, so that the cache holds the
committed tokens', and the next block follows it.

    python examples/block_decoder.py [--fp8-cache] [--requests 2] [--blocks 2] [--prefix 100 | --hybrid]

With --hybrid the cache's pages are given out on the GPU as blocks begin (kv_cache_plan), queries and keys carry
rotary positions (block_rotary), and every second layer has the gated delta rule in the attention's place
(block_delta_rule): its history is read while a block is being resolved, and takes the block in once it is.
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

    def places(self):
        """Positions [R, P] of the block's tokens, and what each request has with them."""
        return self.kv_len[:, None] + torch.arange(self.d.P, dtype=torch.int32, device="cuda"), self.kv_len + self.d.P

    def mixer(self, i: int, L: Layer, pos, seen):
        """The token mixer of layer i over self.x: [T, H]."""
        kd = self.kd
        qkv = (self.x @ L.Wqkv.t()).view(self.T, kd.Hq + 2 * kd.Hkv, kd.D)
        q, k, v = qkv[:, :kd.Hq], qkv[:, kd.Hq:kd.Hq + kd.Hkv], qkv[:, kd.Hq + kd.Hkv:]
        self.rotate(q, k, pos)
        ms.kv_cache_write(kd, self.R, k, v, pos, L.cache, self.kv_ws)
        ms.block_attention(kd, self.R, q, seen, L.cache, self.att, self.kv_ws, kd.D ** -0.5)
        return self.att.view(self.T, -1) @ L.Wo.t()

    def rotate(self, q, k, pos) -> None:
        """(Positions come with the embeddings here.)"""

    def forward(self, record=None, resolved: bool = False) -> None:
        """One pass of the block through the layers; its positions are kv_len .. kv_len + P - 1."""
        d, R = self.d, self.R
        self.resolved = resolved
        pos, seen = self.places()
        ids = torch.where(self.masked.bool(), self.mask_id, self.tokens)
        ms.block_residual_norm(d, self.emb[ids.long()], self.pos_emb.repeat(R, 1), self.h, self.x,
                               w_pre=self.layers[0].attn_in)
        for i, L in enumerate(self.layers):
            if record is not None:
                record.append(dict(h=self.h.clone(), x=self.x.clone()))
            ms.block_residual_norm(d, self.mixer(i, L, pos, seen), self.h, self.h, self.x, w_pre=L.moe_in,
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
        self.begin()
        self.masked.fill_(1)
        rounds = 0
        while rounds < self.d.P and bool(self.masked.any()):
            self.forward()
            ms.lm_head_commit(self.d, self.R, self.x, self.Wlm, threshold, self.tokens, self.masked, self.choice,
                              self.conf, self.accept, self.n_committed, self.ws, logit_scale=logit_scale)
            rounds += 1
        self.forward(resolved=True)  # the committed tokens' keys and values stay
        self.advance()
        return rounds

    def begin(self) -> None:
        """(The pages of all blocks are dealt out in advance here.)"""

    def advance(self) -> None:
        """The block's positions count as cached from here on."""
        self.kv_len += self.d.P

    def check(self) -> None:
        for ws in (self.ws, self.kv_ws):
            word = ms.read_device_error(ws)
            if word != ms.OK:
                raise ms.MoeStepError(word, "device error word")


class HybridDecoder(BlockDecoder):
    """Pages as they are needed, rotary positions in half of every head, and in every second layer the gated delta rule."""

    def __init__(self, d: ms.ModelDims, kd: ms.KvDims, R: int, n_layers: int, seed: int = 0, top_p: float = 0.9):
        super().__init__(d, kd, R, n_layers, seed, top_p)
        g = torch.Generator(device="cuda").manual_seed(seed + 2)
        f32 = dict(dtype=torch.float32, device="cuda")
        self.dd = dd = ms.DeltaDims(Hk=2, Hv=4, Dk=64, Dv=64, n_slots=R)
        self.widths = (dd.Hk * dd.Dk, dd.Hk * dd.Dk, dd.Hv * dd.Dv, dd.Hv, dd.Hv)  # queries, keys, values, decays, rates
        w = lambda *s: (0.02 * torch.randn(s, generator=g, device="cuda")).bfloat16()  # noqa: E731
        self.delta = {i: dict(Win=w(sum(self.widths), d.H), Wout=w(d.H, dd.Hv * dd.Dv),
                              rate=torch.exp(torch.randn(dd.Hv, generator=g, device="cuda") - 3),
                              state=torch.zeros((R, dd.Hv, dd.Dv, dd.Dk), **f32)) for i in range(0, n_layers, 2)}
        self.delta_ws = ms.delta_workspace(dd, R, d.P)
        self.mixed = torch.empty((self.T, dd.Hv, dd.Dv), dtype=torch.bfloat16, device="cuda")
        self.freq = ms.rotary_frequencies(kd.D // 2, 1e4)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table.fill_(-1)
        self.ring = torch.randperm(kd.n_pages, generator=g, device="cuda").to(torch.int32)  # every page is free
        self.head = torch.tensor([0, kd.n_pages], **i32)
        self.pos, self.seen = torch.empty((R, d.P), **i32), torch.zeros(R, **i32)

    def plan(self, n_new) -> None:
        ms.kv_cache_plan(self.kd, self.R, self.kv_len, n_new, self.ring, self.head, self.head, self.table, self.seen, self.pos,
                         self.kv_ws)

    def begin(self) -> None:
        """Pages and positions for a block of every request; where one of them is refused, those of the others go back."""
        self.plan(torch.full_like(self.kv_len, self.d.P))
        self.fresh = (self.kv_len == 0).to(torch.uint8)  # requests that begin, whatever their slots' states hold
        if bool((self.seen != self.kv_len + self.d.P).any()):
            start = self.kv_len.clone()
            self.advance()
            self.plan(start - self.kv_len)
            self.advance()
            raise ms.MoeStepError(ms.EINVAL, "decode_block: no pages left for every request's block")

    def advance(self) -> None:
        self.kv_len.copy_(self.seen)

    def end(self) -> None:
        """Every request ends: its pages go back, its slots may be taken by others."""
        self.plan(-self.kv_len)
        self.advance()

    def places(self):
        return self.pos, self.seen

    def rotate(self, q, k, pos) -> None:
        ms.block_rotary(self.kd, q, k, pos, self.freq, q, k)

    def mixer(self, i: int, L: Layer, pos, seen):
        if i not in self.delta:
            return super().mixer(i, L, pos, seen)
        dd, M = self.dd, self.delta[i]
        q, k, v, a, b = (self.x @ M["Win"].t()).split(self.widths, 1)
        decay = -M["rate"] * torch.nn.functional.softplus(a.float())
        ms.block_delta_rule(dd, self.R, q.unflatten(1, (dd.Hk, dd.Dk)), k.unflatten(1, (dd.Hk, dd.Dk)),
                            v.unflatten(1, (dd.Hv, dd.Dv)), decay, torch.sigmoid(b.float()), M["state"], self.mixed,
                            self.delta_ws, state_out=M["state"] if self.resolved else None, fresh=self.fresh,
                            scale=dd.Dk ** -0.5, qk_eps=1e-6)
        return self.mixed.view(self.T, -1) @ M["Wout"].t()

    def check(self) -> None:
        super().check()
        word = ms.read_device_error(self.delta_ws)
        if word != ms.OK:
            raise ms.MoeStepError(word, "device error word")


def hybrid(R: int, blocks: int, fp8: bool, P: int = 32, seed: int = 0, layers: int = 4) -> HybridDecoder:
    d = ms.ModelDims(H=512, E=32, k=4, I=128, Is=128, V=4096, P=P)
    pages = -(-(blocks * P) // 16)
    kd = ms.KvDims(Hq=8, Hkv=2, D=64, page=16, n_pages=R * pages + 1, max_pages=pages, dtype=ms.FP8 if fp8 else ms.BF16)
    return HybridDecoder(d, kd, R, layers, seed)


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
    ap.add_argument("--prefix", type=int, help="cached positions of random keys and values before the first block (100)")
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--hybrid", action="store_true")
    a = ap.parse_args()
    if a.hybrid and a.prefix is not None:
        ap.error("--prefix writes keys and values only: a --hybrid decoder begins without one")
    prefix = 100 if a.prefix is None else a.prefix
    m = hybrid(a.requests, a.blocks, a.fp8_cache) if a.hybrid else small(a.requests, prefix, a.blocks, a.fp8_cache)
    for b in range(a.blocks):
        rounds = m.decode_block(logit_scale=8.0)
        m.check()
        print(f"block {b}: {rounds} rounds, cached positions {m.kv_len.tolist()}, "
              f"tokens of request 0 {m.tokens[:m.d.P].tolist()}")


if __name__ == "__main__":
    main()
