"""The example decoder's requests: one that begins takes nothing from the one before it, and a block without pages is refused
whole."""
import pytest
import torch

import moe_expert_step_gb300 as ms
from examples.block_decoder import HybridDecoder, hybrid

pytestmark = pytest.mark.gpu


def test_a_new_request_begins_from_nothing():
    """After end() the same decoder gives the tokens of one that has just been made; nothing is cleared by hand."""
    runs = []
    m = hybrid(2, 2, False, seed=5)
    for _ in range(3):
        toks = []
        for _ in range(2):
            m.decode_block(logit_scale=8.0)
            toks.append(m.tokens.clone())
        runs.append(torch.stack(toks))
        m.end()
        m.check()
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def small_pool(R, blocks, pages):
    d = ms.ModelDims(H=512, E=32, k=4, I=128, Is=128, V=4096, P=32)
    kd = ms.KvDims(Hq=8, Hkv=2, D=64, page=16, n_pages=pages, max_pages=2 * blocks)
    return HybridDecoder(d, kd, R, 4, 9)


@pytest.mark.parametrize("R,blocks,pages", [(2, 2, 100), (2, 9, 8), (3, 9, 13)])
def test_a_block_without_pages_is_refused_whole(R, blocks, pages):
    """Two blocks fit; the third passes the tables' end, or the pages that are left (all of it, or that of the last
    request).  Lengths, pages and histories stay, and after end() the decoder serves as at first."""
    m = small_pool(R, blocks, pages)
    first = []
    for _ in range(2):
        m.decode_block(logit_scale=8.0)
        first.append(m.tokens.clone())
    before = [M["state"].clone() for M in m.delta.values()]
    lengths, free = m.kv_len.clone(), int(m.head[1])
    for _ in range(2):
        with pytest.raises(ms.MoeStepError, match="pages"):
            m.decode_block(logit_scale=8.0)
        assert torch.equal(m.kv_len, lengths) and int(m.head[1]) == free
        assert all(torch.equal(a, M["state"]) for a, M in zip(before, m.delta.values()))
    held = [int(p) for r in range(R) for p in m.table[r, :4]]
    ring = m.ring.tolist()
    at = int(m.head[0])
    assert sorted(held + [ring[(at + i) % pages] for i in range(free)]) == list(range(pages))  # every page once
    m.end()
    assert int(m.head[1]) == pages
    for toks in first:
        m.decode_block(logit_scale=8.0)
        assert torch.equal(m.tokens, toks)
    m.check()
