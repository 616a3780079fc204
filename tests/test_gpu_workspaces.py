"""One workspace, made for the largest call, used by every smaller one after another: the same results as with workspaces
of their own."""
import pytest
import torch

from gpu_util import lib, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab", [(14, 151936), (7, 151936), (300, 8192), (140, 8192), (70, 32003)])
def test_logits(rows, vocab):
    q4 = lib()
    x = torch.randn(rows, vocab, device="cuda", generator=torch.Generator(device="cuda").manual_seed(rows))
    ws = torch.full((q4.logits_argmax_workspace_bytes(rows, vocab),), 0x7F, dtype=torch.uint8, device="cuda")
    for n in sorted({1, 2, 5, 6, 7, 13, 14, 25, 63, 64, 65, 128, 129, 140, 256, 257, rows}):
        if n <= rows:
            say("logits workspace", rows, vocab, n)
            assert torch.equal(q4.q4_logits_argmax(x[:n], workspace=ws), x[:n].argmax(1).int())
            assert torch.equal(q4.q4_logits_argmax(x[:n, : vocab // 2], workspace=ws), x[:n, : vocab // 2].argmax(1).int())


@pytest.mark.parametrize("dim,hq,hk", [(128, 32, 8), (64, 8, 2), (256, 8, 4), (96, 40, 8)])
def test_attention(dim, hq, hk):
    """Steps that shrink and grow, over short and long contexts, causal and of trees, in the one workspace."""
    q4 = lib()
    page, columns, tokens = 16, 400, 64
    g = torch.Generator(device="cuda").manual_seed(dim)
    k, v = (torch.randn(columns, hk, page, dim, device="cuda", generator=g).bfloat16() for _ in range(2))
    cache = q4.KVCache(k, v)
    table = torch.randperm(columns, device="cuda", generator=g).int().view(1, -1)
    q = torch.randn(tokens, hq, dim, device="cuda", generator=g).bfloat16()
    mask = torch.tensor([(1 << i + 1) - 1 if i < 63 else -1 for i in range(tokens)], device="cuda").view(-1, 1)
    ws = torch.full((q4.attention_workspace_most(cache, hq, tokens),), 0x7F, dtype=torch.uint8, device="cuda")
    needs = []
    for n in (64, 40, 16, 5, 2, 1, 33, 64):
        for context in (n, 700, 6000):
            batch = q4.KVBatch(table, torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([context], dtype=torch.int32, device="cuda"),
                               max_query_len=n, max_context_len=context)
            say("attention workspace", dim, n, context)
            needs.append(q4.attention_tree_workspace_bytes(cache, batch, hq, n))
            assert torch.equal(q4.q4_attention_tree(cache, batch, q[:n], mask[:n], workspace=ws), q4.q4_attention_tree(cache, batch, q[:n], mask[:n]))
            assert torch.equal(q4.q4_attention_paged(cache, batch, q[:n], workspace=ws), q4.q4_attention_paged(cache, batch, q[:n]))
    assert 0 < max(needs) <= ws.shape[0] and q4.attention_workspace_most(cache, hq, 0) == 0
    with pytest.raises(q4.Q4Error):
        q4.attention_workspace_most(cache, hq + 1, 4)
