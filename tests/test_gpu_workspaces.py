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
