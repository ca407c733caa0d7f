"""Draft verification: large batches."""
import pytest
import torch

from test_gpu_verify import pk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [620, 609])
def test_larger_vocabularies_one_after_another(S):
    # a CTA a request: 8 bytes of shared memory for each 512 tokens, first some 49 KB, then 64 KB
    for V in (3200000, 2 ** 22):
        target = torch.zeros(1, V, device="cuda")
        target[0, V - 3] = 0.25
        out = torch.empty(S, 1, dtype=torch.int64, device="cuda")
        acc = torch.empty(S, dtype=torch.int32, device="cuda")
        starts = torch.ones(S + 1, dtype=torch.int32, device="cuda")           # the first request alone has a row
        starts[0] = 0
        pk().verify_drafts(out, acc, target, torch.empty(S, 0, dtype=torch.int64, device="cuda"), torch.full((S, 1), 0.5, device="cuda"), starts)
        assert out.view(-1).tolist() == [V - 3] + [-1] * (S - 1)
