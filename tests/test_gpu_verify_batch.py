"""Draft verification: large batches, steps without drafts."""
import pytest
import torch

import step_common as sc
from test_gpu_verify import inputs, pk

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


@pytest.mark.parametrize("S", [1, 5, 90])
def test_steps_without_drafts(S):
    # draft_probs as a program keeps them, of no drafts: [S, 0, V]
    target, _, drafted, uniforms, starts = inputs(S, 0, 700, S)
    out = torch.empty(S, 1, dtype=torch.int64, device="cuda")
    acc = torch.empty(S, dtype=torch.int32, device="cuda")
    pk().verify_drafts(out, acc, target.cuda(), drafted.cuda(), uniforms.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"),
                       draft_probs=torch.empty(S, 0, 700, device="cuda"))
    want, accepted, _ = sc.verify(target, None, drafted, uniforms, starts)
    assert out.tolist() == want.tolist() and acc.tolist() == accepted.tolist()
    # and views that are not evenly spaced are still refused
    with pytest.raises(ValueError):
        pk().verify_drafts(torch.empty(2, 3, dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"),
                           torch.ones(6, 8, device="cuda"), torch.zeros(2, 2, dtype=torch.int64, device="cuda"),
                           torch.zeros(2, 3, device="cuda"), torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda"),
                           draft_probs=torch.ones(2, 3, 8, device="cuda")[:, :2])
