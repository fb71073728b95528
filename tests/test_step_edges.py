"""Edges of the step operators: calls that the documentation allows and a plain
step does not make (the operators themselves: test_step_ops.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

from sparse_attention_indexer_02_gb300 import torch_api  # noqa: E402
from test_step_ops import cuda, gpu, lib  # noqa: E402,F401


# ---------------------------------------------------------------------------
# verification of drafts
# ---------------------------------------------------------------------------

def _acceptance(u):
    """What u[i] stands for: clamped to [0, 1], NaN is 0."""
    return 0.0 if math.isnan(u) else min(max(u, 0.0), 1.0)


@gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [9, 16])
@pytest.mark.parametrize("certain", [False, True])
def test_verify_acceptance_numbers_past_their_ends(cuda, dt, V, certain):
    """u[i] below 0, above 1, infinite and NaN, against probabilities (exact in every
    type) of which each is zero, the smaller one, or both are equal."""
    us = [math.nan, -math.inf, -1.0, -0.0, 0.0, 2.0 ** -149, 0.5, 1 - 2.0 ** -24, 1.0, 1 + 2.0 ** -23, 2.0, 8.0, math.inf]
    ps = [0.0, 0.125, 0.25, 0.5, 1.0]
    rows = [(u, p, q) for u in us for p in ps for q in ([1.0] if certain else ps)]
    B, x = len(rows), 4
    target = torch.zeros((B, 2, V), device="cuda")
    target[:, 1, 7] = 1.0
    target[:, 0, x] = torch.tensor([p for _, p, _ in rows], device="cuda")
    target[:, 0, 2] = 0.5
    draft = None
    if not certain:
        draft = torch.zeros((B, 1, V), device="cuda")
        draft[:, 0, x] = torch.tensor([q for _, _, q in rows], device="cuda")
    u = torch.zeros((B, 2), device="cuda")
    u[:, 0] = torch.tensor([r[0] for r in rows], device="cuda")
    got = torch_api.verify_drafts(torch.full((B, 1), x, dtype=torch.int32, device="cuda"), target.to(dt), u,
                                  draft_probs=None if certain else draft.to(dt))
    want = [int(_acceptance(u) * q < p) for u, p, q in rows]
    assert got.num_accepted.tolist() == want
    # refused: the first token with weight left; u[1] = 0 draws it (token 2, it has 0.5 of p alone)
    assert got.tokens.tolist() == [[x, 7] if a else [2, -1] for a in want]
