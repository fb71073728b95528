"""Edges of the step operators: calls that the documentation allows and a plain
step does not make (the operators themselves: test_step_ops.py)."""
import math
import re
import textwrap
import types
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")

from sparse_attention_indexer_02_gb300 import _abi, rotary, serving, torch_api  # noqa: E402
from test_serving_ops import Problem, _cu  # noqa: E402
from test_step_ops import _drafted, cuda, gpu, lib  # noqa: E402,F401


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------

def test_rotary_offsets_are_whole_numbers():
    """A fraction is refused, not cut off."""
    for offset in (1.5, 63.999, -0.5):
        with pytest.raises(ValueError, match="offset"):
            rotary.Rotary(64, offset=offset, device="cpu")
    for offset in (2, 2.0):
        assert rotary.Rotary(64, offset=offset, device="cpu").offset == 2


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


@gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("B,K", [(70, 2), (16, 1), (16, 40), (200, 3)])
@pytest.mark.parametrize("V", [140000, 9001])
@pytest.mark.parametrize("certain", [False, True])
def test_verify_whole_rows_in_every_cluster(cuda, dt, B, K, V, certain):
    """Accepted counts by comparisons of their own, and every entry of the outputs."""
    if B * K * V > 200 * 2 * 140000:
        B = max(1, 200 * 2 * 140000 // (K * V))
    tokens, target, u, draft = _drafted(B, K, V, dt, B + K, spread=1.0)
    g = torch.Generator(device="cuda").manual_seed(V)
    num = torch.randint(-1, K + 2, (B,), generator=g, dtype=torch.int32, device="cuda")
    ctx = torch.randint(0, 9000, (B,), generator=g, dtype=torch.int32, device="cuda")
    got = torch_api.verify_drafts(tokens, target, u, draft_probs=None if certain else draft, num_drafts=num,
                                  context_lens=ctx)
    at = tokens.long()[..., None]
    p = target[:, :K].gather(2, at)[..., 0].double()
    q = torch.ones_like(p) if certain else draft.gather(2, at)[..., 0].double()
    n = num.clamp(0, K)
    refused = ~(u[:, :K].double() * q < p) & (torch.arange(K, device="cuda") < n[:, None])
    acc = torch.where(refused.any(1), refused.int().argmax(1), n).long()
    assert torch.equal(got.num_accepted.long(), acc)
    assert torch.equal(got.next_lens, (ctx + 1 + acc).int())
    # the token after them, in whole units of 2^-45 (no sum passes 2^46)
    i = torch.arange(B, device="cuda")
    unit = lambda x: torch.round(x.double() * 2.0 ** 45).long()  # noqa: E731
    w, k = unit(target[i, acc]), acc.clamp(max=K - 1)
    if certain:
        left = w.scatter(1, tokens[i, k].long()[:, None], 0)
    else:
        left = (w - unit(draft[i, k])).clamp(min=0)
    w = torch.where(((acc < n) & (left.sum(1) > 0))[:, None], left, w)
    # floor(u total) in Python integers (u is no multiple of 2^-24 where it is small)
    point = [math.floor(Fraction(x) * t) for x, t in zip(u[:, K].tolist(), w.sum(1).tolist())]
    point = torch.tensor(point, device="cuda")
    nxt = (w.cumsum(1) <= point[:, None]).sum(1)
    want = torch.full((B, K + 1), -1, device="cuda")
    j = torch.arange(K, device="cuda")
    want[:, :K] = torch.where(j < acc[:, None], tokens.long(), -1)
    want[i, acc] = nxt
    assert torch.equal(got.tokens.long(), want)


# ---------------------------------------------------------------------------
# windows
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
@pytest.mark.parametrize("sinks", [0, 20, 33])
@pytest.mark.parametrize("past", [1, 20, 50, 75])
def test_windows_across_the_tables_end(cuda, form, sinks, past):
    """Rows whose windows begin before the last page's end and end behind it: the
    keys from the window's start to the end of the table, and the sinks."""
    pr = Problem([(384, 40), (64, 3)], 2, 4, 128, 32, "bf16", seed=21)
    cap = 384
    table = pr.table[:, :cap // 32].contiguous()
    out, lse = torch_api.paged_attention(pr.q, pr.kc, pr.vc, table, pr.start, _cu([cap + past, 64]), scale=pr.scale,
                                         return_lse=True, form=form, window=60, sink_tokens=sinks)
    rows = [[t for t in range(min(p + 1, cap)) if t < sinks or t > p - 60] for p in range(cap + past - 40, cap + past)]
    rows += [[t for t in range(p + 1) if t < sinks or t > p - 60] for p in range(61, 64)]
    T, H, D = pr.q.shape
    u = 2.0 ** -8
    for b, (first, n) in enumerate(((0, 40), (40, 3))):
        tok = torch.arange(cap if b == 0 else 64, device="cuda")
        at = table[b].long()[tok // 32] * 32 + tok % 32
        k, v = (c.flatten(0, 1)[at].double() for c in (pr.kc, pr.vc))
        see = torch.zeros((n, len(tok)), dtype=torch.bool, device="cuda")
        for i in range(n):
            see[i, rows[first + i]] = True
        for h in range(H):
            q = pr.q[first:first + n, h].double()
            x = torch.where(see, q @ k[:, h // 4].T * pr.scale, -math.inf)
            z = torch.logsumexp(x, 1)
            p = torch.where(see, torch.exp(x - z.clamp(min=-1e300)[:, None]), 0.0)
            o, mag = p @ v[:, h // 4], p @ v[:, h // 4].abs()
            # half a step of the output and of every probability; scores: D products and sums in fp32
            dx = (D + 2) * 2.0 ** -23 * torch.where(see, q.abs() @ k[:, h // 4].abs().T, 0.0).amax(1) * pr.scale
            slack = 2 * dx + see.sum(1) * 2.0 ** -24 + 2.0 ** -20
            got, gl = out[first:first + n, h].double(), lse[first:first + n, h].double()
            assert ((got - o).abs() <= u * (o.abs() + mag) + mag * slack[:, None]).all(), (b, h)
            empty = see.sum(1) == 0
            assert (got[empty] == 0).all() and (gl[empty] == -math.inf).all()
            assert ((gl - z).abs()[~empty] <= (slack + 2.0 ** -22 * z.abs())[~empty]).all(), (b, h)


# ---------------------------------------------------------------------------
# rounds of drafts
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("K", [1, 3, 20])
def test_documented_rounds_lose_no_page(cuda, K):
    """The lines of serving's text between a verification and the next step, in a
    pool that suffices only if the pages of refused tokens come back."""
    lines = re.search(r"\n\n((?:    [^\n]*\n)*    context_lens = ver\.next_lens\n)", serving.__doc__).group(1)
    B, P, rounds, V = 5, 4, 40, 64
    start = [3, 4, 1, 9, 16]
    # every request's tokens after the last round (three in two rounds), and a round's drafts
    pages = sum(-(-(n + rounds * 3 // 2 + K + 1) // P) for n in start)
    pool = serving.PagedPool(num_pages=pages, page_tokens=P, num_kv_heads=1, head_dim=64)
    g = torch.Generator(device="cuda").manual_seed(K)
    free_pages = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    block_table = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
    maps = torch_api.build_page_maps(_cu([0] * B), _cu(start), free_pages, block_table, page_tokens=P, max_tokens=sum(start))
    free_pages = free_pages[int(maps.pages_used):]
    context_lens, total = _cu(start), list(start)
    for turn in range(rounds):
        maps = torch_api.build_page_maps(context_lens, _cu([K + 1] * B), free_pages, block_table, page_tokens=P,
                                         max_tokens=B * (K + 1))
        assert int(maps.pages_used) <= len(free_pages) and (maps.slots >= 0).all()
        # certain drafts: the first is the target's own in every other round, the second never is
        target = torch.zeros((B, K + 1, V), device="cuda")
        target[:, :, 7] = 1.0
        drafts = torch.full((B, K), 8, dtype=torch.int32, device="cuda")
        drafts[:, 0] = 7 + turn % 2
        ver = torch_api.verify_drafts(drafts, target, torch.full((B, K + 1), 0.5, device="cuda"), context_lens=context_lens)
        names = dict(torch=torch, ver=ver, res=types.SimpleNamespace(maps=maps), pool=pool, block_table=block_table,
                     free_pages=free_pages, context_lens=context_lens)
        exec(textwrap.dedent(lines), names)
        free_pages, context_lens = names["free_pages"], names["context_lens"]
        total = [n + 2 - turn % 2 for n in total]
        assert context_lens.tolist() == total
        live = [block_table[b, :-(-n // P)] for b, n in enumerate(total)]
        assert sorted(torch.cat(live + [free_pages]).tolist()) == list(range(pages))
