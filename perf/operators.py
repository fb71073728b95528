"""Measured cases of the paged serving operators around the sparse-attention indexer.

One decode or prefill step of a model whose attention is steered by the
indexer does, next to the indexer's own scoring and top-k, four things:

  maps    block tables, slots, positions and visible column counts of the
          step's tokens, built on the GPU from the requests' lengths;
  store   the new tokens' keys and values written into the paged cache;
  index   the new compressed index keys written into the paged index cache
          (bf16, or e4m3 with one scale a key);
  attend  attention of the new tokens over the paged cache: every key up to
          the token's own position, or the columns the top-k selected.

`run` computes them either with elementary torch operations in fp32 (own =
False) or with the package's public calls (own = True) on the same state.
"""
import math
import zlib

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
INDEX_DIM = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the step of a small decode batch: 16 requests, one token each (latency of one launch)
        dict(name="maps_decode16", op="maps", requests=16, chunk=1, spread=0, context=32768, page_tokens=64, ratio=4,
             partial=False, pad=0),
        # a large mixed step: 512 requests, a token or a ragged chunk each, 32 K tokens
        dict(name="maps_mixed512", op="maps", requests=512, chunk=64, spread=63, context=8192, page_tokens=16,
             ratio=4, partial=True, pad=77),
        # keys and values of a 36-token verification step (9 requests x 4 rows)
        dict(name="store_verify36", op="store", tokens=36, kv_heads=8, head_dim=128, page_tokens=64, dtype="bf16",
             strided=False),
        # keys and values of a 16 K-token prefill chunk, taken from a fused qkv projection (strided rows)
        dict(name="store_chunk16k", op="store", tokens=16384, kv_heads=8, head_dim=128, page_tokens=64,
             dtype="bf16", strided=True),
        # index keys of 16 decode rows, quantised to e4m3 with a scale a key
        dict(name="index_decode16", op="index", tokens=16, page_cols=64, fp8=True, live=1.0),
        # index keys of a 64 K-token prefill: one token in four completes a column
        dict(name="index_prefill64k", op="index", tokens=65536, page_cols=64, fp8=True, live=0.25),
        # one interactive request, one new token over a short context (latency)
        dict(name="attend_single", op="attend", requests=1, new=1, spread=0, context_lo=1000, context_hi=1000,
             kv_heads=8, group=4, head_dim=128, page_tokens=64, dtype="bf16"),
        # verification of three drafted tokens, 9 requests of 64 K to 128 K tokens
        dict(name="attend_verify9x4", op="attend", requests=9, new=4, spread=0, context_lo=65536, context_hi=131072,
             kv_heads=8, group=4, head_dim=128, page_tokens=64, dtype="bf16"),
        # an 8 K-token prefill chunk that ends a 32 K-token prompt
        dict(name="attend_chunk8k", op="attend", requests=1, new=8192, spread=0, context_lo=24576, context_hi=24576,
             kv_heads=8, group=4, head_dim=128, page_tokens=64, dtype="bf16"),
        # ragged chunks of odd lengths, small heads, small pages, fp16
        dict(name="attend_ragged_fp16", op="attend", requests=7, new=301, spread=290, context_lo=1, context_hi=5000,
             kv_heads=2, group=7, head_dim=64, page_tokens=16, dtype="fp16"),
        # sparse decode: 16 rows at 128 K tokens attend to the indexer's 2048 columns of 4 tokens and the last 64 tokens
        dict(name="select_decode16", op="select", requests=16, new=1, context_lo=131000, context_hi=131072,
             kv_heads=4, group=8, head_dim=128, page_tokens=64, dtype="bf16", k=2048, ratio=4, local=64),
        # sparse prefill: a 512-token chunk at 16 K tokens over 512 columns of 4 tokens a row
        dict(name="select_chunk512", op="select", requests=1, new=512, context_lo=16000, context_hi=16000,
             kv_heads=2, group=16, head_dim=128, page_tokens=64, dtype="bf16", k=512, ratio=4, local=100),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["maps", "store", "index", "attend", "attend", "attend", "select", "select"])
    if op == "maps":
        b = _log_int(rng, 1, 1024)
        chunk = _log_int(rng, 1, max(1, 32768 // b))
        pt, ratio = rng.choice([(8, 1), (16, 4), (20, 4), (64, 4), (64, 2), (128, 4), (1, 1)])
        return dict(op=op, requests=b, chunk=chunk, spread=rng.randrange(0, chunk), context=_log_int(rng, 1, 32768),
                    page_tokens=pt, ratio=ratio, partial=rng.random() < 0.5, pad=rng.choice([0, 1, 100]))
    if op == "store":
        return dict(op=op, tokens=_log_int(rng, 1, 16384), kv_heads=rng.choice([1, 2, 3, 4, 8]),
                    head_dim=rng.choice([64, 128]), page_tokens=rng.choice([1, 16, 20, 64, 128]),
                    dtype=rng.choice(["bf16", "fp16"]), strided=rng.random() < 0.5)
    if op == "index":
        return dict(op=op, tokens=_log_int(rng, 1, 65536), page_cols=rng.choice([1, 4, 16, 20, 64]),
                    fp8=rng.random() < 0.7, live=rng.choice([1.0, 0.5, 0.25]))
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if kv_heads * group > 32:
        kv_heads = max(1, 32 // group)
    heads = dict(kv_heads=kv_heads, group=group, head_dim=rng.choice([64, 128]), dtype=rng.choice(["bf16", "fp16"]))
    if op == "attend":
        if rng.random() < 0.5:  # decode and verification
            b, new = _log_int(rng, 1, 64), rng.randint(1, 8)
            hi = _log_int(rng, 1, min(131072, 600000 // b))
        else:                   # chunks
            b, new = rng.randint(1, 6), _log_int(rng, 9, 1200)
            hi = _log_int(rng, 1, 16384)
        return dict(op=op, requests=b, new=new, spread=rng.randrange(0, new), context_lo=(hi + 1) // 2, context_hi=hi,
                    page_tokens=rng.choice([8, 16, 20, 32, 64, 128, 256]), **heads)
    b = _log_int(rng, 1, 24)
    new = rng.randint(1, 4) if rng.random() < 0.7 else _log_int(rng, 5, max(5, 256 // b))
    hi = _log_int(rng, 1, max(8, min(131072, 600000 // b, 4000000 // (b * new))))
    ratio = rng.choice([1, 2, 4])
    return dict(op=op, requests=b, new=new, context_lo=(hi + 1) // 2, context_hi=hi,
                page_tokens=rng.choice([16, 20, 64, 128]), k=_log_int(rng, 1, 2048), ratio=ratio,
                local=rng.choice([0, 4, 64, 100]), **heads)


# ---------------------------------------------------------------------------
# what a user's program holds before the call
# ---------------------------------------------------------------------------

def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _lengths(case, seed):
    """(context, new) token counts of the case's requests, on the host.  The
    lengths belong to the case, their order to the seed, so that sizes are the
    same for every seed."""
    sizes = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    r = np.random.default_rng(zlib.crc32(sizes.encode()))
    b = case["requests"]
    if case["op"] == "maps":
        ctx = r.integers(max(0, case["context"] // 2), case["context"] + 1, b)
        new = case["chunk"] + r.integers(-case["spread"], case["spread"] + 1, b)
    else:
        ctx = r.integers(case["context_lo"], case["context_hi"] + 1, b)
        new = np.maximum(case["new"] + r.integers(-case.get("spread", 0), 1, b), 1)
    order = np.random.default_rng([seed, 11]).permutation(b)
    return ctx[order], np.maximum(new, 0)[order]


def _generator(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + salt)
    return g


def _randn(shape, dtype, g, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if math.prod(shape) < 1 << 28 else dtype)
    return (x * scale).to(dtype)


def _prepare_maps(case, seed):
    ctx, new = _lengths(case, seed)
    pt = case["page_tokens"]
    have, need = -(-ctx // pt), -(-(ctx + new) // pt)
    max_pages = int(need.max()) + 3
    r = np.random.default_rng([seed, 12])
    pages = r.permutation(int(need.sum()) + 16)
    table = np.full((len(ctx), max_pages), -1, np.int64)
    used = 0
    for b in range(len(ctx)):
        table[b, :have[b]] = pages[used:used + have[b]]
        used += have[b]
    return dict(context=_i32(ctx), new=_i32(new), free=_i32(pages[used:]), table=_i32(table),
                max_tokens=int(new.sum()) + case["pad"])


def _prepare_store(case, seed):
    t, h, d, pt = case["tokens"], case["kv_heads"], case["head_dim"], case["page_tokens"]
    dt, g = DTYPES[case["dtype"]], _generator(seed, 1)
    pages = -(-t // pt) + 2
    r = np.random.default_rng([seed, 13])
    # tokens fill their pages in order, the pages lie anywhere in the pool
    page_of = r.permutation(pages)
    tok = np.arange(t) + r.integers(0, pt)
    slots = page_of[tok // pt] * pt + tok % pt
    slots[r.random(t) < 0.02] = -1          # padding rows
    if case["strided"]:
        both = _randn((t, 3 * h, d), dt, g)
        k, v = both[:, h:2 * h], both[:, 2 * h:]
    else:
        k, v = _randn((t, h, d), dt, g), _randn((t, h, d), dt, g)
    cache = torch.zeros((2, pages, pt, h, d), dtype=dt, device="cuda")
    return dict(k=k, v=v, slots=torch.from_numpy(slots).cuda(), k_cache=cache[0], v_cache=cache[1])


def _prepare_index(case, seed):
    t, pc = case["tokens"], case["page_cols"]
    r = np.random.default_rng([seed, 14])
    n = max(1, int(t * case["live"]))
    live = np.zeros(t, bool)
    live[r.permutation(t)[:n]] = True
    pages = -(-n // pc) + 1
    col = np.arange(n)
    slots = np.full(t, -1, np.int64)
    slots[live] = r.permutation(pages)[col // pc] * pc + col % pc
    keys = _randn((t, INDEX_DIM), torch.bfloat16, _generator(seed, 2), 2.0)
    st = dict(keys=keys, slots=torch.from_numpy(slots).cuda())
    if case["fp8"]:
        st["cache"] = torch.zeros((pages, pc * (INDEX_DIM + 4)), dtype=torch.uint8, device="cuda")
    else:
        st["cache"] = torch.zeros((pages, pc, INDEX_DIM), dtype=torch.bfloat16, device="cuda")
    return st


def _prepare_attend(case, seed):
    ctx, new = _lengths(case, seed)
    h, gq, d, pt = case["kv_heads"], case["group"], case["head_dim"], case["page_tokens"]
    dt, g = DTYPES[case["dtype"]], _generator(seed, 3)
    seq = ctx + new
    need = -(-seq // pt)
    n_pages = int(need.sum())
    r = np.random.default_rng([seed, 15])
    perm = r.permutation(n_pages)
    table = np.full((len(ctx), int(need.max()) + 1), n_pages, np.int64)   # unused entries: the poison page
    used = 0
    for b in range(len(ctx)):
        table[b, :need[b]] = perm[used:used + need[b]]
        used += need[b]
    t = int(new.sum())
    k_cache = _randn((n_pages + 1, pt, h, d), dt, g)
    v_cache = _randn((n_pages + 1, pt, h, d), dt, g)
    k_cache[n_pages], v_cache[n_pages] = math.nan, math.nan
    # logits of standard deviation about 2: some keys stand out, as in trained heads
    q = _randn((t, h * gq, d), dt, g, 2.0)
    start = np.concatenate([[0], np.cumsum(new)])
    st = dict(q=q, k_cache=k_cache, v_cache=v_cache, table=_i32(table), start=_i32(start), seq=_i32(seq),
              lens=[(int(s), int(n)) for s, n in zip(seq, new)], max_new=int(new.max()), scale=1.0 / math.sqrt(d))
    if case["op"] == "select":
        st["selected"] = _select(case, st, g)
    return st


def _select(case, st, g):
    """What the top-k hands over: per row min(k, visible) distinct columns in
    ascending order, then -1."""
    k, ratio, rows = case["k"], case["ratio"], []
    for s, n in st["lens"]:
        pos = torch.arange(s - n, s, device="cuda")
        vis = (pos + 1) // ratio
        cols = max(1, s // ratio)
        score = torch.rand((n, cols), generator=g, device="cuda")
        score.masked_fill_(torch.arange(cols, device="cuda")[None] >= vis[:, None], -1.0)
        top, idx = score.topk(min(k, cols), dim=1)
        idx = torch.where(top >= 0, idx, 1 << 30).sort(dim=1).values
        idx = torch.where(idx < (1 << 30), idx, -1).to(torch.int32)
        out = torch.full((n, k), -1, dtype=torch.int32, device="cuda")
        out[:, :idx.shape[1]] = idx
        rows.append(out)
    return torch.cat(rows)


def prepare(case, seed):
    op = case["op"]
    st = {"maps": _prepare_maps, "store": _prepare_store, "index": _prepare_index, "attend": _prepare_attend,
          "select": _prepare_attend}[op](case, seed)
    st["case"] = case
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        from sparse_attention_indexer_02_gb300 import torch_api
        return _OWN[op](torch_api, state)
    return _PLAIN[op](state)


def _own_maps(api, st):
    c = st["case"]
    m = api.build_page_maps(st["context"], st["new"], st["free"], st["table"], page_tokens=c["page_tokens"],
                            max_tokens=st["max_tokens"], ratio=c["ratio"], partial_cols=c["partial"])
    return (st["table"], m.query_start, m.seq_lens, m.slots, m.positions, m.token_request, m.visible_cols,
            m.column_slots, m.pages_used)


def _own_store(api, st):
    api.store_paged_kv(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"])
    return st["k_cache"], st["v_cache"]


def _index_views(st, pc):
    cache = st["cache"]
    codes = cache[:, :pc * INDEX_DIM].view(torch.float8_e4m3fn).unflatten(1, (pc, INDEX_DIM))
    return codes, cache[:, pc * INDEX_DIM:].view(torch.float32)


def _own_index(api, st):
    c = st["case"]
    if not c["fp8"]:
        api.store_index_keys(st["keys"], st["slots"], st["cache"], page_cols=c["page_cols"])
        return st["cache"]
    from sparse_attention_indexer_02_gb300 import KV_FP8_E4M3
    api.store_index_keys(st["keys"], st["slots"], st["cache"], page_cols=c["page_cols"], kv_dtype=KV_FP8_E4M3,
                         scale_offset=c["page_cols"] * INDEX_DIM)
    return _index_views(st, c["page_cols"])


def _own_attend(api, st):
    c = st["case"]
    kw = {}
    if c["op"] == "select":
        kw = dict(selected=st["selected"], ratio=c["ratio"], local_tokens=c["local"])
    return api.paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["start"], st["seq"],
                               scale=st["scale"], max_new=st["max_new"], return_lse=True, **kw)


def _plain_maps(st):
    c = st["case"]
    pt, ratio, n = c["page_tokens"], c["ratio"], st["max_tokens"]
    ctx, new, table = st["context"].long(), st["new"].long(), st["table"]
    seq = ctx + new
    have, need = (ctx + pt - 1) // pt, (seq + pt - 1) // pt
    take = (need - have).cumsum(0)
    first = take - (need - have)
    j = torch.arange(table.shape[1], device="cuda")[None]
    fresh = (j >= have[:, None]) & (j < need[:, None])
    src = (first[:, None] + j - have[:, None]).clamp(0, st["free"].numel() - 1)
    table = torch.where(fresh, st["free"][src], table)
    start = torch.zeros(len(ctx) + 1, dtype=torch.int64, device="cuda")
    start[1:] = new.cumsum(0)
    t = torch.arange(n, device="cuda")
    live = t < start[-1]
    req = torch.searchsorted(start, t, right=True).sub(1).clamp(max=len(ctx) - 1)
    pos = ctx[req] + t - start[req]
    page = table[req, (pos // pt).clamp(0, table.shape[1] - 1)].long()
    slot = torch.where(live, page * pt + pos % pt, -1)
    vis = (pos + ratio) // ratio if c["partial"] else (pos + 1) // ratio
    done = live & (pos % ratio == ratio - 1)
    i32 = torch.int32
    return (table, start.to(i32), seq.to(i32), slot, torch.where(live, pos, -1).to(i32),
            torch.where(live, req, -1).to(i32), torch.where(live, vis, 0).to(i32),
            torch.where(done, slot // ratio, -1), take[-1:].to(i32))


def _plain_store(st):
    pt = st["k_cache"].shape[1]
    # rows without a slot write the row that slot 0 holds already (or gets): done by selecting the others
    live = (st["slots"] >= 0).nonzero()[:, 0]
    s = st["slots"][live]
    st["k_cache"][s // pt, s % pt] = st["k"][live]
    st["v_cache"][s // pt, s % pt] = st["v"][live]
    return st["k_cache"], st["v_cache"]


def _plain_index(st):
    c = st["case"]
    pc = c["page_cols"]
    live = (st["slots"] >= 0).nonzero()[:, 0]
    s, keys = st["slots"][live], st["keys"][live]
    if not c["fp8"]:
        st["cache"][s // pc, s % pc] = keys
        return st["cache"]
    x = keys.float()
    scale = x.abs().amax(1) / E4M3_MAX
    code = (x / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    codes, scales = _index_views(st, pc)
    codes.view(torch.uint8)[s // pc, s % pc] = code.view(torch.uint8)
    scales[s // pc, s % pc] = scale
    return codes, scales


def _plain_attend(st):
    c = st["case"]
    h, gq, d = c["kv_heads"], c["group"], c["head_dim"]
    out, lse = torch.empty_like(st["q"]), torch.empty(st["q"].shape[:2], dtype=torch.float32, device="cuda")
    t0 = 0
    for b, (s, n) in enumerate(st["lens"]):
        pages = st["table"][b, :-(-s // c["page_tokens"])].long()
        k = st["k_cache"][pages].flatten(0, 1)[:s]
        v = st["v_cache"][pages].flatten(0, 1)[:s]
        for r0 in range(0, n, 1024):        # rows in parts, to bound the score matrix
            m = min(1024, n - r0)
            pos = torch.arange(s - n + r0, s - n + r0 + m, device="cuda")
            key = torch.arange(s, device="cuda")
            seen = key[None] <= pos[:, None]
            if c["op"] == "select":
                sel = st["selected"][t0 + r0:t0 + r0 + m].long()
                cols = -(-s // c["ratio"])
                hit = torch.zeros((m, cols + 1), dtype=torch.bool, device="cuda")
                hit.scatter_(1, torch.where(sel >= 0, sel, cols), True)
                chosen = hit[:, :cols].repeat_interleave(c["ratio"], 1)[:, :s]
                seen &= chosen | (key[None] > pos[:, None] - c["local"])
            rows = slice(t0 + r0, t0 + r0 + m)
            for j in range(h):
                q = st["q"][rows, j * gq:(j + 1) * gq].float().reshape(m * gq, d)
                x = (q @ k[:, j].float().T * st["scale"]).view(m, gq, s)
                x.masked_fill_(~seen[:, None], -math.inf)
                top = x.amax(2, keepdim=True)
                x.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
                tot = x.sum(2, keepdim=True)
                o = (x.view(m * gq, s) @ v[:, j].float()).view(m, gq, d) / torch.where(tot > 0, tot, 1.0)
                out[rows, j * gq:(j + 1) * gq] = o.to(out.dtype)
                lse[rows, j * gq:(j + 1) * gq] = (top + tot.log())[:, :, 0]
        t0 += n
    return out, lse


_OWN = {"maps": _own_maps, "store": _own_store, "index": _own_index, "attend": _own_attend, "select": _own_attend}
_PLAIN = {"maps": _plain_maps, "store": _plain_store, "index": _plain_index, "attend": _plain_attend,
          "select": _plain_attend}


# ---------------------------------------------------------------------------
# work and exact answers
# ---------------------------------------------------------------------------

def work(case):
    """Bytes and operations of one pass: each input read once, each output
    written once."""
    op = case["op"]
    if op == "store":
        return dict(bytes=case["tokens"] * (8 * case["kv_heads"] * case["head_dim"] + 8), flops=0)
    if op == "index":
        n = max(1, int(case["tokens"] * case["live"]))
        out = INDEX_DIM + 4 if case["fp8"] else 2 * INDEX_DIM
        return dict(bytes=case["tokens"] * 8 + n * (2 * INDEX_DIM + out), flops=3 * n * INDEX_DIM if case["fp8"] else 0)
    ctx, new = (x.astype(np.float64) for x in _lengths(case, 0))
    rows = float(new.sum())
    if op == "maps":
        b, pt = case["requests"], case["page_tokens"]
        fresh = float((np.ceil((ctx + new) / pt) - np.ceil(ctx / pt)).sum())
        begun = float(((ctx % pt > 0) & (new > 0)).sum())   # pages the first tokens still fit in
        return dict(bytes=8 * b + 4 * (2 * b + 1) + 8 * fresh + 4 * begun + 28 * (rows + case["pad"]) + 4, flops=0)
    h, gq, d = case["kv_heads"], case["group"], case["head_dim"]
    seen, kept, extra = float((new * (ctx + (new + 1) / 2)).sum()), float((ctx + new).sum()), 0
    if op == "select":
        most = case["k"] * case["ratio"] + case["local"]
        seen = float((new * np.minimum(ctx + (new + 1) / 2, most)).sum())
        kept = float(np.minimum(ctx + new, new * most).sum())
        extra = 4 * rows * case["k"]
    return dict(bytes=4 * kept * h * d + rows * h * gq * (4 * d + 4) + extra, flops=4 * d * h * gq * seen)


def exact(case, seed):
    st = prepare(case, seed)
    return {"maps": _exact_maps, "store": _exact_store, "index": _exact_index, "attend": _exact_attend,
            "select": _exact_attend}[case["op"]](case, st)


def _exact_maps(case, st):
    ctx, new, free = (st[n].tolist() for n in ("context", "new", "free"))
    table = st["table"].cpu().numpy().copy()
    pt, ratio, n = case["page_tokens"], case["ratio"], st["max_tokens"]
    start, taken, rows = [0], 0, []
    for b, (c, m) in enumerate(zip(ctx, new)):
        for j in range(math.ceil(c / pt), math.ceil((c + m) / pt)):
            table[b, j] = free[taken]
            taken += 1
        for p in range(c, c + m):
            slot = int(table[b, p // pt]) * pt + p % pt
            vis = math.ceil((p + 1) / ratio) if case["partial"] else (p + 1) // ratio
            rows.append((slot, p, b, vis, slot // ratio if (p + 1) % ratio == 0 else -1))
        start.append(len(rows))
    rows += [(-1, -1, -1, 0, -1)] * (n - len(rows))
    cols = np.array(rows, np.int64).reshape(n, 5).T
    i32 = np.int32
    return (table, np.array(start, i32), np.array([c + m for c, m in zip(ctx, new)], i32), cols[0],
            cols[1].astype(i32), cols[2].astype(i32), cols[3].astype(i32), cols[4], np.array([taken], i32))


def _exact_store(case, st):
    pt = case["page_tokens"]
    out = []
    for rows, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
        flat = cache.double().flatten(0, 1)
        slots = st["slots"].tolist()
        put = [i for i, s in enumerate(slots) if s >= 0]
        flat[[slots[i] for i in put]] = rows.double()[put]
        out.append(flat.view(-1, pt, *flat.shape[1:]))
    return tuple(out)


def _exact_index(case, st):
    pc, slots = case["page_cols"], st["slots"].tolist()
    put = [i for i, s in enumerate(slots) if s >= 0]
    at = [slots[i] for i in put]
    pages = st["cache"].shape[0]
    x = st["keys"].double()[put]
    codes = torch.zeros((pages * pc, INDEX_DIM), dtype=torch.float64, device="cuda")
    if not case["fp8"]:
        codes[at] = x
        return codes.view(pages, pc, INDEX_DIM)
    scale = x.abs().amax(1) / E4M3_MAX
    y = x / torch.where(scale > 0, scale, 1.0)[:, None]
    # the e4m3 grid: 3 fraction bits, smallest normal exponent -6, nearest with ties to even
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    codes[at] = torch.round(y / step) * step
    scales = torch.zeros(pages * pc, dtype=torch.float64, device="cuda")
    scales[at] = scale
    return codes.view(pages, pc, INDEX_DIM), scales.view(pages, pc)


def _exact_attend(case, st):
    h, gq, d, pt = case["kv_heads"], case["group"], case["head_dim"], case["page_tokens"]
    t, heads = st["q"].shape[:2]
    if 4.0 * d * heads * sum(s * n for s, n in st["lens"]) > 6e12:
        return None
    out = torch.zeros((t, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((t, heads), dtype=torch.float64, device="cuda")
    first = 0
    for b, (s, n) in enumerate(st["lens"]):
        tok = torch.arange(s, device="cuda")
        where = st["table"][b].long()[tok // pt] * pt + tok % pt
        for i0 in range(0, n, 512):
            i1 = min(n, i0 + 512)
            far = tok[None] > torch.arange(s - n + i0, s - n + i1, device="cuda")[:, None]   # after the row's token
            if case["op"] == "select":
                keep = torch.zeros((i1 - i0, s), dtype=torch.bool, device="cuda")
                for i in range(i0, i1):
                    p = s - n + i
                    sel = st["selected"][first + i]
                    sel = sel[sel >= 0].long()
                    at = (sel[:, None] * case["ratio"] + torch.arange(case["ratio"], device="cuda")).flatten()
                    keep[i - i0, at[at < s]] = True
                    keep[i - i0, max(0, p + 1 - case["local"]):p + 1] = True
                far |= ~keep
            for j in range(h):
                k = st["k_cache"].flatten(0, 1)[where, j].double()
                v = st["v_cache"].flatten(0, 1)[where, j].double()
                q = st["q"][first + i0:first + i1, j * gq:(j + 1) * gq].double()
                x = torch.einsum("tgd,sd->gts", q, k) * st["scale"]
                x = torch.where(far[None], -math.inf, x)
                z = torch.logsumexp(x, 2)
                p = torch.exp(x - torch.where(z > -math.inf, z, 0.0)[:, :, None])
                out[first + i0:first + i1, j * gq:(j + 1) * gq] = torch.einsum("gts,sd->tgd", p, v)
                lse[first + i0:first + i1, j * gq:(j + 1) * gq] = z.T
        first += n
    return out, lse
