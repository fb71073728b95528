"""Measured cases of the operators between a layer's projections and the next
tokens: rotary positions, per-head norms with the rotation and the store in one
pass, attention to a sliding window with sinks, and the verification of drafts.

  rotate  queries and keys turned by their positions' angles: the pairs of a
          head (its two halves, or neighbours), all of the head or a part of
          it, frequencies scaled for long contexts;
  norm    queries and keys normalised head by head, then rotated, the keys and
          the values written into the slots of a paged cache;
  window  attention of the new tokens to the last `window` tokens up to their
          own and to the first `sinks` ones, over a paged cache whose pages
          behind the window have gone to other requests;
  verify  drafted tokens accepted or refused against the target's
          probabilities with given random numbers, and the token that follows.

`run` computes them either with elementary torch operations (own = False) or
with the package's public calls (own = True) on the same state.
"""
import math
import zlib

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 16 requests at up to 128 K tokens (latency of one launch)
        dict(name="rotate_decode16", op="rotate", tokens=16, q_heads=32, kv_heads=8, head_dim=128, rot_dim=128, offset=0,
             layout="half", scaling="parts", reach=131072, pad=0, strided=False, dtype="bf16"),
        # a 16 K-token prefill chunk, taken from a fused qkv projection (strided rows)
        dict(name="rotate_chunk16k", op="rotate", tokens=16384, q_heads=32, kv_heads=8, head_dim=128, rot_dim=128,
             offset=0, layout="half", scaling="parts", reach=32768, pad=0, strided=True, dtype="bf16"),
        # index queries of a 2 K-token chunk: 64 heads without keys, neighbours in the last half of the head
        dict(name="rotate_index2k", op="rotate", tokens=2048, q_heads=64, kv_heads=0, head_dim=128, rot_dim=64, offset=64,
             layout="pairs", scaling="linear", reach=131072, pad=3, strided=False, dtype="bf16"),
        # a 36-token verification step (9 requests x 4 rows): norms, rotation, store
        dict(name="norm_verify36", op="norm", tokens=36, q_heads=32, kv_heads=8, head_dim=128, rot_dim=128, offset=0,
             layout="half", scaling="none", reach=131072, pad=0, strided=True, dtype="bf16", norm="rms", page_tokens=64),
        # the same of a 16 K-token prefill chunk
        dict(name="norm_chunk16k", op="norm", tokens=16384, q_heads=32, kv_heads=8, head_dim=128, rot_dim=128, offset=0,
             layout="half", scaling="none", reach=32768, pad=0, strided=True, dtype="bf16", norm="rms", page_tokens=64),
        # one interactive request, one new token, a window shorter than its context (latency)
        dict(name="window_single", op="window", requests=1, new=1, spread=0, context_lo=5000, context_hi=5000,
             window=1024, sinks=4, kv_heads=8, group=4, head_dim=128, page_tokens=64, dtype="bf16"),
        # decode of 64 requests of 64 K to 128 K tokens over the last 4096 of them and 4 sinks
        dict(name="window_decode64", op="window", requests=64, new=1, spread=0, context_lo=65536, context_hi=131072,
             window=4096, sinks=4, kv_heads=8, group=4, head_dim=128, page_tokens=64, dtype="bf16"),
        # an 8 K-token prefill chunk that ends a 32 K-token prompt
        dict(name="window_chunk8k", op="window", requests=1, new=8192, spread=0, context_lo=24576, context_hi=24576,
             window=4096, sinks=64, kv_heads=8, group=4, head_dim=128, page_tokens=64, dtype="bf16"),
        # ragged chunks of odd lengths, small heads, small pages, fp16, a short odd window
        dict(name="window_ragged_fp16", op="window", requests=7, new=301, spread=290, context_lo=1, context_hi=5000,
             window=333, sinks=5, kv_heads=2, group=7, head_dim=64, page_tokens=16, dtype="fp16"),
        # one request's three drafts, a small odd vocabulary (latency)
        dict(name="verify_single3", op="verify", requests=1, drafts=3, ragged=False, vocab=32003, drafted="probs",
             dtype="fp32"),
        # 16 requests with up to seven drafts each from an n-gram lookup (no draft distribution)
        dict(name="verify_lookup16x7", op="verify", requests=16, drafts=7, ragged=True, vocab=131072, drafted="certain",
             dtype="fp32"),
        # a large verification batch: 64 requests x 4 drafts of a draft model
        dict(name="verify_64x4", op="verify", requests=64, drafts=4, ragged=False, vocab=131072, drafted="probs",
             dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rotate", "norm", "window", "window", "window", "verify"])
    if op in ("rotate", "norm"):
        head_dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rot_dim = rng.choice([head_dim, head_dim, head_dim // 2 // 8 * 8, 24])
        kv_heads = rng.choice([1, 2, 3, 4, 8]) if op == "norm" else rng.choice([0, 1, 2, 5, 8])
        q_heads = rng.randint(1, 8) * max(kv_heads, 1)
        most = min(16384, 16384 * 48 * 128 // ((q_heads + 2 * kv_heads) * head_dim))
        return dict(op=op, tokens=_log_int(rng, 1, most), q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                    rot_dim=rot_dim, offset=rng.choice([0, head_dim - rot_dim]), layout=rng.choice(["half", "pairs"]),
                    scaling=rng.choice(["none", "linear", "base", "parts"]), reach=_log_int(rng, 1, 1 << 20),
                    pad=rng.choice([0, 1, 5]), strided=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]),
                    **(dict(norm=rng.choice(["rms", "layer"]), page_tokens=rng.choice([1, 16, 20, 64, 128]))
                       if op == "norm" else {}))
    if op == "verify":
        drafts = rng.choice([0, 1, 2, 3, 4, 7, 15])
        vocab = _log_int(rng, 100, 262144)
        return dict(op=op, requests=_log_int(rng, 1, max(1, min(256, 64 * 5 * 131072 // (vocab * (drafts + 1))))),
                    drafts=drafts, ragged=rng.random() < 0.5, vocab=vocab,
                    drafted=rng.choice(["probs", "probs", "certain"]), dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]))
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if kv_heads * group > 32:
        kv_heads = max(1, 32 // group)
    window = _log_int(rng, 1, 4096)
    if rng.random() < 0.6:  # decode and verification
        b, new = _log_int(rng, 1, 64), rng.randint(1, 8)
        hi = _log_int(rng, 1, 131072)
    else:                   # chunks
        b, new = rng.randint(1, 6), _log_int(rng, 9, 1200)
        hi = _log_int(rng, 1, 32768)
    return dict(op=op, requests=b, new=new, spread=rng.randrange(0, new), context_lo=(hi + 1) // 2, context_hi=hi,
                window=window, sinks=rng.choice([0, 1, 4, 64, 200]), kv_heads=kv_heads, group=group,
                head_dim=rng.choice([64, 128]), page_tokens=rng.choice([8, 16, 20, 32, 64, 128, 256]),
                dtype=rng.choice(["bf16", "fp16"]))


# ---------------------------------------------------------------------------
# what a user's program holds before the call
# ---------------------------------------------------------------------------

def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _generator(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + salt)
    return g


def _randn(shape, dtype, g, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if math.prod(shape) < 1 << 28 else dtype)
    return (x * scale).to(dtype)


# What a model's configuration says of its frequencies.
BASE = 500000.0
SCALING = {"none": None, "linear": dict(kind="linear", factor=4.0), "base": dict(kind="base", factor=8.0),
           "parts": dict(kind="parts", factor=8.0, original=8192, low=1.0, high=32.0)}
MAGNITUDE = {"none": 1.0, "linear": 1.0, "base": 1.0, "parts": 0.1 * math.log(8.0) + 1.0}


def _rotary(case):
    """The handle a user's program makes once for a model."""
    from sparse_attention_indexer_02_gb300 import torch_api
    return torch_api.Rotary(case["rot_dim"], base=BASE, layout=case["layout"], offset=case["offset"],
                            scaling=SCALING[case["scaling"]], magnitude=MAGNITUDE[case["scaling"]])


def _prepare_heads(case, seed):
    t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    rows, dt, g = t + case["pad"], DTYPES[case["dtype"]], _generator(seed, 1)
    r = np.random.default_rng([seed, 21])
    if t > 64:      # a chunk: positions follow one another
        pos = r.integers(0, max(1, case["reach"] - t)) + np.arange(t)
    else:           # rows of many requests
        pos = r.integers(0, case["reach"], t)
    st = dict(positions=_i32(np.concatenate([pos, np.full(case["pad"], -1)])))
    if case["strided"]:
        both = _randn((rows, hq + 2 * hk, d), dt, g)
        st["q"], st["k"], st["v"] = both[:, :hq], both[:, hq:hq + hk], both[:, hq + hk:]
    else:
        st["q"], st["k"], st["v"] = _randn((rows, hq, d), dt, g), _randn((rows, hk, d), dt, g), _randn((rows, hk, d), dt, g)
    # the outputs a captured step keeps; padding rows stay as they are
    st["q_out"] = torch.zeros((rows, hq, d), dtype=dt, device="cuda")
    if case["op"] == "rotate":
        st["k_out"] = torch.zeros((rows, hk, d), dtype=dt, device="cuda")
        if hk == 0:
            st["k"] = st["k_out"] = None
    else:
        for n in ("q_weight", "k_weight"):
            st[n] = (1.0 + _randn((d,), torch.float32, g, 0.2)).to(dt)
        for n in ("q_bias", "k_bias"):
            st[n] = _randn((d,), dt, g, 0.2) if case["norm"] == "layer" else None
        pt = case["page_tokens"]
        pages = -(-t // pt) + 2
        tok = np.arange(t) + r.integers(0, pt)
        slots = r.permutation(pages)[tok // pt] * pt + tok % pt
        st["slots"] = torch.from_numpy(np.concatenate([slots, np.full(case["pad"], -1)]).astype(np.int64)).cuda()
        cache = torch.zeros((2, pages, pt, hk, d), dtype=dt, device="cuda")
        st["k_cache"], st["v_cache"] = cache[0], cache[1]
    if own:
        st["rotary"] = _rotary(case)
    return st


def _lengths(case, seed):
    """(context, new) token counts of the case's requests, on the host.  The
    lengths belong to the case, their order to the seed, so that sizes are the
    same for every seed."""
    sizes = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    r = np.random.default_rng(zlib.crc32(sizes.encode()))
    b = case["requests"]
    ctx = r.integers(case["context_lo"], case["context_hi"] + 1, b)
    new = np.maximum(case["new"] + r.integers(-case["spread"], 1, b), 1)
    order = np.random.default_rng([seed, 11]).permutation(b)
    return ctx[order], new[order]


def _prepare_window(case, seed):
    ctx, new = _lengths(case, seed)
    h, gq, d, pt = case["kv_heads"], case["group"], case["head_dim"], case["page_tokens"]
    dt, g = DTYPES[case["dtype"]], _generator(seed, 3)
    seq = ctx + new
    need = -(-seq // pt)
    # pages no row sees have been freed: their entries name any page, or none
    held = []
    for c, s, n in zip(ctx, seq, need):
        j = np.arange(n)
        held.append((j * pt < min(case["sinks"], s)) | ((j + 1) * pt > c + 1 - case["window"]))
    n_pages = int(sum(m.sum() for m in held))
    r = np.random.default_rng([seed, 15])
    perm = r.permutation(n_pages)
    table = np.full((len(ctx), int(need.max()) + 1), n_pages, np.int64)   # the poison page
    table[r.random(table.shape) < 0.5] = -1
    used = 0
    for b, m in enumerate(held):
        k = int(m.sum())
        table[b, :len(m)][m] = perm[used:used + k]
        used += k
    t = int(new.sum())
    k_cache = _randn((n_pages + 1, pt, h, d), dt, g)
    v_cache = _randn((n_pages + 1, pt, h, d), dt, g)
    k_cache[n_pages], v_cache[n_pages] = math.nan, math.nan
    # logits of standard deviation about 2: some keys stand out, as in trained heads
    q = _randn((t, h * gq, d), dt, g, 2.0)
    start = np.concatenate([[0], np.cumsum(new)])
    return dict(q=q, k_cache=k_cache, v_cache=v_cache, table=_i32(table), start=_i32(start), seq=_i32(seq),
                lens=[(int(s), int(n)) for s, n in zip(seq, new)], max_new=int(new.max()), scale=1.0 / math.sqrt(d))


def _prepare_verify(case, seed):
    b, k, v = case["requests"], case["drafts"], case["vocab"]
    dt, g = DTYPES[case["dtype"]], _generator(seed, 5)
    logits = _randn((b, k + 1, v), torch.float32, g, 2.5)
    st = dict(target=torch.softmax(logits, 2).to(dt), draft=None, num=None)
    # the draft model's distribution: near the target's, as a trained one's
    near = torch.softmax(logits[:, :k] + _randn((b, k, v), torch.float32, g, 0.7), 2)
    if k:
        st["tokens"] = torch.multinomial(near.flatten(0, 1), 1, generator=g).view(b, k).to(torch.int32)
    else:
        st["tokens"] = torch.empty((b, 0), dtype=torch.int32, device="cuda")
    if case["drafted"] == "probs":
        st["draft"] = near.to(dt)
    elif k:         # looked up: often the likeliest token
        best = st["target"][:, :k].argmax(2).to(torch.int32)
        st["tokens"] = torch.where(torch.rand((b, k), generator=g, device="cuda") < 0.7, best, st["tokens"])
        # greedy requests have all their target's weight on one token
        greedy = torch.rand((b,), generator=g, device="cuda") < 0.5
        one = torch.zeros_like(st["target"]).scatter_(2, st["target"].argmax(2, keepdim=True), 1.0)
        st["target"] = torch.where(greedy[:, None, None], one, st["target"])
    r = np.random.default_rng([seed, 25])
    if case["ragged"]:
        st["num"] = _i32(r.integers(0, k + 1, b))
    st["uniforms"] = torch.rand((b, k + 1), generator=g, device="cuda")
    st["context"] = _i32(r.integers(1, 131072, b))
    return st


def prepare(case, seed):
    st = {"rotate": _prepare_heads, "norm": _prepare_heads, "window": _prepare_window,
          "verify": _prepare_verify}[case["op"]](case, seed)
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


def _handle(st):
    if "rotary" not in st:
        st["rotary"] = _rotary(st["case"])
    return st["rotary"]


def _own_rotate(api, st):
    q, k = api.rotate_heads(st["q"], st["k"], st["positions"], _handle(st), q_out=st["q_out"], k_out=st["k_out"])
    return (q,) if k is None else (q, k)


def _own_norm(api, st):
    q = api.rotate_store_kv(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["k_cache"], st["v_cache"],
                            _handle(st), norm=st["case"]["norm"], q_weight=st["q_weight"], k_weight=st["k_weight"],
                            q_bias=st["q_bias"], k_bias=st["k_bias"], eps=EPS, q_out=st["q_out"])
    return q, st["k_cache"], st["v_cache"]


def _own_window(api, st):
    c = st["case"]
    return api.paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["start"], st["seq"],
                               scale=st["scale"], max_new=st["max_new"], return_lse=True, window=c["window"],
                               sink_tokens=c["sinks"])


def _own_verify(api, st):
    r = api.verify_drafts(st["tokens"], st["target"], st["uniforms"], draft_probs=st["draft"], num_drafts=st["num"],
                          context_lens=st["context"])
    return r.tokens, r.num_accepted, r.next_lens


def _inv_freq(case):
    """Angles a position, in radians: base^(-2i/R), scaled as the case says."""
    rot = case["rot_dim"]
    s = SCALING[case["scaling"]] or {}
    base = BASE * s["factor"] ** (rot / (rot - 2)) if s.get("kind") == "base" else BASE
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if s.get("kind") == "linear":
        f = f / s["factor"]
    elif s.get("kind") == "parts":
        turns = s["original"] * f / (2 * math.pi)       # turns over the original context
        keep = np.clip((turns - s["low"]) / (s["high"] - s["low"]), 0.0, 1.0)
        f = f * (keep + (1 - keep) / s["factor"])
    return torch.from_numpy(f).cuda()


def _plain_rotated(x, st, norm=None, w=None, b=None):
    c = st["case"]
    rot, off = c["rot_dim"], c["offset"]
    y = x.float()
    if norm == "rms":
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    elif norm == "layer":
        y = y - y.mean(-1, keepdim=True)
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float() + b.float()
    angle = st["positions"].double()[:, None] * _inv_freq(c)
    m = MAGNITUDE[c["scaling"]]
    cos, sin = (angle.cos() * m).float()[:, None], (angle.sin() * m).float()[:, None]
    z = y[..., off:off + rot]
    if c["layout"] == "half":
        lo, hi = z[..., :rot // 2], z[..., rot // 2:]
        z = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    else:
        lo, hi = z[..., 0::2], z[..., 1::2]
        z = torch.stack([lo * cos - hi * sin, hi * cos + lo * sin], -1).flatten(-2)
    return torch.cat([y[..., :off], z, y[..., off + rot:]], -1).to(x.dtype)


def _live_rows(st, out, y):
    out.copy_(torch.where((st["positions"] >= 0)[:, None, None], y, out))
    return out


def _plain_rotate(st):
    q = _live_rows(st, st["q_out"], _plain_rotated(st["q"], st))
    return (q,) if st["k"] is None else (q, _live_rows(st, st["k_out"], _plain_rotated(st["k"], st)))


def _plain_norm(st):
    n, pt = st["case"]["norm"], st["case"]["page_tokens"]
    q = _live_rows(st, st["q_out"], _plain_rotated(st["q"], st, n, st["q_weight"], st["q_bias"]))
    k = _plain_rotated(st["k"], st, n, st["k_weight"], st["k_bias"])
    live = (st["slots"] >= 0).nonzero()[:, 0]
    s = st["slots"][live]
    st["k_cache"][s // pt, s % pt] = k[live]
    st["v_cache"][s // pt, s % pt] = st["v"][live]
    return q, st["k_cache"], st["v_cache"]


def _plain_window(st):
    c = st["case"]
    h, gq, d, pt = c["kv_heads"], c["group"], c["head_dim"], c["page_tokens"]
    out, lse = torch.empty_like(st["q"]), torch.empty(st["q"].shape[:2], dtype=torch.float32, device="cuda")
    t0 = 0
    for b, (s, n) in enumerate(st["lens"]):
        for r0 in range(0, n, 1024):        # rows in parts, to bound the score matrix
            m = min(1024, n - r0)
            first, last = s - n + r0, s - n + r0 + m - 1
            lo = max(0, first + 1 - c["window"])
            key = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), torch.arange(lo, last + 1, device="cuda")])
            pos = torch.arange(first, last + 1, device="cuda")[:, None]
            seen = (key <= pos) & ((key > pos - c["window"]) | (key < c["sinks"]))
            page = st["table"][b][key // pt].long()
            some = seen.any(0)              # keys of freed pages, that no row sees
            k = torch.where(some[:, None, None], st["k_cache"][page, key % pt], 0)
            v = torch.where(some[:, None, None], st["v_cache"][page, key % pt], 0)
            rows = slice(t0 + r0, t0 + r0 + m)
            for j in range(h):
                q = st["q"][rows, j * gq:(j + 1) * gq].float().reshape(m * gq, d)
                x = (q @ k[:, j].float().T * st["scale"]).view(m, gq, len(key))
                x.masked_fill_(~seen[:, None], -math.inf)
                top = x.amax(2, keepdim=True)
                x.sub_(top).exp_()
                tot = x.sum(2, keepdim=True)
                o = (x.view(m * gq, len(key)) @ v[:, j].float()).view(m, gq, d) / tot
                out[rows, j * gq:(j + 1) * gq] = o.to(out.dtype)
                lse[rows, j * gq:(j + 1) * gq] = (top + tot.log())[:, :, 0]
        t0 += n
    return out, lse


def _plain_verify(st):
    b, k, v = st["target"].shape[0], st["target"].shape[1] - 1, st["target"].shape[2]
    tok, u = st["tokens"].long(), st["uniforms"].double()
    num = torch.full((b,), k, device="cuda") if st["num"] is None else st["num"].long()
    at = torch.arange(b, device="cuda")
    if k:
        p = st["target"][:, :k].gather(2, tok[:, :, None])[:, :, 0].double()
        q = 1.0 if st["draft"] is None else st["draft"].gather(2, tok[:, :, None])[:, :, 0].double()
        ok = (u[:, :k] * q < p) & (torch.arange(k, device="cuda")[None] < num[:, None])
        acc = ok.long().cumprod(1).sum(1)
    else:
        acc = torch.zeros(b, dtype=torch.int64, device="cuda")
    pa = st["target"][at, acc].double()
    rest = pa
    if k:
        i = acc.clamp(max=k - 1)
        if st["draft"] is None:
            q = torch.zeros_like(pa).scatter_(1, tok[at, i][:, None], 1.0)
        else:
            q = st["draft"][at, i].double()
        left = (pa - q).clamp(min=0)
        refused = (acc < num) & (left.sum(1) > 0)
        rest = torch.where(refused[:, None], left, pa)
    cum = rest.cumsum(1)
    following = (cum <= u[:, k:] * cum[:, -1:]).sum(1)
    j = torch.arange(k + 1, device="cuda")[None]
    out = torch.cat([tok, torch.zeros((b, 1), dtype=torch.int64, device="cuda")], 1)
    out = torch.where(j < acc[:, None], out, torch.where(j == acc[:, None], following[:, None], -1))
    i32 = torch.int32
    return out.to(i32), acc.to(i32), (st["context"] + 1 + acc).to(i32)


_OWN = {"rotate": _own_rotate, "norm": _own_norm, "window": _own_window, "verify": _own_verify}
_PLAIN = {"rotate": _plain_rotate, "norm": _plain_norm, "window": _plain_window, "verify": _plain_verify}


# ---------------------------------------------------------------------------
# work and exact answers
# ---------------------------------------------------------------------------

def work(case):
    """Bytes and operations of one pass: each input read once, each output
    written once."""
    op = case["op"]
    if op in ("rotate", "norm"):
        t, h, d = case["tokens"], case["q_heads"] + case["kv_heads"], case["head_dim"]
        moved = 4 * t * h * d + 4 * (t + case["pad"])
        if op == "norm":
            moved += 4 * t * case["kv_heads"] * d + 8 * (t + case["pad"])
        return dict(bytes=moved, flops=t * h * (3 * case["rot_dim"] + (4 * d if op == "norm" else 0)))
    if op == "verify":
        # One row of the target's probabilities a request, and the draft's where a draft is
        # refused (about seven in ten drafts are accepted).
        b, k = case["requests"], case["drafts"]
        refused = 1 - 0.7 ** k if case["drafted"] == "probs" else 0
        size = 4 if case["dtype"] == "fp32" else 2
        return dict(bytes=b * case["vocab"] * size * (1 + refused) + b * (8 * k + 20), flops=2 * b * case["vocab"])
    ctx, new = (x.astype(np.float64) for x in _lengths(case, 0))
    h, gq, d, w, s = case["kv_heads"], case["group"], case["head_dim"], case["window"], case["sinks"]
    pairs = kept = 0.0
    for c, n in zip(ctx, new):
        pos = c + np.arange(int(n))
        pairs += float((np.minimum(pos + 1, w) + np.minimum(s, np.maximum(pos + 1 - w, 0))).sum())
        lo = max(0.0, c + 1 - w)
        kept += c + n - lo + min(s, lo)
    rows = float(new.sum())
    return dict(bytes=float(4 * kept * h * d + rows * h * gq * (4 * d + 4)), flops=float(4 * d * h * gq * pairs))


def exact(case, seed):
    st = prepare(case, seed)
    return {"rotate": _exact_rotate, "norm": _exact_norm, "window": _exact_window, "verify": _exact_verify}[
        case["op"]](case, st)


def _exact_heads(case, st, x, weight=None, bias=None):
    """float64: complex numbers turned by exp(i * angle), the rest as it is."""
    y = x.double()
    if weight is not None:
        if case["norm"] == "layer":
            y = y - y.sum(-1, keepdim=True) / y.shape[-1]
        y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + EPS) * weight.double()
        if bias is not None:
            y = y + bias.double()
    rot, off, s = case["rot_dim"], case["offset"], SCALING[case["scaling"]]
    freq = []
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(BASE))
        if s is not None and s["kind"] == "base":
            f = math.exp(-2.0 * i / rot * (math.log(BASE) + rot / (rot - 2.0) * math.log(s["factor"])))
        elif s is not None and s["kind"] == "linear":
            f /= s["factor"]
        elif s is not None:
            share = (s["original"] / (2 * math.pi / f) - s["low"]) / (s["high"] - s["low"])
            share = min(1.0, max(0.0, share))
            f = (1 - share) * f / s["factor"] + share * f
        freq.append(f)
    angle = st["positions"].double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, MAGNITUDE[case["scaling"]]), angle)
    part = y[..., off:off + rot]
    if case["layout"] == "half":
        z = torch.complex(part[..., :rot // 2], part[..., rot // 2:]) * turn
        part = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(part.reshape(*part.shape[:-1], rot // 2, 2).contiguous()) * turn
        part = torch.view_as_real(z).reshape(part.shape)
    y = y.clone()
    y[..., off:off + rot] = part
    return y


def _exact_rotate(case, st):
    out = []
    for x in (st["q"], st["k"]):
        if x is not None:
            y = _exact_heads(case, st, x)
            y[st["positions"] < 0] = 0.0
            out.append(y)
    return tuple(out)


def _exact_norm(case, st):
    q = _exact_heads(case, st, st["q"], st["q_weight"], st["q_bias"])
    k = _exact_heads(case, st, st["k"], st["k_weight"], st["k_bias"])
    q[st["positions"] < 0] = 0.0
    slots = st["slots"].tolist()
    put = [i for i, s in enumerate(slots) if s >= 0]
    out = [q]
    for rows, cache in ((k, st["k_cache"]), (st["v"].double(), st["v_cache"])):
        flat = cache.double().flatten(0, 1)
        flat[[slots[i] for i in put]] = rows[put]
        out.append(flat.view(cache.shape))
    return tuple(out)


def _exact_window(case, st):
    h, gq, d, pt = case["kv_heads"], case["group"], case["head_dim"], case["page_tokens"]
    w, sinks = case["window"], case["sinks"]
    t, heads = st["q"].shape[:2]
    if 4.0 * d * heads * sum(n * min(s, w + sinks + 512) for s, n in st["lens"]) > 6e12:
        return None
    out = torch.zeros((t, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((t, heads), dtype=torch.float64, device="cuda")
    first = 0
    for b, (s, n) in enumerate(st["lens"]):
        for i0 in range(0, n, 512):
            i1 = min(n, i0 + 512)
            p0, p1 = s - n + i0, s - n + i1         # positions [p0, p1)
            tok = [j for j in range(min(sinks, p1))] + list(range(max(0, p0 - w + 1, min(sinks, p1)), p1))
            tok = torch.tensor(tok, device="cuda")
            back = torch.arange(p0, p1, device="cuda")[:, None] - tok[None]
            hidden = (back < 0) | ((back >= w) & (tok[None] >= sinks))
            where = st["table"][b].long()[tok // pt] * pt + tok % pt
            useful = ~hidden.all(0)
            for j in range(h):
                k = st["k_cache"].flatten(0, 1)[where, j].double()
                v = st["v_cache"].flatten(0, 1)[where, j].double()
                k[~useful], v[~useful] = 0.0, 0.0
                q = st["q"][first + i0:first + i1, j * gq:(j + 1) * gq].double()
                x = torch.einsum("tgd,sd->gts", q, k) * st["scale"]
                x = torch.where(hidden[None], -math.inf, x)
                z = torch.logsumexp(x, 2)
                p = torch.exp(x - z[:, :, None])
                out[first + i0:first + i1, j * gq:(j + 1) * gq] = torch.einsum("gts,sd->tgd", p, v)
                lse[first + i0:first + i1, j * gq:(j + 1) * gq] = z.T
        first += n
    return out, lse


def _exact_verify(case, st):
    b, k = case["requests"], case["drafts"]
    tokens, u = st["tokens"].tolist(), st["uniforms"].double().tolist()
    num = [k] * b if st["num"] is None else st["num"].tolist()
    out = np.full((b, k + 1), -1, np.int32)
    accepted = np.zeros(b, np.int32)
    for r in range(b):
        a = 0
        while a < num[r]:
            x = tokens[r][a]
            q = 1.0 if st["draft"] is None else float(st["draft"][r, a, x])
            if not u[r][a] * q < float(st["target"][r, a, x]):
                break
            a += 1
        weight = st["target"][r, a].double().cpu().numpy()
        if a < num[r]:
            if st["draft"] is None:
                left = weight.copy()
                left[tokens[r][a]] -= 1.0
            else:
                left = weight - st["draft"][r, a].double().cpu().numpy()
            left = np.maximum(left, 0.0)
            if left.any():
                weight = left
        upto = np.cumsum(weight)
        out[r, :a] = tokens[r][:a]
        out[r, a] = np.searchsorted(upto, u[r][k] * upto[-1], side="right")
        accepted[r] = a
    return out, accepted, st["context"].cpu().numpy() + 1 + accepted
