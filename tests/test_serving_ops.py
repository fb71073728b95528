"""Serving operators around the indexer: page maps, paged stores and paged
attention (include/qsa.h) against plain implementations in 64 bits.

Attention tolerances, per output element, from the arithmetic: the fp32 scores
are off by at most dx = (D + 2) * 2^-23 * scale * max_j sum_i |q_i k_ji| (a
truncating accumulator allowed for), so each probability relatively by 2 dx at
most, numerator and denominator together; every probability is rounded to the
16-bit type once (half a step: u = eps / 2) and so is the output; sums of n
terms add n * 2^-24 and the exponentials 2^-20.  With A = sum_j p_j |v_j| the
output is off by at most u (|o| + A) + A (2 dx + n 2^-24 + 2^-20), and for
fp16, whose smallest step is 2^-24, n * 2^-25 * max|v| more.  The
log-sum-exp is off by dx + n 2^-24 + 2^-20 + 2^-22 |lse|."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_02_gb300 as qsa  # noqa: E402
from sparse_attention_indexer_02_gb300 import _abi, torch_api  # noqa: E402
from sparse_attention_indexer_02_gb300 import build as qbuild  # noqa: E402

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load_library()


@pytest.fixture(scope="module")
def cuda(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert qsa.device_status() == 0


# ---------------------------------------------------------------------------
# refusals (host only)
# ---------------------------------------------------------------------------

def _maps_desc(**kw):
    base = dict(num_requests=2, page_tokens=16, max_pages=8, ratio=4, partial_cols=0, reserved=0, table_stride=8,
                num_free=4, max_tokens=10)
    base.update(kw)
    return _abi.PageMapsDesc(*(base[n] for n, _ in _abi.PageMapsDesc._fields_))


def _kv_desc(**kw):
    base = dict(dtype=_abi.HALF_BF16, num_pages=4, page_tokens=16, num_kv_heads=2, head_dim=128, reserved=0,
                k_page_stride=8192, k_token_stride=512, k_head_stride=256, v_page_stride=8192, v_token_stride=512,
                v_head_stride=256)
    base.update(kw)
    return _abi.KvDesc(*(base[n] for n, _ in _abi.KvDesc._fields_))


def _attn_desc(kv=None, **kw):
    base = dict(num_requests=2, num_q_heads=8, max_pages=8, max_new=1, num_selected=0, ratio=1, local_tokens=0,
                form=_abi.ATTN_AUTO, num_tokens=2, table_stride=8, q_token_stride=2048, q_head_stride=256,
                out_token_stride=2048, out_head_stride=256, scale=0.1, reserved=0)
    base.update(kw)
    return _abi.AttnDesc(kv or _kv_desc(), *(base[n] for n, _ in _abi.AttnDesc._fields_[1:]))


def _refused(status, fn, *args, **kw):
    with pytest.raises(qsa.QSAError) as e:
        fn(*args, **kw)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("kw,status", [
    (dict(num_requests=-1), qsa.QSA_ERR_INVALID_ARG),
    (dict(num_requests=16385), qsa.QSA_ERR_UNSUPPORTED),
    (dict(page_tokens=0), qsa.QSA_ERR_INVALID_ARG),
    (dict(max_pages=0), qsa.QSA_ERR_INVALID_ARG),
    (dict(max_pages=1 << 28, table_stride=1 << 28), qsa.QSA_ERR_INVALID_ARG),
    (dict(ratio=3), qsa.QSA_ERR_INVALID_ARG),
    (dict(ratio=0), qsa.QSA_ERR_INVALID_ARG),
    (dict(partial_cols=2), qsa.QSA_ERR_INVALID_ARG),
    (dict(table_stride=7), qsa.QSA_ERR_INVALID_ARG),
    (dict(num_free=-1), qsa.QSA_ERR_INVALID_ARG),
    (dict(max_tokens=-1), qsa.QSA_ERR_INVALID_ARG),
    (dict(reserved=1), qsa.QSA_ERR_INVALID_ARG),
])
def test_page_maps_descriptor_refusals(lib, kw, status):
    _refused(status, _abi.build_page_maps, _maps_desc(**kw), *[16] * 12, stream=0)


@pytest.mark.parametrize("at", range(7))
def test_page_maps_null_and_misaligned(lib, at):
    args = [16] * 12
    args[at] = None
    _refused(qsa.QSA_ERR_INVALID_ARG, _abi.build_page_maps, _maps_desc(), *args, stream=0)
    args[at] = 18 if at < 6 else 20
    _refused(qsa.QSA_ERR_INVALID_ARG, _abi.build_page_maps, _maps_desc(), *args, stream=0)


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(num_pages=0), dict(page_tokens=0), dict(num_kv_heads=0),
                                dict(head_dim=12), dict(head_dim=0), dict(k_page_stride=8), dict(v_token_stride=0),
                                dict(v_head_stride=-256), dict(reserved=1)])
def test_kv_descriptor_refusals(lib, kw):
    d = _kv_desc(**kw)
    _refused(qsa.QSA_ERR_INVALID_ARG, _abi.store_paged_kv, d, 16, 512, 256, 16, 512, 256, 16, 3, 16, 16, stream=0)
    _refused(qsa.QSA_ERR_INVALID_ARG, qsa.plan_attention, _attn_desc(kv=d))


@pytest.mark.parametrize("args", [
    (None, 512, 256, 16, 512, 256, 16, 3, 16, 16), (16, 512, 256, 16, 512, 256, None, 3, 16, 16),
    (16, 512, 256, 16, 512, 256, 16, 3, 16, None), (24, 512, 256, 16, 512, 256, 16, 3, 16, 16),
    (16, 512, 256, 16, 512, 256, 20, 3, 16, 16), (16, 504, 256, 16, 512, 256, 16, 3, 16, 16),
    (16, 512, 256, 16, 512, 0, 16, 3, 16, 16), (16, 512, 256, 16, 512, 256, 16, -1, 16, 16)])
def test_store_refusals(lib, args):
    _refused(qsa.QSA_ERR_INVALID_ARG, _abi.store_paged_kv, _kv_desc(), *args, stream=0)


@pytest.mark.parametrize("desc,keys,stride,slots,n,cache,scales,status", [
    ((0, 4, 16, 64, 4096, 0), 16, 256, 16, 2, 16, None, qsa.QSA_ERR_UNSUPPORTED),
    ((7, 4, 16, 128, 4096, 0), 16, 256, 16, 2, 16, None, qsa.QSA_ERR_INVALID_ARG),
    ((0, 4, 16, 128, 4080, 0), 16, 256, 16, 2, 16, None, qsa.QSA_ERR_INVALID_ARG),
    ((0, 4, 16, 128, 4096, 0), 16, 256, 16, 2, 16, 16, qsa.QSA_ERR_INVALID_ARG),
    ((1, 4, 16, 128, 2112, 2112), 16, 256, 16, 2, 16, None, qsa.QSA_ERR_INVALID_ARG),
    ((1, 4, 16, 128, 2112, 60), 16, 256, 16, 2, 16, 16, qsa.QSA_ERR_INVALID_ARG),
    ((1, 4, 16, 128, 2112, 2112), 24, 256, 16, 2, 16, 16, qsa.QSA_ERR_INVALID_ARG),
    ((1, 4, 16, 128, 2112, 2112), 16, 250, 16, 2, 16, 16, qsa.QSA_ERR_INVALID_ARG),
    ((1, 4, 16, 128, 2112, 2112), 16, 256, None, 2, 16, 16, qsa.QSA_ERR_INVALID_ARG),
    ((1, 0, 16, 128, 2112, 2112), 16, 256, 16, 2, 16, 16, qsa.QSA_ERR_INVALID_ARG)])
def test_index_store_refusals(lib, desc, keys, stride, slots, n, cache, scales, status):
    _refused(status, _abi.store_index_keys, _abi.IndexCacheDesc(*desc), keys, stride, slots, n, cache, scales, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(num_requests=-1), qsa.QSA_ERR_INVALID_ARG), (dict(num_q_heads=7), qsa.QSA_ERR_INVALID_ARG),
    (dict(num_q_heads=0), qsa.QSA_ERR_INVALID_ARG), (dict(num_q_heads=514), qsa.QSA_ERR_INVALID_ARG),
    (dict(max_pages=0), qsa.QSA_ERR_INVALID_ARG), (dict(max_new=-1), qsa.QSA_ERR_INVALID_ARG),
    (dict(num_selected=-1), qsa.QSA_ERR_INVALID_ARG), (dict(ratio=0), qsa.QSA_ERR_INVALID_ARG),
    (dict(local_tokens=-1), qsa.QSA_ERR_INVALID_ARG), (dict(num_selected=1 << 28, ratio=8), qsa.QSA_ERR_INVALID_ARG),
    (dict(form=3), qsa.QSA_ERR_INVALID_ARG), (dict(num_tokens=-1), qsa.QSA_ERR_INVALID_ARG),
    (dict(table_stride=-1), qsa.QSA_ERR_INVALID_ARG), (dict(q_token_stride=24), qsa.QSA_ERR_INVALID_ARG),
    (dict(out_head_stride=0), qsa.QSA_ERR_INVALID_ARG), (dict(scale=0.0), qsa.QSA_ERR_INVALID_ARG),
    (dict(scale=-1.0), qsa.QSA_ERR_INVALID_ARG), (dict(scale=math.inf), qsa.QSA_ERR_INVALID_ARG),
    (dict(scale=math.nan), qsa.QSA_ERR_INVALID_ARG), (dict(reserved=3), qsa.QSA_ERR_INVALID_ARG),
    (dict(form=_abi.ATTN_TILE, num_selected=4), qsa.QSA_ERR_UNSUPPORTED),
    (dict(kv=_kv_desc(head_dim=96), form=0), qsa.QSA_ERR_UNSUPPORTED),
    (dict(kv=_kv_desc(page_tokens=20), form=_abi.ATTN_TILE), qsa.QSA_ERR_UNSUPPORTED)])
def test_attention_descriptor_refusals(lib, kw, status):
    kw = dict(kw)
    d = _attn_desc(kv=kw.pop("kv", None), **kw)
    _refused(status, qsa.plan_attention, d)
    _refused(status, qsa.paged_attention_workspace_bytes, d)
    _refused(status, _abi.paged_attention, d, *[16] * 6, None, 16, 16, 16, 1 << 30, stream=0)


def test_attention_pointer_refusals(lib):
    good = [16] * 6 + [None, 16, 16, 16, 1 << 30]
    for at in (0, 1, 2, 3, 4, 5, 7, 9):
        bad = list(good)
        bad[at] = None
        _refused(qsa.QSA_ERR_INVALID_ARG, _abi.paged_attention, _attn_desc(), *bad, stream=0)
    for at in (0, 1, 2, 7, 9):
        bad = list(good)
        bad[at] = 24
        _refused(qsa.QSA_ERR_INVALID_ARG, _abi.paged_attention, _attn_desc(), *bad, stream=0)
    need = qsa.paged_attention_workspace_bytes(_attn_desc())
    _refused(qsa.QSA_ERR_INVALID_ARG, _abi.paged_attention, _attn_desc(), *good[:-1], need - 1, stream=0)
    _refused(qsa.QSA_ERR_INVALID_ARG, _abi.paged_attention, _attn_desc(), *[16] * 7, *good[7:], stream=0)
    _refused(qsa.QSA_ERR_INVALID_ARG, _abi.paged_attention, _attn_desc(num_selected=4), *good, stream=0)


def test_empty_calls_launch_nothing(lib):
    _abi.paged_attention(_attn_desc(num_requests=0), *[None] * 10, 0, stream=0)
    _abi.paged_attention(_attn_desc(num_tokens=0), *[None] * 10, 0, stream=0)
    _abi.store_paged_kv(_kv_desc(), None, 512, 256, None, 512, 256, None, 0, None, None, stream=0)
    _abi.store_index_keys(_abi.IndexCacheDesc(1, 4, 16, 128, 2112, 2112), None, 256, None, 0, None, None, stream=0)


def test_attention_form_choice(lib):
    """Tiles above 16 query rows a key/value head (here 4 a token), where pages allow them."""
    plan = lambda **kw: qsa.plan_attention(_attn_desc(**kw))  # noqa: E731
    assert plan(max_new=4) == _abi.ATTN_GATHER and plan(max_new=5) == _abi.ATTN_TILE
    assert plan(max_new=0, num_tokens=8) == _abi.ATTN_GATHER and plan(max_new=0, num_tokens=9) == _abi.ATTN_TILE
    for pt, form in ((8, 2), (16, 2), (32, 2), (64, 2), (128, 2), (256, 2), (384, 2), (1, 1), (20, 1), (192, 1)):
        assert plan(max_new=64, kv=_kv_desc(page_tokens=pt)) == form, pt
    assert plan(max_new=64, num_selected=8) == _abi.ATTN_GATHER
    assert plan(max_new=64, form=_abi.ATTN_GATHER) == _abi.ATTN_GATHER
    assert plan(max_new=1, form=_abi.ATTN_TILE) == _abi.ATTN_TILE


def test_torch_api_refuses_wrong_tensors(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kc = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16)
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    ok = dict(q=q, k_cache=kc, v_cache=kc, block_table=i32(2, 4), query_start=i32(3), seq_lens=i32(2))
    for name, t in (("q", q.half()), ("q", q[:, :, :64]), ("v_cache", kc.half()), ("v_cache", kc[:, :8]),
                    ("k_cache", kc.float()), ("block_table", i32(2, 4).long()), ("block_table", i32(4, 2).T),
                    ("query_start", i32(2)), ("seq_lens", i32(2).long()), ("seq_lens", i32(3))):
        with pytest.raises(ValueError, match="must|differ"):
            torch_api.paged_attention(**{**ok, name: t})
    for kw in (dict(selected=i32(2, 4)), dict(selected=i32(3, 0)), dict(out=q.half()), dict(lse=torch.zeros(3, 4))):
        with pytest.raises(ValueError):
            torch_api.paged_attention(**ok, **kw)
    slots = torch.zeros(3, dtype=torch.int64)
    kv = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    for args in ((kv[:2], kv, slots), (kv, kv.half(), slots), (kv, kv, slots.int()), (kv, kv[:, :1], slots)):
        with pytest.raises(ValueError):
            torch_api.store_paged_kv(*args, kc, kc)
    with pytest.raises(ValueError):
        torch_api.store_index_keys(torch.zeros(3, 128), slots, kc, page_cols=16)
    with pytest.raises(ValueError):   # fp8 without the scales' place
        torch_api.store_index_keys(torch.zeros((3, 128), dtype=torch.bfloat16), slots,
                                   torch.zeros((4, 2112), dtype=torch.uint8), page_cols=16, kv_dtype=qsa.KV_FP8_E4M3)
    with pytest.raises(ValueError):   # scales past the page
        torch_api.store_index_keys(torch.zeros((3, 128), dtype=torch.bfloat16), slots,
                                   torch.zeros((4, 2100), dtype=torch.uint8), page_cols=16, kv_dtype=qsa.KV_FP8_E4M3,
                                   scale_offset=2048)
    for args in ((i32(2), i32(3), i32(4), i32(2, 4)), (i32(2), i32(2), i32(4), i32(3, 4)),
                 (i32(2).long(), i32(2), i32(4), i32(2, 4))):
        with pytest.raises(ValueError):
            torch_api.build_page_maps(*args, page_tokens=16, max_tokens=4)


def test_torch_api_refuses_host_tensors(lib):
    """Tensors that fit in every other way, but lie in host memory."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kc = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16)
    kv, slots = torch.zeros((3, 2, 128), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: torch_api.paged_attention(torch.zeros((3, 8, 128), dtype=torch.bfloat16), kc, kc, i32(2, 4),
                                                   i32(3), i32(2)),
                 lambda: torch_api.store_paged_kv(kv, kv, slots, kc, kc),
                 lambda: torch_api.store_index_keys(torch.zeros((3, 128), dtype=torch.bfloat16), slots,
                                                    torch.zeros((4, 16, 128), dtype=torch.bfloat16), page_cols=16),
                 lambda: torch_api.build_page_maps(i32(2), i32(2), i32(4), i32(2, 4), page_tokens=16, max_tokens=4)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    for call in (lambda: torch_api.store_paged_kv(None, kv, slots, kc, kc),
                 lambda: torch_api.build_page_maps(i32(2), i32(2), i32(4), i32(2, 4), page_tokens="16", max_tokens=4),
                 lambda: torch_api.build_page_maps(i32(2), i32(2), i32(4), i32(2, 4), page_tokens=1 << 40,
                                                   max_tokens=4)):
        with pytest.raises((ValueError, TypeError)):
            call()


# ---------------------------------------------------------------------------
# page maps
# ---------------------------------------------------------------------------

def maps_reference(ctx, new, free, table, pt, ratio, partial, max_tokens):
    table = table.copy()
    cap = table.shape[1]
    start, taken, rows, seq = [0], 0, [], []
    for b in range(len(ctx)):
        c, n = max(int(ctx[b]), 0), max(int(new[b]), 0)
        for j in range(min(-(-c // pt), cap), min(-(-(c + n) // pt), cap)):
            table[b, j] = free[taken] if taken < len(free) else -1
            taken += 1
        for p in range(c, c + n):
            page = int(table[b, p // pt]) if p // pt < cap else -1
            slot = page * pt + p % pt if page >= 0 else -1
            done = slot >= 0 and (p + 1) % ratio == 0
            rows.append((slot, p, b, -(-(p + 1) // ratio) if partial else (p + 1) // ratio, slot // ratio if done else -1))
        start.append(start[-1] + n)
        seq.append(c + n)
    rows = (rows + [(-1, -1, -1, 0, -1)] * max(0, max_tokens - len(rows)))[:max_tokens]
    r = np.array(rows, np.int64).reshape(max_tokens, 5)
    return table, start, seq, r, taken


def _cu(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


MAPS = [  # name, ctx, new, page_tokens, ratio, partial, free pages short by, extra table columns, pad
    ("one_token", [0], [1], 16, 4, False, 0, 0, 0),
    ("nothing_new", [5, 0, 32], [0, 0, 0], 16, 4, False, 0, 1, 3),
    ("page_edges", [15, 16, 17, 31, 0, 32], [1, 1, 1, 2, 16, 17], 16, 4, True, 0, 0, 1),
    ("page_of_one", [3, 0, 7], [2, 5, 1], 1, 1, False, 0, 2, 0),
    ("odd_pages", [19, 20, 41, 0], [1, 43, 0, 7], 20, 5, True, 0, 0, 5),
    ("free_list_short", [10, 3, 60], [30, 40, 50], 16, 2, False, 4, 0, 0),
    ("negative_lengths", [-3, 4], [5, -2], 8, 1, False, 0, 0, 2),
    ("past_capacity", [30, 100], [40, 3], 16, 4, False, 0, -2, 0),
    ("many", None, None, 64, 4, False, 0, 1, 100),
]


@gpu
@pytest.mark.parametrize("case", MAPS, ids=[c[0] for c in MAPS])
def test_page_maps(cuda, case):
    name, ctx, new, pt, ratio, partial, short, extra, pad = case
    rng = np.random.default_rng(len(name))
    if ctx is None:
        ctx, new = rng.integers(0, 500, 3000), rng.integers(0, 9, 3000)
    c, n = np.maximum(ctx, 0), np.maximum(new, 0)
    width = max(1, int((-(-(c + n) // pt)).max()) + extra)
    have = np.minimum(-(-c // pt), width)
    table = np.full((len(c), width), -1, np.int64)
    pages = rng.permutation(int((-(-(c + n) // pt)).sum()) + 5)
    used = 0
    for b in range(len(c)):
        table[b, :have[b]] = pages[used:used + have[b]]
        used += have[b]
    want_pages = int((np.minimum(-(-(c + n) // pt), width) - have).sum())
    free = pages[used:used + max(0, want_pages - short)]
    max_tokens = int(n.sum()) + pad
    wide = _cu(np.pad(table, ((0, 0), (0, 3)), constant_values=77))   # rows further apart than their entries
    d_table = wide[:, :width]
    for _ in range(2):   # the second call writes the same again
        got = torch_api.build_page_maps(_cu(ctx), _cu(new), _cu(free), d_table, page_tokens=pt, max_tokens=max_tokens,
                                        ratio=ratio, partial_cols=partial)
        t, start, seq, rows, taken = maps_reference(ctx, new, free, table, pt, ratio, partial, max_tokens)
        assert (d_table.cpu().numpy() == t).all() and (wide[:, width:] == 77).all()
        assert got.query_start.tolist() == start and got.seq_lens.tolist() == seq
        for i, f in enumerate(("slots", "positions", "token_request", "visible_cols", "column_slots")):
            assert (getattr(got, f).cpu().numpy() == rows[:, i]).all(), f
        assert got.pages_used.tolist() == [taken]


@gpu
def test_page_maps_no_requests_and_few_rows(cuda):
    e = _cu([])
    got = torch_api.build_page_maps(e, e, e, torch.zeros((0, 4), dtype=torch.int32, device="cuda"), page_tokens=16,
                                    max_tokens=5)
    assert got.query_start.tolist() == [0] and got.slots.tolist() == [-1] * 5 and got.pages_used.tolist() == [0]
    # fewer output rows than tokens: the rest is counted, not written
    guard = torch.full((9,), 99, dtype=torch.int64, device="cuda")
    out = torch_api.PageMaps(_cu([0, 0]), _cu([0]), guard[:6], _cu([0] * 6), _cu([0] * 6), _cu([0] * 6),
                             _cu([0] * 6, torch.int64), _cu([0]))
    torch_api.build_page_maps(_cu([0]), _cu([8]), _cu([3]), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                              page_tokens=16, max_tokens=6, out=out)
    assert guard.tolist() == [48, 49, 50, 51, 52, 53, 99, 99, 99] and out.query_start.tolist() == [0, 8]


@gpu
def test_page_maps_saturate(cuda):
    """Sums past 2^31 - 1 stay there; such tokens lie past the table and get no slot."""
    big = 2**31 - 1
    got = torch_api.build_page_maps(_cu([big, 2]), _cu([big, big]), _cu([0, 1]),
                                    torch.zeros((2, 2), dtype=torch.int32, device="cuda"), page_tokens=4, max_tokens=8)
    assert got.query_start.tolist() == [0, big, big] and got.seq_lens.tolist() == [big, big]
    assert got.slots.tolist() == [-1] * 8 and got.token_request.tolist() == [0] * 8
    assert got.pages_used.tolist() == [1]


# ---------------------------------------------------------------------------
# stores
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("T,H,D,pt,dt,strided", [
    (1, 1, 64, 1, "bf16", False), (37, 3, 128, 20, "fp16", True), (1000, 8, 128, 64, "bf16", True),
    (33, 2, 8, 16, "bf16", False), (5, 1, 136, 7, "fp16", False), (4097, 1, 64, 16, "bf16", True)])
@pytest.mark.parametrize("head_major", [False, True])
def test_store_paged_kv(cuda, T, H, D, pt, dt, strided, head_major):
    g = torch.Generator(device="cuda").manual_seed(T)
    pages = -(-T // pt) + 3
    base = torch.randn((T, 3 * H, D), generator=g, device="cuda").to(DT[dt])
    k, v = (base[:, H:2 * H], base[:, 2 * H:]) if strided else (base[:, :H].contiguous(), base[:, H:2 * H].contiguous())
    slots = torch.randperm(pages * pt, generator=g, device="cuda")[:T]
    slots[::7] = -1
    if T > 2:
        slots[1], slots[2] = pages * pt, 2**62   # past the cache: skipped
    shape = (2, pages, H, pt, D) if head_major else (2, pages, pt, H, D)
    cache = torch.randn(shape, generator=g, device="cuda").to(DT[dt])
    kc, vc = (cache.permute(0, 1, 3, 2, 4) if head_major else cache).unbind(0)
    want = [kc.clone(), vc.clone()]
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * pt:
            want[0][s // pt, s % pt], want[1][s // pt, s % pt] = k[i], v[i]
    torch_api.store_paged_kv(k, v, slots, kc, vc)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def e4m3_reference(x):
    """(codes uint8, scale) of bf16 rows: fp32 scale and quotient, nearest code, ties to even."""
    x = x.float().cpu()
    scale = x.abs().amax(1) / torch.tensor(448.0)
    y = (x / torch.where(scale > 0, scale, torch.ones(()))[:, None]).clamp(-448, 448)
    codes = y.to(torch.float8_e4m3fn).view(torch.uint8)
    codes[scale == 0] = 0
    return codes, scale


@gpu
def test_store_index_keys_code_borders(cuda):
    """Rows whose quotients lie on and next to the borders between codes, for
    scales of every size: each code is the division's."""
    r = np.random.default_rng(5)
    grid = np.arange(256, dtype=np.uint8)
    val = torch.from_numpy(grid).view(torch.float8_e4m3fn).float().numpy()
    val = np.sort(val[np.isfinite(val)])
    mids = (val[1:] + val[:-1]) / 2
    T = 4096
    amax = torch.from_numpy((r.integers(1, 256, T) * 2.0 ** r.integers(-140, 100, T)).astype(np.float32)).bfloat16().float()
    near = torch.from_numpy(r.choice(mids, (T, 128)).astype(np.float32)) * (amax / 448.0)[:, None]
    bits = near.bfloat16().view(torch.int16) + torch.from_numpy(r.integers(-1, 2, (T, 128)).astype(np.int16))
    keys = bits.view(torch.bfloat16).float().nan_to_num(0.0).clamp(-amax[:, None], amax[:, None]).bfloat16()
    keys[:, 0] = amax.bfloat16()
    cache = torch.zeros((T // 64, 64 * 132), dtype=torch.uint8, device="cuda")
    torch_api.store_index_keys(keys.cuda(), torch.arange(T, device="cuda"), cache, page_cols=64,
                               kv_dtype=qsa.KV_FP8_E4M3, scale_offset=64 * 128)
    codes, scale = e4m3_reference(keys)
    got = cache.cpu()
    assert torch.equal(got[:, 64 * 128:].contiguous().view(torch.float32).flatten(), scale)
    assert torch.equal(got[:, :64 * 128].reshape(T, 128), codes)


@gpu
@pytest.mark.parametrize("T,pc,fp8", [(1, 1, True), (1, 64, False), (100, 4, True), (1001, 64, True), (77, 16, False),
                                      (513, 20, True), (64, 3, True)])
def test_store_index_keys(cuda, T, pc, fp8):
    g = torch.Generator(device="cuda").manual_seed(T + pc)
    pages = -(-T // pc) + 2
    wide = torch.randn((T, 192), generator=g, device="cuda") * torch.exp2(
        torch.randint(-20, 20, (T, 1), generator=g, device="cuda").float())
    keys = wide.to(torch.bfloat16)[:, 64:]
    if T > 10:
        keys[3] = 0
        keys[4] = 2.0 ** -133    # scale below the smallest normal
        keys[5, 1:] = 0
        keys[6] = torch.arange(128, device="cuda") * 3.5   # quotients on code borders
    slots = torch.randperm(pages * pc, generator=g, device="cuda")[:T]
    if T > 10:
        slots[::5] = -1
        slots[1] = pages * pc
    if fp8:
        cache = torch.randint(0, 255, (pages, pc * 132), generator=g, device="cuda", dtype=torch.uint8)
        want = cache.cpu().clone()
        codes, scale = e4m3_reference(keys)
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < pages * pc:
                p, j = s // pc, s % pc
                want[p, j * 128:(j + 1) * 128] = codes[i]
                want[p, pc * 128 + 4 * j:pc * 128 + 4 * j + 4] = scale[i:i + 1].view(torch.uint8)
        torch_api.store_index_keys(keys, slots, cache, page_cols=pc, kv_dtype=qsa.KV_FP8_E4M3, scale_offset=pc * 128)
    else:
        cache = torch.randn((pages, pc, 128), generator=g, device="cuda").to(torch.bfloat16)
        want = cache.cpu().clone()
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < pages * pc:
                want[s // pc, s % pc] = keys[i].cpu()
        torch_api.store_index_keys(keys, slots, cache, page_cols=pc)
    assert torch.equal(cache.cpu(), want)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Problem:
    """Random requests over a shuffled pool; table entries nothing uses, and
    the slots past every request's end, hold NaN."""

    def __init__(self, lens, hkv, group, D, pt, dt, seed=0, head_major=False, strided=False, spread=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        self.lens, self.pt, self.group = lens, pt, group
        need = [-(-max(s, 0) // pt) for s, n in lens]
        total = sum(need)
        shape = (2, total + 1, hkv, pt, D) if head_major else (2, total + 1, pt, hkv, D)
        cache = torch.randn(shape, generator=g, device="cuda").to(DT[dt])
        self.cache = cache.permute(0, 1, 3, 2, 4) if head_major else cache
        self.kc, self.vc = self.cache.unbind(0)
        self.kc[total], self.vc[total] = math.nan, math.nan
        table = np.full((len(lens), max(need + [1]) + 2), total, np.int64)
        perm, used = r.permutation(total), 0
        for b, (s, n) in enumerate(lens):
            table[b, :need[b]] = perm[used:used + need[b]]
            used += need[b]
            if s > 0 and s % pt:
                self.kc[table[b, need[b] - 1], s % pt:] = math.nan
                self.vc[table[b, need[b] - 1], s % pt:] = math.nan
        self.table = _cu(table)
        T = sum(n for _, n in lens)
        H = hkv * group
        q = (torch.randn((T, (3 if strided else 1) * H, D), generator=g, device="cuda") * spread).to(DT[dt])
        self.q = q[:, H:2 * H] if strided else q
        self.start = _cu(np.concatenate([[0], np.cumsum([n for _, n in lens])]))
        self.seq = _cu([s for s, _ in lens])
        self.scale = D ** -0.5

    def run(self, **kw):
        return torch_api.paged_attention(self.q, self.kc, self.vc, self.table, self.start, self.seq,
                                         scale=self.scale, return_lse=True, **kw)

    def check(self, out, lse, selected=None, ratio=1, local=0):
        T, H, D = self.q.shape
        hkv = self.kc.shape[2]
        dt = self.q.dtype
        u = torch.finfo(dt).eps / 2
        t0 = 0
        for b, (s, n) in enumerate(self.lens):
            tok = torch.arange(max(s, 0), device="cuda")
            at = self.table[b].long()[tok // self.pt] * self.pt + tok % self.pt
            k = self.kc.flatten(0, 1)[at].double() if s > 0 else torch.zeros((0, hkv, D), device="cuda").double()
            v = self.vc.flatten(0, 1)[at].double() if s > 0 else torch.zeros((0, hkv, D), device="cuda").double()
            pos = torch.arange(max(s, 0) - n, max(s, 0), device="cuda")
            see = tok[None] <= pos[:, None]
            if selected is not None:
                sel = selected[t0:t0 + n]
                hit = torch.zeros_like(see)
                for i in range(n):
                    c = sel[i][(sel[i] >= 0) & (sel[i].long() * ratio < s)].long()
                    x = (c[:, None] * ratio + torch.arange(ratio, device="cuda")).flatten()
                    hit[i, x[x < s]] = True
                see &= hit | (tok[None] > pos[:, None] - local)
            for h in range(H):
                j = h // self.group
                q = self.q[t0:t0 + n, h].double()
                x = torch.where(see, q @ k[:, j].T * self.scale, -math.inf)
                z = torch.logsumexp(x, 1) if s > 0 else torch.full((n,), -math.inf, device="cuda").double()
                p = torch.where(see, torch.exp(x - z.clamp(min=-1e300)[:, None]), 0.0)
                o, A = p @ v[:, j], p @ v[:, j].abs()
                mag = torch.where(see, q.abs() @ k[:, j].abs().T, 0.0) * self.scale
                dx = (D + 2) * 2.0 ** -23 * (mag.amax(1) if s > 0 else torch.zeros(n, device="cuda"))
                cnt = see.sum(1)
                tol = u * (o.abs() + A) + A * (2 * dx + cnt * 2.0 ** -24 + 2.0 ** -20)[:, None]
                if dt == torch.float16 and s > 0:
                    tol = tol + (cnt * 2.0 ** -25)[:, None] * v[:, j].abs().max() + 2.0 ** -25
                got = out[t0:t0 + n, h].double()
                assert ((got - o).abs() <= tol).all(), (b, h, float(((got - o).abs() - tol).max()))
                empty = cnt == 0
                gl = lse[t0:t0 + n, h].double()
                assert (gl[empty] == -math.inf).all() and (got[empty] == 0).all()
                lt = dx + cnt * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * z.abs()
                assert ((gl - z).abs()[~empty] <= lt[~empty]).all(), (b, h)
            t0 += n


LENS = {
    "one_key": [(1, 1)],
    "decode": [(700, 1), (1, 1), (128, 1), (129, 1), (2000, 1), (17, 1)],
    "verify": [(300, 4), (5, 4), (4, 4), (257, 3), (1030, 1)],
    "chunk": [(200, 200), (513, 130), (64, 64)],
    "ragged": [(90, 33), (0, 0), (1000, 1), (129, 129), (700, 0), (385, 257), (16, 1)],
    "gaps": [(5, 0), (6, 0), (40, 1), (50, 0)],
}


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("hkv,group,D,pt,dt", [
    (1, 1, 128, 64, "bf16"), (2, 4, 128, 16, "bf16"), (2, 7, 64, 8, "fp16"), (1, 16, 64, 128, "bf16"),
    (3, 5, 128, 256, "fp16"), (1, 33, 128, 32, "bf16")])
def test_attention(cuda, form, lens, hkv, group, D, pt, dt):
    pr = Problem(LENS[lens], hkv, group, D, pt, dt, seed=len(lens) * 100 + group)
    out, lse = pr.run(form=form)
    pr.check(out, lse)


@gpu
@pytest.mark.parametrize("pt", [1, 3, 20, 192])
def test_attention_odd_pages(cuda, pt):
    pr = Problem([(333, 2), (41, 5), (7, 7)], 2, 3, 128, pt, "bf16", seed=pt)
    out, lse = pr.run(max_new=7)
    pr.check(out, lse)


@gpu
@pytest.mark.parametrize("form,group", [(f, g) for f in (_abi.ATTN_GATHER, _abi.ATTN_TILE) for g in (65, 100, 128)] +
                         [(_abi.ATTN_GATHER, 256)])
def test_attention_wide_groups(cuda, form, group):
    pr = Problem([(300, 5), (131, 1)], 1, group, 64, 64, "bf16", seed=group)
    out, lse = pr.run(form=form)
    pr.check(out, lse)


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
@pytest.mark.parametrize("hint", [0, 1, 10000])
def test_attention_hint_and_layouts(cuda, form, hint):
    """Strided q and out, a head-major cache, a wrong bound; rows of no request are left alone."""
    pr = Problem([(300, 70), (64, 3)], 2, 4, 128, 32, "bf16", seed=hint, head_major=True, strided=True)
    T, H, D = pr.q.shape
    big = torch.full((T + 3, H + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    torch_api.paged_attention(pr.q, pr.kc, pr.vc, pr.table, pr.start, pr.seq, scale=pr.scale, max_new=hint, form=form,
                              out=big[:T, 1:1 + H], lse=lse)
    pr.check(big[:T, 1:1 + H], lse)
    assert (big[T:] == 7).all() and (big[:, 0] == 7).all() and (big[:, -1] == 7).all()
    short = pr.start.clone()
    short[2] = 71   # two rows of q belong to no request now
    seq = pr.seq.clone()
    seq[1] = 62
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    torch_api.paged_attention(pr.q, pr.kc, pr.vc, pr.table, short, seq, scale=pr.scale, form=form, out=out)
    assert (out[71:] == 7).all() and not (out[70] == 7).all()


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
def test_attention_rows_that_see_nothing(cuda, form):
    """More new tokens than tokens: the first rows lie before position 0."""
    pr = Problem([(40, 40), (3, 8), (0, 2), (200, 1)], 2, 4, 128, 16, "bf16", seed=9)
    out, lse = pr.run(form=form)
    pr.check(out, lse)
    assert (lse[40:45] == -math.inf).all() and (lse[48:50] == -math.inf).all()


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
@pytest.mark.parametrize("B", [33, 390, 1100])
def test_attention_many_requests(cuda, form, B):
    """More requests than a warp, than a CTA, than two rounds of a CTA, some without new tokens."""
    r = np.random.default_rng(B)
    lens = [(int(s), min(int(s), int(n))) for s, n in zip(r.integers(0, 200, B), r.integers(0, 4, B))]
    pr = Problem(lens, 1, 2, 64, 16, "bf16", seed=B)
    out, lse = pr.run(form=form)
    pr.check(out, lse)


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
def test_attention_metadata_out_of_range(cuda, form):
    """Page ids are clamped into the pool, lengths to what the table holds, row
    starts to the rows there are: the results are those of the clamped values."""
    pr = Problem([(300, 40), (64, 3)], 2, 4, 128, 32, "bf16", seed=21)
    pr.kc.nan_to_num_(0.5)
    pr.vc.nan_to_num_(0.5)
    pages = pr.kc.shape[0]
    good = pr.table.clone()
    good[0, 1], good[0, 2], good[1, 0] = 0, pages - 1, pages - 1
    bad = good.clone()
    bad[0, 1], bad[0, 2], bad[1, 0] = -7, 2**31 - 1, pages
    pr.table = good
    want = pr.run(form=form)
    pr.table = bad
    got = pr.run(form=form)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # more tokens than the table's 32 * 12 hold: the keys end there, positions do not
    pr.table = good
    cap = good.shape[1] * 32
    for n in (cap + 40, 2**31 - 1):
        pr.seq = _cu([n, 64])
        far = pr.run(form=form)
        pr.seq = _cu([cap + 40, 64])
        near = pr.run(form=form)
        assert torch.equal(far[0], near[0]) and not far[0].isnan().any()
    pr.seq = _cu([-5, 64])
    neg = pr.run(form=form)
    assert (neg[1][:40] == -math.inf).all() and (neg[0][:40] == 0).all()
    pr.seq = _cu([300, 64])
    pr.start = _cu([0, 40, 10**6])
    late = pr.run(form=form)
    assert torch.equal(late[0], want[0])
    pr.start = _cu([-3, 40, 20])   # decreasing: the second request has no rows
    out = torch.full_like(want[0], 7.0)
    pr.run(form=form, out=out)
    assert torch.equal(out[:40], want[0][:40]) and (out[40:] == 7).all()


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
def test_attention_large_scores(cuda, form):
    """Scores of hundreds: one key takes all; growing maxima along the keys raise m again and again."""
    pr = Problem([(1500, 40)], 1, 4, 128, 64, "bf16", seed=3, spread=30.0)
    ramp = torch.linspace(0.1, 3.0, 1500, device="cuda")
    at = pr.table[0].long()[torch.arange(1500, device="cuda") // 64] * 64 + torch.arange(1500, device="cuda") % 64
    flat = pr.kc.view(-1, 1, 128)
    flat[at] = (flat[at].float() * ramp[:, None, None]).to(torch.bfloat16)
    out, lse = pr.run(form=form)
    pr.check(out, lse)


@gpu
@pytest.mark.parametrize("form,lens,hkv,group,D", [
    (_abi.ATTN_GATHER, [(40000, 1), (3, 1)], 2, 4, 128), (_abi.ATTN_GATHER, [(40000, 1)], 1, 30, 128),
    (_abi.ATTN_GATHER, [(20000, 3)], 1, 9, 64), (_abi.ATTN_TILE, [(30000, 100)], 2, 4, 128),
    (_abi.ATTN_TILE, [(25000, 3)], 1, 11, 64)])
def test_attention_splits_join_the_same_way(cuda, form, lens, hkv, group, D):
    """Long keys over many CTAs, all of them for the cases of one key/value
    head: right, the same bits each time, and the counters zero again."""
    pr = Problem(lens, hkv, group, D, 64, "bf16", seed=5)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    first = pr.run(form=form, workspace=ws)
    pr.check(*first)
    for _ in range(4):
        again = pr.run(form=form, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert int(ws[:_abi.ATTN_COUNTER_BYTES].sum()) == 0


@gpu
def test_attention_one_workspace_serves_both_forms(cuda):
    a = Problem([(9000, 1)], 2, 4, 128, 64, "bf16", seed=6)
    b = Problem([(5000, 64)], 2, 4, 64, 64, "fp16", seed=7)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    for pr in (a, b, a, b, a):
        pr.check(*pr.run(workspace=ws, max_new=pr.lens[0][1]))


@gpu
def test_kept_workspaces_dropped(cuda):
    pr = Problem([(9000, 1)], 2, 4, 128, 64, "bf16", seed=6)
    want = pr.run()
    torch.cuda.synchronize()
    torch_api.drop_attention_workspaces()
    got = pr.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_attention_graph_replays_new_lengths(cuda):
    """Captured once, replayed with lengths, queries and selections written in place."""
    pr = Problem([(900, 1), (450, 1)], 2, 4, 128, 64, "bf16", seed=8)
    st = torch.cuda.Stream()
    for form in (_abi.ATTN_GATHER, _abi.ATTN_TILE):
        pr.run(form=form)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out, lse = pr.run(form=form)
        for s0, s1 in ((900, 450), (3, 449), (128, 1)):
            pr.seq.copy_(_cu([s0, s1]))
            pr.q.mul_(-0.75)
            graph.replay()
            torch.cuda.synchronize()
            pr.lens = [(s0, 1), (s1, 1)]
            pr.check(out, lse)
        pr.seq.copy_(_cu([900, 450]))


@gpu
def test_operators_on_another_stream(cuda):
    """Inputs made on one stream, the call on another that waits for it."""
    pr = Problem([(3000, 1)] * 3, 2, 4, 128, 64, "bf16", seed=10)
    want = pr.run()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for handle in (st, st.cuda_stream):
        got = pr.run(stream=handle)
        st.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def _far_cache(D, dt):
    """Pages 5 GB apart: byte offsets past 32 bits."""
    stride = 5 << 29   # elements of 2 bytes: 5 GiB
    buf = torch.empty(2 * stride + 64 * D, dtype=dt, device="cuda")
    return torch.as_strided(buf, (3, 64, 1, D), (stride, D, D, 1))


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
def test_offsets_past_32_bits(cuda, form):
    D = 128
    pr = Problem([(150, 3)], 1, 4, D, 64, "bf16", seed=11)
    far = _far_cache(D, torch.bfloat16)
    k, v = pr.kc[:3].nan_to_num(), pr.vc[:3].nan_to_num()
    near = torch.zeros_like(v)
    torch_api.store_paged_kv(k.view(192, 1, D), v.view(192, 1, D), torch.arange(192, device="cuda"), far, near)
    assert torch.equal(far, k) and torch.equal(near, v)
    pr.kc, pr.vc = far, near
    pr.table.clamp_(max=2)
    out, lse = pr.run(form=form)
    pr.check(out, lse)


SELECT = [  # lens, hkv, group, D, pt, dt, k, ratio, local
    ([(700, 1), (65, 1), (3, 1)], 2, 4, 128, 64, "bf16", 40, 4, 0),
    ([(700, 4), (30, 2)], 1, 16, 128, 16, "fp16", 100, 4, 64),
    ([(260, 260)], 2, 3, 64, 64, "bf16", 17, 2, 5),
    ([(500, 3)], 1, 40, 128, 20, "bf16", 300, 1, 0),
    ([(2000, 1)] * 5, 1, 8, 128, 64, "bf16", 500, 4, 100),
    ([(129, 129)], 1, 1, 128, 8, "bf16", 1, 8, 1),
    ([(50, 9)], 2, 2, 64, 4, "fp16", 2048, 4, 3),
]


@gpu
@pytest.mark.parametrize("case", SELECT, ids=range(len(SELECT)))
def test_attention_selected(cuda, case):
    lens, hkv, group, D, pt, dt, k, ratio, local = case
    pr = Problem(lens, hkv, group, D, pt, dt, seed=k)
    r = np.random.default_rng(k)
    rows = []
    for s, n in lens:
        for i in range(n):
            cols = r.permutation(-(-s // ratio) + 3)[:k]      # some past the row, some past the request
            row = np.full(k, -1)
            row[r.permutation(k)[:len(cols)]] = cols           # -1 anywhere between
            row[r.random(k) < 0.2] = -1
            rows.append(row)
    rows[0][:] = -1                                            # lists nothing at all
    if k > 1:
        rows[-1][0] = 2**31 - 1
    selected = _cu(np.array(rows))
    out, lse = pr.run(selected=selected, ratio=ratio, local_tokens=local)
    pr.check(out, lse, selected, ratio, local)
    if local == 0:
        assert (lse[0] == -math.inf).all() and (out[0] == 0).all()
    again = pr.run(selected=selected, ratio=ratio, local_tokens=local)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@gpu
def test_selecting_every_column_is_full_attention(cuda):
    pr = Problem([(1000, 2), (77, 1)], 2, 4, 128, 64, "bf16", seed=12)
    selected = torch.arange(250, dtype=torch.int32, device="cuda").repeat(3, 1)
    out, lse = pr.run(selected=selected, ratio=4, local_tokens=0)
    pr.check(out, lse)


# ---------------------------------------------------------------------------
# a step of all of them
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_serving_step(cuda, fp8):
    """Two steps (a prompt, then a decode) from lengths alone: maps, stores,
    scoring, top-k, attention to the selection."""
    from sparse_attention_indexer_02_gb300 import serving

    dev, D, hkv, H, ratio, pt, k = "cuda", 128, 2, 8, 4, 64, 32
    g = torch.Generator(device=dev).manual_seed(1)
    pool = serving.PagedPool(num_pages=40, page_tokens=pt, num_kv_heads=hkv, head_dim=D, ratio=ratio,
                             index_fp8=fp8, device=dev)
    table = torch.full((2, 16), -1, dtype=torch.int32, device=dev)
    ctx = torch.zeros(2, dtype=torch.int32, device=dev)
    perm = torch.randperm(40, generator=g, device=dev).to(torch.int32)
    kept, taken = [[], []], 0
    for B, n in ((1, 203), (2, 130), (2, 1), (2, 4)):   # a prompt, two chunks, a decode, a verification
        T = B * n
        rnd = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
        q, kk, vv, iq, ik = rnd(T, H, D), rnd(T, hkv, D), rnd(T, hkv, D), rnd(T, 4, 128), rnd(T, 128)
        iw = torch.rand((T, 4), generator=g, device=dev)
        new = torch.full((B,), n, dtype=torch.int32, device=dev)
        res = serving.step(pool, table[:B], ctx[:B], new, perm[taken:], q=q, k=kk, v=vv, index_q=iq, index_keys=ik,
                           index_weights=iw, top_k=k, local_tokens=8, max_context=512)
        taken += int(res.maps.pages_used)
        pr = Problem.__new__(Problem)
        pr.lens = [(int(ctx[b]) + n, n) for b in range(B)]
        pr.pt, pr.group, pr.scale = pt, H // hkv, D ** -0.5
        pr.q, pr.kc, pr.vc, pr.table, pr.seq = q, pool.k_cache, pool.v_cache, table, res.maps.seq_lens
        for b in range(B):   # the cache holds what was stored, where the table says
            kept[b].append((kk[b * n:(b + 1) * n], vv[b * n:(b + 1) * n]))
            tok = torch.arange(pr.lens[b][0], device=dev)
            at = table[b].long()[tok // pt] * pt + tok % pt
            assert torch.equal(pool.k_cache.flatten(0, 1)[at], torch.cat([x for x, _ in kept[b]]))
            assert torch.equal(pool.v_cache.flatten(0, 1)[at], torch.cat([x for _, x in kept[b]]))
        assert ((res.selected >= 0).sum(1) == res.maps.visible_cols.clamp(max=k)).all()
        pr.check(res.out, res.lse, res.selected, ratio, 8)
        ctx[:B] += new
