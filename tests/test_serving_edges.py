"""Edges of the serving operators: calls in other orders, on other streams, and
with other layouts and lengths than a plain step's (the operators themselves:
test_serving_ops.py)."""
import os
import subprocess
import sys
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_02_gb300 as qsa  # noqa: E402
from sparse_attention_indexer_02_gb300 import build as qbuild  # noqa: E402
from sparse_attention_indexer_02_gb300 import _abi, serving, torch_api  # noqa: E402
from test_serving_ops import Problem, _cu, cuda, gpu, lib  # noqa: E402,F401


# ---------------------------------------------------------------------------
# page maps directly before a call that reads them early
# ---------------------------------------------------------------------------

def test_page_maps_release_no_kernel_early():
    """The scorers load visible_cols and block_table before they wait for the
    kernel ahead of them, so the kernel that writes both must not release them."""
    with open(os.path.join(qbuild.CSRC, "page_maps.cu")) as f:
        code = [line.split("//")[0] for line in f]
    assert not any("grid_dep_launch" in line or "launch_dependents" in line for line in code)


@gpu
@pytest.mark.parametrize("captured", [False, True])
def test_scoring_directly_after_page_maps(cuda, captured):
    """The maps' table and counts, not what the buffers held before."""
    B, pt, ratio, cols = 64, 64, 4, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    r = np.random.default_rng(1)
    pool = torch.randn((B * 33, pt // ratio, 128), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((B, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand((B, 8), generator=g, device="cuda")
    ctx, new, free, table = _cu([0] * B), _cu([1] * B), _cu([0] * B), _cu(np.zeros((B, 33)))
    out = torch_api.PageMaps(_cu([0] * (B + 1)), _cu([0] * B), _cu([0] * B, torch.int64), _cu([0] * B), _cu([0] * B),
                             _cu([0] * B), _cu([0] * B, torch.int64), _cu([0]))

    def score():
        return torch_api.paged_mqa_logits(q, w, pool, table, out.visible_cols, page_cols=pt // ratio, out_cols=cols)

    def both():
        torch_api.build_page_maps(ctx, new, free, table, page_tokens=pt, max_tokens=B, ratio=ratio, out=out)
        return score()

    both()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = both()
    for _ in range(10):
        c = r.integers(0, 32 * pt, B)
        c[::3] = c[::3] // pt * pt    # these begin a page
        pages = r.permutation(B * 33)
        t = np.zeros((B, 33), np.int64)
        have = -(-c // pt)
        for b in range(B):
            t[b, :have[b]] = pages[b * 32:b * 32 + have[b]]
        ctx.copy_(_cu(c)), free.copy_(_cu(pages[-B:])), table.copy_(_cu(t)), out.visible_cols.zero_()
        if captured:
            graph.replay()
            got = kept
        else:
            got = both()
        torch.cuda.synchronize()
        assert out.visible_cols.tolist() == ((c + 1) // ratio).tolist()
        assert torch.equal(got, score())


# ---------------------------------------------------------------------------
# stream handles
# ---------------------------------------------------------------------------

def test_stream_handle_zero_is_the_default_stream(monkeypatch):
    """ExternalStream(0) is some stream of torch's pool: never made for handle 0."""
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert torch_api._on(0) == "default"
    assert torch_api._on(1234) == ("external", 1234)
    assert torch_api._on("a stream") == "a stream"


@gpu
def test_calls_given_the_default_streams_handle(cuda):
    """The handle of the default stream, from another stream's context: the call is
    ordered with the default stream's work."""
    handle = torch.cuda.default_stream().cuda_stream
    with torch_api._on(handle):
        assert torch.cuda.current_stream().cuda_stream == handle
    with torch.cuda.stream(torch.cuda.Stream()):
        with torch_api._on(handle):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
    k = torch.ones((64, 1, 64), dtype=torch.bfloat16, device="cuda")
    slots, cache = torch.arange(64, device="cuda"), torch.zeros((2, 1, 64, 1, 64), dtype=torch.bfloat16, device="cuda")
    big = torch.ones(1 << 28, device="cuda")
    for i in range(1, 4):
        for _ in range(4):
            big.mul_(1.0)          # the default stream is busy when the call is made
        k.fill_(float(i))
        torch_api.store_paged_kv(k, k, slots, cache[0], cache[1], stream=handle)
        assert (cache == i).all()


# ---------------------------------------------------------------------------
# pages the free list had no more of
# ---------------------------------------------------------------------------

def _short_of_pages(lens, hkv, group, D, pt, dt, lost, seed):
    """A problem some of whose table entries are -1 (lost: of request b, pages
    lost[b]), and the columns of one token, -1 past them, that its rows still
    see.  Page 0, what a clamped -1 would read, holds NaN."""
    pr = Problem(lens, hkv, group, D, pt, dt, seed=seed)
    last = pr.kc.shape[0] - 1
    pr.kc, pr.vc = pr.kc.flip(0), pr.vc.flip(0)     # the page of NaNs first
    pr.table = last - pr.table
    there, held = pr.table.clone(), []
    for b, (s, n) in enumerate(lens):
        gone = [j for j in lost[b] if j * pt < s]
        pr.table[b, gone] = -1
        mine = np.array([t for t in range(max(s, 0)) if t // pt not in gone] or [-1])
        held += [mine] * n
    wide = max(len(m) for m in held)
    cols = np.full((len(held), wide), -1)
    for i, m in enumerate(held):
        cols[i, :len(m)] = m
    return pr, there, _cu(cols)


LOST = {
    "last": ([(700, 1), (70, 3), (5, 2)], [[10], [1], []]),
    "some": ([(700, 4), (300, 1), (64, 64)], [[0, 3, 4, 9], [2], []]),
    "all": ([(130, 2), (64, 1)], [list(range(99)), []]),
    "chunk": ([(900, 300), (513, 130)], [[1, 2, 7, 14], [0, 8]]),
    "long": ([(20000, 3), (9000, 1)], [list(range(0, 400, 3)), list(range(5, 120))]),
}


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
@pytest.mark.parametrize("hkv,group,D,pt,dt", [(2, 4, 128, 64, "bf16"), (1, 7, 64, 8, "fp16"), (1, 2, 128, 32, "fp16"),
                                               (1, 16, 64, 128, "bf16"), (1, 20, 128, 256, "bf16")])
@pytest.mark.parametrize("lost", list(LOST))
def test_attention_does_not_see_missing_pages(cuda, form, lost, hkv, group, D, pt, dt):
    lens, gone = LOST[lost]
    pr, there, cols = _short_of_pages(lens, hkv, group, D, pt, dt, gone, seed=pt)
    out, lse = pr.run(form=form)
    pr.table = there
    pr.check(out, lse, cols, 1, 0)


@gpu
@pytest.mark.parametrize("local", [0, 70])
def test_selected_attention_does_not_see_missing_pages(cuda, local):
    pr, there, cols = _short_of_pages([(700, 4), (300, 1)], 2, 4, 128, 64, "bf16", [[0, 3, 10], [4]], seed=2)
    every = torch.arange(175, dtype=torch.int32, device="cuda").repeat(5, 1)
    out, lse = pr.run(selected=every, ratio=4, local_tokens=local)
    pr.table = there
    pr.check(out, lse, cols, 1, 0)


# ---------------------------------------------------------------------------
# some requests of a larger batch
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("max_new", [1, 64])
def test_attention_of_the_later_requests_of_a_batch(cuda, selected, max_new):
    """Metadata of requests 2 and 3 beside all rows of q: the rows before theirs,
    and past them, are left alone."""
    pr = Problem([(300, 5), (64, 9), (200, 3), (131, 4), (90, 2)], 2, 4, 128, 32, "bf16", seed=31)
    T, H, D = pr.q.shape
    kw = {}
    if selected:
        cols = torch.arange(75, dtype=torch.int32, device="cuda").repeat(T, 1)
        kw = dict(selected=cols, ratio=4, local_tokens=7)
    want = pr.run(max_new=max_new, **kw)
    out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
    torch_api.paged_attention(pr.q, pr.kc, pr.vc, pr.table[2:4], pr.start[2:5], pr.seq[2:4], scale=pr.scale,
                              max_new=max_new, out=out, lse=lse, **kw)
    first, end = int(pr.start[2]), int(pr.start[4])
    u = torch.finfo(torch.bfloat16).eps
    mine = out[first:end].float(), want[0][first:end].float()
    # the same sums split over the CTAs in other places: two roundings of the output apart, and of the terms
    assert ((mine[0] - mine[1]).abs() <= 2 * u * pr.vc.nan_to_num().abs().max().float()).all()
    assert ((lse[first:end] - want[1][first:end]).abs() <= 1e-4).all()
    for x in (out, lse):
        assert (x[:first] == 7).all() and (x[end:] == 7).all()


@gpu
def test_selected_rows_of_no_request(cuda):
    """Decreasing row starts: the rows of the second request are nobody's."""
    pr = Problem([(300, 40), (64, 3)], 2, 4, 128, 32, "bf16", seed=32)
    cols = torch.arange(75, dtype=torch.int32, device="cuda").repeat(43, 1)
    want = pr.run(selected=cols, ratio=4)
    pr.start = _cu([0, 40, 20])
    out = torch.full_like(want[0], 7.0)
    pr.run(selected=cols, ratio=4, out=out)
    assert torch.equal(out[40:], torch.full_like(out[40:], 7.0))
    pr.start = _cu([3, 10, 43])       # rows 0-2 are nobody's
    out = torch.full_like(want[0], 7.0)
    pr.run(selected=cols, ratio=4, out=out)
    assert (out[:3] == 7).all() and not (out[3:] == 7).all(2).any()


# ---------------------------------------------------------------------------
# layouts of what the scoring takes
# ---------------------------------------------------------------------------

def test_scoring_refuses_layouts_it_would_misread(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    ok = dict(q=b16(4, 8, 128), weights=torch.zeros(4, 8), kv_cache=b16(6, 16, 128), block_table=i32(2, 3),
              visible_cols=i32(4))
    bad = [("block_table", i32(2, 5)[:, :3]), ("block_table", i32(2, 3).long()), ("q", b16(4, 16, 128)[:, :8]),
           ("q", b16(4, 8, 128).half()), ("q", torch.zeros(4, 8, 128)), ("weights", b16(4, 8)),
           ("weights", torch.zeros(4, 16)[:, :8]), ("weights", torch.zeros(4, 4)), ("visible_cols", i32(4).long()),
           ("visible_cols", i32(8)[::2]), ("visible_cols", i32(2)), ("next_n_lens", i32(1)),
           ("next_n_lens", i32(2).long()), ("kv_cache", b16(6, 128, 16).transpose(1, 2))]
    for name, t in bad:
        with pytest.raises(ValueError, match="must be"):
            torch_api.paged_mqa_logits(**{**ok, name: t}, page_cols=16, out_cols=32, stream=0)
        with pytest.raises(ValueError, match="must be"):
            torch_api.paged_mqa_topk(**{**ok, name: t}, k=4, page_cols=16, out_cols=32, stream=0)
    for out in (torch.zeros(4, 64)[:, :32], b16(4, 32), torch.zeros(4, 31)):
        with pytest.raises(ValueError, match="out must be"):
            torch_api.paged_mqa_logits(**ok, page_cols=16, out_cols=32, out=out, stream=0)


def test_step_refuses_before_anything_is_launched(lib, monkeypatch):
    def launched(*a, **k):
        raise AssertionError("launched")

    monkeypatch.setattr(torch_api, "build_page_maps", launched)
    pool = serving.PagedPool(num_pages=4, page_tokens=64, num_kv_heads=1, head_dim=64, device="cpu")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    ok = dict(block_table=i32(2, 3), context_lens=i32(2), new_lens=i32(2), free_pages=i32(2), q=b16(4, 2, 64),
              k=b16(4, 1, 64), v=b16(4, 1, 64), index_q=b16(4, 8, 128), index_keys=b16(4, 128),
              index_weights=torch.zeros(4, 8), top_k=4, max_context=64)
    with pytest.raises(AssertionError, match="launched"):
        serving.step(pool, **ok)
    for name, t in (("q", b16(3, 2, 64)), ("q", b16(0, 2, 64)), ("block_table", i32(2, 3).long()),
                    ("index_q", b16(4, 8, 128).half()), ("index_q", b16(2, 8, 128)), ("index_weights", b16(4, 8)),
                    ("index_weights", torch.zeros(4, 4))):
        with pytest.raises(ValueError):
            serving.step(pool, **{**ok, name: t})


def _step_inputs(B, n, hkv, H, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    T = B * n
    return dict(q=rnd(T, H, D), k=rnd(T, hkv, D), v=rnd(T, hkv, D), index_q=rnd(T, 4, 128), index_keys=rnd(T, 128),
                index_weights=torch.rand((T, 4), generator=g, device="cuda"))


def _two_steps(pool, table, B, make, top_k=16):
    """A prompt of 200 tokens a request and two decode steps; the results of each."""
    perm = torch.randperm(pool.k_cache.shape[0], generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    res, ctx, taken = [], 0, 0
    for i, n in enumerate((200, 1, 2)):
        r = serving.step(pool, table, _cu([ctx] * B), _cu([n] * B), perm[taken:], top_k=top_k, local_tokens=4,
                         max_context=256, **make(i, n))
        res.append((r.out, r.lse, r.selected))
        taken += int(r.maps.pages_used)
        ctx += n
    return res


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_step_takes_views(cuda, fp8):
    """Columns of a wider table, index queries and weights out of a fused
    projection: the results of contiguous ones."""
    B, hkv, H, D = 3, 2, 8, 64

    def plain(i, n):
        return _step_inputs(B, n, hkv, H, D, i)

    def views(i, n):
        d = plain(i, n)
        wide = torch.full((B * n, 9, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        wide[:, 2:6] = d["index_q"]
        w = torch.full((B * n, 7), 5.0, device="cuda")
        w[:, 1:5] = d["index_weights"]
        return {**d, "index_q": wide[:, 2:6], "index_weights": w[:, 1:5]}

    new_pool = lambda: serving.PagedPool(num_pages=30, page_tokens=64, num_kv_heads=hkv, head_dim=D, index_fp8=fp8)  # noqa: E731
    want = _two_steps(new_pool(), torch.full((B, 5), -1, dtype=torch.int32, device="cuda"), B, plain)
    wide = torch.full((B, 11), -1, dtype=torch.int32, device="cuda")
    got = _two_steps(new_pool(), wide[:, 3:8], B, views)
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert (wide[:, :3] == -1).all() and (wide[:, 8:] == -1).all()


@pytest.mark.parametrize("pt,ratio", [(4, 4), (8, 4), (12, 4), (20, 4), (64, 4), (6, 2), (7, 1)])
def test_pool_of_any_page_size_suits_the_scoring(lib, pt, ratio):
    pool = serving.PagedPool(num_pages=3, page_tokens=pt, num_kv_heads=1, head_dim=64, ratio=ratio, index_fp8=True,
                             device="cpu")
    assert pool.index.stride(0) % 16 == 0 and pool.index.shape[1] >= 132 * pt // ratio
    desc = _abi.make_desc(1, 1, 4, pool.page_cols, 2, 3, 8, pool.index.stride(0), kv_dtype=qsa.KV_FP8_E4M3,
                          scale_page_stride=pool.index.stride(0))
    qsa.plan_variant(desc)      # raises for a page stride the scorers refuse


@gpu
@pytest.mark.parametrize("pt", [8, 20])
def test_step_over_odd_fp8_pages(cuda, pt):
    """Every complete column selected: the results of 64-token pages, to the roundings
    of sums in another order."""
    B, hkv, H, D = 2, 2, 8, 64
    make = lambda i, n: _step_inputs(B, n, hkv, H, D, i)  # noqa: E731
    got, want = (_two_steps(serving.PagedPool(num_pages=60, page_tokens=p, num_kv_heads=hkv, head_dim=D, index_fp8=True),
                            torch.full((B, 30), -1, dtype=torch.int32, device="cuda"), B, make, top_k=64)
                 for p in (pt, 64))
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a[2], b[2])
        # the output's rounding on both sides and the terms' (values up to 5), bf16
        assert ((a[0].float() - b[0].float()).abs() <= 4 * 2.0 ** -8 * 5).all(), i
        assert ((a[1] - b[1]).abs() <= 1e-4).all(), i


# ---------------------------------------------------------------------------
# kept workspaces
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("flags,clear,dropped", [(8, True, 1), (9, True, 1), (8, False, 0), (0, True, 0), (7, True, 0)])
def test_a_cleared_attention_fault_drops_the_kept_workspaces(monkeypatch, flags, clear, dropped):
    """The fault is the fake's: no kernel has to give up for it."""
    calls = []

    class Library:
        @staticmethod
        def qsa_device_status(word, clear_it):
            word._obj.value = flags
            return 0

    monkeypatch.setattr(_abi, "load_library", Library)
    monkeypatch.setitem(sys.modules, qsa.__name__ + "._qsa_torch",
                        types.SimpleNamespace(drop_workspaces=lambda: calls.append(1)))
    assert qsa.device_status(clear=clear) == flags
    assert len(calls) == dropped
    monkeypatch.delitem(sys.modules, qsa.__name__ + "._qsa_torch")
    assert qsa.device_status(clear=clear) == flags


@gpu
def test_the_kept_workspace_goes_with_a_reported_fault(cuda, monkeypatch):
    """The status word as an attention launch that gave up would set it (by a fake of
    the status call): the workspace kept for the stream is given up, the next call
    makes a new one."""
    pr = Problem([(9000, 1)], 2, 4, 128, 64, "bf16", seed=6)
    want = pr.run()
    real = _abi.load_library().qsa_device_status

    def status(word, clear_it):
        st = real(word, clear_it)
        word._obj.value |= 8
        return st

    before = torch.cuda.memory_allocated()
    monkeypatch.setattr(_abi, "load_library", lambda: types.SimpleNamespace(qsa_device_status=status))
    assert qsa.device_status() & 8
    monkeypatch.undo()
    assert torch.cuda.memory_allocated() < before       # forgotten
    got = pr.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_kept_workspaces_are_bounded(cuda):
    """Calls on 64 streams (torch's pools of both priorities): at most 32 workspaces
    stay, and a stream whose own went still gets right results."""
    pr = Problem([(3000, 1)], 2, 4, 128, 64, "bf16", seed=14)
    out, lse = pr.run()
    torch.cuda.synchronize()
    torch_api.drop_attention_workspaces()
    streams = [torch.cuda.Stream(priority=p) for _ in range(32) for p in (0, -1)]
    assert len({s.cuda_stream for s in streams}) > 40
    o, z = torch.empty_like(out), torch.empty_like(lse)
    before = torch.cuda.memory_allocated()
    for turn in range(2):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            pr.run(stream=s, out=o, lse=z)
            torch.cuda.current_stream().wait_stream(s)
            assert torch.equal(o, out) and torch.equal(z, lse)
    desc = _abi.AttnDesc(_abi.KvDesc(_abi.HALF_BF16, 4, 64, 2, 128, 0, 32768, 512, 256, 32768, 512, 256), 1, 8, 4, 1, 0,
                         1, 0, _abi.ATTN_GATHER, 1, 4, 2048, 256, 2048, 256, 0.1, 0)
    assert torch.cuda.memory_allocated() - before <= 32 * (qsa.paged_attention_workspace_bytes(desc) + 512)
    torch_api.drop_attention_workspaces()
    assert torch.cuda.memory_allocated() <= before


# ---------------------------------------------------------------------------
# tensors of another device
# ---------------------------------------------------------------------------

def test_tensors_of_another_device_are_refused(lib):
    """Tensors that say they are on device 1 (fake ones, without memory) while
    another device, or none, is the current one."""
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    with fake.FakeTensorMode():
        z = lambda dtype, *s: torch.empty(s, dtype=dtype, device="cuda:1")  # noqa: E731
        b16, i32, i64 = torch.bfloat16, torch.int32, torch.int64
        kv, kc, slots, q = z(b16, 3, 2, 128), z(b16, 4, 16, 2, 128), z(i64, 3), z(b16, 3, 8, 128)
        keys, index = z(b16, 3, 128), z(b16, 4, 16, 128)
        two, three, four, table = z(i32, 2), z(i32, 3), z(i32, 4), z(i32, 2, 4)
    if torch.cuda.is_available():
        assert torch.cuda.current_device() != 1
    for call in (lambda: torch_api.store_paged_kv(kv, kv, slots, kc, kc),
                 lambda: torch_api.store_index_keys(keys, slots, index, page_cols=16),
                 lambda: torch_api.build_page_maps(two, two, four, table, page_tokens=16, max_tokens=4),
                 lambda: torch_api.paged_attention(q, kc, kc, table, three, two)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


# ---------------------------------------------------------------------------
# page maps at the end of the range
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("partial", [False, True])
@pytest.mark.parametrize("ratio", [1, 2])
def test_visible_counts_saturate(cuda, ratio, partial):
    """Positions next to and past 2^31 - 1: a count of columns never turns negative."""
    big = 2**31 - 1
    got = torch_api.build_page_maps(_cu([big - 1]), _cu([4]), _cu([0]), _cu([[0]]), page_tokens=2, max_tokens=5,
                                    ratio=ratio, partial_cols=partial)
    pos = [big - 1 + i for i in range(4)]
    vis = [min(big, -(-(p + 1) // ratio) if partial else (p + 1) // ratio) for p in pos]
    assert got.visible_cols.tolist() == vis + [0]
    assert got.positions.tolist() == [min(big, p) for p in pos] + [-1]
    assert got.slots.tolist() == [-1] * 5 and got.column_slots.tolist() == [-1] * 5


# ---------------------------------------------------------------------------
# arguments without a truth value
# ---------------------------------------------------------------------------

def test_flags_without_a_truth_value_are_refused(lib):
    """An error Python raises while a flag is read is the call's own refusal, not a
    result returned with an error pending."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="partial_cols"):
        torch_api.build_page_maps(i32(2), i32(2), i32(4), i32(2, 4), page_tokens=16, max_tokens=4,
                                  partial_cols=np.zeros(2))


@gpu
def test_return_lse_without_a_truth_value_is_refused(cuda):
    pr = Problem([(30, 1)], 1, 2, 64, 16, "bf16", seed=1)
    with pytest.raises(ValueError, match="return_lse"):
        torch_api.paged_attention(pr.q, pr.kc, pr.vc, pr.table, pr.start, pr.seq, return_lse=np.zeros(2))


# ---------------------------------------------------------------------------
# steps whose lengths or pages do not suffice
# ---------------------------------------------------------------------------

def _one_step(new, pages, **kw):
    """A step of 2 requests with 70 tokens each of context and 60 rows in all, over
    64-token pages; page 0 is another request's and holds NaN."""
    pool = serving.PagedPool(num_pages=8, page_tokens=64, num_kv_heads=1, head_dim=64)
    pool.k_cache[0], pool.v_cache[0] = float("nan"), float("nan")
    table = _cu([[1, 2, -1, -1], [3, 4, -1, -1]])
    return serving.step(pool, table, _cu([70, 70]), _cu(new), _cu(pages), top_k=16, local_tokens=8, max_context=256,
                        **_step_inputs(2, 30, 1, 4, 64, 5), **kw), table


@gpu
def test_step_says_whether_lengths_and_pages_sufficed(cuda):
    good, table = _one_step([30, 30], [])
    assert good.valid().item() is True and table.tolist() == [[1, 2, -1, -1], [3, 4, -1, -1]]
    assert not _one_step([20, 40], [5, 6])[0].valid()          # as many rows, shared out otherwise
    assert not _one_step([30, 29], [])[0].valid()
    fine, _ = _one_step([30, 30], [7])
    assert fine.valid() and torch.equal(fine.out, good.out)


@gpu
def test_step_without_enough_pages_reads_no_other_requests(cuda):
    """Requests at a page's end, no page free: their new tokens are nowhere, and the
    rows see the tokens there are, not page 0's."""
    pool = serving.PagedPool(num_pages=8, page_tokens=64, num_kv_heads=1, head_dim=64)
    pool.k_cache.normal_(), pool.v_cache.normal_()
    pool.k_cache[0], pool.v_cache[0] = float("nan"), float("nan")
    pool.index.normal_()
    table = _cu([[1, 2, -1], [3, 4, -1]])
    res = serving.step(pool, table, _cu([128, 128]), _cu([30, 30]), _cu([5]), top_k=16, local_tokens=8, max_context=192,
                       **_step_inputs(2, 30, 1, 4, 64, 5))
    assert not res.valid() and int(res.maps.pages_used) == 2
    assert table.tolist() == [[1, 2, 5], [3, 4, -1]]
    assert not res.out.isnan().any() and not res.lse.isnan().any()
    assert (res.maps.slots[30:] == -1).all() and (res.maps.slots[:30] >= 0).all()


# ---------------------------------------------------------------------------
# the library without torch
# ---------------------------------------------------------------------------

def test_the_library_builds_and_loads_without_torch(lib):
    """As before there was a binding for torch tensors: the C ABI through ctypes needs
    none of it."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "from sparse_attention_indexer_02_gb300 import build\n"
            "build.build()\n"
            "import sparse_attention_indexer_02_gb300 as qsa\n"
            "assert qsa.abi_version() == 1 and qsa.status_string(1)\n")
    root = os.path.dirname(qbuild.PKG)
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
