"""Head norms with rotary positions, windowed attention and draft verification
(include/qsa.h) against plain implementations in 64 bits.

Rotation tolerances, from the arithmetic.  An angle below half a turn is rounded
to fp32 (2^-25 half turns), its frequency to 2^-65 turns and 53 bits (pos * 2^-53
radians): at most 2^-23 + pos 2^-52 together; sine and cosine are off by an ulp of
1 (2^-23) more, times the magnitude m (2^-24).  With e = 2^-21 + pos 2^-52 and
two rounded products and a sum, y = x c + x_p s is off by m (|x| + |x_p|)
(e + 3 * 2^-24).  A norm multiplies by a factor whose square is a sum of D terms
(D * 2^-24 relative, half of it on the root), two roundings of it and of the
weights: (D / 2 + 10) 2^-24 of |n| and |n_p|; the layer norm's mean is off by
D 2^-24 mean|x| and enters every n with the factor.  The output is rounded once,
half a step u of |y| (fp16: 2^-25 at least)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_02_gb300 as qsa  # noqa: E402
from sparse_attention_indexer_02_gb300 import _abi, rotary, torch_api  # noqa: E402
from sparse_attention_indexer_02_gb300 import build as qbuild  # noqa: E402
from test_serving_ops import DT, Problem, _attn_desc, _cu, _kv_desc, _refused  # noqa: E402

gpu = pytest.mark.gpu


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

INVALID, UNSUPPORTED = qsa.QSA_ERR_INVALID_ARG, qsa.QSA_ERR_UNSUPPORTED


def _rotary_desc(**kw):
    base = dict(dtype=_abi.HALF_BF16, head_dim=128, rot_dim=128, rot_offset=0, layout=_abi.ROTARY_HALF,
                norm=_abi.NORM_NONE, weight_f32=0, reserved=0, eps=1e-6, magnitude=1.0, num_tokens=4)
    base.update(kw)
    return _abi.RotaryDesc(*(base[n] for n, _ in _abi.RotaryDesc._fields_))


def _head_rows(**kw):
    base = dict(x=16, out=32, weight=None, bias=None, x_row_stride=512, x_head_stride=256, out_row_stride=512,
                out_head_stride=256, num_heads=2, reserved=0)
    base.update(kw)
    return _abi.HeadRows(*(base[n] for n, _ in _abi.HeadRows._fields_))


def _rotate(desc=None, q=None, k=None, positions=16, freqs=16):
    _abi.rotate_heads(desc or _rotary_desc(), q or _head_rows(), k, positions, freqs, stream=0)


def _rotate_store(desc=None, q=None, k=None, kv=None, v=16, vr=512, vh=256, slots=16, kc=16, vc=16, positions=16):
    _abi.rotate_store_kv(desc or _rotary_desc(), q or _head_rows(), k or _head_rows(out=None), positions, 16,
                         kv or _kv_desc(), v, vr, vh, slots, kc, vc, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=12), INVALID),
    (dict(head_dim=264), UNSUPPORTED), (dict(rot_dim=0), INVALID), (dict(rot_dim=3), INVALID),
    (dict(rot_dim=130), INVALID), (dict(rot_offset=-1), INVALID), (dict(rot_offset=2), INVALID),
    (dict(rot_dim=64, rot_offset=65), INVALID), (dict(rot_dim=64, rot_offset=1, layout=1), INVALID),
    (dict(layout=2), INVALID), (dict(norm=3), INVALID), (dict(weight_f32=2), INVALID), (dict(reserved=1), INVALID),
    (dict(norm=1, eps=-1.0), INVALID), (dict(norm=1, eps=math.nan), INVALID), (dict(norm=2, eps=math.inf), INVALID),
    (dict(magnitude=math.nan), INVALID), (dict(magnitude=math.inf), INVALID), (dict(num_tokens=-1), INVALID)])
def test_rotary_descriptor_refusals(lib, kw, status):
    _refused(status, _rotate, desc=_rotary_desc(**kw))
    _refused(status, _rotate_store, desc=_rotary_desc(**kw))


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(out=None), dict(x=24), dict(out=40), dict(x_row_stride=8), dict(x_head_stride=0),
    dict(out_row_stride=-512), dict(out_head_stride=24), dict(num_heads=0), dict(num_heads=65537), dict(reserved=1),
    dict(weight=16), dict(bias=16)])
def test_rotate_rows_refusals(lib, kw):
    _refused(INVALID, _rotate, q=_head_rows(**kw))
    _refused(INVALID, _rotate, k=_head_rows(**kw))


def test_rotate_other_refusals(lib):
    for kw in (dict(positions=None), dict(freqs=None), dict(positions=18), dict(freqs=20)):
        _refused(INVALID, _rotate, **kw)
    _refused(INVALID, _rotate, desc=_rotary_desc(norm=1), q=_head_rows(bias=16))
    _refused(INVALID, _rotate, desc=_rotary_desc(norm=2, weight_f32=1), q=_head_rows(weight=18))
    for kw in (dict(v=None), dict(v=24), dict(vr=0), dict(vh=24), dict(slots=None), dict(slots=20), dict(kc=None),
               dict(vc=24), dict(k=_head_rows()), dict(kv=_kv_desc(dtype=1)), dict(kv=_kv_desc(head_dim=64)),
               dict(kv=_kv_desc(num_kv_heads=3)), dict(kv=_kv_desc(page_tokens=0)), dict(positions=None)):
        _refused(INVALID, _rotate_store, **kw)


def _verify(positional=None, **kw):
    base = dict(num_requests=2, max_drafts=3, vocab=100, dtype=0, target_request_stride=400, target_row_stride=100,
                draft_request_stride=300, draft_row_stride=100)
    base.update(kw)
    d = _abi.VerifyDesc(*(base[n] for n, _ in _abi.VerifyDesc._fields_))
    _abi.verify_drafts(d, *(positional or [16] * 9), stream=0)


@pytest.mark.parametrize("kw", [
    dict(num_requests=-1), dict(num_requests=65537), dict(max_drafts=-1), dict(max_drafts=1025), dict(vocab=0),
    dict(vocab=(1 << 30) + 1), dict(dtype=3), dict(target_request_stride=-1), dict(target_row_stride=-1),
    dict(draft_request_stride=-1), dict(draft_row_stride=-1)])
def test_verify_descriptor_refusals(lib, kw):
    _refused(INVALID, _verify, **kw)


def test_verify_pointer_refusals(lib):
    for at in (0, 2, 4, 5, 6, 7, 8):  # (5 alone, or 8 alone: context_lens and next_lens go together)
        args = [16] * 9
        args[at] = None
        _refused(INVALID, _verify, args)
    for at in range(9):
        args = [16] * 9
        args[at] = 18
        _refused(INVALID, _verify, args)


@pytest.mark.parametrize("window,sinks,kw", [
    (0, 0, {}), (-1, 0, {}), (4, -1, {}), (4, 0, dict(num_selected=4)), (4, 0, dict(local_tokens=4)),
    (4, 0, dict(num_requests=-1)), (4, 0, dict(scale=0.0))])
def test_window_refusals(lib, window, sinks, kw):
    _refused(INVALID, _abi.paged_attention_window, _attn_desc(**kw), window, sinks, *[16] * 9, 1 << 30, stream=0)


def test_step_calls_of_nothing_launch_nothing(lib):
    _rotate(desc=_rotary_desc(num_tokens=0), q=_head_rows(x=None, out=None), positions=None, freqs=None)
    _rotate_store(desc=_rotary_desc(num_tokens=0), q=_head_rows(x=None, out=None), k=_head_rows(x=None, out=None),
                  v=None, slots=None, kc=None, vc=None, positions=None)
    _verify([None] * 9, num_requests=0)
    _abi.paged_attention_window(_attn_desc(num_requests=0), 4, 1, *[None] * 9, 0, stream=0)


def test_step_tensors_refused(lib):
    z = lambda dt, *s: torch.zeros(s, dtype=dt)  # noqa: E731
    b16, f16, f32, i32, i64 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int64
    rot = rotary.Rotary(128, device="cpu")
    q, k, pos = z(b16, 3, 8, 128), z(b16, 3, 2, 128), z(i32, 3)
    ok = dict(q=q, k=k, positions=pos, rotary=rot)
    for kw in (dict(q=q.float()), dict(q=q[:, :, ::2]), dict(q=q[0]), dict(k=k.half()), dict(k=k[:2]),
               dict(k=k[:, :, :64]), dict(positions=pos.long()), dict(positions=pos[:2]), dict(norm="batch"),
               dict(q_weight=z(b16, 64), norm="rms"), dict(q_weight=z(f16, 128), norm="rms"),
               dict(q_weight=z(b16, 128), k_weight=z(f32, 128), norm="rms"), dict(q_out=z(b16, 3, 7, 128)),
               dict(k_out=z(f16, 3, 2, 128)), dict(k=None, k_out=k), dict(k=None, k_weight=z(b16, 128), norm="rms"),
               dict(eps="1"), dict(q=None)):
        with pytest.raises(ValueError):
            torch_api.rotate_heads(**{**ok, **kw})
    kc, slots = z(b16, 4, 16, 2, 128), z(i64, 3)
    good = dict(q=q, k=k, v=k, positions=pos, slots=slots, k_cache=kc, v_cache=kc, rotary=rot)
    for kw in (dict(k=None), dict(v=None), dict(v=q), dict(slots=pos), dict(slots=slots[:2]), dict(k_cache=kc.half()),
               dict(v_cache=kc[:, :8])):
        with pytest.raises(ValueError):
            torch_api.rotate_store_kv(**{**good, **kw})
    tok, p, u = z(i32, 2, 3), z(f32, 2, 4, 50), z(f32, 2, 4)
    for args, kw in (((tok.long(), p, u), {}), ((tok, p[:, :3], u), {}), ((tok, p.double(), u), {}),
                     ((tok, p.transpose(1, 2), u), {}), ((tok, p, u.double()), {}), ((tok, p, u[:, :3]), {}),
                     ((tok, p, u), dict(draft_probs=p)), ((tok, p, u), dict(draft_probs=p[:, :3].half())),
                     ((tok, p, u), dict(num_drafts=z(i32, 3))), ((tok, p, u), dict(context_lens=z(i64, 2))),
                     ((tok, p, u), dict(out=(None, None, z(i32, 2)))), ((tok, p, u), dict(out=(None, None)))):
        with pytest.raises(ValueError):
            torch_api.verify_drafts(*args, **kw)
    # these fit in every other way, but lie in host memory
    for call in (lambda: torch_api.rotate_heads(**ok), lambda: torch_api.rotate_store_kv(**good),
                 lambda: torch_api.verify_drafts(tok, p, u)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_rotary_refusals_and_frequencies():
    for args, kw in (((3,), {}), ((0,), {}), ((128,), dict(layout="other")), ((128,), dict(scaling=dict(kind="linear"))),
                     ((128,), dict(scaling=dict(kind="far", factor=2.0))), ((128,), dict(base=0.0)),
                     ((128,), dict(scaling=dict(kind="base", factor=-1.0))), ((2,), dict(scaling=dict(kind="base", factor=2.0))),
                     ((128,), dict(frequencies=[1.0])), ((4,), dict(frequencies=[1.0, math.inf])),
                     ((4,), dict(frequencies=[1.0, 0.5], scaling=dict(kind="linear", factor=2.0))),
                     ((128,), dict(magnitude=math.nan)),
                     ((128,), dict(scaling=dict(kind="parts", factor=2.0, original=10, low=4.0, high=4.0)))):
        with pytest.raises(ValueError):
            rotary.Rotary(*args, device="cpu", **kw)
    for kw in ({}, dict(scaling=dict(kind="linear", factor=4.0)), dict(scaling=dict(kind="base", factor=8.0)),
               dict(scaling=dict(kind="parts", factor=8.0, original=4096, low=1.0, high=32.0))):
        r = rotary.Rotary(64, base=500000.0, device="cpu", **kw)
        f = np.array(r.frequencies)
        turns = r.freqs.numpy().view(np.uint64).astype(np.longdouble) / np.longdouble(2) ** 64
        # the quotient's rounding, and that to a whole number of units: half of 2^-64
        assert (np.abs(turns - f / (2 * math.pi)) <= 2.0 ** -53 * f + 2.0 ** -65).all()
        plain = 500000.0 ** (-np.arange(0, 64, 2) / 64)
        if kw.get("scaling", {}).get("kind") == "base":    # the fastest pair as before, the slowest 8 times slower
            assert f[0] == 1.0 and abs(f[-1] / (plain[-1] / 8) - 1) < 1e-12
        elif kw.get("scaling", {}).get("kind") == "parts":
            turned = 4096 * plain / (2 * math.pi)
            assert np.allclose(f[turned > 32], plain[turned > 32], rtol=1e-14)
            assert np.allclose(f[turned < 1], plain[turned < 1] / 8, rtol=1e-14)
    # negative frequencies turn the other way, whole turns a position vanish
    r = rotary.Rotary(4, frequencies=[-math.pi, 2 * math.pi], device="cpu")
    assert r.freqs.tolist() == [-(1 << 63), 0]


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------

def rotated(x, positions, rot, norm=None, w=None, b=None, eps=1e-6):
    """float64 (result, bound on the kernel's error before the last rounding)."""
    D, R, off = x.shape[-1], rot.rot_dim, rot.offset
    y = x.double()
    slack = torch.zeros_like(y)
    if norm:
        mean_abs = y.abs().mean(-1, keepdim=True)
        if norm == "layer":
            y = y - y.mean(-1, keepdim=True)
        f = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        w = torch.ones(D, device=x.device) if w is None else w
        slack = (D / 2 + 10) * 2.0 ** -24 * (y * f * w.double()).abs()
        if norm == "layer":
            slack = slack + 2 * D * 2.0 ** -24 * mean_abs * f * w.double().abs()
        y = y * f * w.double()
        if b is not None:
            y = y + b.double()
            slack = slack + 2.0 ** -23 * b.double().abs()
    pos = positions.double()[:, None, None]
    angle = pos * torch.tensor(rot.frequencies, dtype=torch.float64, device=x.device)
    c, s = angle.cos() * rot.magnitude, angle.sin() * rot.magnitude
    i = torch.arange(R, device=x.device)
    if rot.layout == _abi.ROTARY_HALF:
        pair, partner, sign = i % (R // 2), (i + R // 2) % R, torch.where(i < R // 2, -1.0, 1.0)
    else:
        pair, partner, sign = i // 2, i ^ 1, torch.where(i % 2 == 0, -1.0, 1.0)
    z, zp = y[..., off:off + R], y[..., off:off + R][..., partner]
    out, tol = y.clone(), slack.clone()
    out[..., off:off + R] = z * c[..., pair] + zp * s[..., pair] * sign.double()
    e = 2.0 ** -21 + pos * 2.0 ** -52 + 3 * 2.0 ** -24
    m = abs(rot.magnitude)
    tol[..., off:off + R] = m * ((z.abs() + zp.abs()) * e + (slack[..., off:off + R] + slack[..., off:off + R][..., partner]))
    return out, tol


def near(got, want, tol):
    u = torch.finfo(got.dtype).eps / 2
    bound = tol + u * (want.abs() + tol)
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), float(off.max())


def _positions(T, g, reach=200000):
    pos = torch.randint(0, reach, (T,), generator=g, device="cuda", dtype=torch.int32)
    if T > 3:
        pos[0], pos[1], pos[2] = 0, 2**31 - 1, -1
    return pos


ROTATE = [  # T, q heads, k heads, D, R, offset, layout, dtype
    (1, 1, 1, 128, 128, 0, "half", "bf16"), (5, 32, 8, 128, 128, 0, "half", "bf16"),
    (37, 7, 1, 64, 64, 0, "pairs", "fp16"), (300, 5, 3, 128, 64, 64, "pairs", "bf16"),
    (1001, 9, 2, 96, 24, 0, "half", "bf16"), (64, 4, 4, 80, 40, 40, "half", "fp16"),
    (33, 3, 1, 256, 128, 128, "half", "bf16"), (70, 2, 1, 192, 64, 128, "pairs", "fp16"),
    (9, 6, 2, 8, 2, 6, "pairs", "bf16"), (9, 6, 2, 8, 8, 0, "half", "bf16"), (12, 1, 5, 256, 250, 3, "half", "fp16"),
    (4000, 16, 2, 128, 128, 0, "half", "fp16"), (20, 3, 3, 120, 30, 90, "pairs", "bf16"),
    (6, 65, 1, 16, 16, 0, "half", "bf16")]


@gpu
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("case", ROTATE, ids=range(len(ROTATE)))
def test_rotate_heads(cuda, case, norm):
    T, hq, hk, D, R, off, layout, dt = case
    g = torch.Generator(device="cuda").manual_seed(T + D)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rot = rotary.Rotary(R, base=10000.0, layout=layout, offset=off, magnitude=1.25 if T % 2 else 1.0)
    both = (rnd(T, hq + hk + 1, D) * 3 + (1.5 if norm == "layer" else 0)).to(DT[dt])
    q, k = both[:, :hq], both[:, hq:hq + hk]
    pos = _positions(T, g)
    kw = {}
    if norm:
        wt = torch.float32 if T % 3 == 0 else DT[dt]
        kw = dict(norm=norm, q_weight=(1 + 0.3 * rnd(D)).to(wt), k_weight=(1 + 0.3 * rnd(D)).to(wt), eps=1e-5)
        if norm == "layer":
            kw.update(q_bias=rnd(D).to(wt), k_bias=None if T % 2 else rnd(D).to(wt))
    big = torch.full((2, T + 2, max(hq, hk) + 2, D), 7.0, dtype=DT[dt], device="cuda")
    q_out, k_out = big[0, 1:1 + T, 1:1 + hq], big[1, 1:1 + T, 1:1 + hk]
    got = torch_api.rotate_heads(q, k, pos, rot, q_out=q_out, k_out=k_out, **kw)
    assert got[0].data_ptr() == q_out.data_ptr() and got[1].data_ptr() == k_out.data_ptr()
    live = pos >= 0
    for x, y, n in ((q, q_out, "q"), (k, k_out, "k")):
        want, tol = rotated(x, pos, rot, norm, kw.get(n + "_weight"), kw.get(n + "_bias"), kw.get("eps", 0))
        near(y[live], want[live], tol[live])
        if not norm:    # elements beside the rotated part keep their bits
            assert torch.equal(y[live][..., :off], x[live][..., :off])
            assert torch.equal(y[live][..., off + R:], x[live][..., off + R:])
        assert (y[~live] == 7).all()
    assert (big[:, 0] == 7).all() and (big[:, -1] == 7).all() and (big[:, :, 0] == 7).all()
    assert (big[0, :, 1 + hq:] == 7).all() and (big[1, :, 1 + hk:] == 7).all()
    # new outputs, and in place: the same bits
    a, b = torch_api.rotate_heads(q, k, pos, rot, **kw)
    assert torch.equal(a[live], q_out[live]) and torch.equal(b[live], k_out[live])
    alone, none = torch_api.rotate_heads(q, None, pos, rot, **{n: v for n, v in kw.items() if not n.startswith("k_")})
    assert none is None and torch.equal(alone[live], a[live])
    before = both.clone()
    torch_api.rotate_heads(q, k, pos, rot, q_out=q, k_out=k, **kw)
    assert torch.equal(q[live], a[live]) and torch.equal(k[live], b[live])
    assert torch.equal(both[~live], before[~live]) and torch.equal(both[:, hq + hk:], before[:, hq + hk:])


@gpu
def test_rotation_of_far_positions(cuda):
    """Frequencies whose angles are known exactly, at positions to 2^31 - 1; infinities
    and NaN stay in their pair, and beside the rotated part they keep their bits."""
    pos = _cu([0, 1, 2, 3, 4, 2**30, 2**31 - 1, 1234567891])
    rot = rotary.Rotary(4, frequencies=[math.pi / 2, math.pi], offset=2)
    x = torch.zeros((8, 1, 8), dtype=torch.float16, device="cuda")
    x[..., 2], x[..., 3], x[..., 4], x[..., 5] = 1.0, 2.0, 0.5, 0.25
    x[..., 0], x[..., 1], x[..., 7] = math.inf, math.nan, -math.inf
    y = torch_api.rotate_heads(x, None, pos, rot)[0][:, 0]
    for t, p in enumerate(pos.tolist()):
        c, s = [(1, 0), (0, 1), (-1, 0), (0, -1)][p % 4]
        half = -1.0 if p % 2 else 1.0
        assert y[t, 2:6].tolist() == [c * 1.0 - s * 0.5, 2.0 * half, c * 0.5 + s * 1.0, 0.25 * half]
    assert torch.equal(y.view(torch.int16)[:, [0, 1, 6, 7]], x[:, 0].view(torch.int16)[:, [0, 1, 6, 7]])


@gpu
@pytest.mark.parametrize("layout,R", [("half", 64), ("half", 24), ("pairs", 64)])
def test_heads_of_zeros_and_nan(cuda, layout, R):
    """Heads of zeros with eps 0 aside, a head's NaN stays within it."""
    x = torch.ones((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    x[1, 2, 5], x[2, 0] = math.nan, 0.0
    for norm in (None, "rms", "layer"):
        y = torch_api.rotate_heads(x, None, _cu([1, 2, 3]), rotary.Rotary(R, layout=layout), norm=norm, eps=1e-6)[0]
        assert y[1, 2].isnan().any() and (y[2, 0] == 0).all()
        y[1, 2] = 0
        assert not y.isnan().any()
        assert (norm is None) or layout != "half" or torch.equal(y[0, 0], y[0, 3])


STORE = [  # T, q heads, kv heads, D, R, page_tokens, norm, dtype
    (1, 8, 2, 128, 128, 64, "rms", "bf16"), (36, 32, 8, 128, 128, 64, "rms", "bf16"),
    (301, 6, 3, 64, 32, 20, "layer", "fp16"), (1030, 5, 1, 96, 24, 1, None, "bf16"), (77, 4, 4, 256, 256, 16, "rms", "fp16")]


@gpu
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("case", STORE, ids=range(len(STORE)))
def test_rotate_store_kv(cuda, case, head_major):
    """The same bits as the rotation and the store one after the other; rows
    without a slot, past the cache and of padding store nothing."""
    T, hq, h, D, R, pt, norm, dt = case
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    qkv = rnd(T, hq + 2 * h, D).to(DT[dt])
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
    rot = rotary.Rotary(R, scaling=dict(kind="linear", factor=2.0))
    pos = _positions(T, g, 5000)
    pages = -(-T // pt) + 3
    slots = torch.randperm(pages * pt, generator=g, device="cuda")[:T]
    if T > 9:
        slots[3], slots[4], slots[5] = -1, pages * pt, 2**62
    shape = (2, pages, h, pt, D) if head_major else (2, pages, pt, h, D)
    cache = rnd(*shape).to(DT[dt])
    kc, vc = (cache.permute(0, 1, 3, 2, 4) if head_major else cache).unbind(0)
    kw = {}
    if norm:
        kw = dict(norm=norm, q_weight=rnd(D), k_weight=rnd(D))
    want_q, want_k = torch_api.rotate_heads(q, k, pos, rot, **kw)
    live = pos >= 0
    want = [kc.clone(), vc.clone()]
    torch_api.store_paged_kv(want_k, v, torch.where(live, slots, -1), *want)
    out = torch.full((T, hq, D), 7.0, dtype=DT[dt], device="cuda")
    got = torch_api.rotate_store_kv(q, k, v, pos, slots, kc, vc, rot, q_out=out, **kw)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out[live], want_q[live]) and (out[~live] == 7).all()
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


# ---------------------------------------------------------------------------
# windowed attention
# ---------------------------------------------------------------------------

def windowed(pr, window, sinks, form, **kw):
    """Runs the problem windowed, with NaN in every cache slot no row sees and
    table entries of unseen pages that name the page of NaNs, any page or none;
    checks against its clean caches."""
    kc, vc, table = pr.kc.clone(), pr.vc.clone(), pr.table.clone()
    r = np.random.default_rng(window + sinks)
    bad = [kc.shape[0] - 1, -1, 2**31 - 1, -5]
    seen_slots = torch.zeros(kc.shape[0] * pr.pt, dtype=torch.bool, device="cuda")
    for b, (s, n) in enumerate(pr.lens):
        for j in range(-(-max(s, 0) // pr.pt)):
            tok = np.arange(j * pr.pt, min((j + 1) * pr.pt, s))
            vis = (tok < sinks) | (tok > s - n - window)
            if not vis.any() or n == 0:
                table[b, j] = int(bad[r.integers(0, 4)])
            else:
                seen_slots[int(pr.table[b, j]) * pr.pt + torch.from_numpy(tok[vis] % pr.pt).cuda()] = True
    gone = ~seen_slots.view(-1, pr.pt)
    kc[gone], vc[gone] = math.nan, math.nan
    out, lse = torch_api.paged_attention(pr.q, kc, vc, table, pr.start, pr.seq, scale=pr.scale, return_lse=True,
                                         window=window, sink_tokens=sinks, form=form, **kw)
    T = pr.q.shape[0]
    pr.kc, pr.vc = pr.kc.nan_to_num(), pr.vc.nan_to_num()
    cols = torch.arange(max(sinks, 1), dtype=torch.int32, device="cuda").repeat(T, 1)
    if sinks == 0:
        cols.fill_(-1)
    pr.check(out, lse, cols, 1, window)
    return out, lse


WINDOW_LENS = {
    "one_key": [(1, 1)],
    "decode": [(700, 1), (1, 1), (128, 1), (129, 1), (2000, 1), (17, 1)],
    "verify": [(300, 4), (5, 4), (4, 4), (257, 3), (1030, 1)],
    "chunk": [(200, 200), (813, 430), (64, 64)],
    "ragged": [(90, 33), (0, 0), (1000, 1), (129, 129), (700, 0), (685, 257), (16, 1)],
}


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
@pytest.mark.parametrize("lens", list(WINDOW_LENS))
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (7, 1), (64, 0), (100, 5), (128, 128), (333, 130), (10**6, 4),
                                          (200, 2**31 - 1)])
@pytest.mark.parametrize("hkv,group,D,pt,dt", [
    (1, 1, 128, 64, "bf16"), (2, 7, 64, 8, "fp16"), (1, 16, 64, 128, "bf16"), (1, 20, 128, 256, "fp16")])
def test_windowed_attention(cuda, form, lens, window, sinks, hkv, group, D, pt, dt):
    pr = Problem(WINDOW_LENS[lens], hkv, group, D, pt, dt, seed=len(lens) * 100 + group)
    windowed(pr, window, min(sinks, 2100), form)
    if sinks > 2100:    # every token is a sink: full attention (short items may be divided otherwise)
        pr.check(*pr.run(form=form, window=window, sink_tokens=sinks))


@gpu
@pytest.mark.parametrize("window,new", [(100, 6), (509, 8), (600, 8), (100, 20)])
def test_windowed_attention_of_the_dispatch(cuda, window, new):
    """The form the call chooses itself, on either side of its rule."""
    windowed(Problem([(1500, new), (90, new), (new, new)], 2, 4, 128, 64, "bf16", seed=new), window, 3, _abi.ATTN_AUTO,
             max_new=new)


@gpu
@pytest.mark.parametrize("pt", [1, 3, 20, 192])
def test_windowed_attention_odd_pages(cuda, pt):
    pr = Problem([(333, 2), (41, 5), (7, 7)], 2, 3, 128, pt, "bf16", seed=pt)
    windowed(pr, 50, 5, _abi.ATTN_AUTO, max_new=7)


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
@pytest.mark.parametrize("lens,hkv,group,window,sinks", [
    ([(40000, 1), (3, 1)], 2, 4, 9000, 200), ([(30000, 40)], 1, 8, 20000, 4), ([(9000, 2000)], 2, 4, 1000, 64)])
def test_windows_split_over_the_gpu(cuda, form, lens, hkv, group, window, sinks):
    pr = Problem(lens, hkv, group, 128, 64, "bf16", seed=5)
    a = windowed(pr, window, sinks, form)
    b = pr.run(form=form, window=window, sink_tokens=sinks)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
@pytest.mark.parametrize("B", [33, 390, 1100])
def test_windows_of_many_requests(cuda, form, B):
    r = np.random.default_rng(B)
    lens = [(int(s), min(int(s), int(n))) for s, n in zip(r.integers(0, 400, B), r.integers(0, 4, B))]
    windowed(Problem(lens, 1, 2, 64, 16, "bf16", seed=B), 37, 3, form)


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
@pytest.mark.parametrize("sinks", [0, 20])
def test_windows_past_the_table(cuda, form, sinks):
    """More tokens than the table's 12 pages hold: the keys end there, positions and
    windows do not, and rows whose window lies behind the end see the sinks alone."""
    pr = Problem([(300, 40), (64, 3)], 2, 4, 128, 32, "bf16", seed=21)
    pr.kc.nan_to_num_(0.5)
    pr.vc.nan_to_num_(0.5)
    cap = pr.table.shape[1] * 32
    for n in (cap + 20, cap + 200, 2**31 - 1):
        pr.seq = _cu([n, 64])
        out, lse = pr.run(form=form, window=60, sink_tokens=sinks)
        pr.seq = _cu([min(n, cap + 200), 64])
        want = pr.run(form=form, window=60, sink_tokens=sinks)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and not out.isnan().any()
        if sinks == 0 and n > cap + 100:
            assert (lse[:40] == -math.inf).all() and (out[:40] == 0).all()
    only = torch.arange(20, dtype=torch.int32, device="cuda").repeat(43, 1)
    if sinks:
        sel, z = pr.run(selected=only, ratio=1, local_tokens=0)
        assert ((lse[:40] - z[:40]).abs() <= 1e-4).all()
    pr.seq = _cu([-5, 64])
    out, lse = pr.run(form=form, window=60, sink_tokens=sinks)
    assert (lse[:40] == -math.inf).all() and (out[:40] == 0).all()


@gpu
@pytest.mark.parametrize("form", [_abi.ATTN_GATHER, _abi.ATTN_TILE], ids=["gather", "tile"])
def test_windowed_missing_pages(cuda, form):
    """A missing page inside the window and one of the sinks'."""
    pr = Problem([(700, 4), (300, 130)], 2, 4, 128, 32, "bf16", seed=4)
    there = pr.table.clone()
    pr.table[0, 0] = pr.table[0, 20] = pr.table[1, 6] = -1
    out, lse = pr.run(form=form, window=100, sink_tokens=40)
    pr.table = there
    rows = []
    for (s, n), gone in zip(pr.lens, ([0, 20], [6])):
        for p in range(s - n, s):
            rows.append([t for t in range(p + 1) if (t < 40 or t > p - 100) and t // 32 not in gone])
    wide = max(map(len, rows))
    pr.check(out, lse, _cu([r + [-1] * (wide - len(r)) for r in rows]), 1, 0)


@gpu
def test_windowed_graph_replays_new_lengths(cuda):
    pr = Problem([(900, 1), (450, 1)], 2, 4, 128, 64, "bf16", seed=8)
    st = torch.cuda.Stream()
    cols = torch.arange(3, dtype=torch.int32, device="cuda").repeat(2, 1)
    for form in (_abi.ATTN_GATHER, _abi.ATTN_TILE):
        pr.run(form=form, window=70, sink_tokens=3)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out, lse = pr.run(form=form, window=70, sink_tokens=3)
        for s0, s1 in ((900, 450), (3, 449), (128, 1)):
            pr.seq.copy_(_cu([s0, s1]))
            graph.replay()
            torch.cuda.synchronize()
            pr.lens = [(s0, 1), (s1, 1)]
            pr.check(out, lse, cols, 1, 70)
        pr.seq.copy_(_cu([900, 450]))


# ---------------------------------------------------------------------------
# verification of drafts
# ---------------------------------------------------------------------------

def verified(tokens, target, uniforms, draft=None, num=None, context=None):
    """In Python integers and float64; probabilities in units of 2^-45, as documented."""
    B, K1, V = target.shape
    K = K1 - 1
    clean = lambda x: x.double().nan_to_num(0.0).clamp(0, 1).cpu().numpy()  # noqa: E731
    units = lambda x: [int(v) for v in np.rint(x * 2.0 ** 45)]  # noqa: E731
    t, d = clean(target), None if draft is None else clean(draft)
    u = uniforms.double().nan_to_num(0.0).clamp(0, 1).cpu().numpy()
    out, acc = np.full((B, K1), -1), np.zeros(B, np.int64)
    for b in range(B):
        n = K if num is None else min(max(int(num[b]), 0), K)
        a = 0
        while a < n:
            x = int(tokens[b, a])
            if not (0 <= x < V and u[b, a] * (1.0 if d is None else d[b, a, x]) < t[b, a, x]):
                break
            a += 1
        w = units(t[b, a])
        if a < n:
            x = int(tokens[b, a])
            if d is None:
                left = [0 if j == x else v for j, v in enumerate(w)]
            else:
                left = [max(v - q, 0) for v, q in zip(w, units(d[b, a]))]
            if sum(left):
                w = left
        total, run, nxt = sum(w), 0, -1
        from fractions import Fraction
        # past the last representable u below 1, the largest one of 64 bits
        point = Fraction(float(u[b, K])) * total if u[b, K] < 1 else Fraction(2**64 - 1, 2**64) * total
        for j, v in enumerate(w):
            run += v
            if run > point:
                nxt = j
                break
        out[b, :a] = tokens[b, :a].cpu().numpy()
        out[b, a] = nxt
        acc[b] = a
    lens = None if context is None else [min(max(int(c), 0) + 1 + int(a), 2**31 - 1) for c, a in zip(context, acc)]
    return out, acc, lens


def check_verified(got, want):
    assert (got.tokens.cpu().numpy() == want[0]).all() and (got.num_accepted.cpu().numpy() == want[1]).all()
    assert (got.next_lens is None and want[2] is None) or got.next_lens.tolist() == want[2]


def _drafted(B, K, V, dt, seed, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((B, K + 1, V), generator=g, device="cuda") * spread
    target = logits.softmax(2).to(dt)
    draft = (logits[:, :K] + 0.7 * torch.randn((B, K, V), generator=g, device="cuda")).softmax(2)
    tokens = torch.multinomial(draft.flatten(0, 1), 1, generator=g).view(B, K) if K else torch.empty((B, 0), device="cuda")
    u = torch.rand((B, K + 1), generator=g, device="cuda")
    return tokens.to(torch.int32), target, u, draft.to(dt)


@gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,K,V", [(1, 3, 32003), (5, 0, 1000), (3, 1, 1), (64, 4, 257), (7, 40, 97), (2, 2, 50000),
                                   (300, 2, 8192), (4, 7, 4096)])
@pytest.mark.parametrize("certain", [False, True])
def test_verify_drafts(cuda, dt, B, K, V, certain):
    tokens, target, u, draft = _drafted(B, K, V, dt, B + V)
    draft = None if certain else draft
    num = torch.randint(-1, K + 3, (B,), dtype=torch.int32, device="cuda") if B > 4 else None
    ctx = torch.randint(-3, 9000, (B,), dtype=torch.int32, device="cuda")
    got = torch_api.verify_drafts(tokens, target, u, draft_probs=draft, num_drafts=num, context_lens=ctx)
    check_verified(got, verified(tokens, target, u, draft, num, ctx))
    again = torch_api.verify_drafts(tokens, target, u, draft_probs=draft, num_drafts=num)
    assert again.next_lens is None and torch.equal(again.tokens, got.tokens)


@gpu
def test_verify_strides_and_outputs(cuda):
    """Rows of a wider logits buffer at an odd offset, outputs given, next_lens over context_lens."""
    tokens, target, u, draft = _drafted(6, 3, 1001, torch.float32, 3)
    wide = torch.full((6, 5, 1009), math.nan, device="cuda")
    wide[:, :4, 3:1004] = target
    wide_d = torch.full((3, 6, 1007), math.nan, device="cuda")
    wide_d[:, :, 5:1006] = draft.transpose(0, 1)
    ctx = _cu([5, 0, 2**31 - 2, 2**31 - 1, 7, 8])
    want = verified(tokens, target, u, draft, None, ctx)
    out = torch_api.Verified(torch.zeros((6, 4), dtype=torch.int32, device="cuda"),
                             torch.zeros(6, dtype=torch.int32, device="cuda"), ctx)
    got = torch_api.verify_drafts(tokens, wide[:, :4, 3:1004], u, draft_probs=wide_d[:, :, 5:1006].transpose(0, 1),
                                  context_lens=ctx, out=out)
    check_verified(got, want)
    assert got.tokens.data_ptr() == out.tokens.data_ptr() and ctx.tolist() == want[2]


@gpu
def test_verify_edges(cuda):
    """Random numbers at and past both ends, rows without weight, one-hot rows,
    invalid drafts, NaN, negative and infinite probabilities, equal rows."""
    V, K = 5000, 2
    rows = {
        "onehot_hit": ([7, 8], [(7, 1.0)], [(8, 1.0)], [(9, 1.0)]),
        "onehot_miss": ([6, 8], [(7, 1.0)], [(8, 1.0)], [(9, 1.0)]),
        "empty": ([6, 8], [], [], []),
        "bad_token": ([-1, 3], [(4, 0.5), (4999, 0.5)], [(3, 1.0)], [(2, 1.0)]),
        "past_vocab": ([V, 3], [(0, 0.25), (4999, 0.75)], [(3, 1.0)], [(2, 1.0)]),
        "nan": ([1, 3], [(1, math.nan), (2, -1.0), (17, 0.5), (18, math.inf)], [(3, 1.0)], [(2, 1.0)]),
        "tiny": ([5, 3], [(5, 2.0 ** -46), (40, 2.0 ** -45), (41, 2.0 ** -22 - 2.0 ** -46), (42, 2.0 ** -22), (43, 3 * 2.0 ** -46)], [(3, 1.0)], [(2, 1.0)]),
    }
    us = [0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan, 0.5, 2.0 ** -40]
    for certain in (True, False):
        B = len(rows) * len(us)
        target = torch.zeros((B, K + 1, V), device="cuda")
        tokens = torch.zeros((B, K), dtype=torch.int32, device="cuda")
        u = torch.zeros((B, K + 1), device="cuda")
        for i, (toks, *places) in enumerate(rows.values()):
            for j, x in enumerate(us):
                b = i * len(us) + j
                tokens[b], u[b, K] = _cu(toks), x
                for r, place in enumerate(places):
                    for at, p in place:
                        target[b, r, at] = p
        draft = None if certain else target[:, :K].clone()     # equal rows: nothing left of a refused one
        if draft is not None:
            u[:, :K] = 1.0 - 2.0 ** -24
            u[::2, :K] = 1.0
        got = torch_api.verify_drafts(tokens, target, u, draft_probs=draft)
        check_verified(got, verified(tokens, target, u, draft))


@gpu
@pytest.mark.parametrize("V", [700, 1000])
def test_verify_weights_that_are_no_distribution(cuda, V):
    """Rows of large weights, whose sum is far above 1: still exact."""
    g = torch.Generator(device="cuda").manual_seed(V)
    target = 1 - torch.rand((9, 2, V), generator=g, device="cuda") ** 9
    target[0] = 1.0
    draft = target[:, :1] * torch.rand((9, 1, V), generator=g, device="cuda")
    tokens = torch.randint(0, V, (9, 1), dtype=torch.int32, device="cuda")
    u = torch.rand((9, 2), generator=g, device="cuda")
    for num in (None, _cu([0] * 9)):
        got = torch_api.verify_drafts(tokens, target, u, draft_probs=draft, num_drafts=num)
        check_verified(got, verified(tokens, target, u, draft, num))


@gpu
def test_verified_tokens_are_distributed_as_the_target(cuda):
    """First tokens over many requests of one distribution: within five standard
    deviations of the target's probability, whatever the draft's is."""
    V, N = 8, 40000
    g = torch.Generator(device="cuda").manual_seed(2)
    p = torch.tensor([0.3, 0.05, 0.0, 0.2, 0.15, 0.1, 0.15, 0.05], device="cuda")
    q = torch.tensor([0.1, 0.25, 0.1, 0.0, 0.15, 0.2, 0.1, 0.1], device="cuda")
    tokens = torch.multinomial(q, N, replacement=True, generator=g).view(N, 1).to(torch.int32)
    u = torch.rand((N, 2), generator=g, device="cuda")
    r = torch_api.verify_drafts(tokens, p.expand(N, 2, V), u, draft_probs=q.expand(N, 1, V))
    share = torch.bincount(r.tokens[:, 0].long(), minlength=V).double() / N
    assert ((share - p).abs() <= 5 * (p.double() * (1 - p) / N).sqrt() + 1e-12).all()


@gpu
def test_step_operators_captured_and_on_another_stream(cuda):
    """One graph of rotation, store, windowed attention and verification, replayed with
    other inputs; the same calls given another stream."""
    pr = Problem([(300, 2), (130, 2)], 2, 4, 128, 32, "bf16", seed=14)
    pr.kc.nan_to_num_(0.0)
    pr.vc.nan_to_num_(0.0)
    rot = rotary.Rotary(128)
    qkv = torch.randn((4, 12, 128), device="cuda").to(torch.bfloat16)
    pos = _cu([298, 299, 128, 129])
    slots = torch.tensor([int(pr.table[b, p // 32]) * 32 + p % 32 for b, p in ((0, 298), (0, 299), (1, 128), (1, 129))],
                         device="cuda")
    tokens, target, u, draft = _drafted(2, 1, 3000, torch.float32, 1)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")

    def all_of(stream=None):
        q = torch_api.rotate_store_kv(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], pos, slots, pr.kc, pr.vc, rot, norm="rms",
                                      stream=stream)
        o = torch_api.paged_attention(q, pr.kc, pr.vc, pr.table, pr.start, pr.seq, window=50, sink_tokens=4,
                                      workspace=ws, stream=stream)
        return q, o, torch_api.verify_drafts(tokens, target, u, draft_probs=draft, stream=stream).tokens

    all_of()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = all_of()
    side = torch.cuda.Stream()
    for i in range(3):
        qkv.normal_()
        u.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        cache = pr.kc.clone()
        for s in (None, side, side.cuda_stream):
            pr.kc.zero_()
            side.wait_stream(torch.cuda.current_stream())
            pr.kc.copy_(cache)
            side.wait_stream(torch.cuda.current_stream())
            got = all_of(s)
            torch.cuda.synchronize()
            for a, b in zip(kept, got):
                assert torch.equal(a, b)
            assert torch.equal(cache, pr.kc)


# ---------------------------------------------------------------------------
# runs of them together
# ---------------------------------------------------------------------------

def _plain_window(q, k, v, first, window, sinks):
    """fp64 attention of the last tokens, at positions first.., to keys 0.. ."""
    n, H, D = q.shape
    s = k.shape[0]
    pos = torch.arange(first, first + n, device="cuda")
    j = torch.arange(s, device="cuda")
    see = (j[None] <= pos[:, None]) & ((j[None] > pos[:, None] - window) | (j[None] < sinks))
    kd, vd = (x.double().repeat_interleave(H // x.shape[1], 1) for x in (k, v))
    x = torch.einsum("thd,shd->hts", q.double(), kd) * D ** -0.5
    p = x.masked_fill(~see, -math.inf).softmax(-1)
    return torch.einsum("hts,shd->thd", p, vd), torch.einsum("hts,shd->thd", p, vd.abs())


@gpu
@pytest.mark.parametrize("norm,layout", [("rms", "half"), (None, "pairs")])
def test_speculative_rounds(cuda, norm, layout):
    """Prompts, then rounds of four rows: maps, rotated stores, windowed attention and
    verification, each round's lengths from the last one's on the device.  Refused
    tokens are overwritten; attention is that of the accepted history alone."""
    from sparse_attention_indexer_02_gb300 import serving

    B, K, H, hkv, D, pt, window, sinks, V = 3, 3, 8, 2, 128, 16, 40, 5, 500
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    pool = serving.PagedPool(num_pages=120, page_tokens=pt, num_kv_heads=hkv, head_dim=D, ratio=4)
    how = serving.HeadRotation(torch_api.Rotary(D, layout=layout), norm=norm,
                               q_weight=1 + 0.1 * rnd(D) if norm else None, k_weight=1 + 0.1 * rnd(D) if norm else None)
    table = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    pages = torch.randperm(120, generator=g, device="cuda").to(torch.int32)
    ctx, new = _cu([0, 0, 0]), _cu([70, 3, 41])
    hist, taken = [(torch.empty((0, hkv, D), device="cuda").bfloat16(),) * 2 for _ in range(B)], 0
    for turn in range(7):
        T = int(new.sum())
        q, k, v = rnd(T, H, D), rnd(T, hkv, D), rnd(T, hkv, D)
        maps = torch_api.build_page_maps(ctx, new, pages[taken:], table, page_tokens=pt, max_tokens=T)
        taken += int(maps.pages_used)
        res = serving.windowed(pool, table, maps, q=q, k=k, v=v, window=window, sink_tokens=sinks,
                               max_new=int(new.max()), rotation=how)
        kw = {n: getattr(how, n) for n in ("norm", "q_weight", "k_weight", "eps")}
        qr, kr = torch_api.rotate_heads(q, k, maps.positions, how.rotary, **kw)
        start = maps.query_start.tolist()
        for b in range(B):
            rows = slice(start[b], start[b + 1])
            ks, vs = torch.cat([hist[b][0], kr[rows]]), torch.cat([hist[b][1], v[rows]])
            want, mag = _plain_window(qr[rows], ks, vs, len(hist[b][0]), window, sinks)
            # the rounded output and probabilities, half a step each; scores of about 30 in fp32
            assert ((res.out[rows].double() - want).abs() <= 2.0 ** -8 * (want.abs() + mag) + 1e-4 * mag + 1e-6).all()
        if turn == 0:      # the prompts count as they are
            keep = new.tolist()
            ctx = maps.seq_lens
        else:
            tokens, target, u, draft = _drafted(B, K, V, torch.float32, turn)
            ver = torch_api.verify_drafts(tokens, target, u, draft_probs=draft, context_lens=ctx)
            check_verified(ver, verified(tokens, target, u, draft, None, ctx))
            keep = [1 + a for a in ver.num_accepted.tolist()]
            ctx = ver.next_lens
        hist = [(torch.cat([hist[b][0], kr[start[b]:start[b] + keep[b]]]),
                 torch.cat([hist[b][1], v[start[b]:start[b] + keep[b]]])) for b in range(B)]
        assert ctx.tolist() == [len(h[0]) for h in hist]
        new = _cu([K + 1] * B)


@gpu
def test_serving_step_with_rotation(cuda):
    """The step with a rotation is the step of the rotated queries and keys."""
    from sparse_attention_indexer_02_gb300 import serving

    B, n, H, hkv, D = 2, 40, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    T = B * n
    q, k, v, iq, ik = rnd(T, H, D), rnd(T, hkv, D), rnd(T, hkv, D), rnd(T, 4, 128), rnd(T, 128)
    iw = torch.rand((T, 4), generator=g, device="cuda")
    how = serving.HeadRotation(torch_api.Rotary(64, offset=64, layout="pairs"), "layer", rnd(D), rnd(D), rnd(D), rnd(D))
    irot = torch_api.Rotary(64)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B)
    qr, kr = torch_api.rotate_heads(q, k, pos, how.rotary, norm="layer", q_weight=how.q_weight, k_weight=how.k_weight,
                                    q_bias=how.q_bias, k_bias=how.k_bias, eps=how.eps)
    iqr = torch_api.rotate_heads(iq, None, pos, irot)[0]
    got = []
    for args, kw in (((qr, kr, iqr), {}), ((q, k, iq), dict(rotation=how, index_rotary=irot))):
        pool = serving.PagedPool(num_pages=8, page_tokens=16, num_kv_heads=hkv, head_dim=D, ratio=4)
        table = torch.full((B, 4), -1, dtype=torch.int32, device="cuda")
        res = serving.step(pool, table, _cu([0, 0]), _cu([n, n]), _cu([5, 2, 7, 0, 3, 1, 6, 4]), q=args[0], k=args[1],
                           v=v, index_q=args[2], index_keys=ik, index_weights=iw, top_k=5, local_tokens=8, max_context=64,
                           **kw)
        got.append((res.out, res.lse, res.selected, pool.k_cache, pool.v_cache))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@gpu
def test_rotations_on_two_streams_at_once(cuda):
    """Calls that share their inputs and run beside one another."""
    q = torch.randn((3000, 16, 128), device="cuda").to(torch.bfloat16)
    pos = torch.arange(3000, dtype=torch.int32, device="cuda")
    rots = [rotary.Rotary(128), rotary.Rotary(24, layout="half"), rotary.Rotary(64, layout="pairs", offset=64)]
    want = [torch_api.rotate_heads(q, None, pos, r, norm="rms")[0] for r in rots]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in rots]
    for _ in range(5):
        got = [torch_api.rotate_heads(q, None, pos, r, norm="rms", stream=s)[0] for r, s in zip(rots, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# places of tensors
# ---------------------------------------------------------------------------

def test_step_tensors_of_another_device_are_refused(lib):
    """Tensors that say they are on device 1 (fake ones, without memory)."""
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    with fake.FakeTensorMode():
        z = lambda dtype, *s: torch.empty(s, dtype=dtype, device="cuda:1")  # noqa: E731
        b16, i32 = torch.bfloat16, torch.int32
        q, k, pos, slots, kc = z(b16, 3, 8, 128), z(b16, 3, 2, 128), z(i32, 3), z(torch.int64, 3), z(b16, 4, 16, 2, 128)
        tok, p, u, freqs = z(i32, 2, 3), z(torch.float32, 2, 4, 50), z(torch.float32, 2, 4), z(torch.int64, 64)
    rot = rotary.Rotary(128, device="cpu")
    rot.freqs = freqs
    if torch.cuda.is_available():
        assert torch.cuda.current_device() != 1
    for call in (lambda: torch_api.rotate_heads(q, k, pos, rot),
                 lambda: torch_api.rotate_store_kv(q, k, k, pos, slots, kc, kc, rot),
                 lambda: torch_api.verify_drafts(tok, p, u)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


@gpu
def test_step_tensors_on_two_devices_are_refused(cuda):
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="different devices"):
        torch_api.rotate_heads(q, None, pos, rotary.Rotary(128, device="cpu"))
    with pytest.raises(ValueError, match="different devices"):
        torch_api.rotate_heads(q, q.cpu(), pos, rotary.Rotary(128))
    tok, p, u = _cu([[1, 2]]), torch.rand((1, 3, 50), device="cuda"), torch.rand((1, 3), device="cuda")
    for kw in (dict(draft_probs=p[:, :2].cpu()), dict(num_drafts=torch.ones(1, dtype=torch.int32))):
        with pytest.raises(ValueError, match="different devices"):
            torch_api.verify_drafts(tok, p, u, **kw)


@gpu
def test_rows_and_slots_past_32_bits(cuda):
    """Rows of q and k 3 GB apart, cache pages 5 GiB apart, probabilities 8 GB apart."""
    T, D = 3, 128
    step = 3 << 29                                  # elements of 2 bytes
    far = torch.empty(2 * step + 4 * D, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(far, (T, 2, D), (step, D, 1))
    x.copy_(torch.randn((T, 2, D), device="cuda"))
    q, k, v = x[:, :1], x[:, 1:], x[:, 1:]
    rot, pos = rotary.Rotary(D), _cu([7, 8, 9])
    want = torch_api.rotate_heads(q.contiguous(), k.contiguous(), pos, rot, norm="rms")
    page = 5 << 29
    buf = torch.empty(2 * page + 4 * D, dtype=torch.bfloat16, device="cuda")
    kc = torch.as_strided(buf, (3, 1, 1, D), (page, D, D, 1))
    vc = torch.empty((3, 1, 1, D), dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(far, (T, 1, D), (step, D, 1), 2 * D)
    torch_api.rotate_store_kv(q, k, v, pos, torch.tensor([2, 0, 1], device="cuda"), kc, vc, rot, norm="rms", q_out=out)
    at = [1, 2, 0]                                  # the token that went to each page
    assert torch.equal(out, want[0]) and torch.equal(kc[:, 0], want[1][at]) and torch.equal(vc[:, 0], v[at])
    del buf, kc, far, x, q, k, v, out
    V, gap = 1000, 2 << 30                          # fp32: 8 GB from row to row
    tokens, target, u, draft = _drafted(1, 2, V, torch.float32, 9)
    wide = torch.empty(2 * gap + V, device="cuda")
    rows = torch.as_strided(wide, (1, 3, V), (3 * gap, gap, 1))
    rows.copy_(target)
    for uu in (u, torch.zeros_like(u)):
        check_verified(torch_api.verify_drafts(tokens, rows, uu, draft_probs=draft), verified(tokens, target, uu, draft))


@gpu
def test_first_calls_under_capture(cuda):
    """A process whose first calls of the operators are captured, and then replayed."""
    import subprocess
    import sys

    code = """
import torch
from sparse_attention_indexer_02_gb300 import torch_api
q = torch.randn((5, 8, 128), device="cuda").to(torch.bfloat16)
k = q[:, :2].contiguous()
kc = torch.zeros((2, 4, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
rot, pos, slots = torch_api.Rotary(128), torch.arange(5, dtype=torch.int32, device="cuda"), torch.arange(5, device="cuda")
table, start, seq = i32(0, 1, 2, 3).view(1, 4), i32(0, 5), i32(5)
tok, p, u = i32(3, 4).view(1, 2), torch.softmax(torch.randn((1, 3, 70000), device="cuda"), 2), torch.rand((1, 3), device="cuda")
ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
def run():
    r = torch_api.rotate_store_kv(q, k, k, pos, slots, kc[0], kc[1], rot, norm="rms")
    o = torch_api.paged_attention(r, kc[0], kc[1], table, start, seq, window=3, sink_tokens=1, workspace=ws)
    return r, o, torch_api.verify_drafts(tok, p, u).tokens
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
for a, b in zip(got, run()):
    assert torch.equal(a, b)
print("same")
"""
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                         cwd=qbuild.PKG + "/..")
    assert res.returncode == 0 and "same" in res.stdout, res.stderr[-2000:]


@gpu
def test_window_arguments_refused(cuda):
    pr = Problem([(30, 2)], 2, 4, 128, 16, "bf16", seed=1)
    with pytest.raises(ValueError, match="selected"):
        pr.run(window=4, selected=torch.zeros((2, 1), dtype=torch.int32, device="cuda"))
    for kw in (dict(window=-1), dict(sink_tokens=3), dict(window=3, sink_tokens=-1), dict(window=3, local_tokens=2)):
        with pytest.raises(qsa.QSAError) as e:
            pr.run(**kw)
        assert e.value.status == INVALID
    for kw in (dict(window=1 << 31), dict(window=2.5), dict(window=3, sink_tokens=None)):
        with pytest.raises(ValueError):
            pr.run(**kw)
    windowed(pr, 2**31 - 1, 0, _abi.ATTN_AUTO)


@gpu
@pytest.mark.parametrize("B,K", [(70, 2), (16, 1), (200, 0)])
def test_verify_in_every_cluster(cuda, B, K):
    """Batches that take clusters of every size, over a vocabulary of odd rows too."""
    for V in (140000, 9001):
        tokens, target, u, draft = _drafted(B, K, V, torch.bfloat16 if V > 100000 else torch.float32, B)
        got = torch_api.verify_drafts(tokens, target, u, draft_probs=draft)
        acc = got.num_accepted.long()
        at = torch.arange(B, device="cuda")
        # against integers on the GPU: the row's weights in units, their cumulative sums, the point
        unit = lambda x: torch.round(x.double().clamp(0, 1) * 2.0 ** 45).long()  # noqa: E731
        w = unit(target[at, acc])
        if K:
            left = (w - unit(draft[at, acc.clamp(max=K - 1)])).clamp(min=0)
            some = (acc < K) & (left.sum(1) > 0)
            w = torch.where(some[:, None], left, w)
        cum = w.cumsum(1)
        total = cum[:, -1]
        m = (u[:, K].double() * 2.0 ** 24).long()          # u is a multiple of 2^-24
        # cum > u total  <=>  cum 2^24 > m total, with total = hi 2^24 + lo
        hi, lo = total >> 24, total & ((1 << 24) - 1)
        point = m * hi + ((m * lo) >> 24)
        want = (cum <= point[:, None]).sum(1)
        assert torch.equal(got.tokens[at, acc].long(), want)
