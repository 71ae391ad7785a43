"""The encoder-block operators on the GPU against float64 definitions.

Bounds: an output of a 16-bit or 32-bit type is one rounding (UNIT) from its value, to which come
the float32 arithmetic before it (2^-24 an operation, over sums of n terms at most sqrt-like but
bounded here by a small multiple) and, for attention, the rounding of the probabilities and score
gradients to the tensors' type (UNIT relative to the magnitudes that are summed).
"""
import math
import random

import pytest

torch = pytest.importorskip("torch")

import block_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
E32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from vit_vision_encoder_fusedinputnorm_gb300 import build
    build.build()


def _enc():
    from vit_vision_encoder_fusedinputnorm_gb300 import encoder
    return encoder


def _randn(seed, *shape, dtype=SF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


# ------------------------------------------------------------------ layer norm

NORM_SIZES = [(1, 1), (3, 7), (5, 33), (256, 1280), (70, 1152), (9, 80), (17, 2048), (4, 2056), (33, 1027), (2, 5000),
              (3, 8192), (2, 16384), (2, 16383), (1, 4100), (70, 64), (133, 100), (41, 128), (257, 200), (19, 256),
              (700, 24), (50, 640), (6, 2700), (5, 3584)]


def _norm_tol(x, mean, rstd, w, b, y):
    """Output rounding, and float32 errors of mean, rstd and the line x -> y."""
    big = x.double().abs().amax(1, keepdim=True) * rstd[:, None]
    wa = 1.0 if w is None else w.double().abs()
    ba = 0.0 if b is None else b.double().abs()
    return R.rounding(x.dtype, y) + 16 * E32 * ((1 + big) * wa + ba)


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("rows,width", NORM_SIZES)
def test_layer_norm_and_its_gradients(rows, width, dtype):
    E = _enc()
    x = (_randn(1, rows, width) * (1 + _randn(2, 1, width).abs()) + 2.0).to(dtype)
    w, b = _randn(3, width, dtype=SF), _randn(4, width, dtype=SF)
    dy = _randn(5, rows, width).to(dtype)
    y, mean, rstd = E.layer_norm(x, w, b, 1e-5, stats=True)
    ry, rm, rr = R.layer_norm(x, w, b, 1e-5)
    R.close(y, ry, _norm_tol(x, rm, rr, w, b, ry), "y")
    xm = x.double().abs().amax(1)
    R.close(mean, rm, 16 * E32 * xm, "mean")
    R.close(rstd, rr, 16 * E32 * rr * (1 + xm * rr), "rstd")
    dx, dw, db = E.layer_norm_backward(dy, x, mean, rstd, w)
    rx, rdw, rdb, xh, g = R.layer_norm_backward(dy, x, mean, rstd, w)
    # float32 errors: of xh (its cancellation), of the two means, of the line
    mag = rstd.double()[:, None] * (g.abs() + g.abs().amax(1, keepdim=True) * (1 + xh.abs()) * (1 + xh.abs().amax(1, keepdim=True)))
    off = (1 + xm * rr)[:, None]
    R.close(dx, rx, R.rounding(x.dtype, rx) + 16 * E32 * off * mag, "dx")
    R.close(dw, rdw, 16 * E32 * (dy.double().abs() * (xh.abs() + off)).sum(0), "dweight")
    R.close(db, rdb, 16 * E32 * dy.double().abs().sum(0), "dbias")
    again = E.layer_norm_backward(dy, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again)), "equal calls give equal bits"


@pytest.mark.parametrize("params", [BF, HF, SF, None])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_layer_norm_strides_parameter_types_and_in_place(params, pad):
    E = _enc()
    rows, width = 37, 1280
    wide = _randn(6, rows, width + pad + 8, dtype=BF)
    x = wide[:, pad:pad + width]
    w = None if params is None else _randn(7, width, dtype=params)
    b = None if params is None else _randn(8, width, dtype=params)
    ref = R.layer_norm(x, w, b, 1e-6)
    kept = wide.clone()
    y = E.layer_norm(x, w, b, 1e-6)
    R.close(y, ref[0], _norm_tol(x, ref[1], ref[2], w, b, ref[0]), "y")
    assert torch.equal(wide, kept)
    E.layer_norm(x, w, b, 1e-6, out=x)              # in place, inside the wider rows
    assert torch.equal(x, y)
    assert torch.equal(wide[:, :pad], kept[:, :pad]) and torch.equal(wide[:, pad + width:], kept[:, pad + width:])


def test_layer_norm_no_rows_and_constant_rows():
    E = _enc()
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    assert E.layer_norm(x).shape == (0, 64)
    z = torch.empty(0, device="cuda")
    dx, dw, db = E.layer_norm_backward(x, x, z, z)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    y = E.layer_norm(torch.full((3, 257), 5.0, device="cuda"), eps=1e-6)
    assert not y.any()
    with_nan = _randn(9, 4, 128)
    with_nan[2, 5] = math.nan
    y = E.layer_norm(with_nan)
    assert y[2].isnan().all() and torch.isfinite(y[[0, 1, 3]]).all()


def test_layer_norm_gradient_against_differences():
    E = _enc()
    x, w, b, dy = _randn(10, 6, 96), _randn(11, 96), _randn(12, 96), _randn(13, 6, 96)
    _, mean, rstd = E.layer_norm(x, w, b, 1e-5, stats=True)
    dx, dw, db = E.layer_norm_backward(dy, x, mean, rstd, w)

    def loss(x, w, b):
        return float((R.layer_norm(x, w, b, 1e-5)[0] * dy.double()).sum())
    h = 1e-5
    for t, g, at in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        step = _randn(14 + at, *t.shape).double()
        args = [x.double(), w.double(), b.double()]
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + h * step, args[at] - h * step
        slope = (loss(*up) - loss(*down)) / (2 * h)
        # central differences: h^2 truncation and 1e-16 / h cancellation; gradients: float32
        assert abs(slope - float((g.double() * step).sum())) <= 1e-4 * float((g.double().abs() * step.abs()).sum())


# ------------------------------------------------------------------ rotary positions

def _items(grids):
    table = [(0, 0, t, h, w, 1 if t == 1 else 2 * t) for t, h, w in grids] or [(0,) * 6]
    return (torch.tensor(table, dtype=torch.int32, device="cuda"),
            torch.tensor([len(grids)], dtype=torch.int32, device="cuda"))


def _spans(spans, capacity=0):
    table = list(spans) + [(0, 0, -1, 0)] * max(0, capacity - len(spans)) or [(0, 0, -1, 0)]
    return (torch.tensor(table, dtype=torch.int32, device="cuda"),
            torch.tensor([len(spans)], dtype=torch.int32, device="cuda"))


def _many_spans(n):
    rng = random.Random(n)
    return [(int(rng.random() < 0.2), rng.randint(0, 9), rng.choice([-1, 0, 1, 2]), rng.randint(0, 3)) for _ in range(n)]


GRIDS = [(1, 4, 6), (3, 2, 4), (1, 10, 2)]
SPAN_CASES = {
    "text": ([(1, 5, -1, 0)], []),
    "still_first": ([(1, 0, 0, 1)], GRIDS),
    "prompt": ([(1, 3, 0, 1), (0, 2, 1, 2), (0, 4, -1, 1), (1, 1, 2, 1), (0, 0, 0, 1), (0, 7, -1, 0)], GRIDS),
    "no_flag_and_empty": ([(0, 0, -1, 0), (0, 2, 1, 0), (1, 0, -1, 5), (0, 1, -1, 5)], GRIDS),
    "empty_grid": ([(1, 2, 0, 1), (0, 3, -1, 1)], [(0, 4, 4)]),
    "none": ([], []),
    "many": (_many_spans(257), GRIDS),
    "most": (_many_spans(1024), GRIDS),
}


@pytest.mark.parametrize("name", sorted(SPAN_CASES))
@pytest.mark.parametrize("pad", [0, 13])
def test_mrope_positions(name, pad):
    spans, grids = SPAN_CASES[name]
    total = sum(s[1] + (grids[s[2]][0] * (grids[s[2]][1] // 2) * (grids[s[2]][2] // 2) if s[2] >= 0 else 0) for s in spans)
    st = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    sp, n = _spans(spans, len(spans) + 3 if len(spans) < 1000 else 0)
    pos = _enc().mrope_positions(sp, n, *_items(grids), total + pad, merge=2, status=st)
    assert torch.equal(pos.cpu(), R.positions(spans, grids, 2, total + pad))
    assert st.tolist() == [0, -1]


def test_mrope_positions_device_errors():
    E = _enc()
    st = torch.empty(2, dtype=torch.int32, device="cuda")

    def run(spans, grids, rows, n=None):
        sp, cnt = _spans(spans)
        if n is not None:
            cnt.fill_(n)
        return E.mrope_positions(sp, cnt, *_items(grids), rows, merge=2, status=st).cpu(), st.tolist()
    good = [(1, 2, 0, 1)]
    for bad in [(0, -1, -1, 0), (0, 1, 3, 0), (0, 1, -2, 0), (0, 1, 0, -1), (0, 1, 0, 1 << 20)]:
        pos, code = run(good + [bad, (0, 2, -1, 0)], GRIDS, 10)       # a bad span counts as empty
        assert code == [4, 1] and torch.equal(pos, R.positions(good + [(0, 2, -1, 0)], GRIDS, 2, 10))
    pos, code = run([(1, 1, 0, 1), (0, 1, -1, 0)], [(1, 3, 4)], 4)    # a grid that does not merge
    assert code == [4, 0] and torch.equal(pos, R.positions([(1, 1, -1, 0)], [], 2, 4))
    pos, code = run(good + [(0, 5, -1, 0)], GRIDS, 10)                # more tokens than rows
    assert code == [5, 1] and torch.equal(pos, R.positions(good + [(0, 5, -1, 0)], GRIDS, 2, 10))
    pos, code = run(good, GRIDS, 6, n=2)                              # count over the capacity
    assert code == [4, -1] and (pos == -1).all()
    pos, code = run([(1, 0x7ffffff0, -1, 0), (0, 0x7ffffff0, -1, 0)], [], 3)
    assert code[0] == 5 and torch.equal(pos, R.positions([(1, 3, -1, 0)], [], 2, 3))


ROPE_CASES = [  # rows, q heads, k heads, head_dim, rotary_dim, sections, interleaved
    (1, 28, 4, 128, 128, (16, 24, 24), False),
    (333, 3, 1, 128, 128, (24, 20, 20), True),
    (70, 2, 0, 72, 72, (12, 12, 12), False),
    (5, 0, 3, 80, 40, (10, 5, 5), False),
    (700, 16, 16, 80, 80, (0, 20, 20), False),
    (19, 2, 1, 96, 64, (32,), False),
    (3, 1, 1, 8, 8, (1, 1, 1, 1), True),
    (6, 2, 2, 512, 512, (128, 64, 64), True),
]


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("case", ROPE_CASES)
def test_mrope_apply(case, dtype):
    E = _enc()
    rows, hq, hk, d, rot, sections, inter = case
    axes = E.section_axes(sections, inter)
    assert len(axes) == rot // 2
    g = torch.Generator().manual_seed(rows)
    pos = torch.randint(-3, 1 << 20, (len(sections), rows), generator=g, dtype=torch.int32)
    pos[:, -1] = 0x7fffffff                                  # the largest position
    width = (hq + hk + 1) * d + 4                            # Q | K | something else
    buf = _randn(20, rows, width, dtype=dtype)
    q = buf[:, :hq * d].view(rows, hq, d) if hq else None
    k = buf[:, hq * d:(hq + hk) * d].view(rows, hk, d) if hk else None
    theta = 1e6
    oq, ok = E.mrope_apply(q, k, pos.cuda(), axes, theta=theta)
    kept = buf.clone()
    for x, y in ((q, oq), (k, ok)):
        if x is None:
            assert y is None
            continue
        ref = R.rotate(x, pos, axes, theta)
        # angle: 2^-32 turns, float64's pos * w_i at 2^31 (2^-52 * 2^31); sine and product in float32
        mag = x.double().abs()
        mag = mag + torch.cat([mag[..., rot // 2:rot], mag[..., :rot // 2], 0 * mag[..., rot:]], -1)
        R.close(y, ref, R.rounding(dtype, ref) + (8 * E32 + 2e-6) * mag, "rotated")
        assert torch.equal(y[..., rot:], x[..., rot:])
    E.mrope_apply(q, k, pos.cuda(), axes, theta=theta, q_out=q, k_out=k)      # in place
    for x, y in ((q, oq), (k, ok)):
        if x is not None:
            assert torch.equal(x, y)
    assert torch.equal(buf[:, (hq + hk) * d:], kept[:, (hq + hk) * d:])
    bq, bk = E.mrope_apply(oq, ok, pos.cuda(), axes, theta=theta, inverse=True)
    for x, y in ((oq, bq), (ok, bk)):
        if x is not None:
            ref = R.rotate(x, pos, axes, theta, inverse=True)
            R.close(y, ref, R.rounding(dtype, ref) + (8 * E32 + 2e-6) * 2 * x.double().abs().amax(), "inverse")


def test_mrope_gradient_against_differences():
    # <dout, d rotate(x)> along a direction: the inverse rotation of dout is the gradient
    E = _enc()
    axes = E.section_axes((6, 5, 5))
    pos = torch.randint(0, 500, (3, 11), dtype=torch.int32, device="cuda")
    x, dout, step = _randn(21, 11, 2, 40), _randn(22, 11, 2, 40), _randn(23, 11, 2, 40)
    grad, _ = E.mrope_apply(dout, None, pos, axes, inverse=True)
    h = 1e-3
    up, down = (R.rotate(x.double() + s * h * step.double(), pos, axes, 10000.0) for s in (1, -1))
    slope = float(((up - down) / (2 * h) * dout.double()).sum())
    assert abs(slope - float((grad.double() * step.double()).sum())) <= 1e-5 * float((grad * step).abs().sum())


# ------------------------------------------------------------------ attention

ATTN_CASES = [  # lens_q, lens_k (None: the same), q heads, k heads, head_dim, causal, pad
    ([256], None, 2, 2, 80, False, 0),
    ([1], None, 1, 1, 64, False, 0),
    ([128, 129, 127, 1], None, 2, 2, 64, False, 3),
    ([300, 0, 5, 511], None, 2, 1, 72, False, 40),
    ([640, 257], None, 4, 2, 128, True, 0),
    ([33, 1, 500, 2], None, 7, 1, 128, True, 1),
    ([200, 70], None, 3, 1, 96, True, 0),
    ([5, 300, 40], [300, 7, 0], 4, 2, 64, True, 9),          # rows that see nothing
    ([5, 0, 40], [300, 7, 0], 2, 2, 64, False, 0),           # keys nobody reads, queries without keys
    ([1, 1, 1, 1], [1, 700, 2500, 129], 8, 2, 128, True, 0),  # single tokens, cut key ranges
    ([1, 3], [5000, 4097], 16, 1, 64, True, 2),
    ([2, 130], [1500, 3000], 64, 1, 128, False, 0),
    ([90], [90], 5, 5, 8, True, 0),
    ([150, 20], None, 2, 2, 112, False, 0),
    ([64] * 40, None, 1, 1, 40, False, 0),
    ([1100], None, 1, 1, 88, True, 0),
    ([], [], 2, 2, 64, False, 17),                           # nothing but padding
    ([1] * 30 + [300, 0, 140], [700] * 20 + [90] * 10 + [300, 5, 1000], 4, 2, 128, True, 3),  # short and long ones
    ([70, 1, 200, 0] * 12, None, 2, 2, 80, False, 5),
]


def _attn_inputs(case, dtype, seed=30):
    lq, lk, hq, hk, d, causal, pad = case
    lk = lq if lk is None else lk
    cu = [torch.tensor([0] + list(n), dtype=torch.int32).cumsum(0).int().cuda() for n in (lq, lk)]
    rq, rk = sum(lq) + pad, sum(lk) + pad
    q = _randn(seed, rq, hq, d, dtype=dtype)
    k = _randn(seed + 1, rk, hk, d, dtype=dtype)
    v = (_randn(seed + 2, rk, hk, d) + 0.25).to(dtype)
    return lq, lk, cu, q, k, v


def _score_error(score, d):
    """Absolute error of a scaled score: float32 products summed by the tensor core."""
    return (d + 16) * E32 * (1 + score) * 4 + 2.0 ** -20


def _close_rounded(got, r, name, dtype, err):
    """One rounding of the output, one of each probability or score gradient that it sums, and `err`."""
    tol = R.rounding(dtype, r[name]) + (1.01 * R.UNIT[dtype] + err) * r[name + "_mag"] + R.TINY[dtype] * r[name + "_all"]
    R.close(got, r[name], tol, name)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case", ATTN_CASES)
def test_attention(case, dtype):
    E = _enc()
    lq, lk, cu, q, k, v = _attn_inputs(case, dtype)
    st = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    plan = E.AttentionPlan(*cu, q.shape[0], k.shape[0], case[2], case[3], case[4], causal=case[5], status=st)
    assert st.tolist() == [0, -1]
    st.fill_(-7)
    out, lse = E.attention(q, k, v, plan, lse=True, status=st)
    if q.shape[0]:
        assert st.tolist() == [0, -1]
    r = R.attention(q, k, v, lq, lk, case[5])
    err = _score_error(r["score"], case[4])
    R.close(lse, r["lse"], err + 8 * E32 * (1 + r["lse"].nan_to_num(neginf=0.0).abs()), "lse")
    _close_rounded(out, r, "out", dtype, 2 * err)
    for _ in range(3):
        assert torch.equal(E.attention(q, k, v, plan), out), "equal calls give equal bits"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case", ATTN_CASES)
def test_attention_gradients(case, dtype):
    E = _enc()
    lq, lk, cu, q, k, v = _attn_inputs(case, dtype, seed=40)
    dout = _randn(45, *q.shape, dtype=dtype)
    plan = E.AttentionPlan(*cu, q.shape[0], k.shape[0], case[2], case[3], case[4], causal=case[5])
    out, lse = E.attention(q, k, v, plan, lse=True)
    st = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    got = E.attention_backward(dout, q, k, v, out, lse, plan, status=st)
    if q.shape[0]:
        assert st.tolist() == [0, -1]
    r = R.attention(q, k, v, lq, lk, case[5], dout=dout, out=out)
    for name, g in zip(("dq", "dk", "dv"), got):
        _close_rounded(g, r, name, dtype, 4 * _score_error(r["score"], case[4]))
    again = E.attention_backward(dout, q, k, v, out, lse, plan)
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "equal calls give equal bits"


def test_attention_gradient_against_differences():
    E = _enc()
    case = ([37, 150], None, 4, 2, 64, True, 0)
    lq, lk, cu, q, k, v = _attn_inputs(case, HF, seed=50)
    dout = _randn(55, *q.shape, dtype=HF)
    plan = E.AttentionPlan(*cu, q.shape[0], k.shape[0], 4, 2, 64, causal=True)
    out, lse = E.attention(q, k, v, plan, lse=True)
    grads = E.attention_backward(dout, q, k, v, out, lse, plan)
    h = 1e-4
    for at in range(3):
        args = [q.double(), k.double(), v.double()]
        step = _randn(56 + at, *args[at].shape).double()
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + h * step, args[at] - h * step
        slope = float(((R.attention(*up, lq, lk, True)["out"] - R.attention(*down, lq, lk, True)["out"]) / (2 * h)
                       * dout.double()).sum())
        g = grads[at].double()
        # float16 gradients: a few roundings of each element, at random signs
        assert abs(slope - float((g * step).sum())) <= 32 * R.UNIT[HF] * float((g * step).norm()) + 1e-3


def test_attention_views_of_one_projection_and_another_stream():
    E = _enc()
    lens, h, hk, d = [100, 333], 4, 2, 80
    rows = sum(lens)
    qkv = _randn(60, rows, h + 2 * hk, d, dtype=BF)
    q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    cu = torch.tensor([0, 100, 433], dtype=torch.int32, device="cuda")
    plan = E.AttentionPlan(cu, cu, rows, rows, h, hk, d)
    out, lse = E.attention(q, k, v, plan, lse=True)
    assert torch.equal(out, E.attention(q.contiguous(), k.contiguous(), v.contiguous(), plan))
    wide = torch.zeros((rows, h + 1, d), dtype=BF, device="cuda")
    E.attention(q, k, v, plan, out=wide[:, 1:])
    assert torch.equal(wide[:, 1:], out) and not wide[:, 0].any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = E.attention(q, k, v, plan, stream=side)
    dout = _randn(61, rows, h, d, dtype=BF)
    side.wait_stream(torch.cuda.current_stream())
    there = E.attention_backward(dout, q, k, v, out, lse, plan, stream=side)
    here = E.attention_backward(dout, q, k, v, out, lse, plan)
    torch.cuda.synchronize()
    assert torch.equal(other, out)
    assert all(torch.equal(a, b) for a, b in zip(here, there))


@pytest.mark.parametrize("causal", [False, True])
def test_attention_other_rows_never_leak(causal):
    # NaN and infinities in the padding and in one sequence stay there
    E = _enc()
    case = ([70, 33, 200], None, 2, 1, 64, causal, 60)
    lq, lk, cu, q, k, v = _attn_inputs(case, BF, seed=70)
    dout = _randn(75, *q.shape, dtype=BF)
    plan = E.AttentionPlan(*cu, q.shape[0], k.shape[0], 2, 1, 64, causal=causal)
    out, lse = E.attention(q, k, v, plan, lse=True)
    grads = E.attention_backward(dout, q, k, v, out, lse, plan)
    bad = [t.clone() for t in (q, k, v, dout)]
    for t in bad:
        t[70:103] = math.nan
        t[303:] = math.inf
        t[320:] = math.nan
    bq, bk, bv, bd = bad
    out2, lse2 = E.attention(bq, bk, bv, plan, lse=True)
    keep = torch.cat([torch.arange(0, 70), torch.arange(103, 303)]).cuda()
    assert torch.equal(out2[keep], out[keep]) and torch.equal(lse2[keep], lse[keep])
    assert out2[70:103].isnan().all() and not out2[303:].any() and (lse2[303:] == -math.inf).all()
    o, s = out.clone(), lse.clone()
    o[70:103], s[70:103] = math.nan, math.nan
    o[303:], s[303:] = math.nan, math.nan
    for a, b in zip(grads, E.attention_backward(bd, bq, bk, bv, o, s, plan)):
        assert torch.equal(a[keep], b[keep]) and not b[303:].any()


def test_attention_scores_far_apart_and_infinite():
    # a growing row maximum (the accumulator is rescaled), scores far below it, and infinities
    E = _enc()
    n, d = 700, 64
    q = torch.ones((n, 1, d), dtype=BF, device="cuda")
    k = torch.zeros((n, 1, d), dtype=BF, device="cuda")
    k[:, 0, 0] = torch.linspace(-900, 900, n, device="cuda").to(BF)
    v = _randn(80, n, 1, d, dtype=BF)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    plan = E.AttentionPlan(cu, cu, n, n, 1, 1, d)
    for kk in (k, k.flip(0), k[torch.randperm(n, device="cuda")]):
        out, lse = E.attention(q, kk, v, plan, lse=True, scale=0.5)
        r = R.attention(q, kk, v, [n], [n], False, scale=0.5)
        R.close(lse, r["lse"], 2.0 ** -20 * 512, "lse")
        _close_rounded(out, r, "out", BF, 2.0 ** -10)
    low = k.clone()
    low[:, 0, 0] = torch.finfo(BF).min                       # every score the type's lowest value
    out, lse = E.attention(q, low, v, plan, lse=True, scale=1e-30)
    r = R.attention(q, low, v, [n], [n], False, scale=1e-30)
    _close_rounded(out, r, "out", BF, 2.0 ** -20)
    neg = k.clone()
    neg[:300, 0, 0] = -math.inf                              # keys that weigh nothing
    out, lse = E.attention(q, neg, v, plan, lse=True, scale=0.01)
    ref = E.AttentionPlan(cu, torch.tensor([0, n - 300], dtype=torch.int32, device="cuda"), n, n - 300, 1, 1, d)
    o2, l2 = E.attention(q, neg[300:].contiguous(), v[300:].contiguous(), ref, lse=True, scale=0.01)
    assert torch.isfinite(out.float()).all()
    R.close(out, o2, 4 * R.UNIT[BF] * o2.double().abs().amax(), "out")
    R.close(lse, l2, 2.0 ** -18 * (1 + l2.double().abs()), "lse")


def test_attention_plan_reports_bad_boundaries_and_pads_everything():
    E = _enc()
    st = torch.empty(2, dtype=torch.int32, device="cuda")
    q = _randn(90, 50, 2, 64, dtype=BF)
    good = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    for bad, at in (([0, 30, 20], 1), ([1, 20, 50], 0), ([0, 20, 51], 1), ([0, -1, 50], 0)):
        b = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for cq, ck in ((b, good), (good, b)):
            plan = E.AttentionPlan(cq, ck, 50, 50, 2, 2, 64, status=st)
            assert st.tolist() == [4, at]
            out, lse = E.attention(q, q, q, plan, lse=True)
            assert not out.any() and (lse == -math.inf).all()


def test_attention_graph_replay_with_new_boundaries():
    E = _enc()
    rows, h, d = 600, 2, 80
    q, k, v = (_randn(91 + i, rows, h, d, dtype=BF) for i in range(3))
    dout = _randn(95, rows, h, d, dtype=BF)
    cu = torch.tensor([0, 600, 600, 600], dtype=torch.int32, device="cuda")
    plan = E.AttentionPlan(cu, cu, rows, rows, h, h, d)

    def step():
        plan.update(cu, cu)
        out, lse = E.attention(q, k, v, plan, lse=True)
        return (out, lse) + E.attention_backward(dout, q, k, v, out, lse, plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step()
    for lens in ([100, 200, 300], [600, 0, 0], [1, 0, 450]):
        cu.copy_(torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int())
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, step()):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ together

def test_encoder_block_and_its_gradients():
    # the block in bfloat16 against the same block from float64 definitions, forward and backward
    from vit_vision_encoder_fusedinputnorm_gb300 import block_example as X
    y, dx, block, fe, batch = X.tower()
    hidden, heads = y.shape[1], block.heads
    x, cos, sin = fe.embed_rope(batch, hidden // heads, 10000.0)
    lens = fe.cu_seqlens(batch, 16)[0].diff().tolist()
    p = {n: t.detach().double().requires_grad_(True) for n, t in block.named_parameters()}
    x64 = x.double().requires_grad_(True)

    def turn(t):
        h = t.shape[2] // 2
        c, s = cos.double()[:, None], sin.double()[:, None]
        return torch.cat([t[..., :h] * c - t[..., h:] * s, t[..., h:] * c + t[..., :h] * s], -1)

    def norm(t, w, b):
        return torch.nn.functional.layer_norm(t, (hidden,), w, b, block.eps)
    rows = x.shape[0]
    h = norm(x64, p["norm1_weight"], p["norm1_bias"])
    q, k, v = (h @ p["qkv.weight"].T + p["qkv.bias"]).view(rows, 3 * heads, -1).split(heads, 1)
    q, k, a, at = turn(q), turn(k), [], 0
    for n in lens:
        z = torch.einsum("qhd,khd->hqk", q[at:at + n], k[at:at + n]) * (hidden // heads) ** -0.5
        a.append(torch.einsum("hqk,khd->qhd", z.softmax(-1), v[at:at + n]))
        at += n
    r = x64 + torch.cat(a).reshape(rows, hidden) @ p["proj.weight"].T + p["proj.bias"]
    h = norm(r, p["norm2_weight"], p["norm2_bias"])
    h = torch.nn.functional.gelu(h @ p["fc1.weight"].T + p["fc1.bias"], approximate="tanh")
    y64 = r + h @ p["fc2.weight"].T + p["fc2.bias"]
    y64.square().mean().backward()

    def rel(a, b):
        return float((a.double() - b).norm() / b.norm())
    # some ten roundings to bfloat16 in a row forward, twice that backward
    assert rel(y, y64.detach()) <= 10 * R.UNIT[BF]
    assert rel(dx, x64.grad) <= 20 * R.UNIT[BF]
    for n, t in block.named_parameters():
        assert rel(t.grad, p[n].grad) <= 20 * R.UNIT[BF], n
    fe.close()


def test_example_runs():
    from vit_vision_encoder_fusedinputnorm_gb300 import block_example as X
    X.main()


@pytest.mark.parametrize("lens", [[700, 300], [1] * 9 + [40], [5, 0, 1000]])
def test_attention_plan_with_room_for_more_sequences(lens):
    # the boundaries' capacity says nothing of how long the sequences are: the same bits either way
    E = _enc()
    rows, hq, hk, d = sum(lens), 4, 2, 80
    q, k, v, do = (_randn(90 + i, rows, h, d, dtype=BF) for i, h in enumerate((hq, hk, hk, hq)))
    results = []
    for room in (0, 50):
        cu = torch.tensor([0] + lens + [0] * room, device="cuda").cumsum(0).int()
        plan = E.AttentionPlan(cu, cu, rows, rows, hq, hk, d, causal=True)
        out, lse = E.attention(q, k, v, plan, lse=True)
        results.append((out, lse) + E.attention_backward(do, q, k, v, out, lse, plan))
    assert all(torch.equal(x, y) for x, y in zip(*results))
