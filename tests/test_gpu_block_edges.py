"""Encoder-block operators on the GPU where they could go wrong without an error: memory used again by
the next call, waits that run out, rows far from zero, plans that change, layouts at the edge."""
import math

import pytest

torch = pytest.importorskip("torch")

import block_reference as R  # noqa: E402
import test_gpu_block_ops as T  # noqa: E402

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


def _cu(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).int().cuda()


def test_attention_backward_takes_the_row_values_of_its_own_call():
    # calls back to back in one workspace, each with row values of its own
    from vit_vision_encoder_fusedinputnorm_gb300 import binding as B
    E = _enc()
    lens, h, d = [700, 129, 384], 4, 64
    rows, cu = sum(lens), _cu(lens)
    plan = E.AttentionPlan(cu, cu, rows, rows, h, h, d, causal=True)
    batches, want = [], []
    for i in range(3):
        q, k, v, do = ((1 + i) * _randn(10 * i + j, rows, h, d) for j in range(4))
        q, k, v, do = (t.to(BF) for t in (q, k, v, do))
        out, lse = E.attention(q, k, v, plan, lse=True)
        batches.append((q, k, v, do, out, lse))
        want.append(E.attention_backward(do, q, k, v, out, lse, plan))
    torch.cuda.synchronize()
    work = torch.empty(B.vitfe_attention_backward_workspace(plan.shape), dtype=torch.uint8, device="cuda")
    got = []
    for r in range(10):
        q, k, v, do, out, lse = batches[r % 3]
        g = [torch.empty_like(t) for t in (q, k, v)]
        n = h * d
        B.vitfe_attention_backward(plan.shape, plan.buffer, do, n, q, n, k, n, v, n, out, n, lse, d ** -0.5, g[0], n,
                                   g[1], n, g[2], n, work, None, torch.cuda.current_stream())
        got.append(g)
    torch.cuda.synchronize()
    for r, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[r % 3])), r


# ------------------------------------------------------------------ waits that run out

EXPIRED = [6, -1]
STALL_CASES = [  # lens_q, lens_k, q heads, k heads, head_dim, causal
    ([300, 40], [300, 40], 2, 2, 80, False),                  # two-tile items
    ([1] * 5, [1, 700, 2500, 129, 5000], 4, 2, 128, True),    # one-tile items, cut and joined
]


def _stall(monkeypatch, on):
    if on:
        monkeypatch.setenv("VITFE_WAIT_LIMIT_MS", "50")
        monkeypatch.setenv("VITFE_TEST_STALL_BLOCK_LOADS", "1")
    else:
        monkeypatch.delenv("VITFE_WAIT_LIMIT_MS")
        monkeypatch.delenv("VITFE_TEST_STALL_BLOCK_LOADS")


def _stall_inputs(case):
    E = _enc()
    lq, lk, hq, hk, d, causal = case
    plan = E.AttentionPlan(_cu(lq), _cu(lk), sum(lq), sum(lk), hq, hk, d, causal=causal)
    q, do = (_randn(s, sum(lq), hq, d, dtype=BF) for s in (60, 61))
    k, v = (_randn(s, sum(lk), hk, d, dtype=BF) for s in (62, 63))
    return E, plan, q, k, v, do


@pytest.mark.parametrize("case", STALL_CASES)
def test_attention_reports_a_wait_that_runs_out_and_then_works_again(monkeypatch, case):
    # tiles that never come: every role leaves by the short limit, and the context stays usable
    E, plan, q, k, v, do = _stall_inputs(case)
    st = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    want = E.attention(q, k, v, plan, lse=True)
    grads = E.attention_backward(do, q, k, v, *want, plan)
    _stall(monkeypatch, True)
    missing = E.attention(q, k, v, plan, lse=True, status=st)
    assert st.tolist() == EXPIRED
    st.fill_(-7)
    missing += E.attention_backward(do, q, k, v, *want, plan, status=st)
    assert st.tolist() == EXPIRED
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), missing):      # nor does it take the status to see it
        assert t.isnan().all(), name
    _stall(monkeypatch, False)
    got = E.attention(q, k, v, plan, lse=True, status=st)
    assert st.tolist() == [0, -1]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    st.fill_(-7)
    again = E.attention_backward(do, q, k, v, *want, plan, status=st)
    assert st.tolist() == [0, -1]
    assert all(torch.equal(a, b) for a, b in zip(again, grads))


def test_attention_backward_on_a_long_stretch_of_whole_blocks(monkeypatch):
    # eight sequences of whole key blocks before one that ends inside a block: nothing is cleaned for longer
    # than the limit, which bounds one wait and not the call
    E = _enc()
    lens, h, d = [16384] * 8 + [100], 16, 64
    rows = sum(lens)
    q, k, v, do = (_randn(64 + i, rows, h, d, dtype=BF) for i in range(4))
    plan = E.AttentionPlan(_cu(lens), _cu(lens), rows, rows, h, h, d)
    out, lse = E.attention(q, k, v, plan, lse=True)
    st = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    want = E.attention_backward(do, q, k, v, out, lse, plan, status=st)
    assert st.tolist() == [0, -1]
    monkeypatch.setenv("VITFE_WAIT_LIMIT_MS", "4")
    got = E.attention_backward(do, q, k, v, out, lse, plan, status=st)
    assert st.tolist() == [0, -1]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,width", [(3, 100), (5000, 40), (4000, 1280), (700, 4000), (400, 9001)])
def test_layer_norm_gradients_of_a_wait_that_runs_out_are_nan(monkeypatch, rows, width):
    E = _enc()
    x, dy, w = _randn(70, rows, width, dtype=BF), _randn(71, rows, width, dtype=BF), _randn(72, width)
    _, mean, rstd = E.layer_norm(x, w, stats=True)
    want = E.layer_norm_backward(dy, x, mean, rstd, w)
    _stall(monkeypatch, True)
    for t in E.layer_norm_backward(dy, x, mean, rstd, w):
        assert t.isnan().all()
    _stall(monkeypatch, False)
    got = E.layer_norm_backward(dy, x, mean, rstd, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ layer norm far from zero

@pytest.mark.parametrize("offset", [100.0, 1e4, -1e5])
@pytest.mark.parametrize("rows,width", [(64, 1280), (40, 77), (9, 9000)])
def test_layer_norm_gradients_of_rows_far_from_zero(rows, width, offset):
    # the mean and rstd are given, so nothing of the offset may be left in the gradients.  Roundings, each E32
    # of what it acts on: x - mean, xh, the products and at most 64 + 10 of a sum's additions (32 pairs of
    # columns a thread and the exchanges) over magnitudes whose mean is at most their largest / 2; the rows'
    # sums take at most 16 additions each (rows / groups) and 8 of the groups
    E = _enc()
    x, dy, w = _randn(80, rows, width) + offset, _randn(81, rows, width), _randn(82, width)
    _, mean, rstd = E.layer_norm(x, w, stats=True)
    dx, dw, db = E.layer_norm_backward(dy, x, mean, rstd, w)
    rx, rdw, rdb, xh, g = R.layer_norm_backward(dy, x, mean, rstd, w)
    top = g.abs().amax(1, keepdim=True)
    mag = rstd.double()[:, None] * (g.abs() + top * (1 + xh.abs() * xh.abs().amax(1, keepdim=True)))
    R.close(dx, rx, 48 * E32 * mag, "dx")
    R.close(dw, rdw, 32 * E32 * (dy.double().abs() * xh.abs()).sum(0), "dweight")
    R.close(db, rdb, 32 * E32 * dy.double().abs().sum(0), "dbias")


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("width", [41, 47, 896, 1280, 3584, 9001])
def test_layer_norm_of_rows_of_equal_values_is_the_bias(width, dtype):
    # values of few bits: their sum is exact, so the mean is the value and nothing deviates
    E = _enc()
    values = torch.tensor([0.0, 1.0, 3.0, 7.0, -5.0, 100.0, 1000.0, 200.0, -1.5], device="cuda")
    x = values[:, None].expand(-1, width).contiguous().to(dtype)
    w, b = _randn(83, width), _randn(84, width)
    y, mean, rstd = E.layer_norm(x, w, b, 1e-6, stats=True)
    assert torch.equal(mean, values)
    assert torch.equal(y, b.to(dtype).expand(len(values), -1))
    assert torch.equal(rstd, rstd[:1].expand(len(values))) and abs(float(rstd[0]) * 1e-3 - 1) <= 8 * E32 * 2


# ------------------------------------------------------------------ plans and autograd

def test_gradients_across_an_update_of_the_plan_are_refused():
    E = _enc()
    rows, h, d = 300, 2, 64
    q, k, v = (_randn(90 + i, rows, h, d, dtype=BF).requires_grad_(True) for i in range(3))
    plan = E.AttentionPlan(_cu([100, 200]), _cu([100, 200]), rows, rows, h, h, d)
    out = E.PackedAttention.apply(q, k, v, plan, None)
    plan.update(_cu([250, 50]), _cu([250, 50]))
    with pytest.raises(RuntimeError):
        out.float().sum().backward()
    E.PackedAttention.apply(q, k, v, plan, None).float().sum().backward()
    dout = torch.ones((rows, h, d), dtype=BF, device="cuda")
    out, lse = E.attention(q.detach(), k.detach(), v.detach(), plan, lse=True)
    for t, g in zip((q, k, v), E.attention_backward(dout, q.detach(), k.detach(), v.detach(), out, lse, plan)):
        assert torch.equal(t.grad, g)


@pytest.mark.parametrize("dtype", [BF, SF])
@pytest.mark.parametrize("which", ["q", "k", "both"])
def test_mrope_rotation_and_its_gradient(which, dtype):
    E = _enc()
    rows, d, axes = 21, 32, E.section_axes((6, 5, 5))
    pos = torch.randint(0, 3000, (3, rows), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    q = _randn(95, rows, 4, d, dtype=dtype).requires_grad_(True) if which != "k" else None
    k = _randn(96, rows, 2, d, dtype=dtype).requires_grad_(True) if which != "q" else None
    oq, ok = E.MropeRotation.apply(q, k, pos, axes, 1e4)
    up = {2: _randn(97, rows, 2, d, dtype=dtype), 4: _randn(98, rows, 4, d, dtype=dtype)}
    sum((o * up[o.shape[1]]).float().sum() for o in (oq, ok) if o is not None).backward()
    for x, o in ((q, oq), (k, ok)):
        if x is None:
            assert o is None
            continue
        dx = up[o.shape[1]]
        for got, ref in ((o, R.rotate(x.detach(), pos, axes, 1e4)), (x.grad, R.rotate(dx, pos, axes, 1e4, inverse=True))):
            # angles to 2^-25 turns (float32 phases), then products in float32
            R.close(got.detach(), ref, R.rounding(dtype, ref) + (8 * E32 + 2 * math.pi * 2.0 ** -25) * 2 * 5.0, "rotated")


@pytest.mark.parametrize("theta", [500.0, 1e4, 1e6])
@pytest.mark.parametrize("d", [64, 128, 512])
def test_mrope_angles_are_within_the_stated_bound(theta, d):
    # 2^-26 turns + position * 2^-53 turns; then a sine and a cosine (4 units), two products and a sum in float32,
    # and the float64 reference's own angle (its product's rounding, half a unit of 2^-52, and its exponent's)
    E = _enc()
    pos = torch.tensor([[1, 1000, 32768, 10 ** 6, 8 * 10 ** 6 + 1, 10 ** 8, 2 ** 31 - 1, 2 ** 31 - 2]], dtype=torch.int32)
    rows = pos.shape[1]
    x = torch.zeros((rows, 1, d), device="cuda")
    x[..., :d // 2] = 1.0                                # cos in the first half, sin in the second
    y, _ = E.mrope_apply(x, None, pos.cuda(), [0] * (d // 2), theta=theta)
    at = pos[0].double().cuda()[:, None, None]
    tol = 2 * math.pi * (2.0 ** -26 + at * 2.0 ** -53) + 8 * E32 + at * 2.0 ** -50
    R.close(y, R.rotate(x, pos, [0] * (d // 2), theta), tol, "angles")


# ------------------------------------------------------------------ layouts

def _bytes_off(rows, width, pad, dtype, seed):
    """[rows][width] inside wider rows, `pad` elements in."""
    return _randn(seed, rows, width + pad + 9, dtype=dtype)[:, pad:pad + width]


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("width,pads", [(1280, (0, 0)), (1280, (8, 3)), (1280, (1, 0)), (77, (2, 5)), (2049, (0, 7)),
                                        (64, (8, 16)), (9000, (3, 4))])
def test_layer_norm_gradients_of_rows_inside_wider_ones(width, pads, dtype):
    # x and dout at different distances from 16 bytes, each: the same values as of dense rows
    E = _enc()
    rows = 29
    x, dy = (_bytes_off(rows, width, p, dtype, 100 + i) for i, p in enumerate(pads))
    w = _randn(102, width)
    _, mean, rstd = E.layer_norm(x, w, stats=True)
    dx, dw, db = E.layer_norm_backward(dy, x, mean, rstd, w)
    rx, rdw, rdb, xh, g = R.layer_norm_backward(dy, x, mean, rstd, w)
    top = g.abs().amax(1, keepdim=True)
    mag = rstd.double()[:, None] * (g.abs() + top * (1 + xh.abs() * xh.abs().amax(1, keepdim=True)))
    R.close(dx, rx, R.rounding(dtype, rx) + 48 * E32 * mag, "dx")          # roundings as of rows far from zero
    R.close(dw, rdw, 32 * E32 * (dy.double().abs() * xh.abs()).sum(0), "dweight")
    R.close(db, rdb, 32 * E32 * dy.double().abs().sum(0), "dbias")


@pytest.mark.parametrize("width", [1280, 77, 9000])
@pytest.mark.parametrize("over", ["x", "dout"])
def test_layer_norm_gradient_over_its_input(width, over):
    from vit_vision_encoder_fusedinputnorm_gb300 import binding as B
    E = _enc()
    rows = 2000
    x, dy, w = _randn(110, rows, width, dtype=BF), _randn(111, rows, width, dtype=BF), _randn(112, width)
    _, mean, rstd = E.layer_norm(x, w, stats=True)
    want = E.layer_norm_backward(dy, x, mean, rstd, w)
    dx = x if over == "x" else dy
    dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    size = B.vitfe_layer_norm_workspace(rows, width)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    B.vitfe_layer_norm_backward(dy, width, x, width, B.VITFE_BF16, rows, width, w, B.VITFE_F32, mean, rstd, dx, width,
                                dw, db, work, size, torch.cuda.current_stream())
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), want))


@pytest.mark.parametrize("params", ["both", "weight", "bias", "none"])
def test_layer_norm_function_with_and_without_parameters(params):
    E = _enc()
    x = _randn(115, 33, 96).requires_grad_(True)
    w = _randn(116, 96, dtype=BF).requires_grad_(True) if params in ("both", "weight") else None
    b = _randn(117, 96, dtype=BF).requires_grad_(True) if params in ("both", "bias") else None
    up = _randn(118, 96, 33).t()                                # a gradient that is not contiguous
    y = E.LayerNorm.apply(x, w, b, 1e-5)
    y.backward(up)
    _, mean, rstd = E.layer_norm(x.detach(), w, b, 1e-5, stats=True)
    dx, dw, db = E.layer_norm_backward(up.contiguous(), x.detach(), mean, rstd, w)
    assert torch.equal(x.grad, dx)
    assert w is None or torch.equal(w.grad, dw.to(BF))
    assert b is None or torch.equal(b.grad, db.to(BF))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scale", [0.03, 0.4])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_and_its_gradients_with_a_scale_and_rows_inside_wider_ones(causal, scale, dtype):
    E = _enc()
    lens, hq, hk, d = [130, 257, 1], 4, 2, 72
    rows = sum(lens)

    def wide(seed, h):
        return _randn(seed, rows, h + 1, d, dtype=dtype)[:, 1:]
    q, k, v, do = wide(120, hq), wide(121, hk), wide(122, hk), wide(123, hq)
    plan = E.AttentionPlan(_cu(lens), _cu(lens), rows, rows, hq, hk, d, causal=causal)
    out, lse = E.attention(q, k, v, plan, scale=scale, lse=True, out=wide(124, hq))
    got = E.attention_backward(do, q, k, v, out, lse, plan, scale=scale)
    r = R.attention(q, k, v, lens, lens, causal, scale=scale, dout=do, out=out)
    err = T._score_error(r["score"], d)
    T._close_rounded(out, r, "out", dtype, 2 * err)
    for name, g in zip(("dq", "dk", "dv"), got):
        T._close_rounded(g, r, name, dtype, 4 * err)


def test_packed_attention_function_takes_a_scale_and_any_gradient():
    E = _enc()
    lens, h, d = [100, 60], 2, 64
    rows = sum(lens)
    q, k, v = (_randn(130 + i, rows, h, d, dtype=BF).requires_grad_(True) for i in range(3))
    plan = E.AttentionPlan(_cu(lens), _cu(lens), rows, rows, h, h, d)
    up = _randn(133, h, rows, d, dtype=BF).transpose(0, 1)
    E.PackedAttention.apply(q, k, v, plan, 0.2).backward(up)
    out, lse = E.attention(q.detach(), k.detach(), v.detach(), plan, scale=0.2, lse=True)
    want = E.attention_backward(up.contiguous(), q.detach(), k.detach(), v.detach(), out, lse, plan, scale=0.2)
    assert all(torch.equal(t.grad, g) for t, g in zip((q, k, v), want))


def test_plans_made_again_give_the_same_bits():
    # the order of equal items in a plan may vary from one to the next; what is cut and joined does not
    E = _enc()
    lq, lk, hq, hk, d = [1, 3, 1, 1, 200, 1] * 4, [4000, 4097, 700, 4000, 4000, 2500] * 4, 8, 2, 128
    q, do = (_randn(s, sum(lq), hq, d, dtype=BF) for s in (134, 135))
    k, v = (_randn(s, sum(lk), hk, d, dtype=BF) for s in (136, 137))
    cq, ck = _cu(lq), _cu(lk)
    plan = E.AttentionPlan(cq, ck, sum(lq), sum(lk), hq, hk, d, causal=True)
    want = None
    for _ in range(8):
        plan.update(cq, ck)
        out, lse = E.attention(q, k, v, plan, lse=True)
        got = (out, lse) + E.attention_backward(do, q, k, v, out, lse, plan)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ offsets past 32 bits

def _normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=BF, device="cuda").normal_(generator=g)


def test_layer_norm_past_two_to_the_31_elements():
    E = _enc()
    rows, width, tail = 140000, 16384, 50
    x = _normal(140, rows, width)
    dy = torch.zeros_like(x)
    dy[-tail:] = _normal(141, tail, width)
    w = _randn(142, width)
    y, mean, rstd = E.layer_norm(x, w, stats=True)
    y1, m1, r1 = E.layer_norm(x[-tail:], w, stats=True)
    assert torch.equal(y[-tail:], y1) and torch.equal(mean[-tail:], m1) and torch.equal(rstd[-tail:], r1)
    dx, dw, db = E.layer_norm_backward(dy, x, mean, rstd, w)
    assert torch.equal(dx[-tail:], E.layer_norm_backward(dy[-tail:], x[-tail:], m1, r1, w)[0])
    assert not dx[:-tail].any()
    _, rdw, rdb, xh, _ = R.layer_norm_backward(dy[-tail:], x[-tail:], m1, r1, w)
    a = dy[-tail:].double().abs()
    R.close(dw, rdw, 32 * E32 * (a * xh.abs()).sum(0), "dweight")
    R.close(db, rdb, 32 * E32 * a.sum(0), "dbias")


def test_mrope_past_two_to_the_31_elements():
    E = _enc()
    rows, tail, axes = (1 << 20) + 77, 40, E.section_axes((24, 20, 20))
    q, k = _normal(143, rows, 16, 128), _normal(144, rows, 1, 128)
    pos = torch.arange(3 * rows, dtype=torch.int32, device="cuda").view(3, rows) % 40000
    oq, ok = E.mrope_apply(q, k, pos, axes)
    tq, tk = E.mrope_apply(q[-tail:].contiguous(), k[-tail:].contiguous(), pos[:, -tail:].contiguous(), axes)
    assert torch.equal(oq[-tail:], tq) and torch.equal(ok[-tail:], tk)


def test_attention_over_caches_past_two_to_the_31_elements():
    E = _enc()
    lens, hq, hk, d = [1100000, 700000, 300000, 5000, 777], 16, 8, 128
    rows = sum(lens)
    k, v, q = _normal(145, rows, hk, d), _normal(146, rows, hk, d), _randn(147, len(lens), hq, d, dtype=BF)
    plan = E.AttentionPlan(_cu([1] * len(lens)), _cu(lens), len(lens), rows, hq, hk, d, causal=True)
    out, lse = E.attention(q, k, v, plan, lse=True)
    at = rows
    for i in reversed(range(len(lens))):
        n, at = lens[i], at - lens[i]
        if n > 400000:
            continue
        r = R.attention(q[i:i + 1], k[at:at + n], v[at:at + n], [1], [n], True)
        err = T._score_error(r["score"], d)
        R.close(lse[i:i + 1], r["lse"], err + 8 * E32 * (1 + r["lse"].abs()), "lse")
        T._close_rounded(out[i:i + 1], r, "out", BF, 2 * err)


def test_attention_gradients_past_two_to_the_31_elements():
    E = _enc()
    n, seqs, h, d = 128, 8300, 16, 128
    rows = n * seqs + 60
    lens = [n] * seqs + [60]
    q, k, v, do = (_normal(148 + i, rows, h, d) for i in range(4))
    plan = E.AttentionPlan(_cu(lens), _cu(lens), rows, rows, h, h, d, causal=True)
    out, lse = E.attention(q, k, v, plan, lse=True)
    got = E.attention_backward(do, q, k, v, out, lse, plan)
    last = [t[-60:].contiguous() for t in (q, k, v, do)]
    alone = E.AttentionPlan(_cu([60]), _cu([60]), 60, 60, h, h, d, causal=True)
    o1, l1 = E.attention(*last[:3], alone, lse=True)
    assert torch.equal(out[-60:], o1) and torch.equal(lse[-60:], l1)
    for a, b in zip(got, E.attention_backward(last[3], *last[:3], o1, l1, alone)):
        assert torch.equal(a[-60:], b)


# ------------------------------------------------------------------ streams

def test_a_plan_dropped_before_its_call_has_run_on_another_stream():
    # its memory is not handed out again before that call is done (what would be, is zeroed: an empty plan)
    E = _enc()
    rows, h, d = 700, 2, 64
    cu = _cu([rows])
    q, k, v = (_randn(150 + i, rows, h, d, dtype=BF) for i in range(3))
    do = _randn(153, rows, h, d, dtype=BF)
    keep = E.AttentionPlan(cu, cu, rows, rows, h, h, d)
    want, lse = E.attention(q, k, v, keep, lse=True)
    grads = E.attention_backward(do, q, k, v, want, lse, keep)
    side, size = torch.cuda.Stream(), keep.buffer.numel()
    for inside in (False, True):
        plan = E.AttentionPlan(cu, cu, rows, rows, h, h, d)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)               # some 0.1 s: the call below starts behind it
        if inside:
            with torch.cuda.stream(side):
                out = E.attention(q, k, v, plan)
                got = E.attention_backward(do, q, k, v, want, lse, plan)
        else:
            out = E.attention(q, k, v, plan, stream=side)
            got = E.attention_backward(do, q, k, v, want, lse, plan, stream=side)
        del plan
        taken = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(20)]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and len(taken) == 20
        assert all(torch.equal(a, b) for a, b in zip(got, grads))
