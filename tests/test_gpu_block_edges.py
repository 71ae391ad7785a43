"""Encoder-block operators on the GPU where they could go wrong without an error: memory used again by
the next call, waits that run out, rows far from zero, plans that change, layouts at the edge."""
import math

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
            R.close(got, ref, R.rounding(dtype, ref) + (8 * E32 + 2 * math.pi * 2.0 ** -25) * 2 * 5.0, "rotated")


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
