"""Encoder-block operators, what the torch side has to see to itself (no GPU: the library's calls are
stand-ins where one is reached)."""
import contextlib
import importlib.util

import pytest

torch = pytest.importorskip("torch")

from vit_vision_encoder_fusedinputnorm_gb300 import binding as B  # noqa: E402
from vit_vision_encoder_fusedinputnorm_gb300 import encoder as E  # noqa: E402


def test_the_table_rotation_refuses_other_types_and_tables(monkeypatch):
    # the library's call takes addresses: it would turn any other type's bits as bfloat16
    def never(*args):
        raise AssertionError("the library was called")
    monkeypatch.setattr(B, "vitfe_rope_apply", never)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: None)
    x, cos = torch.zeros(4, 2, 16, dtype=torch.bfloat16), torch.zeros(4, 8)
    for dtype in (torch.float16, torch.float32):
        with pytest.raises(TypeError):
            E.TableRotation.apply(x.to(dtype), cos, cos)
        with pytest.raises(TypeError):
            E.EncoderBlock(32, 2, 64, dtype=dtype, device="cpu")
    for bad in (cos[:3], cos[:, :4], cos.double(), cos.bfloat16(), torch.zeros(8, 4).t(), torch.zeros(4, 16)[:, ::2], cos[0]):
        with pytest.raises(ValueError):
            E.TableRotation.apply(x, bad, cos)
        with pytest.raises(ValueError):
            E.TableRotation.apply(x, cos, bad)
    with pytest.raises(ValueError):
        E.TableRotation.apply(x[0], cos, cos)
    with pytest.raises(ValueError):
        E.TableRotation.apply(x, cos, cos)              # not on the GPU


class _Plan:
    version = 1


def _attention_stand_in(monkeypatch):
    """attention and its gradients by torch, for one head and sequence."""
    def forward(q, k, v, plan, scale=None, lse=False, **_):
        s = (q[:, 0] @ k[:, 0].T) * (1.0 if scale is None else scale)
        return (s.softmax(1) @ v[:, 0])[:, None], s.logsumexp(1)[:, None]

    def backward(dout, q, k, v, out, lse, plan, scale=None, **_):
        p = ((q[:, 0] @ k[:, 0].T) * (1.0 if scale is None else scale) - lse).exp()
        ds = p * (dout[:, 0] @ v[:, 0].T - (dout * out)[:, 0].sum(1, keepdim=True)) * (1.0 if scale is None else scale)
        return (ds @ k[:, 0])[:, None], (ds.T @ q[:, 0])[:, None], (p.T @ dout[:, 0])[:, None]
    monkeypatch.setattr(E, "attention", forward)
    monkeypatch.setattr(E, "attention_backward", backward)


def test_gradients_across_an_update_of_the_plan_are_refused(monkeypatch):
    _attention_stand_in(monkeypatch)
    plan = _Plan()
    q, k, v = (torch.randn(5, 1, 8, requires_grad=True) for _ in range(3))
    E.PackedAttention.apply(q, k, v, plan, 0.3).sum().backward()
    assert q.grad is not None
    out = E.PackedAttention.apply(q, k, v, plan, 0.3)
    plan.version += 1                                    # what update does
    with pytest.raises(RuntimeError):
        out.sum().backward()


def _all_functions(monkeypatch):
    """Each autograd function over stand-ins: name -> a scalar of x."""
    _attention_stand_in(monkeypatch)
    monkeypatch.setattr(E, "layer_norm", lambda x, w, b, eps, stats: (x * w, x.mean(1), x.mean(1)))
    monkeypatch.setattr(E, "layer_norm_backward", lambda dy, x, m, r, w, params: (dy * w, dy.sum(0), dy.sum(0)))
    monkeypatch.setattr(E, "mrope_apply", lambda q, k, pos, axes, theta=1.0, inverse=False: tuple(
        None if t is None else (-1 if inverse else 1) * t.flip(-1) for t in (q, k)))
    monkeypatch.setattr(E.TableRotation, "_turn", staticmethod(lambda x, cos, sin: x * cos + x.flip(-1) * sin))
    one, w, pos = torch.ones(4, 8), torch.ones(8), torch.zeros(3, 4, dtype=torch.int32)

    def heads(x):
        return x[:, None]
    return {
        "LayerNorm": lambda x: E.LayerNorm.apply(x, w, w, 1e-5),
        "MropeRotation": lambda x: torch.cat(E.MropeRotation.apply(heads(x), heads(x), pos, [0] * 4, 10.0)),
        "TableRotation": lambda x: E.TableRotation.apply(heads(x), one[:, None], one[:, None]),
        "PackedAttention": lambda x: E.PackedAttention.apply(heads(x), heads(x), heads(x), _Plan(), 0.3),
    }


def test_gradients_of_gradients_are_refused(monkeypatch):
    # backward's results carry no graph of their own: without a refusal its terms would be missing
    for name, f in _all_functions(monkeypatch).items():
        x = torch.randn(4, 8, requires_grad=True)
        g, = torch.autograd.grad((f(x).square().sum() + x.pow(3).sum()), x, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()
        f(x).square().sum().backward()                   # the first order is as it was
        assert x.grad is not None, name


class _Stream:
    cuda_stream = 5

    def __init__(self, device_index):
        self.device_index = device_index


def test_a_raw_stream_handle_is_one_of_the_tensors_gpu(monkeypatch):
    # the tensors' GPU is 1, the current one is 0: the handle has to be made current on 1
    made, launched = [], []

    class Made:
        def __init__(self, handle, device=None):
            made.append((handle, device))

        def __enter__(self):
            return self

        def __exit__(self, *_):
            return False
    monkeypatch.setattr(E, "_device", lambda *t: 1)
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Made)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: _Stream(1))
    monkeypatch.setattr(E, "_raw_stream", lambda d: _Stream.cuda_stream)
    monkeypatch.setattr(E, "_launch", lambda name, device, *a: launched.append((name, device)))
    x, stat, pos = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(4), torch.zeros(3, 4, dtype=torch.int32)
    q, cu = x.view(4, 2, 8), torch.tensor([0, 4], dtype=torch.int32)
    lse, one = torch.zeros(4, 2), torch.ones(1, dtype=torch.int32)
    plan = E.AttentionPlan(cu, cu, 4, 4, 2, 2, 8, stream=77)
    calls = [
        lambda s: plan.update(cu, cu, stream=s),
        lambda s: E.layer_norm(x, stream=s),
        lambda s: E.layer_norm_backward(x, x, stat, stat, stream=s),
        lambda s: E.mrope_positions(torch.zeros(1, 4, dtype=torch.int32), one, None, None, 4, stream=s),
        lambda s: E.mrope_apply(None, q, pos, [0] * 4, stream=s),
        lambda s: E.attention(q, q, q, plan, stream=s),
        lambda s: E.attention_backward(q, q, q, q, q, lse, plan, stream=s),
    ]
    for f in calls:
        f(77)
    assert made == [(77, 1)] * (len(calls) + 1) and [d for _, d in launched] == [1] * (len(calls) + 1)
    for f in calls:                                      # a stream of another GPU is an error
        with pytest.raises(ValueError):
            f(_Stream(0))


@pytest.mark.parametrize("which", ["q", "k", "both"])
def test_the_rotation_of_q_or_k_alone_has_a_gradient(monkeypatch, which):
    _all_functions(monkeypatch)
    pos = torch.zeros(3, 4, dtype=torch.int32)
    q, k = (torch.randn(4, 1, 8, requires_grad=which in (n, "both")) if which in (n, "both") else None for n in "qk")
    oq, ok = E.MropeRotation.apply(q, k, pos, [0] * 4, 10.0)
    up = torch.randn(4, 1, 8)
    sum((o * up).sum() for o in (oq, ok) if o is not None).backward()
    for x, o in ((q, oq), (k, ok)):
        assert (x is None) == (o is None)
        if x is not None:
            assert torch.equal(x.grad, -up.flip(-1))     # the stand-in's inverse


def test_status_pairs_and_counts_of_the_wrong_size_or_type_are_refused(monkeypatch):
    # a kernel writes two words of status and reads one of a count, whatever the tensor holds
    launched = []
    monkeypatch.setattr(E, "_device", lambda *t: 1)
    monkeypatch.setattr(E, "_current", lambda stream, x: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: _Stream(1))
    monkeypatch.setattr(E, "_raw_stream", lambda d: _Stream.cuda_stream)
    monkeypatch.setattr(E, "_launch", lambda name, *a: launched.append(name))
    x = torch.zeros(4, 2, 8, dtype=torch.bfloat16)
    cu, lse, spans = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(4, 2), torch.zeros(1, 4, dtype=torch.int32)
    one, good = torch.ones(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    plan = E.AttentionPlan(cu, cu, 4, 4, 2, 2, 8, status=good)
    calls = [
        lambda s: E.AttentionPlan(cu, cu, 4, 4, 2, 2, 8, status=s),
        lambda s: plan.update(cu, cu, status=s),
        lambda s: E.mrope_positions(spans, one, None, None, 4, status=s),
        lambda s: E.attention(x, x, x, plan, status=s),
        lambda s: E.attention_backward(x, x, x, x, x, lse, plan, status=s),
    ]
    for f in calls:
        f(good)
    del launched[:]
    for bad in (one, good.long(), good.float(), torch.zeros(4, dtype=torch.int32)[::2]):
        for f in calls:
            with pytest.raises(ValueError):
                f(bad)
    none, items = torch.zeros(0, dtype=torch.int32), torch.zeros(24, dtype=torch.uint8)
    for n, m in ((none, one), (one.long(), one), (one, none), (one, one.float())):
        with pytest.raises(ValueError):
            E.mrope_positions(spans, n, items, m, 4)
    assert not launched


def test_the_module_imports_under_a_torch_without_cuda(monkeypatch):
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name)
    spec = importlib.util.spec_from_file_location(E.__name__ + "_again", E.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    with pytest.raises(ValueError):
        again.layer_norm(torch.zeros(2, 8))              # not on a GPU


def test_a_plan_used_on_another_stream_is_recorded_there(monkeypatch):
    recorded = []
    now = _Stream(1)
    monkeypatch.setattr(E, "_device", lambda *t: 1)
    monkeypatch.setattr(E, "_current", lambda stream, x: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: now)
    monkeypatch.setattr(E, "_raw_stream", lambda d: now.cuda_stream)
    monkeypatch.setattr(E, "_launch", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t, s)))
    x, cu = torch.zeros(4, 2, 8, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    plan = E.AttentionPlan(cu, cu, 4, 4, 2, 2, 8)
    E.attention(x, x, x, plan)
    E.attention_backward(x, x, x, x, x, torch.zeros(4, 2), plan)
    assert not recorded                                  # its own stream
    now.cuda_stream = 9
    E.attention(x, x, x, plan)
    E.attention_backward(x, x, x, x, x, torch.zeros(4, 2), plan)
    assert [(t is plan.buffer, s is now) for t, s in recorded] == [(True, True)] * 2
