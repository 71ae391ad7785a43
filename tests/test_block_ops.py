"""Refusals of the encoder-block operators: host validation, before anything is launched (no GPU)."""
import ctypes

import pytest

from vit_vision_encoder_fusedinputnorm_gb300 import binding as B
from vit_vision_encoder_fusedinputnorm_gb300 import build as vbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    vbuild.build()


def _refused(fn, args, code):
    with pytest.raises(B.VitfeError) as e:
        fn(*args)
    assert e.value.code == code, (fn.__name__, args)


def _with(base, **changes):
    d = dict(base, **changes)
    return list(d.values())


NORM = dict(x=16, xs=64, dtype=0, rows=4, width=64, w=16, b=16, pdtype=2, eps=1e-6, out=16, os=64, mean=16, rstd=16)
GRAD = dict(dout=16, ds=64, x=16, xs=64, dtype=0, rows=4, width=64, w=16, pdtype=2, mean=16, rstd=16, dx=16, dxs=64,
            dw=16, db=16, work=16, size=1 << 20)
POS = dict(spans=16, n=16, cap=4, items=16, n_items=16, cap_items=4, merge=2, rows=10, pos=16, status=16)
ROPE = dict(pos=16, axes=3, axis=bytes(32), rot=64, theta=1e4, inv=0, rows=4, d=64, dtype=0, q=16, hq=2, qs=128, qo=16,
            qos=128, k=16, hk=1, ks=64, ko=16, kos=64)


def test_layer_norm_refusals():
    inval = [dict(x=None), dict(out=None), dict(xs=63), dict(os=63), dict(rows=-1), dict(rows=1 << 31), dict(width=0),
             dict(dtype=3), dict(pdtype=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
             dict(x=17), dict(out=17), dict(w=18), dict(b=18), dict(mean=18), dict(rstd=18)]
    for c in inval:
        _refused(B.vitfe_layer_norm, _with(NORM, **c), 1)
    _refused(B.vitfe_layer_norm, _with(NORM, width=16385, xs=16385, os=16385), 7)
    for c in [dict(x=None), dict(dout=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(work=None),
              dict(work=24), dict(size=4 * 64), dict(xs=10), dict(ds=10), dict(dxs=10), dict(dw=18), dict(db=18),
              dict(dtype=9), dict(rows=-2)]:
        _refused(B.vitfe_layer_norm_backward, _with(GRAD, **c), 1)
    _refused(B.vitfe_layer_norm_backward, _with(GRAD, width=20000, xs=20000, ds=20000, dxs=20000), 7)
    assert B.vitfe_layer_norm_workspace(-1, 10) == 0 and B.vitfe_layer_norm_workspace(10, 0) == 0


def test_mrope_refusals():
    for c in [dict(spans=None), dict(n=None), dict(cap=-1), dict(cap=1025), dict(items=None), dict(n_items=None),
              dict(cap_items=257), dict(cap_items=-1), dict(merge=0), dict(merge=9), dict(rows=-1), dict(pos=None),
              dict(pos=18), dict(items=20), dict(spans=18), dict(status=18)]:
        _refused(B.vitfe_mrope_positions, _with(POS, **c), 1)
    for c in [dict(pos=None), dict(axes=0), dict(axes=5), dict(axis=None), dict(axis=bytes([3] * 32)),
              dict(axis=bytes(31)), dict(rot=60), dict(rot=72), dict(rot=0), dict(theta=0.0), dict(theta=float("inf")),
              dict(rows=-1), dict(d=60), dict(d=520), dict(dtype=3), dict(q=None), dict(qo=None), dict(q=20),
              dict(qs=120), dict(qs=130), dict(qos=127), dict(k=None), dict(ks=60), dict(kos=62), dict(hq=-1),
              dict(hk=5000), dict(dtype=2, q=24)]:
        _refused(B.vitfe_mrope_apply, _with(ROPE, **c), 1)


def _shape(**c):
    d = dict(rows_q=10, rows_k=10, max_seqs=2, heads_q=4, heads_kv=2, head_dim=64, causal=0, dtype=0)
    return B.AttentionShape(*dict(d, **c).values())


def test_attention_refusals():
    inval = [dict(rows_q=-1), dict(rows_k=-1), dict(rows_q=1 << 31), dict(max_seqs=-1), dict(heads_q=0),
             dict(heads_kv=0), dict(heads_kv=3), dict(head_dim=0), dict(head_dim=60), dict(dtype=4)]
    unsup = [dict(head_dim=136), dict(dtype=2), dict(heads_q=130, heads_kv=2), dict(heads_q=8192, heads_kv=8192)]
    for changes, code in [(c, 1) for c in inval] + [(c, 7) for c in unsup]:
        s = _shape(**changes)
        assert B.vitfe_attention_plan_bytes(s) == 0
        assert B.vitfe_attention_workspace(s) == 0 and B.vitfe_attention_backward_workspace(s) == 0
        _refused(B.vitfe_attention_plan, [s, 16, 16, 16], code)
        _refused(B.vitfe_attention, [s, 16, 16, 256, 16, 128, 16, 128, 1.0, 16, 256, 16, 16], code)
    s = _shape()
    for args in [(None, 16, 16), (16, None, 16), (16, 16, None), (18, 16, 16), (16, 16, 24)]:
        _refused(B.vitfe_attention_plan, [s, *args], 1)
    fwd = dict(plan=16, q=16, qs=256, k=16, ks=128, v=16, vs=128, scale=1.0, out=16, os=256, lse=16, work=16, status=16)
    bad = [dict(plan=None), dict(plan=24), dict(q=None), dict(q=24), dict(qs=248), dict(qs=260), dict(k=None),
           dict(ks=120), dict(v=24), dict(vs=132), dict(out=None), dict(os=8), dict(scale=0.0), dict(scale=-1.0),
           dict(scale=float("nan")), dict(lse=18), dict(work=24), dict(status=18)]
    for c in bad:
        _refused(B.vitfe_attention, [s] + _with(fwd, **c), 1)
    grad = dict(plan=16, dout=16, dos=256, q=16, qs=256, k=16, ks=128, v=16, vs=128, out=16, os=256, lse=16, scale=1.0,
                dq=16, dqs=256, dk=16, dks=128, dv=16, dvs=128, work=16, status=16)
    for c in [dict(plan=None), dict(dout=None), dict(dos=8), dict(q=None), dict(out=24), dict(lse=None), dict(dq=None),
              dict(dqs=250), dict(dk=24), dict(dks=64), dict(dv=None), dict(dvs=129), dict(work=None), dict(work=24),
              dict(scale=0.0)]:
        _refused(B.vitfe_attention_backward, [s] + _with(grad, **c), 1)


def test_attention_workspace_is_asked_for_where_key_ranges_may_be_cut():
    assert B.vitfe_attention_workspace(_shape(rows_k=512)) == 0
    s = _shape(rows_k=513)
    assert B.vitfe_attention_workspace(s) > 0
    _refused(B.vitfe_attention, [s, 16, 16, 256, 16, 128, 16, 128, 1.0, 16, 256, 16, None], 1)


def test_shape_struct_layout():
    assert ctypes.sizeof(B.AttentionShape) == 40
    assert B.AttentionShape.max_seqs.offset == 16 and B.AttentionShape.dtype.offset == 36


def test_torch_calls_refuse_what_does_not_fit():
    torch = pytest.importorskip("torch")
    from vit_vision_encoder_fusedinputnorm_gb300 import encoder as E
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        E.layer_norm(x)                                # not on the GPU
    with pytest.raises(ValueError):
        E.layer_norm(x[0])
    with pytest.raises(ValueError):
        E.layer_norm(x.t())
    with pytest.raises(ValueError):
        E.mrope_apply(None, None, None, [0])
    with pytest.raises(TypeError):
        E._dtype(x.double())
    assert E.section_axes((2, 1, 1)) == [0, 0, 1, 2]
    assert E.section_axes((4, 2, 2), True) == [0, 1, 2, 0, 1, 2, 0, 0]
