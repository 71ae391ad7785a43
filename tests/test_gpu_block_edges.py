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
