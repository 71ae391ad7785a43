"""Float64 definitions of the encoder-block operators, and the rounding bounds the tests use."""
import math

import torch

# unit roundoff: half the spacing of values next to 1
# (float16 also has a least spacing, 2^-24, so an absolute rounding of up to TINY)
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def rounding(dtype, y):
    """Bound of one rounding of y to dtype (a hair over, for a value rounded across a binade)."""
    return 1.01 * UNIT[dtype] * y.abs() + TINY[dtype]


def layer_norm(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    return xh * (1 if w is None else w.double()) + (0 if b is None else b.double()), mean[:, 0], rstd[:, 0]


def layer_norm_backward(dy, x, mean, rstd, w):
    dy, x = dy.double(), x.double()
    xh = (x - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy * (1 if w is None else w.double())
    n = x.shape[1]
    dx = rstd.double()[:, None] * (g - g.sum(1, keepdim=True) / n - xh * (g * xh).sum(1, keepdim=True) / n)
    return dx, (dy * xh).sum(0), dy.sum(0), xh, g


def positions(spans, grids, merge, rows):
    """spans: (first, text, item, step); grids: (t, h, w) in patches."""
    out, nxt = [], 0
    for first, text, item, step in spans:
        nxt = 0 if first else nxt
        for _ in range(text):
            out.append((nxt, nxt, nxt))
            nxt += 1
        if item >= 0:
            t, h, w = grids[item][0], grids[item][1] // merge, grids[item][2] // merge
            out += [(nxt + i * step, nxt + y, nxt + x) for i in range(t) for y in range(h) for x in range(w)]
            if t * h * w:
                nxt += max((t - 1) * step + 1, h, w)
    out += [(-1, -1, -1)] * (rows - len(out))
    return torch.tensor(out[:rows], dtype=torch.int32).reshape(-1, 3).T.contiguous()


def rotate(x, pos, axes, theta, inverse=False):
    x = x.double()
    half = len(axes)
    i = torch.arange(half, dtype=torch.float64, device=x.device)
    angle = pos.to(x.device)[torch.tensor(axes, device=x.device)].T.double() * theta ** (-i / half)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None] * (-1 if inverse else 1)
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * half:]], -1)


def attention(q, k, v, lens_q, lens_k, causal, scale=None, dout=None, out=None):
    """Output and log-sum-exp, and with `dout` the gradients; beside each result the sum of the
    magnitudes of what it adds up (`_mag`: what relative rounding errors act on; `_all`: the summed
    factors of the rounded probabilities or score gradients, what absolute ones act on).  `out`: the output that
    the gradient's delta is made of (the rounded one of a forward pass), else the exact one."""
    q, k, v = q.double(), k.double(), v.double()
    hq, hk, d = q.shape[1], k.shape[1], q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    r = {n: torch.zeros_like(t) for n, t in (("out", q), ("out_mag", q), ("dq", q), ("dq_mag", q), ("dk", k),
                                            ("dk_mag", k), ("dv", v), ("dv_mag", v), ("out_all", q), ("dq_all", q),
                                            ("dk_all", k), ("dv_all", v))}
    r["lse"] = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    r["score"] = 0.0
    aq = ak = 0
    for n, m in zip(lens_q, lens_k):
        iq, ik = slice(aq, aq + n), slice(ak, ak + m)
        aq, ak = aq + n, ak + m
        if n == 0 or m == 0:
            continue
        seen = torch.ones((n, m), dtype=torch.bool, device=q.device)
        if causal:
            seen = seen.tril(m - n)
        for h in range(hq):
            j = h // (hq // hk)
            z = (scale * (q[iq, h] @ k[ik, j].T)).masked_fill(~seen, -math.inf)
            lse = torch.logsumexp(z, 1)
            r["lse"][iq, h] = lse
            p = torch.where(seen, torch.exp(z - lse[:, None]), 0.0)
            if seen.any():
                r["score"] = max(r["score"], float(z[seen].abs().max()))
            vj = torch.where(seen.any(0)[:, None], v[ik, j], 0.0)
            r["out"][iq, h] = p @ vj
            r["out_mag"][iq, h] = p @ vj.abs()
            r["out_all"][iq, h] = seen.double() @ vj.abs()
            if dout is None:
                continue
            do = dout[iq, h].double()
            o = r["out"][iq, h] if out is None else out[iq, h].double()
            dp = do @ vj.T
            ds = p * (dp - (do * o).sum(1, keepdim=True)) * scale
            mag = p * (do.abs() @ vj.abs().T + (do * o).abs().sum(1, keepdim=True)) * scale
            r["dv"][ik, j] += p.T @ do
            r["dv_mag"][ik, j] += p.T @ do.abs()
            r["dv_all"][ik, j] += seen.double().T @ do.abs()
            r["dq_all"][iq, h] = seen.double() @ k[ik, j].abs()
            r["dk_all"][ik, j] += seen.double().T @ q[iq, h].abs()
            r["dq"][iq, h] = ds @ k[ik, j]
            r["dq_mag"][iq, h] = mag @ k[ik, j].abs()
            r["dk"][ik, j] += ds.T @ q[iq, h]
            r["dk_mag"][ik, j] += mag.T @ q[iq, h].abs()
    return r


def close(got, ref, tol, name):
    """|got - ref| <= tol elementwise (tol a tensor or a number), with matching infinities."""
    got, ref = got.double().cpu(), ref.double().cpu()
    tol = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(ref)
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(got)), f"{name}: finite in different places"
    assert torch.equal(got[~fin & ~ref.isnan()], ref[~fin & ~ref.isnan()]), f"{name}: infinities differ"
    over = (got[fin] - ref[fin]).abs() - tol[fin]
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{name}: {int((over > 0).sum())} of {over.numel()} over the bound, worst by {float(over.max()):.3e}"
