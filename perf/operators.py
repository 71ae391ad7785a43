"""The encoder-block operators, case by case: layer norm, rotary positions with several axes and
attention over packed sequences, each forward and backward.

`run` computes a case in plain float32 torch (`own` false) or through the library's calls (`own`
true) on the same inputs.  `exact` restates each definition in float64.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
MERGE = 2
THETA = 1e6


# ------------------------------------------------------------------ cases

def _ln(name, op, rows, width, dtype, params):
    return {"name": name, "op": op, "rows": rows, "width": width, "dtype": dtype, "params": params}


def _attn(name, op, lens_q, lens_k, heads, heads_kv, dim, causal, dtype, pad, packed):
    return {"name": name, "op": op, "lens_q": lens_q, "lens_k": lens_k, "heads": heads, "heads_kv": heads_kv,
            "dim": dim, "causal": causal, "dtype": dtype, "pad": pad, "packed": packed}


MIXED = "256,1024,3456,3456,1536,1536,1600,5184"     # patches of the eight mixed stills


def _cache_lens(n, longest):
    """n cache lengths between 1 and `longest`, spread over their logarithm, in a mixed order."""
    lens = [max(1, int(longest ** ((i + 1) / n))) for i in range(n)]
    return [lens[(i * 27 + 5) % n] for i in range(n)]


def listed():
    cache = ",".join(str(v) for v in _cache_lens(64, 32768))
    return [
        # one 224x224 still through a norm of the patch-14 tower: a launch-bound call
        _ln("norm_still", "norm", 256, 1280, "bf16", "bf16"),
        # 64 stills of 1344x1344 through the same norm: the throughput workload's activations
        _ln("norm_stills64", "norm", 589824, 1280, "bf16", "bf16"),
        # fine-tuning on the eight mixed stills: a norm's gradients
        _ln("norm_grad_mixed", "norm_grad", 18048, 1280, "bf16", "f32"),
        # fine-tuning the patch-16 tower with float32 activations over a full bucket
        _ln("norm_grad_bucket", "norm_grad", 65536, 1152, "f32", "f32"),
        # the next token of eight conversations: positions given, one row each
        {"name": "mrope_tokens", "op": "mrope", "rows": 8, "spans": "", "heads": 28, "heads_kv": 4, "dim": 128,
         "rotary": 128, "sections": "16,24,24", "interleaved": False, "inverse": False, "dtype": "bf16"},
        # a packed prompt of text, stills and the 32-frame video: positions built, then Q and K rotated
        {"name": "mrope_prompt", "op": "mrope", "rows": 16384,
         "spans": "14@1,96,96,1;30@1,48,72,1;7|21@16,32,56,2;250|900|5@1,64,64,1;5@1,64,64,1;33", "heads": 32,
         "heads_kv": 8, "dim": 128, "rotary": 128, "sections": "24,20,20", "interleaved": True, "inverse": False,
         "dtype": "bf16"},
        # one 224x224 still through the tower's attention: latency
        _attn("attn_still", "attn", "256", "256", 16, 16, 80, False, "bf16", 0, True),
        # four stills of 1344x1344: the tower's attention at its longest
        _attn("attn_stills4", "attn", "9216,9216,9216,9216", "9216,9216,9216,9216", 16, 16, 80, False, "bf16", 0, True),
        # prompts of different lengths, causal, four query heads to a key head
        _attn("attn_prompt", "attn", "6001,4099,4096,1777,1000,300,17,1", "6001,4099,4096,1777,1000,300,17,1", 32, 8,
              128, True, "bf16", 3, False),
        # one new token of each of 64 conversations over its cached keys and values
        _attn("attn_token", "attn", ",".join(["1"] * 64), cache, 32, 8, 128, True, "bf16", 0, False),
        # fine-tuning on the eight mixed stills: the attention's gradients
        _attn("attn_grad_mixed", "attn_grad", MIXED, MIXED, 16, 16, 80, False, "bf16", 0, False),
        # training on packed prompts, causal, shared key heads: their gradients sum over the group
        _attn("attn_grad_prompt", "attn_grad", "4100,2049,2048,1000,129,2", "4100,2049,2048,1000,129,2", 16, 4, 128,
              True, "f16", 5, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "mrope", "attn", "attn_grad"])
    if op in ("norm", "norm_grad"):
        width = rng.choice([_log(rng, 33, 8192), rng.choice([768, 1024, 1152, 1280, 1536, 2048, 3584, 5120])])
        rows = _log(rng, 1, min(589824, 589824 * 1280 // width // 2))
        return {"op": op, "rows": rows, "width": width, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "params": rng.choice(["bf16", "f32"])}
    if op == "mrope":
        dim = rng.choice([64, 72, 80, 96, 128, 256])
        rotary = rng.choice([dim, dim // 2 // 8 * 8])
        half = rotary // 2
        a = rng.randint(1, half // 3)
        heads_kv = rng.choice([1, 2, 4, 8])
        c = {"op": op, "rows": 1, "spans": "", "heads": heads_kv * rng.randint(1, 8), "heads_kv": heads_kv, "dim": dim,
             "rotary": rotary, "sections": "%d,%d,%d" % (half - 2 * a, a, a), "interleaved": rng.random() < 0.5,
             "inverse": rng.random() < 0.3, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
        if rng.random() < 0.3:
            c["rows"] = _log(rng, 1, 512)
            return c
        total, seqs, most = 0, [], _log(rng, 64, 16384)
        while total < most:
            parts = []
            for _ in range(rng.randint(1, 4)):
                text = _log(rng, 1, max(2, most // 4))
                t, h, w = rng.choice([1, 1, rng.randint(2, 8)]), 2 * _log(rng, 1, 32), 2 * _log(rng, 1, 32)
                seen = rng.random() < 0.7
                parts.append("%d@%d,%d,%d,%d" % (text, t, h, w, rng.randint(1, 4)) if seen else "%d" % text)
                total += text + (t * h * w // 4 if seen else 0)
            seqs.append(";".join(parts))
        c["spans"], c["rows"] = "|".join(seqs), total + rng.choice([0, 0, rng.randint(1, 300)])
        return c
    dim = rng.choice([64, 72, 80, 96, 128, 8 * rng.randint(4, 16)])
    heads_kv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 1, 2, 3, 4, 7, 8]) if heads_kv <= 8 else 1
    n = _log(rng, 1, 48)
    causal = rng.random() < 0.5
    kind = rng.choice(["same", "same", "token", "tail"]) if op == "attn" else "same"
    longest = _log(rng, 16, 32768 if kind == "token" else 8192)
    lens_k = [longest] + [_log(rng, 1, longest) for _ in range(n - 1)]
    rng.shuffle(lens_k)
    lens_q = {"same": lens_k, "token": [1] * n, "tail": [_log(rng, 1, max(2, v)) for v in lens_k]}[kind]

    def cost():
        pairs = sum(a * b for a, b in zip(lens_q, lens_k))
        padded = len(lens_q) * max(lens_q) * max(lens_k)
        return max(pairs * 4 * dim * heads_kv * group * (2.5 if op == "attn_grad" else 1) / 1.2e12,
                   padded * heads_kv * group * 4 / (16e9 if op == "attn" else 6e9), sum(lens_k) * dim * heads_kv / 4e8)
    while cost() > 1 and len(lens_k) > 1:
        at = max(range(len(lens_k)), key=lambda i: lens_q[i] * lens_k[i])
        lens_q, lens_k = lens_q[:at] + lens_q[at + 1:], lens_k[:at] + lens_k[at + 1:]
    while cost() > 1:
        heads_kv, group = max(1, heads_kv // 2), max(1, group // 2)
        lens_k = [max(1, v * 3 // 4) for v in lens_k]
        lens_q = [min(v, lens_k[i]) for i, v in enumerate(lens_q)]
    case = _attn("", op, ",".join(map(str, lens_q)), ",".join(map(str, lens_k)), heads_kv * group, heads_kv, dim, causal,
                 rng.choice(["bf16", "bf16", "f16"]), rng.choice([0, rng.randint(1, 200)]),
                 kind == "same" and rng.random() < 0.5)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _ints(text):
    return [int(v) for v in text.split(",")]


def _axes(case):
    """The axis (0 time, 1 height, 2 width) of each rotated pair: consecutive sections, or height
    and width taken at every third pair while their sections last."""
    s = _ints(case["sections"])
    if not case["interleaved"]:
        return [a for a in range(3) for _ in range(s[a])]
    return [i % 3 if i % 3 and i < 3 * s[i % 3] else 0 for i in range(sum(s))]


def _spans(text):
    """[(first, text tokens, item or -1, time step)], [(t, h, w)] of a spans text."""
    spans, grids = [], []
    for seq in (text.split("|") if text else []):
        for k, part in enumerate(seq.split(";")):
            words, _, grid = part.partition("@")
            t, h, w, step = _ints(grid) if grid else (0, 0, 0, 1)
            spans.append((int(k == 0), int(words), len(grids) if grid else -1, step))
            if grid:
                grids.append((t, h, w))
    return spans, grids


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] in ("norm", "norm_grad"):
        r, n, pt = case["rows"], case["width"], DTYPES[case["params"]]
        # a residual stream: channels of different scale and offset, a few of them large
        scale = 0.5 + normal(n).abs() + 12.0 * (torch.rand(n, generator=g, device="cuda") < 0.01)
        x = torch.empty((r, n), dtype=dt, device="cuda")
        dy = torch.empty((r, n), dtype=dt, device="cuda") if case["op"] == "norm_grad" else None
        shift = 0.3 * normal(n)
        for i in range(0, r, 65536):
            m = min(65536, r - i)
            x[i:i + m] = (normal(m, n) * scale + shift).to(dt)
            if dy is not None:
                dy[i:i + m] = (0.5 * normal(m, n)).to(dt)
        return {"x": x, "dy": dy, "weight": (1 + 0.2 * normal(n)).to(pt), "bias": (0.1 * normal(n)).to(pt)}
    if case["op"] == "mrope":
        spans, grids = _spans(case["spans"])
        s = {"q": normal(case["rows"], case["heads"], case["dim"]).to(dt),
             "k": normal(case["rows"], case["heads_kv"], case["dim"]).to(dt), "pos": None, "spans": None}
        if spans:
            # items as in a vitfe_item table: pixel_offset (8 bytes), t, h, w, frames
            table = [(0, 0, t, h, w, 1 if t == 1 else 2 * t) for t, h, w in grids] or [(0,) * 6]
            s["spans"] = torch.tensor(spans, dtype=torch.int32, device="cuda")
            s["n_spans"] = torch.tensor([len(spans)], dtype=torch.int32, device="cuda")
            s["items"] = torch.tensor(table, dtype=torch.int32, device="cuda")
            s["n_items"] = torch.tensor([len(grids)], dtype=torch.int32, device="cuda")
        else:
            s["pos"] = torch.randint(0, 32768, (3, case["rows"]), generator=g, device="cuda", dtype=torch.int32)
        return s
    lq, lk = _ints(case["lens_q"]), _ints(case["lens_k"])
    rq, rk, hq, hk, d = sum(lq) + case["pad"], sum(lk) + case["pad"], case["heads"], case["heads_kv"], case["dim"]
    # heads of different sharpness; keys share an offset, as those behind a norm and a bias do
    sharp = 0.4 + 1.8 * torch.rand((1, hq, 1), generator=g, device="cuda")
    q, k, v = normal(rq, hq, d) * sharp, normal(rk, hk, d) + 0.5 * normal(1, hk, d), normal(rk, hk, d) + 0.3
    if case["packed"]:
        qkv = torch.cat([q, k, v], 1).to(dt)          # one projection's rows: Q | K | V
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:
        q, k, v = q.to(dt), k.to(dt), v.to(dt)
    cu = [torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda") for n in (lq, lk)]
    s = {"q": q, "k": k, "v": v, "cu_q": cu[0], "cu_k": cu[1], "most_q": max(lq), "most_k": max(lk)}
    if case["op"] == "attn_grad":
        s["dout"] = (0.5 * normal(rq, hq, d)).to(dt)
    return s


def prepare(case, seed):
    state = {**_inputs(case, seed), "case": case}
    if case["op"] == "norm_grad":
        # what a training program keeps from its forward pass
        x = state["x"]
        state["mean"], state["rstd"] = _stats(x)
    if case["op"] == "mrope":
        state["axes"] = _axes(case)
        state["axis"] = torch.tensor(state["axes"], dtype=torch.int64, device="cuda")
        # inverse frequencies theta^(-2i/rotary) in 2^-40 turns, so that positions multiply exactly
        half = case["rotary"] // 2
        turns = THETA ** (-np.arange(half, dtype=np.float64) / half) / (2 * np.pi)
        state["freq"] = torch.tensor(np.rint(turns * 2.0 ** 40).astype(np.int64), device="cuda")
    if case["op"] == "attn_grad":
        out, lse = _attend(state)
        state["out"], state["lse"] = out.to(DTYPES[case["dtype"]]), lse
    if case["op"] in ("attn", "attn_grad") and own:
        # the plan of a batch: made once, used by every layer of the tower
        from vit_vision_encoder_fusedinputnorm_gb300 import encoder
        state["plan"] = encoder.AttentionPlan(state["cu_q"], state["cu_k"], state["q"].shape[0], state["k"].shape[0],
                                              case["heads"], case["heads_kv"], case["dim"], causal=case["causal"])
    return state


# ------------------------------------------------------------------ plain forms

def _stats(x):
    x = x.float()
    mean = x.mean(1)
    return mean, torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS)


def _norm(s):
    x = s["x"]
    mean, rstd = _stats(x)
    y = (x.float() - mean[:, None]) * rstd[:, None] * s["weight"].float() + s["bias"].float()
    return {"y": y.to(x.dtype), "mean": mean, "rstd": rstd}


def _norm_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    dweight, dbias = (dy * xhat).sum(0), dy.sum(0)
    dxhat = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (dxhat - dxhat.mean(1, keepdim=True) - xhat * (dxhat * xhat).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": dweight, "dbias": dbias}


def _positions(s, rows):
    """[3][rows] int32: text advances all axes together; an item's merged patches take
    (start + group * step, start + row, start + column), and what follows starts past all three."""
    first, text, item, step = s["spans"].long().unbind(1)
    grid = s["items"].long()[item.clamp(min=0)]
    has = (item >= 0).long()
    t, h, w = grid[:, 2] * has, grid[:, 3] // MERGE * has, grid[:, 4] // MERGE * has
    count = text + t * h * w
    end = count.cumsum(0)
    reach = torch.maximum((t - 1) * step + 1, torch.maximum(h, w)) * (t * h * w > 0)
    before = (text + reach).cumsum(0) - text - reach
    base = before - torch.where(first > 0, before, 0).cummax(0).values
    row = torch.arange(rows, device=end.device)
    at = torch.searchsorted(end, row, right=True).clamp(max=len(end) - 1)
    local = row - (end - count)[at] - text[at]
    hw, wide = (h * w)[at].clamp(min=1), w[at].clamp(min=1)
    start = base[at] + text[at]
    seen = torch.stack([start + local // hw * step[at], start + local % hw // wide, start + local % wide])
    pos = torch.where(local < 0, start + local, seen)
    return torch.where(row < end[-1], pos, -1).int()


def _rotate(x, cos, sin, rotary):
    half = rotary // 2
    f = x.float()
    a, b = f[..., :half], f[..., half:rotary]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, f[..., rotary:]], -1).to(x.dtype)


def _mrope(s):
    c = s["case"]
    pos = s["pos"] if s["pos"] is not None else _positions(s, c["rows"])
    phase = (pos.long()[s["axis"]].T * s["freq"]) & (2 ** 40 - 1)            # [rows][pairs], a turn is 2^40
    angle = (phase - ((phase >> 39) << 40)).float() * (2 * math.pi / 2.0 ** 40)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None] * (-1 if c["inverse"] else 1)
    return {"pos": pos, "q": _rotate(s["q"], cos, sin, c["rotary"]), "k": _rotate(s["k"], cos, sin, c["rotary"])}


def _padded(x, cu, most):
    """[batch][most][heads][dim] float32 of packed rows, zeros past each sequence's end."""
    at = cu[:-1, None] + torch.arange(most, device=cu.device)
    live = at < cu[1:, None]
    return x.float()[at.clamp(max=x.shape[0] - 1)] * live[:, :, None, None], at, live


def _scores(s):
    """Padded Q, K, V, the probabilities [batch][kv head][group][q][k] and their log-sum-exp."""
    c = s["case"]
    q, at, live_q = _padded(s["q"], s["cu_q"], s["most_q"])
    k, _, live_k = _padded(s["k"], s["cu_k"], s["most_k"])
    v, at_k, _ = _padded(s["v"], s["cu_k"], s["most_k"])
    b, n, hq, d = q.shape
    hk = k.shape[2]
    q = q.view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    k, v = k.permute(0, 2, 1, 3)[:, :, None], v.permute(0, 2, 1, 3)[:, :, None]
    p = (q * d ** -0.5).reshape(b, hk, -1, d) @ k[:, :, 0].transpose(-1, -2)
    p = p.view(b, hk, hq // hk, n, -1)
    hidden = ~live_k[:, None, :]
    if c["causal"]:
        # the last query sees every key: query i of n sees keys up to i + (keys - n)
        lens = (s["cu_k"].diff() - s["cu_q"].diff())[:, None, None]
        reach = torch.arange(n, device=q.device)[:, None] + lens
        hidden = hidden | (torch.arange(p.shape[-1], device=q.device) > reach)
    p.masked_fill_(hidden[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, 1.0, total))
    lse = (top + total.log())[..., 0]
    return q, k, v, p, lse, at, live_q, at_k, live_k


def _unpad(x, at, live, rows, fill=0.0):
    """Packed rows of a padded [batch][rows][...] tensor; rows of no sequence hold `fill`."""
    out = torch.full((rows,) + tuple(x.shape[2:]), fill, dtype=x.dtype, device=x.device)
    out[at[live]] = x[live]
    return out


def _attend(s):
    """Attention's float32 output [rows][heads][dim] and log-sum-exp [rows][heads]."""
    q, k, v, p, lse, at, live, _, _ = _scores(s)
    b, hk, g, n, d = q.shape
    o = (p.reshape(b, hk, g * n, -1) @ v[:, :, 0]).view(b, hk, g, n, d)
    rows = s["q"].shape[0]
    return (_unpad(o.permute(0, 3, 1, 2, 4).reshape(b, n, hk * g, d), at, live, rows),
            _unpad(lse.permute(0, 3, 1, 2).reshape(b, n, hk * g), at, live, rows, -math.inf))


def _attn_grad(s):
    q, k, v, p, _, at, live, at_k, live_k = _scores(s)
    b, hk, g, n, d = q.shape
    m, dt = k.shape[3], s["q"].dtype

    def heads(x):
        return _padded(x, s["cu_q"], n)[0].view(b, n, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * n, d)

    do, o = heads(s["dout"]), heads(s["out"])
    p = p.view(b, hk, g * n, m)
    dv = p.transpose(-1, -2) @ do
    ds = do @ v[:, :, 0].transpose(-1, -2)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    scale = d ** -0.5
    dq = (ds @ k[:, :, 0]) * scale
    dk = ds.transpose(-1, -2) @ q.reshape(b, hk, g * n, d) * scale
    dq = dq.view(b, hk, g, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, hk * g, d)
    dk, dv = dk.permute(0, 2, 1, 3), dv.permute(0, 2, 1, 3)
    return {"dq": _unpad(dq, at, live, s["q"].shape[0]).to(dt), "dk": _unpad(dk, at_k, live_k, s["k"].shape[0]).to(dt),
            "dv": _unpad(dv, at_k, live_k, s["v"].shape[0]).to(dt)}


# ------------------------------------------------------------------ one pass

def _run_own(s):
    from vit_vision_encoder_fusedinputnorm_gb300 import encoder
    c = s["case"]
    if c["op"] == "norm":
        y, mean, rstd = encoder.layer_norm(s["x"], s["weight"], s["bias"], EPS, stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if c["op"] == "norm_grad":
        dx, dweight, dbias = encoder.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if c["op"] == "mrope":
        pos = s["pos"]
        if pos is None:
            pos = encoder.mrope_positions(s["spans"], s["n_spans"], s["items"], s["n_items"], c["rows"], merge=MERGE)
        q, k = encoder.mrope_apply(s["q"], s["k"], pos, s["axes"], theta=THETA, inverse=c["inverse"])
        return {"pos": pos, "q": q, "k": k}
    if c["op"] == "attn":
        out, lse = encoder.attention(s["q"], s["k"], s["v"], s["plan"], lse=True)
        return {"out": out, "lse": lse}
    dq, dk, dv = encoder.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["plan"])
    return {"dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "attn":
        out, lse = _attend(state)
        return {"out": out.to(state["q"].dtype), "lse": lse}
    return {"norm": _norm, "norm_grad": _norm_grad, "mrope": _mrope, "attn_grad": _attn_grad}[op](state)


def _pairs(case):
    """Query-key pairs that the mask leaves, over all sequences."""
    n = 0
    for a, b in zip(_ints(case["lens_q"]), _ints(case["lens_k"])):
        short = min(a, b)
        n += a * b if not case["causal"] else short * (b - short) + short * (short + 1) // 2
    return n


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] in ("norm", "norm_grad"):
        r, n, p = case["rows"], case["width"], BYTES[case["params"]]
        if case["op"] == "norm":
            return {"bytes": 2 * r * n * e + 2 * n * p + 8 * r, "flops": 8 * r * n}
        return {"bytes": 3 * r * n * e + n * p + 8 * n + 8 * r, "flops": 14 * r * n}
    if case["op"] == "mrope":
        r, h = case["rows"], case["heads"] + case["heads_kv"]
        return {"bytes": 2 * r * h * case["dim"] * e + 12 * r, "flops": 3 * r * h * case["rotary"]}
    rq, rk = sum(_ints(case["lens_q"])) + case["pad"], sum(_ints(case["lens_k"])) + case["pad"]
    q, kv, stat = rq * case["heads"] * case["dim"] * e, rk * case["heads_kv"] * case["dim"] * e, 4 * rq * case["heads"]
    mm = 2 * case["dim"] * case["heads"] * _pairs(case)          # one product over the mask's pairs
    if case["op"] == "attn":
        return {"bytes": 2 * q + 2 * kv + stat, "flops": 2 * mm}
    return {"bytes": 4 * q + 4 * kv + stat, "flops": 5 * mm}


# ------------------------------------------------------------------ float64

def _exact_positions(case):
    spans, grids = _spans(case["spans"])
    rows, nxt = [], 0
    for first, text, item, step in spans:
        nxt = 0 if first else nxt
        rows += [(nxt + i,) * 3 for i in range(text)]
        nxt += text
        if item >= 0:
            t, h, w = grids[item][0], grids[item][1] // MERGE, grids[item][2] // MERGE
            rows += [(nxt + i * step, nxt + y, nxt + x) for i in range(t) for y in range(h) for x in range(w)]
            nxt += max((t - 1) * step + 1, h, w)
    rows += [(-1, -1, -1)] * (case["rows"] - len(rows))
    return np.array(rows, dtype=np.int32).T.copy()


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("norm", "norm_grad"):
        y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        mean, rstd = (torch.empty(case["rows"], dtype=torch.float64, device="cuda") for _ in range(2))
        dw, db = (torch.zeros(case["width"], dtype=torch.float64, device="cuda") for _ in range(2))
        w, b = s["weight"].double(), s["bias"].double()
        for i in range(0, case["rows"], 32768):
            j = slice(i, i + 32768)
            x = s["x"][j].double()
            mean[j] = x.mean(1)
            rstd[j] = 1 / torch.sqrt(x.var(1, unbiased=False) + EPS)
            z = (x - mean[j, None]) * rstd[j, None]
            if case["op"] == "norm":
                y[j] = z * w + b
                continue
            dy = s["dy"][j].double()
            dw += torch.einsum("rn,rn->n", dy, z)
            db += dy.sum(0)
            gz = dy * w
            y[j] = rstd[j, None] * (gz - gz.mean(1, keepdim=True) - z * torch.einsum("rn,rn->r", gz, z)[:, None] / case["width"])
        return {"y": y, "mean": mean, "rstd": rstd} if case["op"] == "norm" else {"dx": y, "dweight": dw, "dbias": db}
    if case["op"] == "mrope":
        pos = s["pos"].cpu().numpy() if s["pos"] is not None else _exact_positions(case)
        half = case["rotary"] // 2
        angle = pos[np.array(_axes(case))].T * THETA ** (-2.0 * np.arange(half) / case["rotary"])
        turn = torch.from_numpy(np.exp((-1j if case["inverse"] else 1j) * angle)).cuda()[:, None]

        def rotated(x):
            x = x.double()
            z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
            return torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)
        return {"pos": pos, "q": rotated(s["q"]), "k": rotated(s["k"])}
    lq, lk = _ints(case["lens_q"]), _ints(case["lens_k"])
    hq, hk, d = case["heads"], case["heads_kv"], case["dim"]
    grad = case["op"] == "attn_grad"
    if 4 * d * hq * sum(a * b for a, b in zip(lq, lk)) * (2.5 if grad else 1) > 4e12:
        return None
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    aq, ak = 0, 0
    for n, m in zip(lq, lk):
        iq, ik = slice(aq, aq + n), slice(ak, ak + m)
        aq, ak = aq + n, ak + m
        seen = None
        if case["causal"]:
            seen = torch.ones((n, m), dtype=torch.bool, device="cuda").tril(m - n)
        for h in range(hq):
            j = h * hk // hq
            z = q[iq, h] @ k[ik, j].T / math.sqrt(d)
            z = z if seen is None else z.masked_fill(~seen, -math.inf)
            lse[iq, h] = torch.logsumexp(z, 1)
            p = torch.exp(z - torch.nan_to_num(lse[iq, h], neginf=0.0)[:, None])
            out[iq, h] = p @ v[ik, j]
            if grad:
                do = s["dout"][iq, h].double()
                dv[ik, j] += p.T @ do
                dz = p * (do @ v[ik, j].T - (do * out[iq, h]).sum(1, keepdim=True)) / math.sqrt(d)
                dq[iq, h] = dz @ k[ik, j]
                dk[ik, j] += dz.T @ q[iq, h]
    return {"dq": dq, "dk": dk, "dv": dv} if grad else {"out": out, "lse": lse}
