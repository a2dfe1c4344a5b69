"""Cases of the attention block's operators, and their plain forms.

Hybrid stacks put attention over a sliding window between the recurrent layers.  Four operators of
such a layer, each with its directions:

* ``attn``: causal attention of H query heads over G key/value heads, softmax(scale q k^T) v, with
  or without a window, and the logarithm of every row's sum.  Query t of T stands at key S - T + t
  of S.  Whole sequences (``attn``), packed ones with the keys that they go on from
  (``attn_packed``), and the gradients of both (``attn_bwd``, ``attn_bwd_packed``), which recompute
  the probabilities from the logarithms.
* ``step``: one token a sequence over a cache that keeps the last C tokens: token p lies in slot
  p mod C, and the step writes its own key and value there.
* ``rotary``: rotary positions on the first channels of the heads of q and k, halves or
  interleaved pairs, from a table of frequencies.
* ``rms``: root-mean-square norm of x + residual, with an output in the input's type or in 8 bits
  with a scale for each row (``rms8``), and its gradients (``rms_bwd``).
"""
import math

import torch

own = False

EPS = 1e-6
E4M3 = 448.0  # the largest value in 8 bits
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases ----------------------------------------------------------------------------------

def listed():
    return [
        # the training shape's batch through one attention layer with a window of 2048 tokens
        dict(name="attn_train", op="attn", dtype="bf16", n=8, length=4096, past=0, heads=16, groups=8, d=128, window=2048),
        # one long document, all of it visible
        dict(name="attn_long", op="attn", dtype="bf16", n=1, length=32768, past=0, heads=16, groups=2, d=128, window=0),
        # a serving batch of mixed prompts, each behind the keys it goes on from, heads of 64
        dict(name="attn_prompts", op="attn_packed", dtype="bf16", n=16, median=512, most=4096, past=256, heads=32, groups=4,
             d=64, window=0),
        # gradients at the training shape
        dict(name="attn_bwd_train", op="attn_bwd", dtype="bf16", n=8, length=4096, past=0, heads=16, groups=8, d=128,
             window=2048),
        # gradients of a batch of documents of mixed lengths, packed, a key head for each query head
        dict(name="attn_bwd_packed", op="attn_bwd_packed", dtype="bf16", n=16, median=512, most=4096, past=0, heads=12,
             groups=12, d=64, window=0),
        # a small check of the gradients in fp32 with ragged last tiles
        dict(name="attn_bwd_fp32", op="attn_bwd", dtype="fp32", n=2, length=333, past=0, heads=4, groups=2, d=64, window=100),
        # one token for each of a full decoding batch, caches of a window
        dict(name="step_batch", op="step", dtype="bf16", n=256, cache=2048, heads=16, groups=2, d=128, window=2048),
        # one token for a few users with long caches: latency
        dict(name="step_few", op="step", dtype="bf16", n=3, cache=16384, heads=16, groups=2, d=128, window=0),
        # the queries and keys of attn_train, half of each head rotated
        dict(name="rotary_train", op="rotary", dtype="bf16", n=8, length=4096, heads=16, groups=8, d=128, rot=64,
             interleaved=False, far=0),
        # one token for a decoding batch at far positions, interleaved pairs
        dict(name="rotary_step", op="rotary", dtype="fp32", n=255, length=1, heads=16, groups=2, d=128, rot=128,
             interleaved=True, far=1000000),
        # the norm in front of a layer's projections in 8 bits
        dict(name="rms8_prompts", op="rms8", dtype="bf16", rows=32768, width=2048),
        # the norm's gradients at the training shape
        dict(name="rms_bwd_train", op="rms_bwd", dtype="bf16", rows=32768, width=2048),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "attn_packed", "attn_bwd", "attn_bwd", "attn_bwd_packed", "step", "step", "rotary",
                     "rms", "rms8", "rms_bwd"))
    c = dict(op=op, dtype="bf16" if op == "rms8" else rng.choice(("bf16", "bf16", "fp32")))
    small = c["dtype"] == "fp32"
    if op.startswith("attn") or op in ("step", "rotary"):
        c.update(d=rng.choice((64, 128)), heads=rng.choice((1, 2, 6, 8, 12, 16, 20)))
        c["groups"] = rng.choice([g for g in (1, 2, 3, 4, 8, 16) if c["heads"] % g == 0])
    if op in ("attn", "attn_bwd"):
        # no more pairs of tokens than a small multiple of the training shape's
        pairs = (1 << (26 if small else 30)) // c["heads"]
        c["n"] = _log_uniform(rng, 1, 16)
        longest = max(2, int(math.sqrt(pairs / c["n"])))
        c["length"] = _log_uniform(rng, 1, longest)
        c["past"] = rng.choice((0, _log_uniform(rng, 1, longest))) if op == "attn" else 0
        c["window"] = rng.choice((0, _log_uniform(rng, 1, 4096)))
    elif op in ("attn_packed", "attn_bwd_packed"):
        c["n"] = _log_uniform(rng, 1, 32)
        longest = max(64, int(math.sqrt((1 << (25 if small else 30)) / c["heads"] / c["n"])))
        c["median"] = _log_uniform(rng, 8, max(9, longest // 8))
        c["most"] = 8 * c["median"]
        c["past"] = rng.choice((0, _log_uniform(rng, 8, longest // 2))) if op == "attn_packed" else 0
        c["window"] = rng.choice((0, _log_uniform(rng, 16, 4096)))
    elif op == "step":
        c["n"] = _log_uniform(rng, 1, 160)
        c["cache"] = _log_uniform(rng, 16, min(32768, (1 << (22 if small else 24)) // (c["n"] * c["groups"])))
        c["window"] = rng.choice((0, _log_uniform(rng, 1, c["cache"])))
    elif op == "rotary":
        c["n"] = _log_uniform(rng, 1, 16)
        c["length"] = _log_uniform(rng, 1, 32768 // c["n"] * 16 // max(16, c["heads"]))
        c.update(rot=c["d"] // rng.choice((1, 2, 4)), interleaved=rng.choice((False, True)), far=rng.choice((0, 1000000)))
    elif op in ("rms", "rms8", "rms_bwd"):
        c["width"] = _log_uniform(rng, 16, 8192)
        c["rows"] = _log_uniform(rng, 1, min(32768, 2 ** 25 // c["width"]))
    return c


def _spread(case, median, most, salt):
    """Lengths of a packed case: log-normal around the median, between 1 and the most.  They are the
    case's own, whatever the seed of the values."""
    g = torch.Generator("cpu").manual_seed(case["n"] * 1009 + median + salt)
    z = torch.randn(case["n"], generator=g, dtype=torch.float64)
    return [int(v) for v in (z.exp() * median).round().clamp(1, most).tolist()]


def _lengths(case):
    """Queries and keys of every sequence."""
    if not case["op"].endswith("packed"):
        return [case["length"]] * case["n"], [case["length"] + case["past"]] * case["n"]
    tq = _spread(case, case["median"], case["most"], 0)
    past = _spread(case, case["past"], 8 * case["past"], 77) if case["past"] else [0] * case["n"]
    return tq, [a + b for a, b in zip(tq, past)]


def _places(case):
    """The position of every sequence's token in a step: from an empty cache to one written over and over."""
    g = torch.Generator("cpu").manual_seed(case["n"] * 31 + case["cache"])
    return [int(v) for v in (torch.rand(case["n"], generator=g, dtype=torch.float64) * 2 * case["cache"]).tolist()]


def _pairs(tq, tk, window):
    """Pairs of a query and a key that it sees."""
    w = window or tk
    full = max(0, tk - max(w, tk - tq + 1) + 1)  # queries at positions w - 1 and on see w keys
    rest = tq - full
    first = tk - tq + 1
    return full * w + rest * first + rest * (rest - 1) // 2


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("attn"):
        h, g, d = case["heads"], case["groups"], case["d"]
        tq, tk = _lengths(case)
        pairs = sum(_pairs(a, b, case["window"]) for a, b in zip(tq, tk))
        nq, nk = sum(tq) * h * d * es, sum(tk) * g * d * es
        stats = sum(tq) * h * 4
        if "bwd" in op:  # q, o and its gradient, k, v read; three gradients written
            return {"bytes": 4 * nq + 4 * nk + stats, "flops": 10.0 * pairs * h * d}
        return {"bytes": 2 * nq + 2 * nk + stats, "flops": 4.0 * pairs * h * d}
    if op == "step":
        h, g, d = case["heads"], case["groups"], case["d"]
        seen = sum(min(p + 1, case["cache"], case["window"] or case["cache"]) for p in _places(case))
        tokens = case["n"] * (2 * h + 2 * g) * d * es
        return {"bytes": 2 * seen * g * d * es + tokens + 8 * case["n"], "flops": 4.0 * seen * h * d}
    if op == "rotary":
        t = case["n"] * case["length"] * (case["heads"] + case["groups"])
        # channels that are not rotated are part of the result too
        return {"bytes": 2 * t * case["d"] * es + 8 * case["n"] * case["length"], "flops": 3.0 * t * case["rot"]}
    r, w = case["rows"], case["width"]
    if op == "rms_bwd":  # dy, the sum and its own gradient read; the gradients of x and gamma written
        return {"bytes": 4 * r * w * es + 4 * r + 8 * w, "flops": 9.0 * r * w}
    out = r * w + 4 * r if op == "rms8" else r * w * es
    return {"bytes": 3 * r * w * es + out + 4 * r + 4 * w, "flops": 5.0 * r * w}


# ---- inputs ---------------------------------------------------------------------------------

def _offsets(lengths, dev):
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, dtype=torch.int64, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    dt = TYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device=dev) * (hi - lo) + lo

    s = dict(case=case)
    if op.startswith("attn") or op in ("step", "rotary"):
        h, gr, d = case["heads"], case["groups"], case["d"]
    if op.startswith("attn"):
        packed = op.endswith("packed")
        tq, tk = _lengths(case)
        lead_q = (sum(tq),) if packed else (case["n"], tq[0])
        lead_k = (sum(tk),) if packed else (case["n"], tk[0])
        if lead_q == lead_k:  # parts of the one output of the layer's projection
            s["q"], s["k"], s["v"] = _parts(normal(*lead_q, (h + 2 * gr) * d).to(dt), h, gr, d)
        else:
            s["q"], s["k"], s["v"] = (normal(*lead, n, d).to(dt) for lead, n in ((lead_q, h), (lead_k, gr), (lead_k, gr)))
        if packed:
            s["cu_q"], s["cu_k"] = _offsets(tq, dev), _offsets(tk, dev)
        if "bwd" in op:
            s["d_o"] = normal(*lead_q, h, d).to(dt)
            s["o"], s["lse"] = _plain_attn(s)  # what the forward pass has kept
    elif op == "step":
        n, c = case["n"], case["cache"]
        s["q"], s["k"], s["v"] = _parts(normal(n, (h + 2 * gr) * d).to(dt), h, gr, d)
        s["k_cache"], s["v_cache"] = (normal(n, c, gr, d).to(dt) for _ in range(2))
        s["positions"] = torch.tensor(_places(case), dtype=torch.int64, device=dev)
    elif op == "rotary":
        n, t = case["n"], case["length"]
        s["q"], s["k"], _ = _parts(normal(n, t, (h + 2 * gr) * d).to(dt), h, gr, d)
        half = case["rot"] // 2
        # a base of 10000, the slow half of the frequencies divided by 4 for long contexts
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        s["freq"] = torch.where(torch.arange(half) >= half // 2, freq / 4, freq).float().to(dev)
        s["positions"] = None
        if case["far"]:
            first = torch.randint(0, case["far"], (n, 1), generator=g, device=dev)
            s["positions"] = first + torch.arange(t, device=dev)
    else:
        r, w = case["rows"], case["width"]
        s["gamma"] = uniform(0.5, 1.5, w)
        if op == "rms_bwd":
            s["h"] = (2 * normal(r, w)).to(dt)
            s["dy"], s["dh"] = normal(r, w).to(dt), normal(r, w).to(dt)
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(-1) + EPS).float()
        else:
            s["x"], s["residual"] = normal(r, w).to(dt), (2 * normal(r, w)).to(dt)
    return s


def _parts(qkv, h, g, d):
    q, k, v = qkv.split((h * d, g * d, g * d), -1)
    return q.unflatten(-1, (h, d)), k.unflatten(-1, (g, d)), v.unflatten(-1, (g, d))


# ---- one pass -------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import gated_delta_rule_gdn2_amd as gdn2

    c = s["case"]
    op = c["op"]
    window = c.get("window") or None
    if op == "attn":
        return gdn2.attn_fwd(s["q"], s["k"], s["v"], window=window)
    if op == "attn_packed":
        return gdn2.attn_fwd_varlen(s["q"], s["k"], s["v"], s["cu_q"], cu_seqlens_k=s["cu_k"], window=window)
    if op == "attn_bwd":
        return gdn2.attn_bwd(s["d_o"], s["q"], s["k"], s["v"], s["o"], s["lse"], window=window)
    if op == "attn_bwd_packed":
        return gdn2.attn_bwd_varlen(s["d_o"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu_q"], window=window)
    if op == "step":
        o = gdn2.attn_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["positions"], window=window)
        return o, s["k_cache"], s["v_cache"]
    if op == "rotary":
        return gdn2.rotary(s["q"], s["k"], s["freq"], s["positions"], interleaved=c["interleaved"])
    if op == "rms":
        return gdn2.rms_norm(s["x"], s["gamma"], EPS, residual=s["residual"])
    if op == "rms8":
        return gdn2.rms_norm_fp8(s["x"], s["gamma"], EPS, residual=s["residual"])
    return gdn2.rms_norm_bwd(s["dy"], s["h"], s["gamma"], s["rstd"], dh=s["dh"])


def _run_plain(s):
    op = s["case"]["op"]
    if op in ("attn", "attn_packed"):
        return _plain_attn(s)
    if op in ("attn_bwd", "attn_bwd_packed"):
        return _plain_attn_bwd(s)
    return {"step": _plain_step, "rotary": _plain_rotary, "rms": _plain_rms, "rms8": _plain_rms8, "rms_bwd": _plain_rms_bwd}[op](s)


def _rows(x, cu, longest):
    """[sequences, heads, longest, ...] in 32 bits: packed sequences one below the other, what lies
    behind a short one's end left to the mask."""
    if cu is not None:
        at = cu[:-1, None] + torch.arange(longest, device=x.device)
        x = x[at.clamp(max=x.shape[0] - 1)]
    return x.transpose(1, 2).float().contiguous()


def _tokens(x, cu, total):
    """Back to tokens: [sequences, heads, longest, ...] to [total, heads, ...]."""
    if cu is None:
        return x.transpose(1, 2).contiguous()
    token = torch.arange(total, device=x.device)
    seq = torch.searchsorted(cu, token, right=True) - 1
    return x[seq, :, token - cu[seq]]


def _hidden(s):
    """True where a query does not see a key: [sequences or 1, 1, queries, keys]."""
    c, dev = s["case"], s["q"].device
    tq, tk = _lengths(c)
    if "cu_q" in s:
        nq, nk = (s[n][1:] - s[n][:-1] for n in ("cu_q", "cu_k"))
    else:
        nq, nk = torch.tensor([tq[0]], device=dev), torch.tensor([tk[0]], device=dev)
    key = torch.arange(max(tk), device=dev)
    place = (nk - nq)[:, None, None] + torch.arange(max(tq), device=dev)[:, None]
    hidden = (key > place) | (key >= nk[:, None, None])
    if c["window"]:
        hidden |= key <= place - c["window"]
    return hidden[:, None]


def _wide(s):
    c = s["case"]
    tq, tk = _lengths(c)
    cu_q, cu_k = s.get("cu_q"), s.get("cu_k")
    share = c["heads"] // c["groups"]
    q = _rows(s["q"], cu_q, max(tq))
    k, v = (_rows(s[n], cu_k, max(tk)).repeat_interleave(share, 1) for n in ("k", "v"))
    return q, k, v


def _plain_attn(s):
    q, k, v = _wide(s)
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(1 / math.sqrt(s["case"]["d"]))
    p.masked_fill_(_hidden(s), -math.inf)
    most = p.amax(-1, keepdim=True)
    p.sub_(most).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total
    lse = (most + torch.log(total))[..., 0]
    cu, total = s.get("cu_q"), s["q"].shape[0]
    return _tokens(o, cu, total).to(s["q"].dtype), _tokens(lse, cu, total)


def _plain_attn_bwd(s):
    c = s["case"]
    tq, _ = _lengths(c)
    cu_q, cu_k = s.get("cu_q"), s.get("cu_k")
    scale = 1 / math.sqrt(c["d"])
    q, k, v = _wide(s)
    d_o, o, lse = (_rows(s[n], cu_q, max(tq)) for n in ("d_o", "o", "lse"))
    hidden = _hidden(s)
    if cu_q is not None:  # rows behind a sequence's end have no part in the sums over queries
        behind = torch.arange(max(tq), device=q.device)[:, None] >= (cu_q[1:] - cu_q[:-1])[:, None, None]
        hidden = hidden | behind[:, None]
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(scale).sub_(lse[..., None]).exp_()
    p.masked_fill_(hidden, 0.0)
    dv = torch.matmul(p.transpose(-1, -2), d_o)
    ds = torch.matmul(d_o, v.transpose(-1, -2).contiguous()).sub_((d_o * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    del p
    ds.masked_fill_(hidden, 0.0)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q)
    share = (c["groups"], c["heads"] // c["groups"])
    dk, dv = (x.unflatten(1, share).sum(2) for x in (dk, dv))
    kind = s["q"].dtype
    dq = _tokens(dq, cu_q, s["q"].shape[0])
    dk, dv = (_tokens(x, cu_k, s["k"].shape[0]) for x in (dk, dv))
    return {"dq": dq.to(kind), "dk": dk.to(kind), "dv": dv.to(kind)}


def _plain_step(s):
    c = s["case"]
    n, size, h, g, d = c["n"], c["cache"], c["heads"], c["groups"], c["d"]
    place = s["positions"]
    row = torch.arange(n, device=place.device)
    s["k_cache"][row, place % size] = s["k"]
    s["v_cache"][row, place % size] = s["v"]
    # the token in a slot: the last one not behind this step's whose position gives the slot
    slot = torch.arange(size, device=place.device)
    back = (place[:, None] - slot) % size
    hidden = (back > place[:, None]) | (back >= (c["window"] or size))
    k, v = (s[x].permute(0, 2, 1, 3).float().contiguous() for x in ("k_cache", "v_cache"))  # [n, g, size, d]
    q = s["q"].reshape(n, g, h // g, d).float()
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).masked_fill_(hidden[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.reshape(n, h, d).to(s["q"].dtype), s["k_cache"], s["v_cache"]


def _plain_rotary(s):
    c, dev = s["case"], s["q"].device
    place = s["positions"] if s["positions"] is not None else torch.arange(c["length"], device=dev).expand(c["n"], -1)
    angle = place[..., None].double() * s["freq"].double()
    cos, sin = (f(angle).float()[..., None, :] for f in (torch.cos, torch.sin))
    rot, half = c["rot"], c["rot"] // 2

    def turned(x):
        y = x.float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["interleaved"] else (y[..., :half], y[..., half:rot])
        first, second = a * cos - b * sin, a * sin + b * cos
        pair = torch.stack((first, second), -1).flatten(-2) if c["interleaved"] else torch.cat((first, second), -1)
        return torch.cat((pair, y[..., rot:]), -1).to(x.dtype)

    return turned(s["q"]), turned(s["k"])


def _plain_rms_rows(s):
    total = s["x"].float() + s["residual"].float()
    rstd = 1 / torch.sqrt((total * total).mean(-1, keepdim=True) + EPS)
    return total * rstd * s["gamma"], total.to(s["residual"].dtype), rstd[:, 0]


def _plain_rms(s):
    y, total, rstd = _plain_rms_rows(s)
    return y.to(s["x"].dtype), total, rstd


def _plain_rms8(s):
    y, total, rstd = _plain_rms_rows(s)
    scale = y.abs().amax(-1) / E4M3
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (y / scale[:, None]).clamp(-E4M3, E4M3).to(torch.float8_e4m3fn), scale, total, rstd


def _plain_rms_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    u, v = s["h"].float() * rstd, dy * s["gamma"]
    dx = s["dh"].float() + rstd * (v - u * (u * v).mean(-1, keepdim=True))
    return {"dx": dx.to(s["h"].dtype), "dgamma": (dy * u).sum(0)}


# ---- 64 bits --------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("attn"):
        return _exact_attn(s)
    if op == "step":
        return _exact_step(s)
    if op == "rotary":
        return _exact_rotary(s)
    if op == "rms_bwd":
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        v = dy * s["gamma"].double()
        dx = s["dh"].double() + r * v - h * r ** 3 * (h * v).sum(-1, keepdim=True) / h.shape[-1]
        return {"dx": dx, "dgamma": torch.einsum("rw,rw,r->w", dy, h, r[:, 0])}
    h = s["x"].double() + s["residual"].double()
    rstd = torch.rsqrt(torch.linalg.vecdot(h, h)[:, None] / h.shape[-1] + EPS)
    y = h * rstd * s["gamma"].double()
    if op == "rms":
        return y, h, rstd[:, 0]
    scale = torch.linalg.vector_norm(y, ord=math.inf, dim=-1) / E4M3
    scale[scale == 0] = 1
    return y / scale[:, None], scale, h, rstd[:, 0]


def _exact_attn(s):
    """Sequence by sequence and head by head, the probabilities of 4096 queries at a time."""
    c = s["case"]
    tq, tk = _lengths(c)
    share, scale, window, d = c["heads"] // c["groups"], c["d"] ** -0.5, c["window"] or 1 << 40, c["d"]
    bwd = "bwd" in c["op"]
    names = ("q", "k", "v") + (("d_o",) if bwd else ())
    flat = {n: s[n].reshape(-1, *s[n].shape[-2:]) for n in names}
    like = dict(dtype=torch.float64, device=s["q"].device)
    o, lse = torch.empty(flat["q"].shape, **like), torch.empty(flat["q"].shape[:2], **like)
    grads = {n: torch.zeros(flat[n].shape, **like) for n in ("q", "k", "v")} if bwd else None
    at_q = at_k = 0
    for a, b in zip(tq, tk):
        rows, cols = slice(at_q, at_q + a), slice(at_k, at_k + b)
        for h in range(c["heads"]):
            k, v = (flat[n][cols, h // share].double() for n in ("k", "v"))
            for lo in range(0, a, 4096):
                hi = min(a, lo + 4096)
                part = slice(at_q + lo, at_q + hi)
                q = flat["q"][part, h].double()
                ago = torch.arange(b - a + lo, b - a + hi, device=q.device)[:, None] - torch.arange(b, device=q.device)
                score = torch.where((ago >= 0) & (ago < window), q @ k.T * scale, -math.inf)
                lse[part, h] = torch.logsumexp(score, -1)
                p = torch.softmax(score, -1)
                if not bwd:
                    o[part, h] = p @ v
                    continue
                g = flat["d_o"][part, h].double()
                dp = g @ v.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
                grads["q"][part, h] = ds @ k
                grads["k"][cols, h // share] += ds.T @ q
                grads["v"][cols, h // share] += p.T @ g
        at_q, at_k = at_q + a, at_k + b
    if bwd:
        return {"d" + n: v.reshape(s[n].shape) for n, v in grads.items()}
    return o.reshape(s["q"].shape), lse.reshape(s["q"].shape[:-1])


def _exact_step(s):
    c = s["case"]
    share, size = c["heads"] // c["groups"], c["cache"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    keys, values = s["k_cache"].clone(), s["v_cache"].clone()
    for n, place in enumerate(_places(c)):
        keys[n, place % size], values[n, place % size] = s["k"][n], s["v"][n]
        seen = range(max(0, place + 1 - min(size, c["window"] or size)), place + 1)
        slots = torch.tensor([p % size for p in seen], device=o.device)
        k, v = (x[n, slots].double().repeat_interleave(share, 1) for x in (keys, values))  # [seen, h, d]
        p = torch.softmax((k * s["q"][n].double()).sum(-1) * c["d"] ** -0.5, 0)
        o[n] = (p[..., None] * v).sum(0)
    return o, keys.double(), values.double()


def _exact_rotary(s):
    c = s["case"]
    n, t, rot = c["n"], c["length"], c["rot"]
    place = s["positions"] if s["positions"] is not None else torch.arange(t, device=s["q"].device).repeat(n, 1)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=place.device), place.double()[..., None] * s["freq"].double())
    out = []
    for x in (s["q"], s["k"]):
        y = x.double()
        if c["interleaved"]:
            pairs = torch.view_as_complex(y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous())
            y = torch.cat((torch.view_as_real(pairs * turn[:, :, None]).flatten(-2), y[..., rot:]), -1)
        else:
            pairs = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn[:, :, None]
            y = torch.cat((pairs.real, pairs.imag, y[..., rot:]), -1)
        out.append(y)
    return tuple(out)
