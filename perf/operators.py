"""Cases of the state space block's operators, and their plain forms.

Three operators, each with its directions:

* ``scan``: the selective state space scan over prompts (``scan``: sequences of one length, or
  packed ones with the states they continue from) and over single tokens (``step``).  Per head,
  with dt = softplus(raw + bias) and a state S of dk rows and dv columns:
  ``S_t = exp(dt_t A) S_{t-1} + dt_t B_t x_t^T``, ``y_t = S_t^T C_t + D x_t``.
  B and C are shared by the heads of a group.
* ``conv``: the causal depthwise convolution of four taps with bias and SiLU in front of it, over
  prompts (one length, or packed with the last three inputs of each) and single tokens.
* ``norm``: layer norm, forward (``norm``) and backward (``norm_bwd``).

The plain form of the scan works on blocks of 64 tokens: products inside a block, one state a
block, and one matrix of decays that joins the blocks.  ``exact`` walks the recurrence token by
token in 64 bits.
"""
import math

import torch

own = False

BLOCK = 64
TAPS = 4
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases ----------------------------------------------------------------------------------

def listed():
    return [
        # the training shape's batch of full sequences through one layer
        dict(name="scan_train", op="scan", dtype="bf16", n=8, length=4096, heads=16, groups=1, dk=128, dv=128),
        # one long document: few heads, many tokens
        dict(name="scan_long", op="scan", dtype="bf16", n=1, length=32768, heads=16, groups=1, dk=128, dv=128),
        # a serving batch of mixed prompts that continue from states, heads of 64 channels
        dict(name="scan_prompts", op="scan_packed", dtype="bf16", n=64, median=512, most=4096, heads=32, groups=2,
             dk=128, dv=64),
        # a small check in fp32 with a ragged last block
        dict(name="scan_fp32", op="scan", dtype="fp32", n=2, length=333, heads=2, groups=1, dk=64, dv=64),
        # one token for each of a full decoding batch
        dict(name="step_batch", op="step", dtype="bf16", n=256, heads=16, groups=1, dk=128, dv=128),
        # one token for a few users: latency
        dict(name="step_few", op="step", dtype="fp32", n=3, heads=16, groups=2, dk=128, dv=64),
        # the channels that feed scan_train
        dict(name="conv_train", op="conv", dtype="bf16", n=8, length=4096, channels=2304),
        # packed prompts in fp32 that continue from the inputs kept before
        dict(name="conv_prompts", op="conv_packed", dtype="fp32", n=64, median=512, most=4096, channels=2560),
        # one token for a decoding batch
        dict(name="conv_step", op="conv_step", dtype="bf16", n=256, channels=2304),
        # the norm in front of a layer at the training shape, and its gradients
        dict(name="norm_train", op="norm", dtype="bf16", rows=32768, width=2048),
        dict(name="norm_bwd_train", op="norm_bwd", dtype="bf16", rows=32768, width=2048),
        # a width that is no multiple of a wave's, an odd number of rows, fp32
        dict(name="norm_bwd_odd", op="norm_bwd", dtype="fp32", rows=1001, width=1540),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("scan", "scan", "scan_packed", "step", "conv", "conv_packed", "conv_step", "norm", "norm_bwd"))
    c = dict(op=op, dtype=rng.choice(("bf16", "bf16", "fp32")))
    if op in ("scan", "scan_packed", "step"):
        c.update(dk=rng.choice((64, 128)), dv=rng.choice((64, 128)), heads=rng.choice((1, 2, 6, 8, 12, 16, 24)))
        c["groups"] = rng.choice([g for g in (1, 2, 3, 4, 8) if c["heads"] % g == 0])
    if op in ("conv", "conv_packed", "conv_step"):
        c["channels"] = 8 * _log_uniform(rng, 8, 512)
    if op in ("scan", "conv"):
        tokens = (4096 if c["dtype"] == "fp32" else 32768) * 16 // max(16, c.get("heads", 16))
        c["n"] = _log_uniform(rng, 1, 16)
        c["length"] = _log_uniform(rng, 1, tokens // c["n"])
    elif op in ("scan_packed", "conv_packed"):
        most = (128 if c["dtype"] == "fp32" else 512) * 2048 // max(2048, c.get("heads", 1) * c.get("dv", 1))
        c.update(n=_log_uniform(rng, 1, 64), median=_log_uniform(rng, 8, most))
        c["most"] = 8 * c["median"]
    elif op in ("step", "conv_step"):
        c["n"] = _log_uniform(rng, 1, 160)
    elif op in ("norm", "norm_bwd"):
        c["width"] = _log_uniform(rng, 16, 8192)
        c["rows"] = _log_uniform(rng, 1, min(32768, 2 ** 25 // c["width"]))
    return c


def _lengths(case):
    """Prompt lengths of a packed case: log-normal around the median, between 1 and the most.  They
    are the case's own, whatever the seed of the values."""
    g = torch.Generator("cpu").manual_seed(case["n"] * 1009 + case["median"])
    z = torch.randn(case["n"], generator=g, dtype=torch.float64)
    return [int(v) for v in (z.exp() * case["median"]).round().clamp(1, case["most"]).tolist()]


def _tokens(case):
    return sum(_lengths(case)) if case["op"].endswith("packed") else case["n"] * case.get("length", 1)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("scan", "scan_packed", "step"):
        h, g, dk, dv, t = case["heads"], case["groups"], case["dk"], case["dv"], _tokens(case)
        states = case["n"] * h * dk * dv * 4
        token = t * es * (2 * h * dv + 2 * g * dk + h)
        # x, B, C and dt read, y written; the final states written, and read too where they go on
        return {"bytes": token + 12 * h + states * (1 if op == "scan" else 2), "flops": 4.0 * t * h * dk * dv}
    if op in ("conv", "conv_packed", "conv_step"):
        t, ch = _tokens(case), case["channels"]
        # the inputs that the next token needs are written, and read too where a call goes on
        state = (1 if op == "conv" else 2) * case["n"] * (TAPS - 1) * ch * es
        return {"bytes": 2 * t * ch * es + state + 20 * ch, "flops": 2.0 * TAPS * t * ch}
    r, d = case["rows"], case["width"]
    if op == "norm":
        return {"bytes": 2 * r * d * es + 8 * r + 8 * d, "flops": 7.0 * r * d}
    return {"bytes": 3 * r * d * es + 8 * r + 12 * d, "flops": 11.0 * r * d}


# ---- inputs ---------------------------------------------------------------------------------

def _packed(case, dev):
    ends = [0]
    for n in _lengths(case):
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

    def silu(v):
        return v * torch.sigmoid(v)

    s = dict(case=case)
    if op in ("scan", "scan_packed", "step"):
        h, gr, dk, dv = case["heads"], case["groups"], case["dk"], case["dv"]
        lead = (case["n"], case["length"]) if op == "scan" else (_tokens(case),)
        # x, B and C are parts of the convolution's one output; dt is a projection of its own
        s["xbc"] = silu(normal(*lead, h * dv + 2 * gr * dk)).to(dt)
        s["dt"] = normal(*lead, h).mul_(0.5).to(dt)
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), h))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it is the step
        s["a"] = -uniform(1.0, 16.0, h)
        s["d"] = uniform(0.5, 1.5, h)
        if op != "scan":
            s["state"] = normal(case["n"], h, dk, dv).mul_(0.1)
        if op == "scan_packed":
            s["cu"] = _packed(case, dev)
    elif op in ("conv", "conv_packed", "conv_step"):
        ch = case["channels"]
        lead = (case["n"], case["length"]) if op == "conv" else (_tokens(case),)
        s["x"] = normal(*lead, ch).to(dt)
        s["taps"] = uniform(-0.5, 0.5, ch, TAPS)
        s["bias"] = uniform(-0.2, 0.2, ch)
        if op != "conv":
            s["state"] = normal(case["n"], TAPS - 1, ch).to(dt)
        if op == "conv_packed":
            s["cu"] = _packed(case, dev)
    else:
        r, d = case["rows"], case["width"]
        s["x"] = (normal(r, d) + uniform(0.2, 1.0, r, 1)).to(dt)
        s["gamma"] = uniform(0.5, 1.5, d)
        s["beta"] = uniform(-0.5, 0.5, d)
        if op == "norm_bwd":
            s["dy"] = normal(r, d).to(dt)
            wide = s["x"].double()  # the statistics that the forward pass has kept
            mean = wide.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = torch.rsqrt((wide - mean[:, None]).square().mean(-1) + EPS).float()
    return s


def _split(s):
    """x, B and C of the convolution's output: views, one stride between tokens."""
    c = s["case"]
    h, g, dk, dv = c["heads"], c["groups"], c["dk"], c["dv"]
    x, b, cm = s["xbc"].split((h * dv, g * dk, g * dk), -1)
    return x.unflatten(-1, (h, dv)), b.unflatten(-1, (g, dk)), cm.unflatten(-1, (g, dk))


# ---- one pass -------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import gated_delta_rule_gdn2_amd as gdn2

    op = s["case"]["op"]
    if op in ("scan", "scan_packed", "step"):
        x, b, c = _split(s)
        if op == "scan":
            return gdn2.ssm_fwd(x, s["dt"], b, c, s["a"], s["d"], s["dt_bias"])
        if op == "scan_packed":
            return gdn2.ssm_fwd_varlen(x, s["dt"], b, c, s["a"], s["cu"], s["d"], s["dt_bias"], s["state"])
        return gdn2.ssm_step(x, s["dt"], b, c, s["a"], s["state"], s["d"], s["dt_bias"]), s["state"]
    if op == "conv":
        return gdn2.short_conv(s["x"], s["taps"], s["bias"])
    if op == "conv_packed":
        return gdn2.short_conv_varlen(s["x"], s["taps"], s["cu"], s["bias"], s["state"])
    if op == "conv_step":
        return gdn2.short_conv_step(s["x"], s["taps"], s["state"], s["bias"]), s["state"]
    if op == "norm":
        return gdn2.layer_norm(s["x"], s["gamma"], s["beta"], EPS)
    return gdn2.layer_norm_bwd(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"])


def _run_plain(s):
    op = s["case"]["op"]
    if op in ("scan", "scan_packed"):
        return _plain_scan(s)
    if op == "step":
        return _plain_step(s)
    if op in ("conv", "conv_packed"):
        return _plain_conv(s)
    if op == "conv_step":
        return _plain_conv_step(s)
    return _plain_norm(s) if op == "norm" else _plain_norm_bwd(s)


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_scan(s):
    c = s["case"]
    h, g, dk, dv, n = c["heads"], c["groups"], c["dk"], c["dv"], c["n"]
    x, b, cm = _split(s)
    dev, kind = x.device, x.dtype
    lead = x.shape[:-2]
    x, b, cm = x.reshape(-1, h, dv).float(), b.reshape(-1, g, dk).float(), cm.reshape(-1, g, dk).float()
    dt = _softplus(s["dt"].reshape(-1, h).float() + s["dt_bias"])
    total = x.shape[0]
    # blocks of 64 tokens, each of one sequence; the last of a sequence may be short
    if c["op"] == "scan":
        cu = torch.arange(n + 1, device=dev) * c["length"]
        nb = n * -(-c["length"] // BLOCK)
    else:
        cu = s["cu"]
        nb = total // BLOCK + n  # no fewer than there are
    blocks = (cu[1:] - cu[:-1] + BLOCK - 1) // BLOCK
    first = torch.cumsum(blocks, 0) - blocks
    ids = torch.arange(nb, device=dev)
    seq = torch.searchsorted(first + blocks, ids, right=True).clamp(max=n - 1)
    token = cu[seq, None] + (ids - first[seq])[:, None] * BLOCK + torch.arange(BLOCK, device=dev)  # [nb, 64]
    live = (token < cu[seq + 1][:, None]) & (ids < first[-1] + blocks[-1])[:, None]
    at = token.clamp(max=total - 1)
    at = torch.where(live, at, torch.zeros_like(at))
    mask = live[..., None]
    dtb = torch.where(mask, dt[at], 0.0)                                                # [nb, 64, h]
    xb = torch.where(mask[..., None], x[at], 0.0)
    bb = torch.where(mask[..., None], b[at], 0.0).transpose(1, 2).contiguous()          # [nb, g, 64, dk]
    cb = torch.where(mask[..., None], cm[at], 0.0).transpose(1, 2).contiguous()
    # decays: sums of logarithms in 64 bits
    cum = torch.cumsum(dtb.double() * s["a"].double(), 1).permute(0, 2, 1)              # [nb, h, 64]
    low = torch.ones(BLOCK, BLOCK, dtype=torch.bool, device=dev).tril()
    pair = torch.where(low, cum[..., :, None] - cum[..., None, :], -math.inf).float().exp()
    dx = (xb * dtb[..., None]).permute(0, 2, 1, 3).contiguous()                         # [nb, h, 64, dv]
    grams = torch.matmul(cb, bb.transpose(-1, -2).contiguous())                         # [nb, g, 64, 64]
    hb = bb.repeat_interleave(h // g, 1)
    hc = cb.repeat_interleave(h // g, 1)
    y = torch.matmul(grams.repeat_interleave(h // g, 1) * pair, dx)
    del pair, grams
    # a block's own state, and every block's start from those before it and the sequence's first
    rest = (cum[..., -1:] - cum).float().exp()
    states = torch.matmul((hb * rest[..., None]).transpose(-1, -2).contiguous(), dx)    # [nb, h, dk, dv]
    start = s["state"] if c["op"] == "scan_packed" else torch.zeros(n, h, dk, dv, device=dev)
    every = torch.cat((start, states)).permute(1, 0, 2, 3).reshape(h, n + nb, dk * dv)
    gone = torch.cumsum(cum[..., -1], 0).permute(1, 0)                                  # [h, nb], through block i
    before = gone - cum[..., -1].permute(1, 0)
    zero = torch.zeros(h, 1, dtype=gone.dtype, device=dev)
    past = torch.cat((zero, gone), 1)                                                   # before block i, i = 0 .. nb
    own_first = past[:, first]
    source = torch.cat((own_first, gone), 1)
    target = torch.cat((before, past[:, first + blocks]), 1)                            # starts, then finals
    every_seq = torch.arange(n, device=dev)
    src_seq, dst_seq = torch.cat((every_seq, seq)), torch.cat((seq, every_seq))
    src_at, dst_at = torch.cat((every_seq * 0 - 1, ids)), torch.cat((ids, every_seq * 0 + nb))
    joined = (src_seq[None, :] == dst_seq[:, None]) & (src_at[None, :] < dst_at[:, None])
    joined = joined & torch.cat((torch.ones_like(every_seq), (ids < first[-1] + blocks[-1]).long())).bool()[None, :]
    carry = torch.where(joined, target[:, :, None] - source[:, None, :], -math.inf).float().exp()
    carried = torch.matmul(carry, every).reshape(h, nb + n, dk, dv).permute(1, 0, 2, 3)
    y = y + torch.matmul(hc * cum.float().exp()[..., None], carried[:nb].contiguous())
    y = y.permute(0, 2, 1, 3) + s["d"][:, None] * xb
    # places of no token write to a row of their own, behind the last one
    out = torch.zeros(total + 1, h, dv, device=dev)
    out[torch.where(live, token, torch.full_like(token, total))] = y
    return out[:total].to(kind).reshape(*lead, h, dv), carried[nb:].contiguous()


def _plain_step(s):
    c = s["case"]
    x, b, cm = _split(s)
    kind = x.dtype
    h, g = c["heads"], c["groups"]
    x, b, cm = x.float(), b.float().repeat_interleave(h // g, 1), cm.float().repeat_interleave(h // g, 1)
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    s["state"].mul_(torch.exp(dt * s["a"])[..., None, None]).add_(b[..., :, None] * (x * dt[..., None])[..., None, :])
    y = (s["state"] * cm[..., :, None]).sum(-2) + s["d"][:, None] * x
    return y.to(kind), s["state"]


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_conv(s):
    c = s["case"]
    n, ch, dev = c["n"], c["channels"], s["x"].device
    x = s["x"].reshape(-1, ch).float()
    total = x.shape[0]
    if c["op"] == "conv":
        cu = torch.arange(n + 1, device=dev) * c["length"]
        kept = torch.zeros(n, TAPS - 1, ch, device=dev)
    else:
        cu, kept = s["cu"], s["state"].float()
    # each sequence's kept inputs in front of its own: row i of it is its input i - 3
    seq = torch.searchsorted(cu, torch.arange(total, device=dev), right=True) - 1
    rows = torch.empty(total + n * (TAPS - 1), ch, device=dev)
    place = torch.arange(total, device=dev) + (seq + 1) * (TAPS - 1)
    rows[place] = x
    head = cu[:-1] + torch.arange(n, device=dev) * (TAPS - 1)
    rows[head[:, None] + torch.arange(TAPS - 1, device=dev)] = kept
    t = s["taps"]
    u = s["bias"] + t[:, 0] * rows[place - 3] + t[:, 1] * rows[place - 2] + t[:, 2] * rows[place - 1] + t[:, 3] * rows[place]
    y = _silu(u).to(s["x"].dtype).reshape(s["x"].shape)
    tail = cu[1:] + torch.arange(n, device=dev) * (TAPS - 1)
    return y, rows[tail[:, None] + torch.arange(TAPS - 1, device=dev)].to(s["x"].dtype)


def _plain_conv_step(s):
    x, t, st = s["x"].float(), s["taps"], s["state"].float()
    u = s["bias"] + t[:, 0] * st[:, 0] + t[:, 1] * st[:, 1] + t[:, 2] * st[:, 2] + t[:, 3] * x
    s["state"].copy_(torch.cat((st[:, 1:], x[:, None]), 1))
    return _silu(u).to(s["x"].dtype), s["state"]


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    off = x - mean
    rstd = 1 / torch.sqrt((off * off).mean(-1, keepdim=True) + EPS)
    y = off * rstd * s["gamma"] + s["beta"]
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_norm_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["gamma"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


# ---- 64 bits --------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "scan_packed", "step"):
        return _exact_scan(s)
    if op in ("conv", "conv_packed", "conv_step"):
        return _exact_conv(s)
    x, gamma = s["x"].double(), s["gamma"].double()
    if op == "norm":
        var, mean = torch.var_mean(x, dim=-1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        return (x - mean[:, None]) * rstd[:, None] * gamma + s["beta"].double(), mean, rstd
    dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    u, v = (x - mean) * rstd, dy * gamma
    dx = rstd * (v - (v.sum(-1, keepdim=True) + u * (u * v).sum(-1, keepdim=True)) / x.shape[-1])
    return {"dx": dx, "dgamma": (dy * u).sum(0), "dbeta": dy.sum(0)}


def _rows_of(s, v):
    """[sequences, longest, ...] of a token tensor (any values behind a sequence's end), and the lengths."""
    c = s["case"]
    if not c["op"].endswith("packed"):
        v = v if c["op"] in ("scan", "conv") else v[:, None]
        return v, [v.shape[1]] * v.shape[0]
    lengths = _lengths(c)
    longest = max(lengths)
    at = s["cu"][:-1, None] + torch.arange(longest, device=v.device)
    return v[at.clamp(max=v.shape[0] - 1)], lengths


def _tokens_of(s, v, lengths):
    if not s["case"]["op"].endswith("packed"):
        return v if s["case"]["op"] in ("scan", "conv") else v[:, 0]
    return torch.cat([v[i, :n] for i, n in enumerate(lengths)])


def _exact_scan(s):
    c = s["case"]
    h, g, dk, dv, n = c["heads"], c["groups"], c["dk"], c["dv"], c["n"]
    x, b, cm = (v.double() for v in _split(s))
    raw = s["dt"].double() + s["dt_bias"].double()
    dt = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
    (x, lengths), b, cm, dt = _rows_of(s, x), _rows_of(s, b)[0], _rows_of(s, cm)[0], _rows_of(s, dt)[0]
    a, d = s["a"].double(), s["d"].double()
    state = s["state"].double() if "state" in s else torch.zeros(n, h, dk, dv, dtype=torch.float64, device=x.device)
    state = state.reshape(n, g, h // g, dk, dv).clone()
    decay = torch.exp(dt * a).reshape(n, -1, g, h // g, 1, 1)
    put = (x * dt[..., None]).reshape(n, -1, g, h // g, 1, dv)
    ends = torch.tensor(lengths, device=x.device)
    ragged = len(set(lengths)) > 1
    y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for t in range(max(lengths)):
        new = state * decay[:, t] + b[:, t, :, None, :, None] * put[:, t]
        state = torch.where((t < ends)[:, None, None, None, None], new, state) if ragged else new
        y[:, t] = (state * cm[:, t, :, None, :, None]).sum(-2).reshape(n, h, dv)
    y += d[:, None] * x
    return _tokens_of(s, y, lengths), state.reshape(n, h, dk, dv)


def _exact_conv(s):
    x, lengths = _rows_of(s, s["x"].double())
    n, longest, ch = x.shape
    kept = s["state"].double() if "state" in s else torch.zeros(n, TAPS - 1, ch, dtype=torch.float64, device=x.device)
    row = torch.cat((kept, x), 1)
    u = s["bias"].double().expand(x.shape).clone()
    for j in range(TAPS):
        u += s["taps"].double()[:, j] * row[:, j:j + longest]
    y = _tokens_of(s, u * torch.sigmoid(u), lengths)
    return y, torch.stack([row[i, m:m + TAPS - 1] for i, m in enumerate(lengths)])
