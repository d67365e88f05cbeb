"""Cases of the gated delta rule on given q, k and v, the RMS norm and the tokens' log probabilities.

Each case is one pass of one operator as a serving loop calls it: prompts, a window of drafted tokens with the
state read only, or a single token a sequence. ``run`` computes the plain form, or the framework's kernels where
``own`` is set.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


def listed():
    return [
        # one long prompt of a layer with 16 q/k heads and 32 value heads of 128: few rows, many tokens
        dict(name="delta_long_prompt", op="delta", batch=1, seq_len=4096, hq=16, hv=32, d=128, io="bf16", gate="f32",
             state="f32", pool=4, pad=0, ragged=False, update=True),
        # eight prompts of different lengths, one row of padding
        dict(name="delta_prompts", op="delta", batch=8, seq_len=777, hq=16, hv=32, d=128, io="f16", gate="f16",
             state="f32", pool=64, pad=1, ragged=True, update=True),
        # small heads, everything in 32 bits
        dict(name="delta_small_heads", op="delta", batch=2, seq_len=509, hq=4, hv=8, d=64, io="f32", gate="f32",
             state="f32", pool=3, pad=0, ragged=False, update=True),
        # a window of drafted tokens, the state only read
        dict(name="delta_window", op="delta", batch=16, seq_len=5, hq=16, hv=32, d=128, io="bf16", gate="bf16",
             state="f32", pool=48, pad=2, ragged=False, update=False),
        # one token of each of 64 sequences, and of one
        dict(name="delta_step", op="delta_step", batch=64, hq=16, hv=32, d=128, io="bf16", gate="bf16", state="f32",
             pool=128, pad=0),
        dict(name="delta_step_single", op="delta_step", batch=1, hq=16, hv=32, d=128, io="bf16", gate="f32",
             state="bf16", pool=4, pad=0),
        # in front of an 8-bit projection: the residual is added, one scale a token
        dict(name="norm_prompts", op="norm", rows=4099, n=2048, group=2048, io="bf16", out="e4m3", block=2048,
             residual="bf16", gate="none", unit=True),
        # behind the recurrence: 32 heads of 128, gated after the norm
        dict(name="norm_heads", op="norm", rows=4096, n=4096, group=128, io="bf16", out="bf16", block=0,
             residual="none", gate="after", unit=False),
        # one token of each of 64 sequences, the residual kept in 32 bits, scales of 128 columns
        dict(name="norm_step", op="norm", rows=64, n=5120, group=5120, io="f16", out="e4m3", block=128,
             residual="f32", gate="none", unit=False),
        # every token of a prompt, three alternatives
        dict(name="logprobs_prompt", op="logprobs", rows=2039, vocab=32000, io="bf16", top=3, masked=False),
        # the nodes of a verify window over a large vocabulary, masked by a grammar in places
        dict(name="logprobs_window", op="logprobs", rows=128, vocab=131072, io="f32", top=20, masked=True),
        # one token of one sequence
        dict(name="logprobs_single", op="logprobs", rows=1, vocab=131072, io="f32", top=5, masked=False),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def pick(*of):
        return rng.choice(of)

    op = pick("delta", "delta", "delta_step", "norm", "norm", "logprobs")
    io = pick("f32", "f16", "bf16", "bf16")
    if op == "norm":
        group, groups = pick((size(64, 16384), 1), (size(64, 16384), 1), (pick(32, 64, 128, 256), size(2, 64)))
        out = pick(io, io, "e4m3")
        n = group * groups
        block = 0 if out != "e4m3" else n if groups > 1 or n % 128 else pick(n, 128)
        return dict(op=op, rows=min(size(1, 16384), (1 << 24) // n), n=n, group=group, io=io, out=out, block=block,
                    residual=pick("none", io, "f32") if groups == 1 else "none",
                    gate=pick("none", "none", "after", "before"), unit=pick(True, False))
    if op == "logprobs":
        vocab = size(1000, 131072)
        return dict(op=op, rows=min(size(1, 4096), (1 << 25) // vocab), vocab=vocab, io=io, top=size(1, 24),
                    masked=pick(True, False))
    d = pick(32, 64, 128, 128, 256)
    ratio = pick(1, 2, 2, 4, 8)
    hv = max(ratio, size(2, 32) // ratio * ratio)
    batch = size(1, 64)
    case = dict(op=op, batch=batch, hq=hv // ratio, hv=hv, d=d, io=io, gate=pick(io, "f32"),
                state=pick("f32", "f32", "f16", "bf16"), pool=batch + size(1, 32), pad=rng.randint(0, batch // 4))
    if op == "delta":
        case.update(seq_len=min(size(1, 4096), max(1, (1 << 30) // (batch * hv * d * d))), ragged=pick(True, False),
                    update=pick(True, True, False))
    return case


# ---------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------
class _Draws:
    """Seeded values on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0):
        return torch.randn(shape, generator=self.g, device="cuda") * std

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def rows(self, pool, batch, pad):
        """Distinct rows of the pool's first pool - 1, the last `pad` entries of the batch padding."""
        i = torch.randperm(pool - 1, generator=self.g, device="cuda")[:batch].to(torch.int32)
        if pad:
            i[batch - pad:] = -1
        return i

    def lengths(self, batch, most, ragged):
        if not ragged:
            return None
        return torch.randint(max(1, most // 8), most + 1, (batch,), generator=self.g, device="cuda",
                             dtype=torch.int32)


def prepare(case, seed):
    r = _Draws(seed)
    return {"delta": _delta_inputs, "delta_step": _delta_inputs, "norm": _norm_inputs,
            "logprobs": _logprobs_inputs}[case["op"]](case, r)


def _delta_inputs(c, r):
    b, t, hq, hv, d = c["batch"], c.get("seq_len", 1), c["hq"], c["hv"], c["d"]
    io = _DT[c["io"]]
    # q | k | v of one convolution's output, b | a of one projection's
    qkv = torch.nn.functional.silu(r.normal(b, t, (2 * hq + hv) * d)).to(io)
    ba = r.normal(b, t, 2 * hv).to(_DT[c["gate"]])
    s = dict(op=c["op"], q=qkv[..., :hq * d].unflatten(-1, (hq, d)),
             k=qkv[..., hq * d:2 * hq * d].unflatten(-1, (hq, d)), v=qkv[..., 2 * hq * d:].unflatten(-1, (hv, d)),
             b=ba[..., :hv], a=ba[..., hv:], A_log=torch.log(r.uniform(hv, lo=1.0, hi=16.0)),
             dt_bias=torch.log(torch.expm1(torch.exp(r.uniform(hv, lo=math.log(1e-3), hi=math.log(0.1))))),
             state=r.normal(c["pool"], hv, d, d, std=0.1).to(_DT[c["state"]]), rows=r.rows(c["pool"], b, c["pad"]),
             lengths=r.lengths(b, t, c.get("ragged")), update=c.get("update", True),
             out=torch.empty(b, t, hv, d, dtype=io, device="cuda"))
    if c["op"] == "delta_step":
        s.update({k: s[k][:, 0] for k in ("q", "k", "v", "a", "b", "out")})
    return s


def _norm_inputs(c, r):
    rows, n, io = c["rows"], c["n"], _DT[c["io"]]
    # channels of different scale, a few of them large, as activations have them
    spread = torch.exp(r.normal(n, std=0.7))
    return dict(op="norm", x=(r.normal(rows, n) * spread).to(io), group=c["group"], unit=c["unit"], gate=c["gate"],
                weight=(r.normal(c["group"], std=0.2) + (0.0 if c["unit"] else 1.0)).to(io),
                residual=None if c["residual"] == "none" else r.normal(rows, n, std=2.0).to(_DT[c["residual"]]),
                z=None if c["gate"] == "none" else r.normal(rows, 2 * n).to(io)[:, n:],
                out=torch.empty(rows, n, dtype=_DT[c["out"]], device="cuda"), block=c["block"],
                scales=torch.empty(rows, n // c["block"], device="cuda") if c["block"] else None)


def _logprobs_inputs(c, r):
    rows, v = c["rows"], c["vocab"]
    logits = r.normal(rows, v, std=3.0)
    # the token that was sampled: the largest of a noisy copy
    noise = -torch.log(-torch.log(r.uniform(rows, v, lo=1e-6, hi=1.0 - 1e-6)))
    if c["masked"]:  # a third of the rows may only answer with a part of the vocabulary, one of them with a token
        keep = torch.rand((rows, v), generator=r.g, device="cuda") < 0.05
        keep[0] = False
        keep[:, 7] = True
        logits[::3] = torch.where(keep[::3], logits[::3], -math.inf)
    tokens = (logits + noise).argmax(1).to(torch.int32)
    return dict(op="logprobs", logits=logits.to(_DT[c["io"]]), tokens=tokens,
                logprobs=torch.empty(rows, device="cuda"), entropy=torch.empty(rows, device="cuda"),
                top_ids=torch.empty(rows, c["top"], dtype=torch.int32, device="cuda"),
                top_logprobs=torch.empty(rows, c["top"], device="cuda"))


# ---------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "logprobs":
        return _plain_logprobs(s)
    return _plain_delta(s)


def _own(s):
    import linear_rnn_recurrent_amd as lib
    if s["op"] == "delta":
        lib.ssu_delta_prefill(s["q"], s["k"], s["v"], s["a"], s["b"], s["state"], s["out"], A_log=s["A_log"],
                              dt_bias=s["dt_bias"], context_lengths=s["lengths"], state_indices=s["rows"],
                              update_state=s["update"])
        return s["out"], s["state"]
    if s["op"] == "delta_step":
        lib.ssu_delta_decode(s["q"], s["k"], s["v"], s["a"], s["b"], s["state"], s["out"], A_log=s["A_log"],
                             dt_bias=s["dt_bias"], state_indices=s["rows"])
        return s["out"], s["state"]
    if s["op"] == "norm":
        lib.ssu_rms_norm(s["x"], s["weight"], s["out"], residual=s["residual"], z=s["z"], scales=s["scales"],
                         group_size=s["group"], unit_offset=s["unit"], gate_first=s["gate"] == "before")
        return s["out"], s["scales"], s["residual"]
    lib.ssu_token_logprobs(s["logits"], s["tokens"], s["logprobs"], entropy=s["entropy"], top_ids=s["top_ids"],
                           top_logprobs=s["top_logprobs"])
    return s["logprobs"], s["entropy"], s["top_ids"], s["top_logprobs"]


def _plain_delta(s):
    """Tokens in chunks of up to 64: products within a chunk for all chunks at once, then chunk after chunk."""
    step = s["op"] == "delta_step"
    q, k, v, a, beta = (s[n][:, None].float() if step else s[n].float() for n in ("q", "k", "v", "a", "b"))
    b, t, hv, d = v.shape
    pool = s["state"]
    live = s["rows"] >= 0
    row = torch.where(live, s["rows"], pool.shape[0] - 1).long()  # padding reads the last, which nobody owns
    old = pool[row]
    length = torch.full_like(s["rows"], t) if s["lengths"] is None else s["lengths"]
    length = torch.where(live, length, 0)
    there = (torch.arange(t, device=v.device) < length[:, None])[..., None]
    g = torch.where(there, -torch.exp(s["A_log"]) * torch.nn.functional.softplus(a + s["dt_bias"]), 0.0)
    beta = torch.where(there, torch.sigmoid(beta), 0.0)
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6) * d ** -0.5
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)

    c = min(64, t)
    n = -(-t // c)

    def chunks(x):  # [b, t, h, ...] -> [b, hv, n, c, ...], behind the end zeros
        x = x.repeat_interleave(hv // x.shape[2], 2) if x.shape[2] < hv else x
        x = torch.cat([x, x.new_zeros(b, n * c - t, *x.shape[2:])], 1)
        return x.transpose(1, 2).unflatten(2, (n, c)).contiguous()

    q, k, v, g, beta = chunks(q), chunks(k), chunks(v), chunks(g), chunks(beta)
    total = g.cumsum(-1)
    at = torch.arange(c, device=v.device)
    upto = at[:, None] >= at
    decay = torch.exp(torch.where(upto, total[..., :, None] - total[..., None, :], -math.inf))
    kt = k.transpose(-1, -2).contiguous()
    power = torch.where(at[:, None] > at, beta[..., None] * decay * (k @ kt), 0.0)
    inverse = torch.eye(c, device=v.device) - power  # (I + L)^-1 = (I - L)(I + L^2)(I + L^4)...
    reach = 2
    while reach < c:
        power = power @ power
        inverse = inverse + inverse @ power
        reach *= 2
    begin = torch.exp(total)[..., None]
    fresh = inverse @ (beta[..., None] * v)
    seen = inverse @ (beta[..., None] * begin * k)
    within = decay * (q @ kt)
    q = q * begin
    end = torch.exp(total[..., -1:] - total)[..., None]
    kt = (k * end).contiguous()
    last = begin[..., -1:, :]
    state = old.float().transpose(-1, -2).contiguous()  # [b, hv, key, value]
    outs = []
    for i in range(n):
        u = fresh[:, :, i] - seen[:, :, i] @ state
        outs.append(q[:, :, i] @ state + within[:, :, i] @ u)
        state = last[:, :, i] * state + kt[:, :, i].transpose(-1, -2) @ u
    out = torch.stack(outs, 2).flatten(2, 3)[:, :, :t].transpose(1, 2)
    out = torch.where(there[..., None], out, 0.0).to(s["v"].dtype)
    if s["update"]:
        keep = (length > 0)[:, None, None, None]
        pool[row] = torch.where(keep, state.transpose(-1, -2).to(pool.dtype), old)
    return (out[:, 0] if step else out), pool


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
        s["residual"].copy_(h)
    z = None if s["z"] is None else s["z"].float()
    gate = None if z is None else z * torch.sigmoid(z)
    if s["gate"] == "before":
        h = h * gate
    rows, n = h.shape
    parts = h.unflatten(1, (n // s["group"], s["group"]))
    w = s["weight"].float() + (1.0 if s["unit"] else 0.0)
    y = (parts * torch.rsqrt((parts * parts).mean(-1, keepdim=True) + 1e-6) * w).flatten(1)
    if s["gate"] == "after":
        y = y * gate
    if s["scales"] is None:
        return y.to(s["out"].dtype), None, s["residual"]
    blocks = y.unflatten(1, (n // s["block"], s["block"]))
    scales = (blocks.abs().amax(-1) / 448.0).clamp_min(2.0 ** -126)
    return (blocks / scales[..., None]).flatten(1).to(s["out"].dtype), scales, s["residual"]


def _plain_logprobs(s):
    x = s["logits"].float()
    most = x.amax(-1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(-1, keepdim=True)
    norm = torch.log(total) + most
    mean = torch.where(e > 0, e * (x - most), 0.0).sum(-1) / total[:, 0]
    given = x.gather(1, s["tokens"].long()[:, None])
    best, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    k = s["top_ids"].shape[1]
    return ((given - norm)[:, 0], torch.log(total)[:, 0] - mean, ids[:, :k].to(torch.int32), best[:, :k] - norm)


# ---------------------------------------------------------------------------------------------------------
# What a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        e = _SIZE[c["io"]]
        sides = e + _SIZE[c["out"]] + (e if c["gate"] != "none" else 0)
        sides += 2 * _SIZE[c["residual"]] if c["residual"] != "none" else 0
        scales = 4 * c["rows"] * (c["n"] // c["block"]) if c["block"] else 0
        return {"bytes": c["rows"] * c["n"] * sides + c["group"] * e + scales, "flops": 6 * c["rows"] * c["n"]}
    if c["op"] == "logprobs":
        return {"bytes": c["rows"] * (c["vocab"] * _SIZE[c["io"]] + 12 + 8 * c["top"]),
                "flops": 6 * c["rows"] * c["vocab"]}
    b, t, hq, hv, d = c["batch"], c.get("seq_len", 1), c["hq"], c["hv"], c["d"]
    live = b - c["pad"]
    mean = 0.5625 if c.get("ragged") else 1.0  # lengths are even between an eighth of seq_len and all of it
    toks = live * t * mean
    io = _SIZE[c["io"]]
    sides = 2 if c.get("update", True) else 1
    return {"bytes": toks * ((2 * hq + hv) * d * io + 2 * hv * _SIZE[c["gate"]]) + b * t * hv * d * io
            + sides * live * hv * d * d * _SIZE[c["state"]], "flops": toks * hv * 7 * d * d}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "logprobs": _exact_logprobs}.get(case["op"], _exact_delta)(s)


def _exact_delta(s):
    """Token by token."""
    step = s["op"] == "delta_step"
    get = {n: (s[n][:, None] if step else s[n]).double() for n in ("q", "k", "v", "a", "b")}
    b, t, hv, d = get["v"].shape
    per = hv // get["q"].shape[2]
    pool = s["state"].double()
    lengths = [t] * b if s["lengths"] is None else s["lengths"].tolist()
    counts = torch.tensor([0 if r < 0 else n for r, n in zip(s["rows"].tolist(), lengths)], device=pool.device)
    S = pool[s["rows"].long().clamp_min(0)]
    dt = get["a"] + s["dt_bias"].double()
    dt = torch.where(dt > 40.0, dt, torch.log1p(torch.exp(dt.clamp_max(40.0))))
    alpha = torch.exp(-torch.exp(s["A_log"].double()) * dt)
    beta = 1.0 / (1.0 + torch.exp(-get["b"]))
    out = torch.zeros(b, t, hv, d, dtype=torch.float64, device=pool.device)
    heads = torch.arange(hv, device=pool.device) // per
    for i in range(t):
        go = (i < counts)[:, None, None]
        qi, ki = (x[:, i] / torch.sqrt((x[:, i] ** 2).sum(-1, keepdim=True) + 1e-6) for x in (get["q"], get["k"]))
        qi, ki = qi[:, heads], ki[:, heads]
        new = S * alpha[:, i, :, None, None]
        u = beta[:, i, :, None] * (get["v"][:, i] - (new * ki[:, :, None]).sum(-1))
        new = new + u[..., None] * ki[:, :, None]
        out[:, i] = torch.where(go, (new * qi[:, :, None]).sum(-1) / math.sqrt(d), 0.0)
        S = torch.where(go[..., None], new, S)
    if s["update"]:
        for i, n in enumerate(counts.tolist()):
            if n:
                pool[int(s["rows"][i])] = S[i]
    return (out[:, 0] if step else out), pool


def _exact_norm(s):
    h = s["x"].double()
    left = None
    if s["residual"] is not None:
        h = h + s["residual"].double()
        left = h
    if s["gate"] == "before":
        h = h * (s["z"].double() / (1.0 + torch.exp(-s["z"].double())))
    rows, n = h.shape
    parts = h.reshape(rows, -1, s["group"])
    rms = torch.sqrt((parts ** 2).sum(-1) / s["group"] + 1e-6)
    w = s["weight"].double() + (1.0 if s["unit"] else 0.0)
    y = (parts / rms[..., None] * w).reshape(rows, n)
    if s["gate"] == "after":
        y = y * (s["z"].double() / (1.0 + torch.exp(-s["z"].double())))
    if s["scales"] is None:
        return y, None, left
    blocks = y.reshape(rows, -1, s["block"])
    scales = torch.clamp(blocks.abs().max(-1).values / 448.0, min=2.0 ** -126)
    v = blocks / scales[..., None]
    # three bits behind the leading one, none below 2^-9
    lead = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    ulp = torch.exp2(lead - 3.0)
    return (torch.round(v / ulp) * ulp).reshape(rows, n), scales, left


def _exact_logprobs(s):
    x = s["logits"].double()
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    entropy = -torch.where(p > 0, p * (x - lse[:, None]), 0.0).sum(-1)
    given = x[torch.arange(x.shape[0], device=x.device), s["tokens"].long()] - lse
    best = torch.topk(x, s["top_ids"].shape[1], -1).values - lse[:, None]
    return given, entropy, None, best
