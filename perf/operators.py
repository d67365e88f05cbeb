"""Cases of the causal convolution, the per-channel selective scan and draft verification.

Each case is one pass of one operator as a serving loop calls it: a prompt (``seq_len`` tokens of every
sequence), a single token a sequence (``step``), a window of drafted tokens with the state read only, or the
verification of drafted tokens. ``run`` computes the plain form, or the framework's kernels where ``own`` is set.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # the convolution in front of the heads' state update: 5,120 channels of x, 128 of B, 128 of C,
        # eight prompts of different lengths padded to 512 tokens
        dict(name="conv_prompts", op="conv", batch=8, seq_len=512, dim=5376, width=4, io="bf16", state="bf16",
             pool=64, pad=0, ragged=True, update=True),
        # one long prompt, x a half of the input projection's output
        dict(name="conv_long_prompt", op="conv", batch=1, seq_len=4099, dim=5120, width=4, io="bf16",
             state="bf16", pool=4, pad=0, ragged=False, update=True),
        # a window of drafted tokens, the state only read
        dict(name="conv_window", op="conv", batch=32, seq_len=5, dim=2560, width=3, io="f16", state="f16",
             pool=48, pad=3, ragged=False, update=False),
        # one token of each of 64 sequences
        dict(name="conv_step", op="conv_step", batch=64, dim=5376, width=4, io="bf16", state="bf16", pool=256,
             pad=0),
        # one long prompt of a per-channel model: few rows, work split over time
        dict(name="scan_long_prompt", op="scan", batch=1, seq_len=2048, dim=5120, dstate=16, groups=1, io="bf16",
             dt="bf16", state="f32", pool=4, pad=0, ragged=False, update=True, gate=True),
        # eight prompts of different lengths, one row of padding
        dict(name="scan_prompts", op="scan", batch=8, seq_len=777, dim=2560, dstate=16, groups=1, io="f16",
             dt="f32", state="f32", pool=16, pad=1, ragged=True, update=True, gate=True),
        # a wide state in groups, everything in 32 bits
        dict(name="scan_wide_state", op="scan", batch=2, seq_len=509, dim=1536, dstate=64, groups=2, io="f32",
             dt="f32", state="f32", pool=3, pad=0, ragged=False, update=True, gate=False),
        # a window of drafted tokens, the state only read
        dict(name="scan_window", op="scan", batch=16, seq_len=5, dim=5120, dstate=16, groups=1, io="bf16",
             dt="bf16", state="f32", pool=32, pad=2, ragged=False, update=False, gate=True),
        # one token of each of 64 sequences, and of one
        dict(name="scan_step", op="scan_step", batch=64, dim=5120, dstate=16, groups=1, io="bf16", dt="bf16",
             state="f32", pool=128, pad=0, gate=True),
        dict(name="scan_step_single", op="scan_step", batch=1, dim=1536, dstate=16, groups=1, io="bf16",
             dt="f32", state="f32", pool=4, pad=0, gate=True),
        # seven drafted tokens of each of 64 sequences over a large vocabulary, drafts sampled from a small model
        dict(name="verify_chains", op="verify", batch=64, tokens=8, vocab=131072, probs="f32", tree=False,
             draft=True, pad=0),
        # draft trees over a vocabulary of ordinary size, drafts the most probable tokens
        dict(name="verify_trees", op="verify", batch=16, tokens=64, vocab=32000, probs="bf16", tree=True,
             draft=False, pad=1),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def pick(*of):
        return rng.choice(of)

    op = pick("conv", "conv_step", "scan", "scan", "scan_step", "verify")
    batch = size(1, 64)
    io = pick("f32", "f16", "bf16")
    if op == "conv":
        dim = size(64, 8192)
        seq = min(size(1, 4099), max(1, (1 << 24) // (batch * dim)))
        return dict(op=op, batch=batch, seq_len=seq, dim=dim, width=pick(2, 3, 4, 4, 5, 8), io=io,
                    state=pick(io, "f32"), pool=batch + size(1, 64), pad=rng.randint(0, batch // 4),
                    ragged=pick(True, False), update=pick(True, True, False))
    if op == "conv_step":
        return dict(op=op, batch=batch, dim=size(64, 8192), width=pick(2, 3, 4, 4, 5, 8), io=io,
                    state=pick(io, "f32"), pool=batch + size(1, 64), pad=rng.randint(0, batch // 4))
    if op == "verify":
        tree = pick(True, False)
        tokens = size(2, 64) if tree else size(1, 16)
        vocab = min(size(1000, 131072), (1 << 26) // (batch * tokens))
        return dict(op=op, batch=batch, tokens=tokens, vocab=vocab, probs=io, tree=tree,
                    draft=False if tree else pick(True, True, False), pad=rng.randint(0, batch // 4))
    groups = pick(1, 1, 1, 2, 4)
    dim = groups * size(max(1, 64 // groups), 8192 // groups)
    dstate = pick(8, 16, 16, 16, 24, 32, 64, 128)
    case = dict(op=op, batch=batch, dim=dim, dstate=dstate, groups=groups, io=io, dt=pick(io, "f32"),
                state=pick("f32", "f32", "f16", "bf16"), pool=batch + size(1, 32),
                pad=rng.randint(0, batch // 4), gate=pick(True, False))
    if op == "scan":
        case.update(seq_len=min(size(1, 2048), max(1, (1 << 27) // (batch * dim * dstate))),
                    ragged=pick(True, False), update=pick(True, True, False))
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
        i = torch.cat([i, i.new_full((batch - i.numel(),), -1)])
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
    return {"conv": _conv_inputs, "conv_step": _conv_inputs, "scan": _scan_inputs, "scan_step": _scan_inputs,
            "verify": _verify_inputs}[case["op"]](case, r)


def _conv_inputs(c, r):
    b, t, d, w = c["batch"], c.get("seq_len", 1), c["dim"], c["width"]
    io = _DT[c["io"]]
    x = r.normal(b, t, 2 * d).to(io)[..., :d]  # the first half of the input projection's output
    s = dict(op=c["op"], x=x, weight=r.normal(d, w, std=w ** -0.5).to(io), bias=r.normal(d, std=0.1).to(io),
             conv_state=r.normal(c["pool"], d, w - 1).to(_DT[c["state"]]),
             rows=r.rows(c["pool"], b, c["pad"]), lengths=r.lengths(b, t, c.get("ragged")),
             update=c.get("update", True), out=torch.empty(b, t, d, dtype=io, device="cuda"))
    if c["op"] == "conv_step":
        s["x"], s["out"] = s["x"][:, 0], s["out"][:, 0]
    return s


def _scan_inputs(c, r):
    b, t, d, n, g = c["batch"], c.get("seq_len", 1), c["dim"], c["dstate"], c["groups"]
    io = _DT[c["io"]]
    rank = d // 32
    low = r.normal(b, t, rank + 2 * g * n).to(io)  # dt's low-rank part, B and C of one projection
    s = dict(op=c["op"], x=torch.nn.functional.silu(r.normal(b, t, d)).to(io),
             A=-torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * r.uniform(d, n, lo=0.8, hi=1.25),
             B=low[..., rank:rank + g * n].unflatten(-1, (g, n)), C=low[..., rank + g * n:].unflatten(-1, (g, n)),
             dt=r.normal(b, t, d, std=0.5).to(_DT[c["dt"]]),
             dt_bias=torch.log(torch.expm1(torch.exp(r.uniform(d, lo=math.log(1e-3), hi=math.log(0.1))))),
             D=r.normal(d), z=r.normal(b, t, 2 * d).to(io)[..., d:] if c["gate"] else None,
             state=r.normal(c["pool"], d, n).to(_DT[c["state"]]), rows=r.rows(c["pool"], b, c["pad"]),
             lengths=r.lengths(b, t, c.get("ragged")), update=c.get("update", True),
             out=torch.empty(b, t, d, dtype=io, device="cuda"))
    if c["op"] == "scan_step":
        s.update({k: s[k][:, 0] for k in ("x", "B", "C", "dt", "z", "out") if s[k] is not None})
    return s


def _verify_inputs(c, r):
    b, t, v = c["batch"], c["tokens"], c["vocab"]
    dt = _DT[c["probs"]]
    logits = r.normal(b, t, v, std=4.0)
    p = logits.softmax(-1).to(dt)
    s = dict(op="verify", target_probs=p, uniforms=r.uniform(b, t).clamp_max_(1 - 2.0 ** -24),
             accepted=torch.empty(b, dtype=torch.int32, device="cuda"),
             next=torch.empty(b, dtype=torch.int32, device="cuda"),
             path=torch.empty(b, t, dtype=torch.int32, device="cuda"),
             draft_probs=None, parents=None,
             lengths=torch.randint(1, t + 1, (b,), generator=r.g, device="cuda", dtype=torch.int32))
    s["lengths"][::2] = t
    if c["pad"]:
        s["lengths"][b - c["pad"]:] = 0
    first = torch.randint(0, v, (b, 1), generator=r.g, device="cuda")
    if c["tree"]:
        # every node but the root hangs under an earlier one; a node's j-th child is the j-th most probable
        # token of a noisy copy of its distribution
        gc = torch.Generator().manual_seed(r.g.initial_seed())
        par = (torch.rand(b, t, generator=gc) * torch.arange(t).clamp_max(24)).long()
        par[:, 0] = -1
        same = (par[:, :, None] == par[:, None, :]) & (torch.arange(t)[None] < torch.arange(t)[:, None])
        rank = same.sum(-1).cuda()
        s["parents"] = par.to(torch.int32).cuda()
        k = min(v, int(rank.max()) + 1)
        top = (logits + r.normal(b, t, v)).topk(k, -1).indices
        at = s["parents"].long().clamp_min(0)
        tok = top.gather(1, at[..., None].expand(b, t, k)).gather(2, rank.clamp_max(k - 1)[..., None])[..., 0]
        s["tokens"] = torch.cat([first, tok[:, 1:]], 1).to(torch.int32)
    else:
        q = (logits[:, :t - 1] + r.normal(b, t - 1, v)).softmax(-1)
        tok = torch.multinomial(q.reshape(-1, v), 1, generator=r.g).reshape(b, t - 1) if t > 1 else first[:, :0]
        s["tokens"] = torch.cat([first, tok], 1).to(torch.int32)
        if c["draft"]:
            s["draft_probs"] = q.to(dt)
    return s


# ---------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    if s["op"] in ("conv", "conv_step"):
        return _plain_conv(s)
    if s["op"] in ("scan", "scan_step"):
        return _plain_scan(s)
    return _plain_verify(s)


def _own(s):
    import linear_rnn_recurrent_amd as lib
    if s["op"] == "conv":
        lib.ssu_conv_prefill(s["x"], s["weight"], s["bias"], s["conv_state"], s["out"], silu=True,
                             context_lengths=s["lengths"], state_indices=s["rows"], update_state=s["update"])
        return s["out"], s["conv_state"]
    if s["op"] == "conv_step":
        lib.ssu_conv_decode(s["x"], s["weight"], s["bias"], s["conv_state"], s["out"], silu=True,
                            state_indices=s["rows"])
        return s["out"], s["conv_state"]
    if s["op"] == "scan":
        lib.ssu_scan_prefill(s["x"], s["A"], s["B"], s["C"], s["dt"], s["state"], s["out"],
                             dt_bias=s["dt_bias"], D=s["D"], z=s["z"], dt_softplus=True,
                             context_lengths=s["lengths"], state_indices=s["rows"], update_state=s["update"])
        return s["out"], s["state"]
    if s["op"] == "scan_step":
        lib.ssu_scan_decode(s["x"], s["A"], s["B"], s["C"], s["dt"], s["state"], s["out"],
                            dt_bias=s["dt_bias"], D=s["D"], z=s["z"], dt_softplus=True,
                            state_indices=s["rows"])
        return s["out"], s["state"]
    lib.ssu_draft_verify(s["tokens"], s["target_probs"], s["uniforms"], s["accepted"], s["next"],
                         draft_probs=s["draft_probs"], parent_ids=s["parents"], context_lengths=s["lengths"],
                         accepted_node_ids=s["path"])
    return s["accepted"], s["next"], s["path"]


def _live(rows, pool_rows):
    """Whether each row is none of padding, and the pool row it reads (padding: the last, which nobody owns)."""
    live = rows >= 0
    return live, torch.where(live, rows, pool_rows - 1).long()


def _plain_conv(s):
    step = s["op"] == "conv_step"
    x = s["x"].float()
    x = x[:, None] if step else x
    b, t, d = x.shape
    pool = s["conv_state"]
    live, row = _live(s["rows"], pool.shape[0])
    old = pool[row]
    window = torch.cat([old.float().transpose(1, 2), x], 1)
    w = s["weight"].shape[1]
    y = (window.unfold(1, w, 1) * s["weight"].float()).sum(-1) + s["bias"].float()
    y = y * torch.sigmoid(y)
    length = torch.full_like(s["rows"], t) if s["lengths"] is None else s["lengths"]
    length = torch.where(live, length, 0).long()
    there = torch.arange(t, device=x.device) < length[:, None]
    out = torch.where(there[..., None], y, 0.0).to(s["x"].dtype)
    if s["update"]:
        at = length[:, None] + torch.arange(w - 1, device=x.device)
        new = window.gather(1, at[..., None].expand(b, w - 1, d)).transpose(1, 2)
        pool[row] = torch.where(live[:, None, None], new.to(pool.dtype), old)
    return (out[:, 0] if step else out), pool


def _plain_scan(s):
    step = s["op"] == "scan_step"
    x, dt, B, C, z = (None if s[k] is None else s[k].float() for k in ("x", "dt", "B", "C", "z"))
    if step:
        x, dt, B, C = x[:, None], dt[:, None], B[:, None], C[:, None]
        z = None if z is None else z[:, None]
    b, t, d = x.shape
    g = B.shape[2]
    pool = s["state"]
    live, row = _live(s["rows"], pool.shape[0])
    old = pool[row]
    length = torch.full_like(s["rows"], t) if s["lengths"] is None else s["lengths"]
    length = torch.where(live, length, 0)
    there = torch.arange(t, device=x.device) < length[:, None]
    dt = torch.nn.functional.softplus(dt + s["dt_bias"])
    dt = torch.where(there[..., None], dt, 0.0)  # tokens behind a sequence's end leave the state
    decay = torch.exp(dt[..., None] * s["A"])
    heads = B.repeat_interleave(d // g, 2)
    state = (dt * x)[..., None] * heads
    state[:, 0] += decay[:, 0] * old.float()
    del heads
    # state[i] = decay[i] state[i-1] + state[i] for all i, by doubling the reach of each token
    reach = 1
    while reach < t:
        state = torch.cat([state[:, :reach], torch.addcmul(state[:, reach:], decay[:, reach:], state[:, :-reach])], 1)
        if 2 * reach < t:
            decay = torch.cat([decay[:, :reach], decay[:, reach:] * decay[:, :-reach]], 1)
        reach *= 2
    y = (state * C.repeat_interleave(d // g, 2)).sum(-1) + s["D"] * x
    if z is not None:
        y = y * (z * torch.sigmoid(z))
    out = torch.where(there[..., None], y, 0.0).to(s["x"].dtype)
    if s["update"]:
        keep = live & (length > 0)
        pool[row] = torch.where(keep[:, None, None], state[:, -1].to(pool.dtype), old)
    return (out[:, 0] if step else out), pool


def _plain_verify(s):
    p, u, tok = s["target_probs"], s["uniforms"].double(), s["tokens"].long()
    b, t, v = p.shape
    node = torch.arange(t, device=p.device)
    length = s["lengths"]
    there = node < length[:, None]
    if s["parents"] is None:
        parent = (node - 1).expand(b, t)
    else:
        parent = s["parents"].long()
    above = parent.clamp_min(0)
    there = there & (parent >= 0)
    at = p.flatten(1).gather(1, above * v + tok).double()  # p of each drafted token where it was drafted
    older = (parent[:, :, None] == parent[:, None, :]) & (node[None] < node[:, None]) & there[:, None, :]
    if s["draft_probs"] is not None:
        odds = s["draft_probs"].flatten(1).gather(1, (node[:-1] * v) + tok[:, 1:]).double()
        accept = torch.cat([there[:, :1], u[:, 1:] * odds < at[:, 1:]], 1) & there
        removed_of = None
    else:
        again = (older & (tok[:, :, None] == tok[:, None, :])).any(-1)  # a token that a sibling had before
        at = torch.where(again | ~there, 0.0, at)
        removed = torch.matmul(older.double(), at[..., None])[..., 0]
        accept = (u * (1.0 - removed) < at) & there
        removed_of = at
    chosen = accept & ~(older & accept[:, None, :]).any(-1)
    # on the path: chosen, and all its ancestors; by doubling
    on = chosen | (node == 0)
    up = above
    reach = 1
    while reach < t:
        on = on & on.gather(1, up)
        up = up.gather(1, up)
        reach *= 2
    some = length > 0
    on = on & (node < length[:, None])
    count = torch.where(some, on.sum(1), 0)
    path = torch.sort(torch.where(on, node, t), 1).values
    path = torch.where(node < count[:, None], path, -1)
    last = path.gather(1, (count - 1).clamp_min(0)[:, None])[:, 0].clamp_min(0)
    full = p[torch.arange(b, device=p.device), last].double()
    weight = full.clone()
    if s["draft_probs"] is not None:
        if t > 1:
            rejected = last + 1 < length
            q = s["draft_probs"][torch.arange(b, device=p.device), last.clamp_max(t - 2)].double()
            weight = torch.where(rejected[:, None], (full - q).clamp_min(0.0), full)
    else:
        child = there & (parent == last[:, None])
        weight.scatter_reduce_(1, tok, torch.where(child, 0.0, math.inf).double(), "amin")
    weight = torch.where((weight > 0).any(1, keepdim=True), weight, full)
    sums = weight.cumsum(1)
    drawn = (sums > u[:, :1] * sums[:, -1:]).to(torch.uint8).argmax(1)
    nxt = torch.where(some, drawn, -1)
    return count.to(torch.int32), nxt.to(torch.int32), path.to(torch.int32)


# ---------------------------------------------------------------------------------------------------------
# What a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    b = c["batch"]
    live = b - c["pad"]
    if c["op"] == "verify":
        rows = 2 if c["draft"] else 1
        e = _SIZE[c["probs"]]
        return {"bytes": live * (rows * c["vocab"] * e + c["tokens"] * (12 + 2 * e)),
                "flops": live * c["vocab"] * (1 + rows)}
    t, d = c.get("seq_len", 1), c["dim"]
    mean = 0.5625 if c.get("ragged") else 1.0  # lengths are even between an eighth of seq_len and all of it
    toks = live * t * mean
    io, st = _SIZE[c["io"]], _SIZE[c["state"]]
    sides = 2 if c.get("update", True) else 1
    if c["op"] in ("conv", "conv_step"):
        w = c["width"]
        return {"bytes": toks * d * io + b * t * d * io + d * (w + 1) * io + sides * live * d * (w - 1) * st,
                "flops": toks * d * (2 * w + 4)}
    n, g = c["dstate"], c["groups"]
    per = d * ((2 if c["gate"] else 1) * io + _SIZE[c["dt"]]) + 2 * g * n * io
    return {"bytes": toks * per + b * t * d * io + d * (n + 2) * 4 + sides * live * d * n * st,
            "flops": toks * d * (7 * n + 12)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("conv", "conv_step"):
        return _exact_conv(s)
    if case["op"] in ("scan", "scan_step"):
        return _exact_scan(s)
    return _exact_verify(s)


def _counts(s, b, t):
    lengths = [t] * b if s["lengths"] is None else s["lengths"].tolist()
    return [0 if r < 0 else max(0, min(t, n)) for r, n in zip(s["rows"].tolist(), lengths)]


def _exact_conv(s):
    step = s["op"] == "conv_step"
    x = (s["x"][:, None] if step else s["x"]).double()
    weight, bias = s["weight"].double(), s["bias"].double()
    pool = s["conv_state"].double()
    b, t, d = x.shape
    out = torch.zeros(b, t, d, dtype=torch.float64, device=x.device)
    for i, n in enumerate(_counts(s, b, t)):
        if n == 0:
            continue
        row = int(s["rows"][i])
        seen = torch.cat([pool[row].t(), x[i, :n]], 0)
        acc = bias.repeat(n, 1)
        for j in range(weight.shape[1]):
            acc += weight[:, j] * seen[j:j + n]
        out[i, :n] = acc / (1.0 + torch.exp(-acc))
        if s["update"]:
            pool[row] = seen[n:].t()
    return (out[:, 0] if step else out), pool


def _exact_scan(s):
    step = s["op"] == "scan_step"
    get = {k: None if s[k] is None else (s[k][:, None] if step else s[k]) for k in ("x", "dt", "B", "C", "z")}
    x, dt = get["x"].double(), get["dt"].double() + s["dt_bias"].double()
    dt = torch.where(dt > 40.0, dt, torch.log1p(torch.exp(dt.clamp_max(40.0))))
    pool, A = s["state"].double(), s["A"].double()
    b, t, d = x.shape
    counts = _counts(s, b, t)
    length = torch.tensor(counts, device=x.device)
    rows = s["rows"].long().clamp_min(0)
    h = pool[rows]
    group = torch.arange(d, device=x.device) // (d // get["B"].shape[2])
    out = torch.zeros(b, t, d, dtype=torch.float64, device=x.device)
    for k in range(t):
        go = (k < length)[:, None]
        Bk, Ck = get["B"][:, k].double()[:, group], get["C"][:, k].double()[:, group]
        nh = h * torch.exp(dt[:, k, :, None] * A) + Bk * (dt[:, k] * x[:, k])[..., None]
        h = torch.where(go[..., None], nh, h)
        y = (h * Ck).sum(-1) + s["D"].double() * x[:, k]
        if get["z"] is not None:
            zk = get["z"][:, k].double()
            y = y * zk / (1.0 + torch.exp(-zk))
        out[:, k] = torch.where(go, y, 0.0)
    if s["update"]:
        for i, n in enumerate(counts):
            if n:
                pool[int(s["rows"][i])] = h[i]
    return (out[:, 0] if step else out), pool


def _exact_verify(s):
    b, t, v = s["target_probs"].shape
    tok, u, lengths = s["tokens"].tolist(), s["uniforms"].double().tolist(), s["lengths"].tolist()
    parents = None if s["parents"] is None else s["parents"].tolist()
    accepted, drawn, paths = [], [], []
    for i in range(b):
        n = lengths[i]
        if n <= 0:
            accepted.append(0)
            drawn.append(-1)
            paths.append([-1] * t)
            continue

        def dist(which, k):
            return s[which][i, k].double().cpu().numpy()

        at, p, w = 0, dist("target_probs", 0), None
        path = [0]
        if s["draft_probs"] is not None:
            w = p
            for k in range(1, n):
                q = dist("draft_probs", k - 1)
                if not u[i][k] * q[tok[i][k]] < p[tok[i][k]]:
                    w = np.maximum(p - q, 0.0)
                    break
                path.append(k)
                p = w = dist("target_probs", k)
        else:
            w, left = p.copy(), 1.0
            for k in range(1, n):
                par = parents[i][k] if parents is not None else k - 1
                if par != at:
                    continue
                if u[i][k] * left < w[tok[i][k]]:
                    at = k
                    path.append(k)
                    p = dist("target_probs", k)
                    w, left = p.copy(), 1.0
                else:
                    left -= w[tok[i][k]]
                    w[tok[i][k]] = 0.0
        if not w.any():
            w = p
        c = np.cumsum(w)
        accepted.append(len(path))
        drawn.append(int(np.argmax(c > u[i][0] * c[-1])))
        paths.append(path + [-1] * (t - len(path)))
    return tuple(torch.tensor(a, dtype=torch.int32) for a in (accepted, drawn, paths))
