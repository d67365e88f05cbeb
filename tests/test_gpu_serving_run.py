"""One layer of a gated-delta-rule model as a serving loop runs it, through the calls of this
library: norm with the residual, convolution, delta rule, gated norm, log probabilities, draft
verification and the commit of what was accepted. Every stage is checked against the fp64 oracle on
the inputs that it got."""
import numpy as np
import pytest
import torch

import linear_rnn_recurrent_amd as L
from oracle import sequence, serving
from sequence_helpers import U, check, conv_bound, f64

pytestmark = pytest.mark.gpu

HQ, HV, D, HIDDEN, VOCAB, W = 2, 4, 64, 256, 1500, 4
QKV = (2 * HQ + HV) * D


class Layer:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).cuda()  # noqa: E731
        self.embed = r(VOCAB, HIDDEN).bfloat16()
        self.norm_w, self.out_w = r(HIDDEN, std=0.1).bfloat16(), (1 + r(D, std=0.1)).bfloat16()
        self.w_in = r(HIDDEN, QKV + HV * D + 2 * HV, std=HIDDEN ** -0.5).bfloat16()
        self.w_out = r(HV * D, HIDDEN, std=(HV * D) ** -0.5).bfloat16()
        self.conv_w, self.conv_b = r(QKV, W, std=0.5).bfloat16(), r(QKV, std=0.1).bfloat16()
        self.A_log = torch.log(torch.rand(HV, generator=g) * 15 + 1).cuda()
        self.dt_bias = (torch.rand(HV, generator=g) * 2 - 5).cuda()
        self.pools = torch.zeros(6, QKV, W - 1, dtype=torch.bfloat16, device="cuda"), \
            torch.zeros(6, HV, D, D, device="cuda")

    def window(self, tokens, rows, *, update, lengths=None, look=False):
        """Logits of tokens [b, t]; the layer's states advance with update."""
        b, t = tokens.shape
        conv, ssm = self.pools
        x = self.embed[tokens.long()]
        residual = torch.zeros(b, t, HIDDEN, device="cuda")
        n = torch.empty_like(x)
        L.ssu_rms_norm(x, self.norm_w, n, residual=residual, unit_offset=True)
        y = (n.flatten(0, 1) @ self.w_in).unflatten(0, (b, t))
        qkv, z, ba = y[..., :QKV], y[..., QKV:QKV + HV * D], y[..., QKV + HV * D:]
        before = conv.clone(), ssm.clone()
        u = torch.empty(b, t, QKV, dtype=torch.bfloat16, device="cuda")
        L.ssu_conv_prefill(qkv, self.conv_w, self.conv_b, conv, u, context_lengths=lengths, state_indices=rows,
                           update_state=update)
        o = torch.empty(b, t, HV, D, dtype=torch.bfloat16, device="cuda")
        q, k = (u[..., i * HQ * D:(i + 1) * HQ * D].unflatten(-1, (HQ, D)) for i in range(2))
        v = u[..., 2 * HQ * D:].unflatten(-1, (HV, D))
        L.ssu_delta_prefill(q, k, v, ba[..., HV:], ba[..., :HV], ssm, o, A_log=self.A_log, dt_bias=self.dt_bias,
                            context_lengths=lengths, state_indices=rows, update_state=update)
        m = torch.empty(b, t, HV * D, dtype=torch.bfloat16, device="cuda")
        L.ssu_rms_norm(o.flatten(2), self.out_w, m, z=z, group_size=D)
        h = (m.flatten(0, 1) @ self.w_out).unflatten(0, (b, t))
        f = torch.empty_like(h)
        L.ssu_rms_norm(h, self.norm_w, f, residual=residual, unit_offset=True)
        logits = f.float() @ self.embed.float().t()
        self.commit = (qkv, q, k, v, ba)
        if look:
            self.check(x, n, residual, h, qkv, u, before, q, k, v, ba, o, z, m, f, lengths, rows, update)
        return logits

    def check(self, x, n, residual, h, qkv, u, before, q, k, v, ba, o, z, m, f, lengths, rows, update):
        rel = (HIDDEN / 2 + 24) * U
        y, _ = serving.rms_norm(f64(x), f64(self.norm_w), unit=True)
        check(n, y, rel * np.abs(y), torch.bfloat16, "norm")
        conv, ssm = f64(before[0]), f64(before[1])
        ctx, idx = None if lengths is None else f64(lengths), f64(rows)
        y, mag = sequence.causal_conv(f64(qkv), f64(self.conv_w), f64(self.conv_b), conv, ctx=ctx, idx=idx, update=update)
        check(u, y, conv_bound(y, mag, W), torch.bfloat16, "convolution")
        y, bound, sbound = serving.gated_delta(f64(q), f64(k), f64(v), f64(ba[..., HV:]), f64(ba[..., :HV]), ssm,
                                               A_log=f64(self.A_log), dt_bias=f64(self.dt_bias), ctx=ctx, idx=idx,
                                               update=update)
        check(o, y, bound, torch.bfloat16, "delta rule")
        if update:
            check(self.pools[1], ssm, sbound[..., None] + 0 * ssm, torch.float32, "state")
        y, _ = serving.rms_norm(f64(o.flatten(2)), f64(self.out_w), z=f64(z), group=D)
        check(m, y, (D / 2 + 24 + np.abs(f64(z))) * U * np.abs(y), torch.bfloat16, "gated norm")
        y, left = serving.rms_norm(f64(h), f64(self.norm_w), residual=f64(x), unit=True)
        check(residual, left, U * np.abs(left), torch.float32, "residual")
        inv = 1 / np.sqrt((left ** 2).mean(-1, keepdims=True))
        loss = U * (np.abs(f64(x)) + np.abs(f64(h))) * inv * (1 + np.abs(f64(self.norm_w)))
        check(f, y, rel * np.abs(y) + loss, torch.bfloat16, "second norm")


@pytest.mark.parametrize("prompt", [7, 90])
def test_prompt_window_verification_commit(prompt):
    layer = Layer(1)
    g = torch.Generator().manual_seed(2)
    b, t = 3, 6
    rows = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    lengths = torch.tensor([prompt, prompt // 2, 1], dtype=torch.int32).cuda()
    tokens = torch.randint(0, VOCAB, (b, prompt), generator=g).int().cuda()
    layer.window(tokens, rows, update=True, lengths=lengths, look=True)
    after_prompt = [p.clone() for p in layer.pools]

    # drafts: the model's own choices along the window, one of them spoiled
    drafts = torch.randint(0, VOCAB, (b, t), generator=g).int().cuda()
    for i in range(1, t):
        logits = layer.window(drafts, rows, update=False)
        drafts[:, i] = logits[:, i - 1].argmax(-1).int()
    drafts[1, 3] = (drafts[1, 3] + 7) % VOCAB
    logits = layer.window(drafts, rows, update=False, look=True)
    for p, q in zip(layer.pools, after_prompt):
        assert torch.equal(p, q)

    # the drafts are the likeliest tokens: log probabilities, alternatives, entropy of each position
    new = lambda *s, **k: torch.empty(b, t, *s, device="cuda", **k)  # noqa: E731
    lp, ent, ids, best = new(), new(), new(4, dtype=torch.int32), new(4)
    following = torch.cat([drafts[:, 1:], torch.full((b, 1), -1, dtype=torch.int32, device="cuda")], 1)
    L.ssu_token_logprobs(logits, following, lp, entropy=ent, top_ids=ids, top_logprobs=best)
    ref = serving.token_logprobs(f64(logits), f64(following), 4)
    assert (f64(ids) == ref[2]).all()
    for got, want in ((lp, ref[0]), (ent, ref[1]), (best, ref[3])):
        fine = np.isfinite(want)
        assert (np.abs(f64(got)[fine] - want[fine]) <= 60 * U * (1 + np.abs(want[fine]) + np.log(VOCAB))).all()
    assert torch.isinf(lp[:, -1]).all()
    assert (ids[0, :t - 1, 0] == drafts[0, 1:]).all()

    # sharpened so that the argmax all but surely stands; the spoiled draft does not
    probs = torch.softmax(logits * 40.0, -1)
    accepted, nxt = (torch.empty(b, dtype=torch.int32, device="cuda") for _ in range(2))
    uniforms = torch.full((b, t), 0.5, device="cuda")
    L.ssu_draft_verify(drafts, probs, uniforms, accepted, nxt, state_indices=rows)
    assert accepted.tolist()[1] == 3 and min(accepted.tolist()) >= 3

    # commit of the accepted lengths without outputs: as those tokens run for themselves
    qkv, q, k, v, ba = layer.commit
    conv, ssm = layer.pools
    L.ssu_conv_prefill(qkv, layer.conv_w, layer.conv_b, conv, None, state_indices=rows, context_lengths=accepted)
    L.ssu_delta_prefill(None, k, v, ba[..., HV:], ba[..., :HV], ssm, None, A_log=layer.A_log, dt_bias=layer.dt_bias,
                        state_indices=rows, context_lengths=accepted)
    committed = [p.clone() for p in layer.pools]
    for p, q0 in zip(layer.pools, after_prompt):
        p.copy_(q0)
    layer.window(drafts, rows, update=True, lengths=accepted, look=True)
    assert torch.equal(layer.pools[0], committed[0])
    assert torch.equal(layer.pools[1], committed[1])
