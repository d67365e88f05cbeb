"""A per-channel model's decode loop with drafted windows, as a server runs it:
convolution and scan over the fed window with the state read only, verification,
then the commit of the accepted tokens, all on device results. Afterwards the
pools are those of prefills of exactly the accepted tokens."""
import pytest
import torch

import oracle
from linear_rnn_recurrent_amd import (ssu_conv_decode, ssu_conv_prefill, ssu_draft_verify,
                                      ssu_scan_decode, ssu_scan_prefill, verify_workspace_bytes)
from gpu_helpers import assert_bitwise
from sequence_helpers import check, conv_inputs, f64, scan_bound, scan_inputs, verify_inputs

pytestmark = pytest.mark.gpu

B, T, D, N, V = 4, 5, 192, 16, 400


class Loop:
    def __init__(self):
        self.c = conv_inputs(1, batch=B, seq_len=T, channels=D, width=4, pool=B + 2, io="f32",
                             idx=[5, 0, -1, 3])
        self.s = scan_inputs(2, batch=B, seq_len=T, dim=D, dstate=N, pool=B + 2, io="f32")
        self.s["idx"] = self.c["idx"]
        self.v = verify_inputs(3, batch=B, tokens=T, vocab=V, sharp=6.0)
        self.conv_out, self.out = torch.empty_like(self.c["x"]), torch.empty_like(self.s["x"])
        self.acc = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.next = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")

    def conv(self, out, **kw):
        ssu_conv_prefill(self.c["x"], self.c["weight"], self.c["bias"], self.c["conv_state"], out,
                         state_indices=self.c["idx"], **kw)

    def scan(self, out, **kw):
        s = self.s
        ssu_scan_prefill(self.conv_out, s["A"], s["B"], s["C"], s["dt"], s["state"], out,
                         dt_bias=s["dt_bias"], D=s["D"], z=s["z"], state_indices=s["idx"], **kw)

    def step(self):
        self.conv(self.conv_out, update_state=False)
        self.scan(self.out, update_state=False)
        ssu_draft_verify(self.v["tokens"], self.v["target"], self.v["uniforms"], self.acc, self.next,
                         draft_probs=self.v["draft"], state_indices=self.c["idx"], workspace=self.ws)
        self.conv(None, context_lengths=self.acc)
        self.scan(None, context_lengths=self.acc)

    def pools(self):
        return self.c["conv_state"], self.s["state"]


def test_window_verify_commit():
    m = Loop()
    conv0, scan0 = (p.clone() for p in m.pools())
    m.step()
    torch.cuda.synchronize()
    acc = f64(m.acc)
    want = oracle.draft_verify(f64(m.v["tokens"]), f64(m.v["target"]), f64(m.v["uniforms"]),
                               draft=f64(m.v["draft"]), idx=f64(m.c["idx"]))
    assert acc.tolist() == want[0].tolist() and f64(m.next).tolist() == want[1].tolist()
    assert acc[2] == 0 and acc.max() > 1 and acc.max() < T + 1
    cs = f64(conv0).copy()
    oracle.causal_conv(f64(m.c["x"]), f64(m.c["weight"]), f64(m.c["bias"]), cs, ctx=acc,
                       idx=f64(m.c["idx"]))
    assert_bitwise(m.c["conv_state"], torch.from_numpy(cs).float(), "conv pool")
    ss = f64(scan0).copy()
    s = m.s
    _, _, smag = oracle.channel_scan(f64(m.conv_out), f64(s["A"]), f64(s["B"]), f64(s["C"]),
                                     f64(s["dt"]), ss, dt_bias=f64(s["dt_bias"]), D=f64(s["D"]),
                                     z=f64(s["z"]), ctx=acc, idx=f64(s["idx"]))
    check(s["state"], ss, scan_bound(smag, T, 0), torch.float32, "scan pool")


def test_window_loop_in_a_graph():
    eager, g = Loop(), torch.cuda.CUDAGraph()
    starts = [p.clone() for p in eager.pools()]
    for _ in range(3):
        eager.step()
    m = Loop()
    m.step()  # warm up
    with torch.cuda.graph(g):
        m.step()
    for rep in range(2):
        for p, s in zip(m.pools(), starts):
            p.copy_(s)
        torch.cuda.synchronize()
        for _ in range(3):
            g.replay()
            torch.cuda.synchronize()
        for a, b in zip(m.pools(), eager.pools()):
            assert_bitwise(a, b, f"pools, round {rep}")
        assert_bitwise(m.out, eager.out, "window outputs")


def test_prompt_then_single_tokens():
    """A prompt through both prefills, then tokens one at a time, is the prompt
    with those tokens appended."""
    full = 21
    c = conv_inputs(4, batch=2, seq_len=full, channels=D, width=4, io="f32")
    s = scan_inputs(5, batch=2, seq_len=full, dim=D, dstate=N, io="f32")
    s["idx"] = c["idx"]
    kw = dict(dt_bias=s["dt_bias"], D=s["D"], state_indices=c["idx"])
    ref_c, ref_s = c["conv_state"].clone(), s["state"].clone()
    mid, want = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    ssu_conv_prefill(c["x"], c["weight"], c["bias"], ref_c, mid, state_indices=c["idx"])
    ssu_scan_prefill(mid, s["A"], s["B"], s["C"], s["dt"], ref_s, want, z=s["z"], **kw)
    k = 16
    m1, o1 = torch.empty_like(mid[:, :k]), torch.empty_like(mid[:, :k])
    ssu_conv_prefill(c["x"][:, :k], c["weight"], c["bias"], c["conv_state"], m1,
                     state_indices=c["idx"])
    ssu_scan_prefill(m1, s["A"], s["B"][:, :k], s["C"][:, :k], s["dt"][:, :k], s["state"], o1,
                     z=s["z"][:, :k], **kw)
    for t in range(k, full):
        m2, o2 = torch.empty_like(mid[:, t]), torch.empty_like(mid[:, t])
        ssu_conv_decode(c["x"][:, t], c["weight"], c["bias"], c["conv_state"], m2,
                        state_indices=c["idx"])
        assert_bitwise(m2, mid[:, t].contiguous(), f"conv, token {t}")
        ssu_scan_decode(m2, s["A"], s["B"][:, t], s["C"][:, t], s["dt"][:, t], s["state"], o2,
                        z=s["z"][:, t], **kw)
    assert_bitwise(c["conv_state"], ref_c, "conv pool")
    # two evaluations of the same recurrence; 40 bounds every state's terms here (20 tokens of
    # |B dt' x| well below 1 each plus a start below 6)
    ref = f64(ref_s)
    check(s["state"], ref, 2 * scan_bound(abs(ref) * 0 + 40.0, full, 0), torch.float32, "scan pool")
