"""The first calls of a process on a 4-bit cache and at a verification step's end are captured: what the library
asks of the runtime once, it may ask during a capture.  And two captured steps replayed at once on two streams."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STEP = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import relative_bias_hybrid_gb300.inkattn as ia
from relative_bias_hybrid_gb300 import inputs as gen
from relative_bias_hybrid_gb300.step import AttentionStep, VerifyStep


class Step:
    # a decode, a prefill and a step's end over V tokens; its outputs, and the states that it changes in place
    def __init__(self, seed, V):
        self.w = w = gen.custom("capture", Hq=16, Hkv=2, q_lens=[9, 3], prefix_lens=[700, 40], rel_extent=64)
        self.x = x = gen.make_inputs(w, seed=seed, device="cuda", kv_dtype="i4")
        self.decode = AttentionStep(w, x, mode="decode", num_splits=3)
        self.prefill = AttentionStep(w, x, mode="prefill")
        self.prefill.attn.q = self.decode.q_out.data_ptr()
        self.before = [x["conv_state_k"].clone(), x["conv_state_v"].clone()]
        xv = gen.make_verify_inputs(w, V, seed=seed, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed)
        logits = 3 * torch.randn((w.N_tok, V), generator=g, device="cuda")
        self.after = [torch.zeros_like(s) for s in self.before]
        self.end = VerifyStep(w, xv, logits, [(x["k"], self.before[0], self.after[0]), (x["v"], self.before[1], self.after[1])])
        wide = 3 * torch.randn((330, 8200), generator=g, device="cuda")
        self.many = torch.empty_like(wide)
        self.p_many = ia.token_probs_params(logits=wide, probs=self.many, temperature=torch.ones(330, device="cuda"))

    def run(self, stream=None):
        self.decode.run(stream)
        self.prefill.run_attention(stream)
        self.end.run(stream)
        ia.inkattn_token_probs(self.p_many, stream)

    def reset(self):
        for s, b in zip((self.x["conv_state_k"], self.x["conv_state_v"]), self.before):
            s.copy_(b)
        for t in self.outputs():
            t.zero_()

    def outputs(self):
        return [self.decode.out, self.prefill.out, self.end.probs, self.end.n_new, self.end.tokens, *self.after, self.many]

    def status(self):
        return self.decode.device_status() | self.prefill.device_status() | self.end.device_status()
"""

FIRST = STEP + r"""
step = Step(1, 50001)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step.run()
for t in step.outputs():
    t.zero_()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in step.outputs()]
assert step.status() == 0 and all(bool(t.any()) for t in got)
step.reset()
step.run()
torch.cuda.synchronize()
assert step.status() == 0 and all(torch.equal(a, b) for a, b in zip(got, step.outputs()))
print("FIRST CALLS CAPTURED")
"""

TWO = STEP + r"""
steps = [Step(s, 30011) for s in (1, 2)]
want = []
for step in steps:
    step.run()
    torch.cuda.synchronize()
    want.append([t.clone() for t in step.outputs()])
streams, graphs = [torch.cuda.Stream() for _ in steps], [torch.cuda.CUDAGraph() for _ in steps]
for step, s, g in zip(steps, streams, graphs):
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        step.run(s)
for _ in range(5):
    for step in steps:
        step.reset()
    torch.cuda.synchronize()
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for step, w in zip(steps, want):
        assert step.status() == 0 and all(torch.equal(a, b) for a, b in zip(w, step.outputs()))
print("TWO REPLAYED AT ONCE")
"""


@pytest.mark.parametrize("text, said", [(FIRST, "FIRST CALLS CAPTURED"), (TWO, "TWO REPLAYED AT ONCE")],
                         ids=["first_calls", "two_at_once"])
def test_captured(text, said):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", text, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and said in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
