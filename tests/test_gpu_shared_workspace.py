"""One workspace for calls of every kind in turn, and one that held other data.

The calls run in a process of their own, so that their numbers, by which the
counters of a workspace tell calls apart, begin anew."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
import numpy as np
import torch
import speculative_decoding_verification_23_gb300 as sv
from speculative_decoding_verification_23_gb300 import workload as W
from speculative_decoding_verification_23_gb300.device_batch import to_device

which = sys.argv[1]
batch = W.make_batch(B=6, V=50000, K=[0, 1, 3, 5, 8, 2], dtype="bf16", seed=5, rho=[0.3, 0.6, 0.8, 0.9, 0.95, 0.99],
                     temperature=[0.5, 0.7, 1.0, 1.3, 0.9, 0.6], rep_penalty=1.0, hist_len=4, top_p=1.0, tv_budget=0.2)
db = to_device(batch)
drafts = int(batch.cu_draft[-1])
g = torch.Generator(device="cuda").manual_seed(1)
beams = []
for i in range(20):
    z = (3 * torch.randn(6 * 4, 50000, generator=g, device="cuda")).bfloat16()
    beams.append(sv.make_beam_args(logits=z, V=50000, scores=-torch.rand(6, 4, generator=g, device="cuda"), keep=4))
need = max(sv.spec_workspace_bytes(6, drafts, 50000), sv.spec_beam_workspace_bytes(beams[0]))
shared = torch.zeros(need, dtype=torch.uint8, device="cuda")
other = {"greedy": lambda ws: sv.spec_verify_greedy(db.args(), workspace=ws),
         "confidence": lambda ws: sv.spec_draft_confidence(db.args(), 0.3, workspace=ws),
         "resident": lambda ws: sv.spec_verify_sample(db.args(flags=sv.SPEC_PREFER_RESIDENT), workspace=ws),
         "streaming": lambda ws: sv.spec_verify_sample(db.args(flags=sv.SPEC_PREFER_STREAMING), workspace=ws)}[which]
got = []
for a in beams:
    one = [x.clone() for x in sv.spec_beam_select(a, workspace=shared)]
    got.append((one, [x.clone() for x in other(shared)]))
torch.cuda.synchronize()
for a, (one, two) in zip(beams, got):
    apart = [torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = sv.spec_beam_select(a, workspace=apart[0])
    assert all(torch.equal(x, y) for x, y in zip(one, want)), "beams"
    assert int(one[3].abs().max()) == 0
    want = other(apart[1])
    assert all(torch.equal(x, y) for x, y in zip(two, want)), which
print("equal")
"""


@pytest.mark.parametrize("which", ["greedy", "confidence", "resident", "streaming"])
def test_beams_and_a_verify_call_share_a_workspace(which):
    r = subprocess.run([sys.executable, "-c", PROGRAM, which], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "equal", (r.stdout + r.stderr)[-2000:]


HELD = """
import sys
import torch
import speculative_decoding_verification_23_gb300 as sv
from speculative_decoding_verification_23_gb300 import workload as W
from speculative_decoding_verification_23_gb300.device_batch import to_device

if sys.argv[1] == "greedy":
    batch = W.make_batch(B=5, V=20000, K=[0, 1, 3, 5, 2], dtype="bf16", seed=5, rho=0.9, temperature=0.7,
                         rep_penalty=1.0, hist_len=4, top_p=1.0, tv_budget=0.2)
    db = to_device(batch)
    need = sv.spec_workspace_bytes(5, int(batch.cu_draft[-1]), 20000)
    total = int(batch.cu_draft[-1]) + 5
    outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (total, 5, 5)]
    names = ("out_tokens", "out_accepted", "out_status")
    run = lambda ws: sv.spec_verify_greedy(db.args(), workspace=ws, **dict(zip(names, outs)))
else:
    g = torch.Generator(device="cuda").manual_seed(1)
    z = (3 * torch.randn(5 * 4, 20000, generator=g, device="cuda")).bfloat16()
    a = sv.make_beam_args(logits=z, V=20000, scores=torch.zeros(5, 4, device="cuda"), keep=4)
    need = sv.spec_beam_workspace_bytes(a)
    outs = [torch.empty(5, 4, device="cuda"), *(torch.empty(5, 4, dtype=torch.int32, device="cuda") for _ in range(2)),
            torch.empty(5, dtype=torch.int32, device="cuda")]
    names = ("out_scores", "out_parents", "out_tokens", "out_status")
    run = lambda ws: sv.spec_beam_select(a, workspace=ws, **dict(zip(names, outs)))
def call(ws):
    for x in outs:
        x.fill_(-9)
    return run(ws)
want = [x.clone() for x in call(torch.zeros(need, dtype=torch.uint8, device="cuda"))]
ws = torch.empty(need, dtype=torch.uint8, device="cuda")
words = ws[:need // 8 * 8].view(torch.int32).view(-1, 2)
for n in range(2, 200):
    words[:, 0] = (n << 24 | 0x8005) - (1 << 32 if n > 127 else 0)  # a float of exponent n, before a zero
    words[:, 1] = 0
    for x, y in zip(want, call(ws)):
        assert torch.equal(x, y), n
print("equal")
"""


@pytest.mark.parametrize("which", ["greedy", "beams"])
def test_a_workspace_that_held_floats(which):
    r = subprocess.run([sys.executable, "-c", HELD, which], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "equal", (r.stdout + r.stderr)[-2000:]
