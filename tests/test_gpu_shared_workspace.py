"""One workspace for calls of every kind in turn.

The calls run in a process of their own, so that each kind of call is as old
as the others when they meet: the counters of a workspace tell calls apart by
their numbers."""
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
