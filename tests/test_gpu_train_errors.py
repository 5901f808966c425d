"""A call of a training-step operator that fails on the host leaves no CUDA error behind, which
the thread's next CUDA call would report as its own.  The failure: a launch into a stream capture
that has been invalidated (an error of the runtime on the host; nothing runs).  In a child process,
which keeps its broken capture to itself."""
import os
import subprocess
import sys

import pytest

from tests import gpu_util as G

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import os, sys, torch
from mixture_experts_layer_16_gb300 import MoEBalanceLoss, MoEGradClip, MoELayerNorm
from mixture_experts_layer_16_gb300.binding import MoEError
x = torch.randn(8, 64, device="cuda")
w, dw, db, y, z = (torch.ones(s, device="cuda") for s in (64, 64, 64, (8, 64), 1))
n, c, h = MoELayerNorm(8, 64, "fp32"), MoEGradClip(2), MoEBalanceLoss(8, 64, 2)
idx, dl = torch.zeros(8, 2, dtype=torch.int32, device="cuda"), torch.ones(2, device="cuda")
n.forward(x, w, w, y=y)
h.forward(x, idx)
calls = dict(
    norm_forward=lambda s: n.forward(x, w, w, y=y, stream=s),
    norm_backward=lambda s: n.backward(y, x, w, out=(d, dw, db), stream=s),
    balance_forward=lambda s: h.forward(x, idx, stream=s),
    balance_backward=lambda s: h.backward(x, dl, dlogits=d, stream=s),
    norm=lambda s: c.norm([x], stream=s),
    clip=lambda s: c.clip([x], 1.0, out=[d], stream=s))
d = torch.empty_like(x)
s, other = torch.cuda.Stream(), torch.cuda.Stream()
z.add_(1)
torch.cuda.synchronize()
with torch.cuda.stream(s):
    g = torch.cuda.CUDAGraph()
    g.capture_begin(capture_error_mode="relaxed")
    try:
        s.synchronize()          # not allowed in a capture: it is invalid from here on
    except RuntimeError:
        pass
    try:
        calls[sys.argv[1]](s)
        why = "the call went through"
    except MoEError:
        why = ""
    with torch.cuda.stream(other):
        try:
            z.add_(1)
        except RuntimeError as e:
            why += "the next call: " + str(e).splitlines()[0]
print(why or "clean", flush=True)
os._exit(0)
"""


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("call", ["norm_forward", "norm_backward", "balance_forward",
                                  "balance_backward", "norm", "clip"])
def test_failed_call_leaves_no_error(call):
    r = subprocess.run([sys.executable, "-c", CHILD, call], capture_output=True, text=True, cwd=ROOT,
                       env=dict(os.environ, PYTHONPATH=ROOT), timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip() == "clean", r.stdout
