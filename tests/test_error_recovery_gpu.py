"""A call that fails in CUDA is reported once: the next call, whichever it is, reports its own launches only.
The failure is a launch on a stream whose capture is void, which CUDA refuses on the host.  In a process of its
own, because the void capture stays with torch."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
import mhc_hyper_connections_b200 as mhc
T, n, d = 9, 4, 64
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda")
X, F, H, W, x = r(T, n, d), r(T, d), r(T, n * n + 2 * n), r(32, d), r(T, d)
Hs, w = H[None].contiguous(), r(d)
out = lambda: [torch.empty_like(X), torch.empty(1, T, 2, device="cuda"), torch.empty_like(x), torch.empty(T, 32, device="cuda")]
ws = torch.empty(max(1, mhc.mhc_linear_workspace_bytes(T, d, 32, torch.float32)), dtype=torch.uint8, device="cuda")
calls = [lambda o: mhc.mhc_post(X, F, H, o[0]), lambda o: mhc.mhc_amax_gain(Hs, o[1]),
         lambda o: mhc.mhc_layer_norm(x, w, None, 1e-5, o[2]), lambda o: mhc.mhc_linear(x, W, None, o[3], workspace=ws)]
ref = out()
for c in calls:
    c(ref)
got = out()
torch.cuda.synchronize()
for c in calls:
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph.capture_begin()
        try:
            torch.cuda.synchronize()     # refused, and the capture is void
        except RuntimeError:
            pass
        for fail in calls[2:]:
            try:
                fail(got)
                raise SystemExit("a launch on a void capture went through")
            except mhc.MhcError as e:
                assert e.status == 6, e
        try:
            graph.capture_end()
        except RuntimeError:
            pass
    c(got)                               # its own status, not the one before
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, ref))
assert mhc.mhc_device_status() == 0
print("recovered")
"""


def test_an_error_is_reported_once():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "recovered" in r.stdout, r.stdout + r.stderr
