"""The library's first call in a process, with work pending on the default stream and on
device memory that is not zero: what the set-up clears is clear before the call's kernel
runs on a stream that does not wait for the default one."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys, torch
import bit_weight_only_w4a16_gb300 as w4
blocks = [torch.full((1 << 28,), 0x01010101, dtype=torch.int32, device="cuda") for _ in range(4)]
x = torch.randn(64, 20000, device="cuda")
t = torch.arange(64, dtype=torch.int32, device="cuda")
want = torch.log_softmax(x.double(), 1).gather(1, t.long()[:, None])[:, 0]
ids = x.argmax(1)
out = [torch.full((64,), 7.0, device="cuda"), None, torch.zeros(64, 1, device="cuda"),
       torch.full((64, 1), -5, dtype=torch.int32, device="cuda")]
s = torch.cuda.Stream()
torch.cuda.synchronize()
del blocks
torch.cuda.empty_cache()
torch.cuda._sleep(1_000_000_000)  # about half a second of the default stream
if sys.argv[1] == "init":
    w4.init()
w4.w4_logprobs(x, t, 1, out=out, stream=s)
s.synchronize()
assert (out[0].double() - want).abs().max().item() < 1e-4
assert torch.equal(out[3][:, 0].long(), ids)
torch.cuda.synchronize()
assert w4.device_error() == 0
w4.w4_logprobs(x, t, 1, out=out, stream=s)
s.synchronize()
assert (out[0].double() - want).abs().max().item() < 1e-4
print("ok")
"""


@pytest.mark.parametrize("first", ["init", "call"])
def test_first_call_on_a_side_stream(first):
    r = subprocess.run([sys.executable, "-c", CODE, first], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
