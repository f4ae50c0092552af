"""The binding beside torch builds that lack the device names it prefers.  No GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_without_the_raw_stream_names():
    """Types are still told apart, wrong ones refused, and the stream comes from torch's public call."""
    _run("""
import torch, torch._C
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from block_wise_int4_amd import mnb
assert mnb._dtype_code(torch.zeros(1, dtype=torch.float16)) == mnb.MNB_F16
assert mnb._dtype_code(torch.zeros(1)) == mnb.MNB_F32
try:
    mnb._dtype_code(torch.zeros(1, dtype=torch.float64))
    raise SystemExit("a double was taken")
except ValueError:
    pass
x = torch.zeros((2, 64), dtype=torch.float16)
try:
    mnb.mnb_rms_norm(x, x[0], x, 1e-5)
    raise SystemExit("a host tensor was taken")
except ValueError:
    pass
class S:
    cuda_stream = 12
torch.cuda.current_stream = lambda: S
assert mnb._stream(None).value == 12 and mnb._stream(S).value == 12 and mnb._stream(7).value == 7
""")


def test_size_queries_keep_the_last_variant():
    """The last call that enqueued work, or was a no-op, is still named after a query."""
    _run("""
import ctypes
from block_wise_int4_amd import mnb
from tests.test_decoder_abi import desc, norm
assert norm(m=0) == 0 and mnb.mnb_last_variant() == "noop"
assert mnb.mnb_kv4_cache_bytes(desc()) > 0 and mnb.mnb_last_variant() == "noop"
assert mnb.mnb_attention_kv4_workspace_bytes(desc(), 1, 1, 1, 100000) > 0 and mnb.mnb_last_variant() == "noop"
assert mnb.mnb_attention_kv4_workspace_bytes(desc(), 0, 0, 0, 0) == 0 and mnb.mnb_last_variant() == "noop"
assert norm(m=-1) != 0 and mnb.mnb_last_error()
mnb.mnb_kv4_cache_bytes(desc())
assert mnb.mnb_last_error() == "" and mnb.mnb_last_variant() == "noop"
""")
