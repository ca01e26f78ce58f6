"""The binding with plain device addresses and a stream handle needs no torch (CPU, a process of its own)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.modules["torch"] = None          # an import of it fails
from layer_lstm_b200 import binding as b
d = b.make_desc(8, 16, batch=2, seq_len=3)
assert b.lstm_workspace_size(d) > 0
one = [256]
# refused on the host: the workspace is no multiple of 256 bytes
assert b.lstm_forward(d, 256, 0, 0, one, one, one, one, 256, 256, 256, 264, None, 0, 1 << 30, 0) == b.LSTM_ERR_INVALID_ARG
n = b.make_norm_desc(4, 8)
assert b.lstm_layer_norm_workspace_size(n) > 0
assert b.lstm_layer_norm_forward(n, 256, 256, 256, 257, 256, 256, 0) == b.LSTM_ERR_INVALID_ARG
assert b.lstm_layer_norm_backward(n, 256, 256, 256, 256, 256, 256, 256, 256, 264, 0, 1 << 30) == b.LSTM_ERR_INVALID_ARG
a = b.make_attention_desc(2, 1, 2, 8, 8)
assert b.lstm_linear_attention_workspace_size(a) > 0
assert b.lstm_linear_attention_forward(a, 257, 256, 256, 256, 0, 256, 0, 256, 0, 1 << 30) == b.LSTM_ERR_INVALID_ARG
assert b.lstm_linear_attention_step(a, 257, 256, 256, 256, 256, 256, 0) == b.LSTM_ERR_INVALID_ARG
w = b.make_adamw_desc(1)
assert b.lstm_adamw_step(w, [4], [258], None, one, one, one, None, None, 256, None, 0) == b.LSTM_ERR_INVALID_ARG
assert "torch" not in [m for m in sys.modules if sys.modules[m] is not None]
print("ok")
"""


def test_addresses_need_no_torch():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=120, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
