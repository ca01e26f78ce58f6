"""A bounded wait of the tensor-core linear attention that gives up ends the call with LSTM_ERR_TIMEOUT in the
status word and leaves the context usable (GPU).  One block withholds one chunk's arrivals
(LSTM_B200_DEBUG_SKIP_ARRIVAL), the wait limit is 20 ms (LSTM_B200_WAIT_TIMEOUT_NS): every other wait of that
block ends by the flag which the loads' warp sets, products and copies in flight have ended long before.  Each
case runs in a fresh process because both settings are read once per process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("skip,which,size", [
    ("att:0:0", "forward", (1, 64, 2, 64, 64)),          # one chunk: the loads' warp is already past its loads
    ("att:3:1", "forward", (4, 300, 3, 128, 128)),       # in the middle of a row
    ("att:147:2", "forward", (64, 300, 8, 64, 64)),      # many items a block
    ("att:1:1", "backward", (2, 400, 2, 128, 64)),       # products of two kernels' sizes
    ("att:0:1", "forward", (1, 40000, 1, 64, 64)),       # segments of three chunks
], ids=["one_chunk", "row", "items", "backward", "segments"])
def test_withheld_arrival_times_out(skip, which, size, cuda_lib):
    env = dict(os.environ, LSTM_B200_WAIT_TIMEOUT_NS="20000000", LSTM_B200_DEBUG_SKIP_ARRIVAL=skip)
    r = subprocess.run([sys.executable, os.path.join(HERE, "attention_timeout_check.py"), which, *map(str, size)],
                       capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "LSTM_ERR_TIMEOUT" in r.stdout
