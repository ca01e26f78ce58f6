"""The give-up path of the tensor-core linear attention, run in a fresh process (the wait limit and the fault
injection are read once per process).

argv: "forward" or "backward", batch, steps, heads, key size, value size.  The environment sets
LSTM_B200_WAIT_TIMEOUT_NS (a few ms) and LSTM_B200_DEBUG_SKIP_ARRIVAL="att:<block>:<chunk>": that block withholds
one chunk's weighed values, every role of it comes to a stop, its loads' warp gives up, all roles leave, and the
call ends with LSTM_ERR_TIMEOUT in the status word.  The stream and the context stay usable, and what lies around
the outputs stays as it was.  Exit code 0 on success."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

from layer_lstm_b200 import binding  # noqa: E402

PAD = 256


def main():
    which, B, T, H, dk, dv = sys.argv[1], *(int(a) for a in sys.argv[2:7])
    bf = torch.bfloat16

    def framed(*shape, dt=bf):
        n = int(torch.Size(shape).numel())
        whole = torch.full((n + 2 * PAD,), 3.0, device="cuda", dtype=dt)
        return whole, whole[PAD:PAD + n].view(shape)

    n = lambda *s: torch.randn(s, device="cuda").to(bf)  # noqa: E731
    q, k, v, go = n(B, T, H, dk), n(B, T, H, dk), n(B, T, H, dv), n(B, T, H, dv)
    ld = torch.full((H,), -0.05, device="cuda")
    d = binding.make_attention_desc(B, T, H, dk, dv, dtype=binding.LSTM_BF16)
    ws = torch.full((binding.lstm_linear_attention_workspace_size(d),), 255, device="cuda", dtype=torch.uint8)
    if which == "forward":
        outs = [framed(B, T, H, dv), framed(B, H, dk, dv, dt=torch.float32)]
        binding.check(binding.lstm_linear_attention_forward(d, q, k, v, ld, None, outs[0][1], outs[1][1], ws))
    else:
        outs = [framed(B, T, H, dk), framed(B, T, H, dk), framed(B, T, H, dv), framed(B, H, dk, dv, dt=torch.float32)]
        binding.check(binding.lstm_linear_attention_backward(d, q, k, v, ld, None, go, None, *(o for _, o in outs), ws))
    st = binding.lstm_query_status(ws)
    print("status", binding.status_string(st))
    total = float(torch.arange(10, device="cuda", dtype=torch.float32).sum().item())
    torch.cuda.synchronize()
    kept = all(bool((w[:PAD] == 3.0).all() and (w[-PAD:] == 3.0).all()) for w, _ in outs)
    print("kept", kept)
    sys.exit(0 if st == binding.LSTM_ERR_TIMEOUT and total == 45.0 and kept else 1)


if __name__ == "__main__":
    main()
