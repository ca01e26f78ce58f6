"""optim.AdamW.read_state on a stream of its own makes its outputs there (GPU): memory that the current stream
gave back, with work on it still to come, is not written to beside that work."""
import pytest
import torch

from layer_lstm_b200.optim import AdamW

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_outputs_belong_to_the_stream(bits, handle, cuda_lib):
    n = 1 << 20
    opt = AdamW([torch.randn(n, device="cuda")], [torch.randn(n, device="cuda")], state_bits=bits)
    opt.step()
    want = [t.clone() for t in opt.read_state()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    other = [torch.empty(n, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)      # some 50 ms
    for t in other:
        t.fill_(7.0)
    del t, other
    got = opt.read_state(stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
