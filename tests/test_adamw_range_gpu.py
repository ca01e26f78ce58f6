"""lstm_adamw_step at the borders of the hyperparameters it accepts (GPU): elements whose gradient and moments
are zero keep their parameter, whatever eps and the step size."""
import pytest
import torch

from layer_lstm_b200.optim import AdamW

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kw", [dict(eps=2.0 ** -126), dict(eps=2.0 ** 126), dict(lr=1e37, beta1=0.9),
                                dict(beta1=1 - 2.0 ** -53, beta2=1 - 2.0 ** -53)])
def test_zero_gradients_move_nothing(kw, bits, cuda_lib):
    p = torch.randn(1000, device="cuda")
    p0, g = p.clone(), torch.zeros(1000, device="cuda")
    opt = AdamW([p], [g], state_bits=bits, weight_decay=0.0, **kw)
    for _ in range(2):
        opt.step()
    assert torch.equal(p, p0)
