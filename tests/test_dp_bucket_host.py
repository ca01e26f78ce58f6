"""dp.GradBucket.adopt moves a problem's gradients: whoever holds the gradient tensors follows them (CPU)."""
import types

import torch

from layer_lstm_b200 import binding, dp
from layer_lstm_b200.optim import AdamW


def _problem(n=2):
    z = lambda *s: torch.full(s, float("nan"))  # noqa: E731
    return types.SimpleNamespace(dw_ih=[z(12, 4) for _ in range(n)], dw_hh=[z(12, 3) for _ in range(n)],
                                 db_ih=[z(12) for _ in range(n)], db_hh=[z(12) for _ in range(n)])


def test_tensors_taken_before_see_the_bucket():
    prob = _problem()
    held = prob.dw_ih + prob.dw_hh + prob.db_ih
    bucket = dp.GradBucket.adopt(prob, bias=True)
    for i, g in enumerate(prob.dw_ih + prob.dw_hh + prob.db_ih):
        g.fill_(i + 1.0)
    for i, (a, b) in enumerate(zip(held, prob.dw_ih + prob.dw_hh + prob.db_ih)):
        assert a.data_ptr() == b.data_ptr() and a.shape == b.shape and (a == i + 1.0).all()
    assert bucket.flat.numel() == sum(t.numel() for t in held)


def test_optimizer_made_before_reads_the_bucket(monkeypatch):
    got = []
    monkeypatch.setattr(binding, "lstm_adamw_step", lambda desc, numel, *a: got.append(list(a[2])) or binding.LSTM_OK)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    prob = _problem()
    grads = prob.dw_ih + prob.dw_hh + prob.db_ih + prob.db_hh
    opt = AdamW([torch.zeros(g.shape) for g in grads], grads)
    bucket = dp.GradBucket.adopt(prob, bias=True)

    def step():
        for g in prob.dw_ih + prob.dw_hh + prob.db_ih:
            g.fill_(2.0)

    dp.train_step(step, bucket, 1, optimizer=opt)
    want = [t.data_ptr() for t in bucket.views + prob.db_hh]
    assert got == [want]
    assert all((g == 2.0).all() for g in opt.grads)
