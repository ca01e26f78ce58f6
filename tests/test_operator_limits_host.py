"""Sizes past which the operators' 32-bit column offsets would wrap are refused before anything is enqueued (CPU)."""
import pytest

from layer_lstm_b200 import binding
from test_linear_attention_host import _bwd as att_bwd
from test_linear_attention_host import _fwd as att_fwd
from test_linear_attention_host import _step as att_step
from test_norm_host import _bwd as norm_bwd
from test_norm_host import _fwd as norm_fwd

MOST = 1 << 30


@pytest.mark.parametrize("cols", [MOST + 1, 2 ** 31 - 256, 2 ** 31 - 1])
def test_norm_columns(cols):
    d = binding.make_norm_desc(1, cols)
    assert binding.lstm_layer_norm_workspace_size(d) == 0
    # (a NULL x or grad_y keeps a library without this check from starting anything)
    for x in (None, 256):
        assert norm_fwd(d, x=x) == binding.LSTM_ERR_UNSUPPORTED
        assert norm_bwd(d, gy=x) == binding.LSTM_ERR_UNSUPPORTED


def test_norm_at_the_border():
    d = binding.make_norm_desc(1, MOST)
    assert binding.lstm_layer_norm_workspace_size(d) >= 8 * MOST
    assert norm_fwd(d, x=None) == binding.LSTM_ERR_INVALID_ARG
    assert norm_bwd(d, gy=None) == binding.LSTM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(heads=MOST // 128 + 1, key_size=128, value_size=1),
                                dict(heads=MOST // 64 + 1, key_size=1, value_size=64),
                                dict(heads=1 << 28, key_size=8, value_size=8)])
def test_attention_row_width(kw):
    d = binding.make_attention_desc(1, 1, **kw)
    assert binding.lstm_linear_attention_workspace_size(d) == 0
    # (a NULL q keeps a library without this check from starting anything)
    for q in (None, 256):
        for call in (att_fwd, att_bwd, att_step):
            assert call(d, q=q) == binding.LSTM_ERR_UNSUPPORTED


def test_attention_at_the_border():
    d = binding.make_attention_desc(1, 1, MOST // 128, 128, 128)
    assert binding.lstm_linear_attention_workspace_size(d) > 0
    for call in (att_fwd, att_bwd, att_step):
        assert call(d, q=None) == binding.LSTM_ERR_INVALID_ARG
