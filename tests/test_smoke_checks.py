"""smoke() fails where values that it compares are no numbers."""
import numpy as np
import pytest

import oracle
from __graft_entry__ import _outside, smoke


def test_no_number_is_outside_every_bound():
    nan = float("nan")
    assert _outside(np.array([0.0, nan]), 1.0) and _outside(nan, 1.0) and _outside(np.array([0.5, 2.0]), 1.0)
    assert _outside(np.array([0.5, 0.5]), np.array([1.0, 0.1])) and _outside(float("inf"), 1.0)
    assert _outside(0.5, nan)
    assert not _outside(np.array([0.5, 1.0]), 1.0) and not _outside(0.0, 0.0) and not _outside(np.zeros(0), 1.0)


@pytest.mark.gpu
def test_smoke_passes_and_names_its_errors(capsys):
    smoke()
    out = capsys.readouterr().out
    assert out.startswith("smoke ok") and "layer norm" in out and "embedding" in out


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["residual_add_ln", "norm_gather", "bias_gelu_tanh", "bias_gelu_tanh_bwd",
                                  "window_bias_mask_add", "position_bias", "position_bias_bwd", "group_norm_act",
                                  "group_norm_act_bwd"])
def test_smoke_fails_where_the_oracle_gives_no_number(monkeypatch, name):
    plain = getattr(oracle, name)

    def spoil(out):
        if isinstance(out, (tuple, list)):
            return type(out)(spoil(part) for part in out)
        if isinstance(out, np.ndarray) and out.dtype.kind == "f":
            out = out.copy()
            out.reshape(-1)[-1] = np.nan
        return out

    def spoilt(*args, **kw):
        return spoil(plain(*args, **kw))

    monkeypatch.setattr(oracle, name, spoilt)
    with pytest.raises(AssertionError):
        smoke()
