"""What `MoEBlock` refuses before it makes anything, without a GPU."""
import math

import pytest

from routing_dispatch_grouped_router_gb300 import block

SHAPE = (4, 128, 4, 128, 2)


@pytest.mark.parametrize("kw,word", [
    (dict(residual_scale=0.9), "residual_scale"), (dict(residual_scale=math.nan), "residual_scale"),
    (dict(dropout=-0.1), "dropout"), (dict(dropout=1.01), "dropout"),
    (dict(dropout=math.nan), "dropout"), (dict(post_norm=True, dropout=-1.0), "dropout")])
def test_refused(kw, word):
    with pytest.raises(ValueError, match=word):
        block.MoEBlock(*SHAPE, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(residual_scale=1), dict(dropout=0),
                                dict(dropout=1.0, site=(1 << 32) - 1),
                                dict(post_norm=True, residual_scale=0.5, dropout=0.1)])
def test_taken(kw, monkeypatch):
    monkeypatch.setattr(block.api, "MoELayer", lambda *a, **k: None)
    b = block.MoEBlock(*SHAPE, **kw)
    assert b.residual_scale == kw.get("residual_scale", 1.0)
    assert b.dropout == kw.get("dropout", 0.0)
