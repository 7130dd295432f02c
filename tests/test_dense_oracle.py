"""The 64-bit forms that the operators around the experts are tested against."""
from __future__ import annotations

import pytest
import torch

from . import _dense as d


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_an_expert_out_of_service_has_no_weight(score, renorm):
    """Out of service by its logit or by its bias, one alone of four is left."""
    l = torch.tensor([[1.0, 2.0, 3.0, -torch.inf]])
    bias = torch.tensor([0.0, torch.nan, -torch.inf, 0.0])
    idx, w = d.topk64(l, 4, bias=bias, score=score, renorm=renorm)
    assert idx.tolist() == [[0, 1, 2, 3]]
    own = torch.sigmoid(l[0, 0].double()) if score == "sigmoid" else torch.softmax(l.double(), -1)[0, 0]
    want = 1.0 if renorm else float(own)
    assert w[0, 1:].tolist() == [0.0] * 3 and abs(float(w[0, 0]) - want) < 1e-15
