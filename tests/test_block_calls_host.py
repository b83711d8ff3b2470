"""Calls of the operators around the routed experts that the binding refuses (no GPU needed)."""
import pytest
import torch

import dequant_iqk_moe_amd as q
from test_block_host import Fake

F32, I8, I32 = torch.float32, torch.int8, torch.int32


def _weights():
    w = q.Int8Weights(torch.zeros(2, 4, 16, dtype=I8), torch.zeros(2, 4))
    w.codes, w.scales = Fake((2, 4, 16), I8), Fake((2, 4), F32)
    return w


@pytest.mark.parametrize("grouped,which", [(g, m) for g in (False, True) for m in
                                           ("codes", "scales", "x", "x_scales", "workspace", "y") + ("offsets",) * g])
def test_products_refuse_another_device(grouped, which, monkeypatch):
    """Each tensor of the call, those that the weights consist of among them."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    w = _weights()
    given = dict(x=Fake((3, 16), I8), x_scales=Fake((3,), F32), workspace=Fake((1 << 20,), torch.uint8), y=Fake((3, 4), F32))
    if grouped:
        given["offsets"] = Fake((3,), I32)
    for t in (*given.values(), w.codes, w.scales):
        t.at = 0
    (given[which] if which in given else getattr(w, which)).at = 1
    with pytest.raises(q.IqkValueError, match="cuda:1"):
        (q.int8_grouped if grouped else q.int8_linear)(w, **given)
