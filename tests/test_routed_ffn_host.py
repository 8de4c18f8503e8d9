"""What RoutedFFN refuses before it touches the GPU (no GPU)."""

import pytest
import torch

import moe_fp8_grouped_amd as m
from moe_fp8_grouped_amd.pipeline import RoutedFFN

BF, F32 = torch.bfloat16, torch.float32
T, E, El, H, I, K = 6, 8, 4, 64, 32, 2


def arguments(**kw):
    a = dict(x=torch.zeros(T, H, dtype=BF), logits=torch.zeros(T, E, dtype=F32), w0=torch.zeros(El, H, I, dtype=BF),
             w1=torch.zeros(El, H, I, dtype=BF), wo=torch.zeros(El, I, H, dtype=BF), k=K)
    a.update(kw)
    return a


BAD = {
    "logits must": [dict(logits=torch.zeros(T, E, dtype=torch.float16)), dict(logits=torch.zeros(T, E, dtype=torch.float64)),
                    dict(logits=torch.zeros(T + 1, E)), dict(logits=torch.zeros(T, 2 * E)[:, :E])],
    "x must": [dict(x=torch.zeros(T, H)), dict(x=torch.zeros(T, H, dtype=torch.float16)), dict(x=torch.zeros(T, 2 * H, dtype=BF)[:, ::2])],
    "w0 must": [dict(w0=torch.zeros(El, H, I)), dict(w0=torch.zeros(El, H + 32, I, dtype=BF))],
    "w1 must": [dict(w1=torch.zeros(El, H, I + 32, dtype=BF)), dict(w1=torch.zeros(El + 1, H, I, dtype=BF))],
    "wo must": [dict(wo=torch.zeros(El, H, I, dtype=BF)), dict(wo=torch.zeros(El, H, I, dtype=BF).transpose(1, 2))],
    "select_bias must": [dict(select_bias=torch.zeros(E, dtype=BF)), dict(select_bias=torch.zeros(E - 1)), dict(select_bias=torch.zeros(2 * E)[::2])],
    "k must": [dict(k=0), dict(k=E + 1)],
    "local experts": [dict(group_offset=-1), dict(group_offset=5)],
    "dimensions": [dict(x=torch.zeros(T * H, dtype=BF)), dict(logits=torch.zeros(T * E)), dict(w0=torch.zeros(El, H * I, dtype=BF))],
    "rows must": [dict(rows=m.MOE_BF16)],
}


@pytest.mark.parametrize("match,kw", [(k, v) for k, vs in BAD.items() for v in vs], ids=lambda v: v if isinstance(v, str) else "-".join(v))
def test_refused(match, kw):
    with pytest.raises(ValueError, match=match):
        RoutedFFN(**arguments(**kw))


def test_what_is_allowed_gets_past_the_checks():
    for kw in (dict(), dict(w0=torch.zeros(El, I, H, dtype=BF).transpose(1, 2)), dict(logits=torch.zeros(T, E, dtype=BF), select_bias=torch.zeros(E), group_offset=4)):
        with pytest.raises(ValueError, match="GPU memory"):          # the quantizer's, where these tensors end
            RoutedFFN(**arguments(**kw))


@pytest.mark.parametrize("dout", [torch.zeros(T, H), torch.zeros(T + 1, H, dtype=BF), torch.zeros(H, T, dtype=BF).t()])
def test_gradients_of_another_kind_are_refused(dout):
    layer = RoutedFFN.__new__(RoutedFFN)
    layer.few, layer.T, layer.H, layer.x = False, T, H, torch.zeros(T, H, dtype=BF)
    with pytest.raises(ValueError, match="dout must"):
        layer.router_backward(dout)
