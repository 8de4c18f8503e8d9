"""What BlockScaledFFN refuses before it touches the GPU (no GPU)."""

import pytest
import torch

from moe_fp8_grouped_amd.pipeline import BlockScaledFFN

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
T, E, El, H, I, K = 6, 8, 4, 64, 32, 2


def arguments(**kw):
    a = dict(x=torch.zeros(T, H, dtype=BF), logits=torch.zeros(T, E, dtype=F32), w0=torch.zeros(El, H, I, dtype=BF),
             w1=torch.zeros(El, H, I, dtype=BF), wo=torch.zeros(El, I, H, dtype=BF), k=K)
    a.update(kw)
    return a


BAD = {
    "logits must": [dict(logits=torch.zeros(T, E, dtype=torch.float16)), dict(logits=torch.zeros(T + 1, E)), dict(logits=torch.zeros(T, 2 * E)[:, :E])],
    "x must": [dict(x=torch.zeros(T, H)), dict(x=torch.zeros(T, 2 * H, dtype=BF)[:, ::2])],
    "w0 must": [dict(w0=torch.zeros(El, H, I)), dict(w0=torch.zeros(El, H + 16, I, dtype=BF))],
    "w1 must": [dict(w1=torch.zeros(El, H, I + 16, dtype=BF)), dict(w1=torch.zeros(El + 1, H, I, dtype=BF))],
    "wo must": [dict(wo=torch.zeros(El, H, I, dtype=BF)), dict(wo=torch.zeros(El, H, I, dtype=BF).transpose(1, 2))],
    "select_bias must": [dict(select_bias=torch.zeros(E, dtype=BF)), dict(select_bias=torch.zeros(E - 1))],
    "seq_offsets must": [dict(seq_offsets=torch.zeros(3, dtype=torch.int64)), dict(seq_offsets=torch.zeros(6, dtype=I32)[::2])],
    "seq_offsets holds": [dict(seq_offsets=torch.zeros(1, dtype=I32)), dict(seq_offsets=torch.zeros(2, 2, dtype=I32))],
    "k must": [dict(k=0), dict(k=E + 1)],
    "local experts": [dict(group_offset=-1), dict(group_offset=5)],
    "m_cap must": [dict(m_cap=-1)],
    "multiples of 16": [dict(x=torch.zeros(T, 72, dtype=BF), w0=torch.zeros(El, 72, I, dtype=BF), w1=torch.zeros(El, 72, I, dtype=BF), wo=torch.zeros(El, I, 72, dtype=BF))],
    "grad_dtype must": [dict(grad_dtype=torch.float16)],
    "dimensions": [dict(x=torch.zeros(T * H, dtype=BF)), dict(logits=torch.zeros(T * E)), dict(w0=torch.zeros(El, H * I, dtype=BF))],
}


@pytest.mark.parametrize("match,kw", [(k, v) for k, vs in BAD.items() for v in vs], ids=lambda v: v if isinstance(v, str) else "-".join(v))
def test_refused(match, kw):
    with pytest.raises(ValueError, match=match):
        BlockScaledFFN(**arguments(**kw))


def test_what_is_allowed_gets_past_the_checks():
    for kw in (dict(), dict(w0=torch.zeros(El, I, H, dtype=BF).transpose(1, 2)), dict(balance_weight=0.1, seq_offsets=torch.zeros(3, dtype=I32)),
               dict(logits=torch.zeros(T, E, dtype=BF), select_bias=torch.zeros(E), group_offset=4, grad_dtype=BF)):
        with pytest.raises(ValueError, match="GPU memory"):          # the quantizer's, where these tensors end
            BlockScaledFFN(**arguments(**kw))


@pytest.mark.parametrize("dout", [torch.zeros(T, H), torch.zeros(T + 1, H, dtype=BF), torch.zeros(H, T, dtype=BF).t()])
def test_gradients_of_another_kind_are_refused(dout):
    layer = BlockScaledFFN.__new__(BlockScaledFFN)
    layer.T, layer.H, layer.x = T, H, torch.zeros(T, H, dtype=BF)
    with pytest.raises(ValueError, match="dout must"):
        layer.backward(dout)
