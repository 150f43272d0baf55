"""What the pre-norm block refuses before anything is launched (no GPU): the layer
behind it works on a fixed number of tokens and reads raw addresses."""

from types import SimpleNamespace

import pytest
import torch

from sparse_mixture_experts_softmax_gb300.block import BlockState, MoEBlock
from sparse_mixture_experts_softmax_gb300.norm import LayerNorm, NormGrads, NormOut

T, D = 8, 16


class _Norm(LayerNorm):
    """A norm whose calls return tensors of the right kind without a kernel."""

    def forward(self, x, delta=None, stats=True, out=None):
        rows = torch.zeros(x.shape[0])
        return NormOut(None, torch.zeros(x.shape, dtype=self.z_type), rows, rows)

    def backward(self, dz, h, mean, rstd, dres=None, out=None):
        return NormGrads(dz, self.gamma, None)


class _Layer:
    def __init__(self, dtype="f32"):
        self.cfg, self.dtype, self.calls = SimpleNamespace(T=T, D=D), dtype, 0
        self.w_gate = torch.zeros(2, D)

    def forward(self, x, y=None):
        self.calls += 1
        return torch.zeros(T, D)

    def backward(self, x, dy, dx=None):
        self.calls += 1
        return dx


def _block(dtype="f32"):
    return MoEBlock(_Norm(torch.ones(D), z_dtype=dtype), _Layer(dtype))


def _state(t=T, z=torch.float32, d=D):
    return BlockState(torch.zeros(t, d), torch.zeros(t, d, dtype=z), torch.zeros(t), torch.zeros(t))


@pytest.mark.parametrize("rows", [0, 1, T - 1, T + 1])
def test_forward_takes_the_layers_tokens_only(rows):
    b = _block()
    with pytest.raises(ValueError, match="8 tokens"):
        b.forward(torch.zeros(rows, D))
    assert b.layer.calls == 0
    b.forward(torch.zeros(T, D))
    assert b.layer.calls == 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_checks_what_the_layer_reads(dtype):
    b, z = _block(dtype), torch.bfloat16 if dtype == "bf16" else torch.float32
    other = torch.float32 if dtype == "bf16" else torch.bfloat16
    for bad in (torch.zeros(T, D, dtype=torch.bfloat16), torch.zeros(T, D, dtype=torch.float64),
                torch.zeros(T - 1, D), torch.zeros(T, D + 1), torch.zeros(T * D),
                torch.zeros(D, T).t()):
        with pytest.raises(ValueError, match="dout"):
            b.backward(_state(z=z), bad)
    for bad in (_state(t=T - 1, z=z), _state(z=other), _state(z=z, d=D + 8)):
        with pytest.raises(ValueError, match="state.z"):
            b.backward(bad, torch.zeros(T, D))
    assert b.layer.calls == 0
    b.backward(_state(z=z), torch.zeros(T, D))
    assert b.layer.calls == 1


def test_norm_and_layer_share_a_device():
    layer = _Layer()
    layer.w_gate = torch.zeros(2, D, device="meta")
    with pytest.raises(ValueError, match="meta"):
        MoEBlock(_Norm(torch.ones(D)), layer)
