"""A call launches on the current GPU: tensors of another one are refused before
the library is entered (the current device is a stand-in, no GPU is used)."""

from types import SimpleNamespace

import pytest
import torch

from sparse_mixture_experts_softmax_gb300 import binding as B
from sparse_mixture_experts_softmax_gb300.layer import MoELayer


class _Library:
    """Counts calls; every entry point returns MOE_OK."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return B.MOE_OK
        return call


@pytest.fixture
def library(monkeypatch):
    fake = _Library()
    monkeypatch.setattr(B, "lib", lambda: fake)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 77 + i)
    monkeypatch.setattr(B, "_ptr", lambda t: None)
    monkeypatch.setattr(B, "_stream", lambda s: s)
    return fake


def _tensor(index):
    """What the binding looks at of a tensor on GPU `index`."""
    return SimpleNamespace(device=torch.device("cuda", index), numel=lambda: 0)


def test_stream_of_another_device(library):
    assert B._stream_on(None, torch.device("cuda", 0)) == 77
    assert B._stream_on(5, torch.device("cuda", 0)) == 5
    for stream in (None, 5):
        with pytest.raises(ValueError, match="cuda:1"):
            B._stream_on(stream, torch.device("cuda", 1))


def test_block_bindings(library):
    t0, t1 = _tensor(0), _tensor(1)
    cfg, ncfg, w = B.make_config(4, 16, 8, 8, 2), B.make_norm_config(4, 16), B.moe_weights()
    calls = [lambda t: B.moe_norm_forward(ncfg, t, None, t, None, None, t),
             lambda t: B.moe_norm_backward(ncfg, t, t, t, t, t, None, t, t, None, t),
             lambda t: B.moe_decode(cfg, w, t, t, t),
             lambda t: B.moe_decode_init(cfg, t), lambda t: B.moe_decode_status(cfg, t)]
    for n, call in enumerate(calls):
        call(t0)
        assert library.calls == n + 1
        with pytest.raises(ValueError, match="cuda:1"):
            call(t1)
        assert library.calls == n + 1


def test_layer_of_another_device(library):
    la = MoELayer.__new__(MoELayer)
    for name in ("w1", "w2", "w3", "b1", "b2", "logit_bias", "corr_bias", "ws1", "ws3", "ws2",
                 "w1_lp", "w3_lp", "w2_lp", "ws1_lp", "ws3_lp", "ws2_lp", "dw_gate"):
        setattr(la, name, None)
    la.dtype, la.cfg, la.grads, la.d_loss = "f32", B.make_config(4, 16, 8, 8, 2), B.moe_grads(), None
    for index, refused in ((0, False), (1, True)):
        la.device = torch.device("cuda", index)
        la.w_gate = la.dw_gate = la.workspace = t = _tensor(index)
        for call in (lambda: la.forward(t, t), lambda: la.backward(t, t),
                     lambda: la.train_step(t, t, 0.1)):
            before = library.calls
            if refused:
                with pytest.raises(ValueError, match="cuda:1"):
                    call()
                assert library.calls == before
            else:
                call()
                assert library.calls == before + 1
