"""Workspaces with no room for sums in parts: the layer's own regions alone.  Every call accepts
them and gives what it gives otherwise, within the same tolerances."""
import pytest
import torch

import test_gpu_q8 as base
from test_gpu_q8 import dev, gen
from test_q8_workspace_cpu import FEW

pytestmark = pytest.mark.gpu


class Bare:
    """The binding with workspaces of given sizes, a red zone behind them."""

    def __init__(self, sm, forward, backward):
        self.sm, self.sizes, self.all = sm, (forward, backward), []

    def __getattr__(self, name):
        return getattr(self.sm, name)

    def make(self, n):
        t = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
        t[n:] = 0x5A
        self.all.append(t)
        return t[:n]

    def workspace(self, cfg):
        return self.make(self.sizes[0])

    def backward_workspace(self, cfg):
        return self.make(self.sizes[1])

    def intact(self):
        return all((t[-4096:] == 0x5A).all() for t in self.all)


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


@pytest.mark.parametrize("sizes,forward,backward", FEW)
def test_calls_in_the_layers_own_regions(sm, sizes, forward, backward):
    w = Bare(sm, forward, backward)
    base.test_ffn_q8(w, *sizes, False)
    base.check_ffn_checkpoint(w, *sizes, (), 0, False)
    if sizes != FEW[2][0]:
        base.test_ffn_backward_q8(w, *sizes, (), 0)
    else:
        # d_ff > 16 d_model and more slots than tokens: the regions left idle do not hold the
        # hidden values' mask
        with pytest.raises(sm.SwitchError) as e:
            base.test_ffn_backward_q8(w, *sizes, (), 0)
        assert e.value.status == 3
    assert w.intact() and len(w.all) >= 3


@pytest.mark.parametrize("sizes,forward,backward", FEW[:2])
def test_the_layer_in_its_own_regions(sm, sizes, forward, backward):
    T, d, F, N, cf = sizes
    w = Bare(sm, forward, backward)
    g = gen(T)
    x, dout = (dev(torch.randn(T, d, generator=g).bfloat16()) for _ in range(2))
    w_r = dev(torch.randn(N, d, generator=g) * 0.1)
    w1 = dev((torch.randn(N, F, d, generator=g) * d ** -0.5).bfloat16())
    w2 = dev((torch.randn(N, d, F, generator=g) * F ** -0.5).bfloat16())

    def run(m):
        cfg = sm.config(T, d, F, N, cf, flags=sm.FLAG_TRAINING)
        ws = m.backward_workspace(cfg)
        o = [torch.empty_like(t) for t in (x, x, w_r, w_r[:, 0].contiguous(), w1, w2)]
        sm.switch_layer_forward(cfg, x, w_r, None, w1, w2, o[0], None, None, None, None, ws)
        c = sm.checkpoint(cfg)
        sm.switch_checkpoint_save(cfg, ws, c)
        sm.switch_checkpoint_load(cfg, x, c, ws)
        sm.switch_layer_backward(cfg, x, w_r, None, w1, w2, dout, 1.0, *o[1:], None, ws)
        assert sm.switch_get_device_error(ws)[0] == 0
        return o

    assert all(torch.equal(a, b) for a, b in zip(run(w), run(sm)))
    assert w.intact()
    # forward only, in the forward's size
    cfg = sm.config(T, d, F, N, cf)
    out = torch.empty_like(x)
    sm.switch_layer_forward(cfg, x, w_r, None, w1, w2, out, None, None, None, None, w.workspace(cfg))
    assert w.intact() and torch.isfinite(out).all()
