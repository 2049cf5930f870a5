"""What a checkpoint of the layer's kept state holds, byte by byte, and that the backward pass
from it is the backward pass of that state."""
import pytest
import torch

import q8_ref as ref
from test_gpu_q8 import dev, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


@pytest.mark.parametrize("flags", [0, 512, 16])
@pytest.mark.parametrize("T,d,F,N,cf", [(900, 128, 320, 6, 1.0), (300, 192, 256, 3, 0.5), (5, 64, 64, 2, 8.0)])
def test_load_gives_the_state_with_rounded_hidden_rows(sm, T, d, F, N, cf, flags):
    """Into a workspace of 0xFF a load writes the forward's bytes again, but for the hidden
    rows: those are the forward's, taken to 8 bits and back by the plain form.  The forward's
    own workspace with its hidden rows rounded the same way gives the same gradients."""
    cfg = sm.config(T, d, F, N, cf, flags=flags | sm.FLAG_TRAINING)
    C = sm.switch_capacity((2 if flags & 512 else 1) * T, N, cf)
    g = gen(T)
    x = dev(torch.randn(T, d, generator=g).bfloat16())
    w_r = dev(torch.randn(N, d, generator=g) * 0.1)
    w1 = dev((torch.randn(N, F, d, generator=g) * 0.1).bfloat16())
    w2 = dev((torch.randn(N, d, F, generator=g) * 0.1).bfloat16())
    dout = dev(torch.randn(T, d, generator=g).bfloat16())
    out = torch.empty_like(x)
    counts = torch.empty(N, dtype=torch.int32, device="cuda")

    def backward(ws):
        o = [torch.empty_like(x), torch.empty_like(w_r), torch.empty(N, device="cuda"),
             torch.empty_like(w1), torch.empty_like(w2)]
        sm.switch_layer_backward(cfg, x, w_r, None, w1, w2, dout, 1.0, *o, None, ws)
        assert sm.switch_get_device_error(ws)[0] == 0
        return o

    ws = sm.backward_workspace(cfg)
    sm.switch_layer_forward(cfg, x, w_r, None, w1, w2, out, None, None, counts, None, ws)
    c = sm.checkpoint(cfg)
    sm.switch_checkpoint_save(cfg, ws, c)
    kept = torch.clamp(counts.cpu(), max=C).tolist()
    filled = []
    for fill in (255, 0x11):                         # what a load writes stands over either
        w = torch.full_like(ws, fill)
        w[:256] = 0
        sm.switch_checkpoint_load(cfg, x, c, w)
        assert sm.switch_get_device_error(w)[0] == 0
        filled.append(w)
    b, wrote = filled[0], filled[0] == filled[1]
    wrote[:256] = False
    # the hidden rows lie before the experts' outputs, which end the forward's regions; all
    # that differs from the forward's bytes lies in them
    size, unit = N * C * F * 2, 1024
    at = sm.switch_workspace_size(cfg) - -(-N * C * d * 2 // unit) * unit - -(-size // unit) * unit
    differs = torch.nonzero(wrote & (b != ws))[:, 0]
    assert at <= int(differs[0]) and int(differs[-1]) < at + size

    def rows(w):
        return w[at:at + size].view(torch.bfloat16).view(N, C, F)

    for e, n in enumerate(kept):
        q, s = ref.quantize(rows(ws)[e, :n].cpu().double(), positive=True)
        rows(ws)[e, :n] = (q * ref.spread(s, F)).bfloat16().cuda()
        assert torch.equal(rows(ws)[e, :n], rows(b)[e, :n])
    # and the routing, the probabilities and the dispatched rows were written back
    assert int(wrote.sum()) >= 4 * T * N + 2 * d * sum(kept) + 2 * F * sum(kept) + 4 * (3 * T + N + N * C)
    got, want = backward(b), backward(ws)
    for name, u, v in zip(("dx", "dw_r", "db_r", "dw1", "dw2"), got, want):
        assert torch.equal(u, v), name
