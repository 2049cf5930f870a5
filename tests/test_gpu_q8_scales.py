"""The 8-bit FFN with scales far from one on either side of a product: what counts is the
product of the two scales, also where a block's sum times one of them alone leaves fp32's
range, and on the paths for few tokens and for many alike."""
import pytest
import torch

import q8_ref as ref
from test_gpu_q8 import check, dev, ffn_inputs, ffn_q8_want

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


# powers of two on the rows, on W1 and on W2: W1's scale near fp32's largest and the rows' as
# far below; the other way round, W1's near its smallest; hidden rows far below one and W2's
# scale far above
SHIFTS = [(-103, 125, -10), (110, -110, 0), (-47, -42, 115)]


@pytest.mark.parametrize("T", [1, 8, 9, 200])
@pytest.mark.parametrize("shifts", SHIFTS)
def test_opposite_scales(sm, T, shifts):
    d, F, N = 256, 384, 2
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, 2.0, 41 + T)
    a = [ref.to_q8(x), ref.as_q8(*ref.quantize_weights(w1)), ref.as_q8(*ref.quantize_weights(w2))]
    for (q, s), k in zip(a, shifts):
        b = s.view(torch.uint8)
        moved = b.int() + k
        assert 1 <= int(moved.min()) and int(moved.max()) <= 254
        b.copy_(moved.to(torch.uint8))
    cfg = sm.config(T, d, F, N, 2.0)
    ws = sm.workspace(cfg)
    y = torch.zeros(N, C, d, dtype=torch.bfloat16, device="cuda")
    sm.switch_expert_ffn_q8(cfg, *map(dev, a[0]), dev(slot), dev(counts), *map(dev, a[1]),
                            *map(dev, a[2]), y, ws)
    assert sm.switch_get_device_error(ws)[0] == 0
    xv, w1v, w2v = ref.rows(*a[0]), ref.weights(*a[1]), ref.weights(*a[2])
    for e in range(N):
        n = int(kept[e])
        if n:
            want, tol = ffn_q8_want(xv[slot.view(N, C)[e, :n].long()], w1v[e], w2v[e])
            check(y[e, :n], want, tol, f"expert {e}")
