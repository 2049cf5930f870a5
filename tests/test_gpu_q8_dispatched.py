"""More rows than the config has tokens.  Rows that lie in their slots already are bounded by the
slots alone: where those are many, nothing about a call depends on the tokens.  And slots may
name a token more than once."""
import pytest
import torch

import q8_ref as ref
from test_gpu_q8 import check, dev, ffn_inputs, ffn_q8_want, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


# (tokens, capacity factor) twice with the same capacity: few tokens against many; a sum that
# goes in parts, whose number depends on the rows
@pytest.mark.parametrize("one,two,d,F,N,counts", [
    ((8, 10.0), (80, 1.0), 512, 1024, 2, (37, 12)), ((1, 160.0), (160, 1.0), 320, 640, 4, (40, 0, 23, 8)),
    ((20, 15.0), (300, 1.0), 64, 4672, 1, (300,)), ((9, 80.0), (720, 1.0), 128, 9472, 2, (360, 211))])
def test_tokens_of_the_config_do_not_matter(sm, one, two, d, F, N, counts):
    C = sm.switch_capacity(one[0], N, one[1])
    assert C == sm.switch_capacity(two[0], N, two[1])
    _, _, _, _, _, w1, w2 = ffn_inputs(4, d, F, N, 1.0, d + F)
    x = torch.randn(N * C, d, generator=gen(d)).double()
    xq, xs = map(dev, ref.to_q8(x))
    w1q, w1s = map(dev, ref.as_q8(*ref.quantize_weights(w1)))
    w2q, w2s = map(dev, ref.as_q8(*ref.quantize_weights(w2)))
    x, w1, w2 = dev(x.bfloat16()), dev(w1.bfloat16()), dev(w2.bfloat16())
    dy = dev(torch.randn(N, C, d, generator=gen(F)).bfloat16())
    n = dev(torch.tensor(counts, dtype=torch.int32))

    def run(T, cf):
        cfg = sm.config(T, d, F, N, cf, flags=sm.FLAG_ROWS_DISPATCHED)
        ws = sm.backward_workspace(cfg)
        y = [torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        cx, ch = sm.q8_rows(N * C, d), sm.q8_rows(N * C, F)
        dw1, dw2 = torch.empty_like(w1), torch.empty_like(w2)
        sm.switch_expert_ffn_q8(cfg, xq, xs, None, n, w1q, w1s, w2q, w2s, y[0], ws)
        sm.switch_expert_ffn_checkpoint(cfg, x, None, n, w1, w2, y[1], *cx, *ch, ws)
        sm.switch_expert_ffn_backward_q8(cfg, *cx, *ch, n, w1, w2, dy, y[2], dw1, dw2, ws)
        assert sm.switch_get_device_error(ws)[0] == 0
        # (the weight gradients' sums go in parts by the tokens that an expert is due)
        return y + [t.view(torch.uint8) for t in (*cx, *ch)]

    assert all(torch.equal(a, b) for a, b in zip(run(*one), run(*two)))


@pytest.mark.parametrize("T", [3, 8, 9])
def test_tokens_named_more_than_once(sm, T):
    """Slots that hold a few tokens again and again: more rows than the paths for few tokens
    take at a time."""
    d, F, N = 192, 320, 2
    cf = 40 / T
    C = sm.switch_capacity(T, N, cf)
    counts = (19, 8)
    _, _, _, _, x, w1, w2 = ffn_inputs(T, d, F, N, 1.0, 29)
    slot = torch.randint(0, T, (N, C), generator=gen(T), dtype=torch.int32)
    xq, xs = ref.to_q8(x)
    w1q, w1s = ref.as_q8(*ref.quantize_weights(w1))
    w2q, w2s = ref.as_q8(*ref.quantize_weights(w2))
    cfg = sm.config(T, d, F, N, cf)
    ws = sm.workspace(cfg)
    y = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
    sm.switch_expert_ffn_q8(cfg, dev(xq), dev(xs), dev(slot.view(-1)),
                            dev(torch.tensor(counts, dtype=torch.int32)), dev(w1q), dev(w1s),
                            dev(w2q), dev(w2s), y, ws)
    assert sm.switch_get_device_error(ws)[0] == 0
    xv, w1v, w2v = ref.rows(xq, xs), ref.weights(w1q, w1s), ref.weights(w2q, w2s)
    for e, n in enumerate(counts):
        assert (y[e, n:] == -7).all()
        want, tol = ffn_q8_want(xv[slot[e, :n].long()], w1v[e], w2v[e])
        check(y[e, :n], want, tol, f"expert {e}")
