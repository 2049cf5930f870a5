"""A NaN among the hidden values: it stays NaN, in y and in the 8-bit rows, and touches no
other value and no scale, however many tokens the call has and however its sums are taken."""
import pytest
import torch

import q8_ref as ref
from test_gpu_q8 import dev, ffn_inputs

pytestmark = pytest.mark.gpu
NAN = 127                                            # e4m3's NaN, without the sign


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


def bits(t):
    return t.view(torch.uint8)


# few tokens; tiles; both products in parts
@pytest.mark.parametrize("T,d,F,N", [(3, 128, 320, 2), (8, 1024, 640, 1), (9, 128, 320, 2),
                                     (300, 192, 320, 3), (20, 5632, 5696, 1)])
def test_ffn_q8(sm, T, d, F, N):
    """A NaN in one feature's weights makes every row of that expert NaN; a NaN in a token's row
    that token's; the other rows keep their bits."""
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, float(N), 3 * T + d)
    xq, xs = map(dev, ref.to_q8(x))
    w1q, w1s = map(dev, ref.as_q8(*ref.quantize_weights(w1)))
    w2q, w2s = map(dev, ref.as_q8(*ref.quantize_weights(w2)))
    cfg = sm.config(T, d, F, N, float(N))
    ws = sm.workspace(cfg)

    def run(rows, weights):
        y = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
        sm.switch_expert_ffn_q8(cfg, rows, xs, dev(slot), dev(counts), weights, w1s, w2q, w2s, y, ws)
        assert sm.switch_get_device_error(ws)[0] == 0
        return y

    want = run(xq, w1q)
    assert torch.isfinite(want).all()
    e = int(counts.argmax())
    n = int(kept[e])
    bad = w1q.clone()
    bits(bad)[e, F - 3, 5] = NAN
    got = run(xq, bad)
    assert torch.isnan(got[e, :n]).all()
    got[e, :n] = want[e, :n]
    assert torch.equal(got, want)
    t = int(slot.view(N, C)[e, n - 1])
    bad = xq.clone()
    bits(bad)[t, d - 2] = NAN
    got = run(bad, w1q)
    assert torch.isnan(got[e, n - 1]).all()
    got[e, n - 1] = want[e, n - 1]
    assert torch.equal(got, want)


# tiles (a block of 128 features whole, and one of 64), and sums in parts
@pytest.mark.parametrize("T,d,F,N", [(200, 128, 320, 2), (37, 2368, 2432, 1)])
def test_checkpoint(sm, T, d, F, N):
    """Features whose weights hold a NaN, one of them the only one of its 32 neighbours that
    the scale could overlook: their codes are NaN, all other codes and all scales are those
    of the same features at zero."""
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, 1.0, 5 * T + d)
    x, w1, w2 = dev(x.bfloat16()), dev(w1.bfloat16()), dev(w2.bfloat16())
    w1[:, 33] *= 64                                  # the largest of its block, beside a NaN
    feats = [34, 128, F - 1]
    cfg = sm.config(T, d, F, N, 1.0)
    ws = sm.workspace(cfg)

    def run(weights):
        y = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
        (xq, xs), (hq, hs) = sm.q8_rows(N * C, d), sm.q8_rows(N * C, F)
        sm.switch_expert_ffn_checkpoint(cfg, x, dev(slot), dev(counts), weights, w2, y, xq, xs, hq, hs, ws)
        assert sm.switch_get_device_error(ws)[0] == 0
        return y, bits(hq).view(N, C, F), bits(hs).view(N, C, -1)

    zero, bad = w1.clone(), w1.clone()
    zero[0, feats] = 0
    bad[0, feats, 7] = float("nan")
    y0, q0, s0 = run(zero)
    y1, q1, s1 = run(bad)
    n = int(kept[0])
    assert n > 0 and torch.isfinite(y0).all()
    assert torch.equal(s1, s0)
    assert ((q1[0, :n][:, feats] & 127) == NAN).all() and (q0[0, :n][:, feats] == 0).all()
    q1[0, :n, feats] = 0
    assert torch.equal(q1, q0)
    assert torch.isnan(y1[0, :n]).all()
    assert torch.equal(y1[1:], y0[1:]) and torch.equal(y1[0, n:], y0[0, n:])


def test_block_of_nan(sm):
    """A whole block of NaN has the scale of a block of zeros, by tiles and in parts alike."""
    for T, d, F in ((40, 128, 256), (37, 2368, 2432)):
        C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, 1, 1.0, 9)
        x, w1, w2 = dev(x.bfloat16()), dev(w1.bfloat16()), dev(w2.bfloat16())
        w1[0, 128:256, 0] = float("nan")
        cfg = sm.config(T, d, F, 1, 1.0)
        ws = sm.workspace(cfg)
        y = torch.zeros(1, C, d, dtype=torch.bfloat16, device="cuda")
        (xq, xs), (hq, hs) = sm.q8_rows(C, d), sm.q8_rows(C, F)
        sm.switch_expert_ffn_checkpoint(cfg, x, dev(slot), dev(counts), w1, w2, y, xq, xs, hq, hs, ws)
        assert ((bits(hq)[:, 128:256] & 127) == NAN).all() and (bits(hs)[:, 1] == 27).all()
        assert (bits(hs)[:, 0] > 27).all() and ((bits(hq)[:, :128] & 127) != NAN).all()
