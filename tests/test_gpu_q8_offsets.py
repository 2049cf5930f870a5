"""Rows whose offsets pass 32 bits: more than 2^31 values and 2^32 bytes in a tensor.  What the
calls make of the last rows has to be what they make of those rows alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("T,d", [(600001, 4096), (140001, 16384)])
def test_norm(sm, T, d):
    """Register-held and wide rows; the rows' codes pass 2^31 bytes."""
    n = 77
    g = torch.Generator("cuda").manual_seed(d)
    gain = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    x, r = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    x[-n:], r[-n:] = rand(g, n, d), rand(g, n, d)

    def run(x, r):
        t = len(x)
        cfg = sm.config(t, d, 64, 1, 1.0)
        y, rstd, q = torch.empty_like(x), torch.empty(t, device="cuda"), sm.q8_rows(t, d)
        sm.switch_residual_norm(cfg, x, r, gain, 1e-6, r, y, *q, rstd)       # (z in r's buffer)
        dx, dg = torch.empty_like(x), torch.empty(d, device="cuda")
        sm.switch_residual_norm_backward(cfg, r, gain, rstd, y, None, dx, dg, sm.norm_workspace(cfg))
        terms = (y[-n:].double() * r[-n:].double() * rstd[-n:, None].double()).abs().sum(0)
        return [v[-n:].view(torch.uint8) for v in (r, y, dx, rstd, *q)], dg, terms

    small = run(x[-n:].clone(), r[-n:].clone())
    big = run(x, r)
    assert all(torch.equal(a, b) for a, b in zip(small[0], big[0]))
    # the other rows are zeros: dgain is the last rows', n values (and three roundings in each)
    # in another order, off by at most so many half steps of the terms' sizes on either side
    off = (small[1].double() - big[1].double()).abs()
    assert (off <= 2 * (n + 3) * 2.0 ** -24 * small[2]).all()


def test_expert_ffns(sm):
    """Hidden rows of 2^32 codes, in bf16 twice the bytes; dispatched rows of one expert.  The last
    rows' own batch has the same config, so the same sums in the same order: the same bits, the
    weight gradients' too, as the other rows' dy is zero and their number fills whole stages."""
    T, d, F, n = 66048, 64, 65536, 192
    assert (T - n) % 64 == 0 and T * F > 2 ** 32
    g = torch.Generator("cuda").manual_seed(3)
    w1, w2 = rand(g, 1, F, d) * d ** -0.5, rand(g, 1, d, F) * F ** -0.5
    cfg = sm.config(T, d, F, 1, 1.0, flags=sm.FLAG_ROWS_DISPATCHED)
    ws = sm.backward_workspace(cfg)
    wq = sm.q8_weights(1, F, d), sm.q8_weights(1, d, F)
    sm.switch_quantize_weights(cfg, w1, w2, *wq[0], *wq[1])
    x, dy = rand(g, T, d), torch.zeros(1, T, d, dtype=torch.bfloat16, device="cuda")
    dy[:, -n:] = rand(g, 1, n, d)
    a, h = sm.q8_rows(T, d), sm.q8_rows(T, F)

    def run(x, dy, rows):
        c = torch.tensor([rows], dtype=torch.int32, device="cuda")
        y, yq, dx = (torch.zeros_like(dy) for _ in range(3))
        dw1, dw2 = torch.empty_like(w1), torch.empty_like(w2)
        sm.switch_expert_ffn_checkpoint(cfg, x, None, c, w1, w2, y, *a, *h, ws)
        sm.switch_expert_ffn_q8(cfg, *a, None, c, *wq[0], *wq[1], yq, ws)
        sm.switch_expert_ffn_backward_q8(cfg, *a, *h, c, w1, w2, dy, dx, dw1, dw2, ws)
        assert sm.switch_get_device_error(ws)[0] == 0
        last = slice(rows - n, rows)
        return [v.view(torch.uint8)[last].clone() for v in (*a, *h)] + \
            [v[0, last].clone() for v in (y, yq, dx)] + [dw1, dw2]

    big = run(x, dy, T)
    assert all(v.view(torch.uint8).any() for v in big)
    small = run(x.roll(n, 0), dy.roll(n, 1), n)
    assert all(torch.equal(u, v) for u, v in zip(small, big))
