"""Products over many tiles and sums in parts: what the accumulators' hand-over and the parts'
scratch have to keep apart."""
import ctypes

import pytest
import torch

import q8_ref as ref
from test_gpu_q8 import check, dev, ffn_q8_want, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


@pytest.mark.parametrize("d,F", [(128, 6144), (6144, 128)])
@pytest.mark.parametrize("counts", [(2048, 2048), (1907, 2045)])
def test_many_wide_tiles_a_pair(sm, d, F, counts):
    """16 token tiles of 256 (or 240) tokens by 24 feature tiles, five and more in a row for
    each of 74 CTA pairs: two such tiles share TMEM columns, and each accumulator is used
    again and again."""
    N, C = 2, 2048
    g = torch.Generator("cuda").manual_seed(d)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    x = rand(N * C, d).bfloat16()
    w1, w2 = (rand(N, F, d) * d ** -0.5).bfloat16(), (rand(N, d, F) * F ** -0.5).bfloat16()
    n = dev(torch.tensor(counts, dtype=torch.int32))
    cfg = sm.config(N * C, d, F, N, 1.0, flags=sm.FLAG_ROWS_DISPATCHED)
    ws = sm.workspace(cfg)
    a, b = sm.q8_weights(N, F, d), sm.q8_weights(N, d, F)
    sm.switch_quantize_weights(cfg, w1, w2, *a, *b)
    (xq, xs), (hq, hs) = sm.q8_rows(N * C, d), sm.q8_rows(N * C, F)
    y = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
    sm.switch_expert_ffn_checkpoint(cfg, x, None, n, w1, w2, y, xq, xs, hq, hs, ws)
    y.fill_(-7.0)
    sm.switch_expert_ffn_q8(cfg, xq, xs, None, n, *a, *b, y, ws)
    again = torch.full_like(y, -7.0)
    sm.switch_expert_ffn_q8(cfg, xq, xs, None, n, *a, *b, again, ws)
    assert sm.switch_get_device_error(ws)[0] == 0
    assert torch.equal(y, again)
    xv = ref.rows(xq, xs).view(N, C, d).cuda()
    w1v, w2v = ref.weights(*a).cuda(), ref.weights(*b).cuda()
    for e, k in enumerate(counts):
        want, tol = ffn_q8_want(xv[e, :k], w1v[e], w2v[e])
        check(y[e, :k], want.cpu(), tol.cpu(), f"expert {e}")
        assert (y[e, k:] == -7).all()


def launches(call):
    """Kernels of a call, counted in its captured graph."""
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    n = ctypes.c_size_t(0)
    get = ctypes.CDLL("libcuda.so.1").cuGraphGetNodes
    assert get(ctypes.c_void_p(g.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    g.instantiate()
    return n.value, g


# (sizes, products in parts: of the 8-bit FFN, of the FFN with checkpoint, of the backward)
SPLITS = [((20, 5632, 5696, 1, 1.0), 2, 2, 2), ((8000, 128, 192, 3, 2.0), 0, 0, 1),
          ((300, 64, 4672, 1, 1.0), 1, 1, 1), ((700, 320, 832, 6, 1.25), 0, 0, 0)]


@pytest.mark.parametrize("sizes,q8,fwd,bwd", SPLITS)
def test_parts_are_taken_and_repeat(sm, sizes, q8, fwd, bwd):
    """Each product whose sum goes in parts adds a launch: hidden and out rows of both FFNs,
    da and dx, the weight gradients.  All outputs keep their bits: again, over scratch that
    holds NaN, on another stream, and from captured graphs."""
    T, d, F, N, cf = sizes
    C = sm.switch_capacity(T, N, cf)
    g = gen(d + F)
    x = dev(torch.randn(T, d, generator=g).bfloat16())
    dy = dev(torch.randn(N, C, d, generator=g).bfloat16())
    w1 = dev((torch.randn(N, F, d, generator=g) * d ** -0.5).bfloat16())
    w2 = dev((torch.randn(N, d, F, generator=g) * F ** -0.5).bfloat16())
    counts, slot, _ = ref.routing(T, N, C, 6)
    counts, slot = dev(counts), dev(slot)
    cfg = sm.config(T, d, F, N, cf)
    ws = sm.backward_workspace(cfg)
    tq, ts = sm.q8_rows(T, d)
    (xq, xs), (hq, hs) = sm.q8_rows(N * C, d), sm.q8_rows(N * C, F)
    (w1q, w1s), (w2q, w2s) = sm.q8_weights(N, F, d), sm.q8_weights(N, d, F)
    sm.switch_quantize_weights(cfg, w1, w2, w1q, w1s, w2q, w2s)
    sm.switch_residual_norm(cfg, x, None, None, 1e-6, None, None, tq, ts, None)
    out = [torch.zeros_like(t) for t in (dy, dy, dy, w1, w2)] + [t.view(torch.uint8) for t in (xq, hq, hs)]
    calls = [
        lambda: sm.switch_expert_ffn_q8(cfg, tq, ts, slot, counts, w1q, w1s, w2q, w2s, out[0], ws),
        lambda: sm.switch_expert_ffn_checkpoint(cfg, x, slot, counts, w1, w2, out[1], xq, xs, hq, hs, ws),
        lambda: sm.switch_expert_ffn_backward_q8(cfg, xq, xs, hq, hs, counts, w1, w2, dy, *out[2:5], ws)]

    def run():
        for c in calls:
            c()

    def same():
        torch.cuda.synchronize()
        assert sm.switch_get_device_error(ws)[0] == 0
        ok = [torch.equal(a, b) for a, b in zip(out, want)]
        for t in out[:5]:
            t.zero_()
        ws[256:] = 255
        return all(ok)

    ws[256:] = 255
    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    assert all(torch.isfinite(t).all() and t.abs().max() > 0 for t in want[:5])
    assert same()
    run()
    assert same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    assert same()
    graphs = [launches(c) for c in calls]
    for _ in range(2):
        for _, gr in graphs:
            gr.replay()
        assert same()
    # gather and two products; copy and two products; unpacking, da, dx and both gradients
    assert [n for n, _ in graphs] == [3 + q8, 3 + fwd, 4 + bwd]
