"""The residual norm over so many rows that a block takes several in turn, in each of its
kernels, and over long columns of the gain's gradient.

Tolerances.  A row's sum is taken by W warps (the fewest of 1, 2, 4, 8 that hold it in V 16-byte
vectors a lane, V = 2 forward and 4 backward; 256 threads for wider rows): a lane adds n values in
sequence, then come 5 steps across the warp and W across the warps, each off by 2^-24 at most of
sums of magnitudes.  1 / rms halves that (the root) and adds the mean's two roundings (halved), the
root's and the quotient's; y two products more.  dx: the sum, and at most 12 roundings of products
and sums behind it.  dgain: a lane adds every blocks-th row, or runs of 64 rows that are added in
turn, then at most 8 rows of a block, 10 parts in sequence and 5 steps across a warp, and 3
roundings are in each term."""
import math

import pytest
import torch

import q8_ref as ref
from test_gpu_q8 import check

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -24


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


def lanes(d, dtype, vecs):
    """Values that a lane adds in sequence, warps of a row, whether rows are wide."""
    per = 8 if dtype == torch.bfloat16 else 4
    nv = (d + per - 1) // per
    for v in (vecs, 4):
        for w in (1, 2, 4, 8):
            if nv <= 32 * v * w:
                return v * per, w, False
    return math.ceil(nv / 256) * per, 8, True


def check_on_gpu(got, want, tol, what):
    assert torch.isfinite(got).all(), what
    worst = ((got.double() - want).abs() - tol).max().item()
    assert worst <= 0, f"{what}: {worst} above its tolerance"


# (W, V) = (1, 2), (2, 2), (4, 2), (8, 2), (8, 4) and wide forward; 1, 1, 2, 4, 8 warps and wide
# backward: each with three rounds or more of the blocks that a launch has at most
LONG = [(30001, 64, torch.bfloat16), (15001, 1024, torch.bfloat16), (7003, 2048, torch.bfloat16),
        (3001, 4096, torch.bfloat16), (3001, 8192, torch.bfloat16), (8001, 8256, torch.bfloat16),
        (15001, 516, torch.float32), (7003, 772, torch.float32), (3001, 2048, torch.float32),
        (3001, 4096, torch.float32), (7300, 4100, torch.float32)]


@pytest.mark.parametrize("T,d,dtype", LONG)
def test_rows_in_turn(sm, T, d, dtype):
    g = torch.Generator("cuda").manual_seed(T + d)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    size = torch.exp(2 * rand(T, 1))
    x, r = (size * rand(T, d)).to(dtype), (size * rand(T, d)).to(dtype)
    gain = 1 + 0.3 * rand(d)
    cfg = sm.config(T, d, 64, 1, 1.0, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    z, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    yq, ys = sm.q8_rows(T, d)
    sm.switch_residual_norm(cfg, x, r, gain, 1e-6, z, y, yq, ys, rstd)
    assert torch.equal(z, (x.float() + r.float()).to(dtype))
    n, w, _ = lanes(d, dtype, 2)
    tol_r = ((n + 5 + w + 2) / 2 + 2) * F32
    h = z.double()
    want_r = 1 / torch.sqrt((h * h).mean(1) + 1e-6)
    check_on_gpu(rstd, want_r, tol_r * want_r, "rstd")
    want = h * want_r[:, None] * gain.double()
    rel = tol_r + 2 * F32
    check_on_gpu(y, want, (ref.HALF[dtype] * (1 + rel) + rel) * want.abs(), "y")
    s = torch.exp2(ys.view(torch.uint8).double() - 127)
    b = s.shape[1]
    amax = torch.nn.functional.pad(want, (0, b * 128 - d)).reshape(T, b, 128).abs().amax(2)
    assert (448 * s >= amax * (1 - rel)).all()
    assert ((s == 2.0 ** -100) | (224 * s < amax * (1 + rel))).all()
    full = ref.spread(s, d)
    tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * full) + 2 * rel * want.abs()
    check_on_gpu(yq.float().double() * full, want, tol, "8-bit y")
    del yq, ys, full, tol, want

    dy, ds = rand(T, d).to(dtype), rand(T, d).to(dtype)
    dx, dg = torch.empty_like(x), torch.empty(d, device="cuda")
    sm.switch_residual_norm_backward(cfg, z, gain, rstd, dy, ds, dx, dg, sm.norm_workspace(cfg))
    n, w, wide = lanes(d, dtype, 4)
    q, rr = dy.double(), rstd.double()[:, None]
    t = q * gain.double()
    c = (t * h).mean(1, keepdim=True)
    want = rr * t - h * rr ** 3 * c + ds.double()
    mag = (rr * t).abs() + h.abs() * rr ** 3 * (t * h).abs().mean(1, keepdim=True) + ds.double().abs()
    check_on_gpu(dx, want, ref.HALF[dtype] * want.abs() + (n + 5 + w + 12) * F32 * mag, "dx")
    p = q * h * rr
    check_on_gpu(dg, p.sum(0), gain_steps(T, w, wide) * F32 * p.abs().sum(0), "dgain")


def gain_steps(T, w, wide):
    rows = 8 // w                                    # of a block at a time
    turns = 64 + math.ceil(T / 64 / 64) if wide else math.ceil(T / (296 * rows))
    return turns + 8 + 10 + 5 + 3


@pytest.mark.parametrize("T,d,dtype", [(65536, 4100, torch.float32), (65536, 1024, torch.float32)])
def test_gain_gradient_of_long_columns(sm, T, d, dtype):
    """Every term of a column is alike, so that a running sum's roundings lean the same way: a
    thousand terms in sequence are 170 2^-24 off here, runs of 64 of them 12."""
    x = torch.full((T, d), 1.0, dtype=dtype, device="cuda")
    dy = torch.full((T, d), 0.7, dtype=dtype, device="cuda")
    rstd = torch.full((T,), 1.0, device="cuda")
    cfg = sm.config(T, d, 64, 1, 1.0, dtype="f32")
    dg = torch.empty(d, device="cuda")
    sm.switch_residual_norm_backward(cfg, x, None, rstd, dy, None, None, dg, sm.norm_workspace(cfg))
    want = T * dy[0, 0].double().cpu()
    n, w, wide = lanes(d, dtype, 4)
    check(dg, want.expand(d), gain_steps(T, w, wide) * F32 * want, "dgain")
