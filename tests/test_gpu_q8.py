"""The residual norm, the 8-bit expert FFN and the 8-bit checkpoints on the
GPU, against plain 64-bit forms.

Tolerances, derived once:
* a rounding to a type is off by at most half a step, relative to the value
  (bf16 2^-8, fp32 2^-24, e4m3 2^-4, or half of 2^-9 scales where e4m3 is
  subnormal);
* a sum of n products in fp32 is off by at most n 2^-24 of the sum of their
  magnitudes;
* the norm's 1 / rms takes at most 32 sequential additions a lane and 8 across
  (64 2^-24 = 2^-18 relative with the root, the quotient and the products);
* a hidden value whose exact value lies within its own fp32 error of the middle
  between two codes may take either: one step (2^-3 of the value at most),
  weighted with |w2|, is allowed for exactly those values, and twice that for
  the blocks whose maximum lies that near to a change of scale.
"""
import numpy as np
import pytest
import torch

import q8_ref as ref

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -24


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


def dev(t, dtype=None):
    return (t if dtype is None else t.to(dtype)).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check(got, want, tol, what):
    got = got.cpu().double()
    assert torch.isfinite(got).all(), what
    worst = ((got - want).abs() - tol).max().item() if got.numel() else 0.0
    assert worst <= 0, f"{what}: {worst} above its tolerance"


# -------------------------------------------------------------------- norm

def norm_inputs(T, d, dtype, seed, residual):
    g = gen(seed)
    size = torch.exp(2 * torch.randn(T, 1, generator=g))
    x = (size * torch.randn(T, d, generator=g)).to(dtype)
    r = (size * torch.randn(T, d, generator=g)).to(dtype) if residual else None
    return x, r, 1 + 0.3 * torch.randn(d, generator=g)


SHAPES = [(1, 64, torch.bfloat16), (3, 128, torch.bfloat16), (130, 192, torch.bfloat16),
          (67, 1024, torch.bfloat16), (9, 1088, torch.bfloat16), (5, 4096, torch.bfloat16),
          (7, 8192, torch.bfloat16), (4, 8256, torch.bfloat16), (2, 20480, torch.bfloat16),
          (1, 4, torch.float32), (33, 100, torch.float32), (17, 512, torch.float32),
          (18, 516, torch.float32), (6, 2052, torch.float32), (3, 4100, torch.float32),
          (2, 10244, torch.float32), (6000, 64, torch.bfloat16)]


@pytest.mark.parametrize("T,d,dtype", SHAPES)
@pytest.mark.parametrize("residual,gain", [(True, True), (False, True), (True, False)])
def test_norm(sm, T, d, dtype, residual, gain):
    x, r, g = norm_inputs(T, d, dtype, 7 * T + d, residual)
    x[T // 2] = 0                                    # a row of zeros: eps alone
    if residual:
        r[T // 2] = 0
    cfg = sm.config(T, d, 64, 1, 1.0, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    z = torch.empty_like(x, device="cuda")
    y, rstd = torch.empty_like(z), torch.empty(T, device="cuda")
    yq, ys = sm.q8_rows(T, d)
    sm.switch_residual_norm(cfg, dev(x), dev(r) if residual else None, dev(g) if gain else None,
                            1e-6, z, y, yq, ys, rstd)
    held = (x.float() + r.float()).to(dtype) if residual else x
    assert torch.equal(z.cpu(), held)
    h = held.double()
    want_r = 1 / torch.sqrt((h * h).mean(1) + 1e-6)
    check(rstd, want_r, 2.0 ** -18 * want_r, "rstd")
    want = h * want_r[:, None] * (g.double() if gain else 1.0)
    check(y, want, (ref.HALF[dtype] + 2.0 ** -18) * want.abs(), "y")
    # 8 bits: the scale is right for the maximum (up to its fp32 error), each
    # value within half a step
    s = ref.scales(ys)
    b = s.shape[1]
    amax = torch.nn.functional.pad(want, (0, b * 128 - d)).reshape(T, b, 128).abs().amax(2)
    assert (448 * s >= amax * (1 - 2.0 ** -18)).all()
    assert ((s == 2.0 ** -100) | (224 * s < amax * (1 + 2.0 ** -18))).all()
    full = ref.spread(s, d)
    tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * full) + 2.0 ** -17 * want.abs()
    check(ref.rows(yq, ys), want, tol, "8-bit y")
    # each output alone gives the same bits; z may be the residual's or x's buffer
    y2 = torch.empty_like(y)
    own = dev(r) if residual else dev(x)
    sm.switch_residual_norm(cfg, dev(x), own if residual else None, dev(g) if gain else None, 1e-6,
                            own if residual else None, y2, None, None, None)
    assert torch.equal(y2, y)
    if residual:
        assert torch.equal(own, z)
    q2, s2 = sm.q8_rows(T, d)
    sm.switch_residual_norm(cfg, dev(x), dev(r) if residual else None, dev(g) if gain else None,
                            1e-6, None, None, q2, s2, None)
    assert torch.equal(q2.view(torch.uint8), yq.view(torch.uint8))
    assert torch.equal(s2.view(torch.uint8), ys.view(torch.uint8))


@pytest.mark.parametrize("T,d,dtype", SHAPES)
@pytest.mark.parametrize("dsum,gain", [(True, True), (False, True), (True, False)])
def test_norm_backward(sm, T, d, dtype, dsum, gain):
    x, s, g = norm_inputs(T, d, dtype, 11 * T + d, True)
    dy = torch.randn(T, d, generator=gen(T + d)).to(dtype)
    rstd = torch.rsqrt(x.double().square().mean(1) + 1e-6).float()
    cfg = sm.config(T, d, 64, 1, 1.0, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    ws = sm.norm_workspace(cfg).fill_(255)           # nothing in it has to be zero
    dx, dg = torch.empty_like(x, device="cuda"), torch.empty(d, device="cuda")
    args = (dev(x), dev(g) if gain else None, dev(rstd), dev(dy), dev(s) if dsum else None)
    sm.switch_residual_norm_backward(cfg, *args, dx, dg, ws)
    z, y, r = x.double(), dy.double(), rstd.double()[:, None]
    t = y * (g.double() if gain else 1.0)
    part = s.double() if dsum else torch.zeros_like(z)
    want = r * t - z * r ** 3 * (t * z).mean(1, keepdim=True) + part
    size = (r * t).abs() + z.abs() * r ** 3 * (t * z).abs().mean(1, keepdim=True) + part.abs()
    check(dx, want, ref.HALF[dtype] * want.abs() + 2.0 ** -17 * size, "dx")
    p = y * z * r
    check(dg, p.sum(0), (T + 64) * F32 * p.abs().sum(0) + 1e-30, "dgain")
    # each alone, dx in dy's buffer, again: the same bits
    d2, g2 = args[3].clone(), torch.empty_like(dg)
    sm.switch_residual_norm_backward(cfg, args[0], args[1], args[2], d2, args[4], d2, g2, ws)
    assert torch.equal(d2, dx) and torch.equal(g2, dg)
    d3 = torch.empty_like(dx)
    sm.switch_residual_norm_backward(cfg, *args, d3, None, None)
    assert torch.equal(d3, dx)
    g3 = torch.empty_like(dg)
    sm.switch_residual_norm_backward(cfg, *args, None, g3, ws)
    assert torch.equal(g3, dg)


def test_norm_backward_by_differences(sm):
    """The gradients against central differences of the forward's formula in 64 bits."""
    T, d = 4, 132
    x, _, g = norm_inputs(T, d, torch.float32, 3, False)
    dy = torch.randn(T, d, generator=gen(4))
    cfg = sm.config(T, d, 64, 1, 1.0, dtype="f32")
    rstd = torch.empty(T, device="cuda")
    sm.switch_residual_norm(cfg, dev(x), None, dev(g), 1e-5, None, torch.empty(T, d, device="cuda"),
                            None, None, rstd)
    dx, dg = torch.empty(T, d, device="cuda"), torch.empty(d, device="cuda")
    sm.switch_residual_norm_backward(cfg, dev(x), dev(g), rstd, dev(dy), None, dx, dg,
                                     sm.norm_workspace(cfg))

    def value(xv, gv):
        return (xv / torch.sqrt((xv * xv).mean(1, keepdim=True) + 1e-5) * gv * dy.double()).sum()

    h = 1e-6
    for t, c in ((0, 0), (1, 77), (3, 131)):
        s = h * x[t].double().abs().mean()
        up, dn = x.double().clone(), x.double().clone()
        up[t, c] += s
        dn[t, c] -= s
        num = (value(up, g.double()) - value(dn, g.double())) / (2 * s)
        # fp32's part as above, the difference's own: s^2 and 2^-52 / s of the value's size
        assert abs(num - dx[t, c].item()) <= 1e-4 * dx[t].abs().max().item()
        up, dn = g.double().clone(), g.double().clone()
        up[c] += h
        dn[c] -= h
        num = (value(x.double(), up) - value(x.double(), dn)) / (2 * h)
        assert abs(num - dg[c].item()) <= 1e-4 * dg.abs().max().item()


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("N,F,d", [(1, 64, 64), (3, 320, 192), (2, 256, 1024)])
def test_quantize_weights(sm, N, F, d):
    cfg = sm.config(8, d, F, N, 1.0)
    w1 = (torch.randn(N, F, d, generator=gen(F)) * torch.exp(
        torch.randn(N, F, 1, generator=gen(d)))).bfloat16()
    w2 = torch.randn(N, d, F, generator=gen(N)).bfloat16()
    w2[0, :64] = 0
    b1, b2 = sm.q8_weights(N, F, d), sm.q8_weights(N, d, F)
    sm.switch_quantize_weights(cfg, dev(w1), dev(w2), *b1, *b2)
    for w, (q, s) in ((w1, b1), (w2, b2)):
        wq, wsc = ref.quantize_weights(w.double())
        assert torch.equal(ref.scales(s), wsc) and torch.equal(ref.codes(q), wq)
    only = sm.q8_weights(N, d, F)
    sm.switch_quantize_weights(cfg, None, dev(w2), None, None, *only)
    assert torch.equal(only[0].view(torch.uint8), b2[0].view(torch.uint8))


# ------------------------------------------------------------- 8-bit FFN

def ffn_inputs(T, d, F, N, cf, seed, dead=()):
    from oracle.switch_oracle import capacity
    C = capacity(T, N, cf)
    counts, slot, kept = ref.routing(T, N, C, seed, dead)
    g = gen(seed)
    x = torch.randn(T, d, generator=g).double() * torch.exp(torch.randn(T, 1, generator=g))
    w1 = torch.randn(N, F, d, generator=g).double() * (0.1 / d) ** 0.5
    w2 = torch.randn(N, d, F, generator=g).double() * (0.1 / F) ** 0.5
    return C, counts, slot, kept, x, w1, w2


def ffn_q8_want(x, w1, w2):
    """64-bit FFN of decoded rows through 8-bit hidden rows, and the tolerance of a bf16 y."""
    h = (x @ w1.T).clamp(min=0)
    err = x.shape[1] * F32 * (x.abs() @ w1.abs().T)
    q, s = ref.quantize(h)
    full = ref.spread(s, h.shape[1])
    step = torch.exp2(torch.floor(torch.log2((h / full).clamp(min=2.0 ** -6))) - 3)
    off = (h / full / step) % 1.0
    near = ((off - 0.5).abs() * step * full <= err) & (h + err > 0)
    loose = torch.where(near, step * full, torch.zeros_like(h))
    # blocks whose maximum is that near to a change of scale
    b = s.shape[1]
    pad = (0, b * 128 - h.shape[1])
    a = torch.nn.functional.pad(h, pad).reshape(-1, b, 128).amax(2)
    ea = torch.nn.functional.pad(err, pad).reshape(-1, b, 128).amax(2)
    border = (torch.minimum((a - 448 * s).abs(), (a - 224 * s).abs()) <= ea)
    loose = torch.where(ref.spread(border, h.shape[1]), 2 * step * full, loose)
    hv = q * full
    y = hv @ w2.T
    tol = 2.0 ** -8 * y.abs() + h.shape[1] * F32 * (hv.abs() @ w2.abs().T) + loose @ w2.abs().T
    return y, tol * 1.001 + 1e-30


FFN = [(1, 64, 64, 1, 1.0), (2, 128, 128, 1, 4.0), (300, 64, 128, 2, 1.0), (700, 320, 832, 6, 1.25),
       (513, 192, 320, 3, 2.0), (40, 1088, 704, 16, 8.0), (1000, 512, 1024, 4, 0.5),
       (8, 1024, 2048, 64, 32.0), (260, 2560, 640, 1, 1.0), (3000, 256, 2304, 12, 1.0)]


@pytest.mark.parametrize("T,d,F,N,cf", FFN)
@pytest.mark.parametrize("dispatched", [False, True])
def test_ffn_q8(sm, T, d, F, N, cf, dispatched):
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, cf, T + d + F)
    xq, xs = ref.to_q8(x)
    w1q, w1s = ref.as_q8(*ref.quantize_weights(w1))
    w2q, w2s = ref.as_q8(*ref.quantize_weights(w2))
    cfg = sm.config(T, d, F, N, cf, flags=sm.FLAG_ROWS_DISPATCHED if dispatched else 0)
    ws = sm.workspace(cfg)
    ws[256:] = 255                                   # scratch may hold anything (NaN codes here)
    y = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
    dq, ds = xq, xs
    if dispatched:
        t = slot.clamp(min=0).long()
        dq, ds = xq.view(torch.uint8)[t], xs.view(torch.uint8)[t]
        dq[slot < 0], ds[slot < 0] = 127, 255        # NaN behind the last token
    sm.switch_expert_ffn_q8(cfg, dev(dq), dev(ds), None if dispatched else dev(slot), dev(counts),
                            dev(w1q), dev(w1s), dev(w2q), dev(w2s), y, ws)
    assert sm.switch_get_device_error(ws)[0] == 0
    xv, w1v, w2v = ref.rows(xq, xs), ref.weights(w1q, w1s), ref.weights(w2q, w2s)
    for e in range(N):
        n = int(kept[e])
        assert (y[e, n:] == -7).all(), "rows behind the last token are left as they were"
        if n:
            want, tol = ffn_q8_want(xv[slot.view(N, C)[e, :n].long()], w1v[e], w2v[e])
            check(y[e, :n], want, tol, f"expert {e}")


def test_ffn_q8_scale_range(sm):
    """Rows of very different sizes, zero rows and weights far from one: the scales carry it."""
    T, d, F, N = 200, 256, 384, 2
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, 1.0, 5)
    x *= torch.exp2(torch.randint(-40, 41, (T, 1), generator=gen(1)).double())
    x[::7] = 0
    x[:, 128:] *= 2.0 ** -20                         # a second block far below the first
    w1[:, 128:] *= 2.0 ** 12
    xq, xs = ref.to_q8(x)
    w1q, w1s = ref.as_q8(*ref.quantize_weights(w1))
    w2q, w2s = ref.as_q8(*ref.quantize_weights(w2 * 2.0 ** -15))
    cfg = sm.config(T, d, F, N, 1.0)
    ws = sm.workspace(cfg)
    y = torch.zeros(N, C, d, dtype=torch.bfloat16, device="cuda")
    sm.switch_expert_ffn_q8(cfg, dev(xq), dev(xs), dev(slot), dev(counts), dev(w1q), dev(w1s),
                            dev(w2q), dev(w2s), y, ws)
    xv, w1v, w2v = ref.rows(xq, xs), ref.weights(w1q, w1s), ref.weights(w2q, w2s)
    for e in range(N):
        n = int(kept[e])
        want, tol = ffn_q8_want(xv[slot.view(N, C)[e, :n].long()], w1v[e], w2v[e])
        check(y[e, :n], want, tol, f"expert {e}")


def test_ffn_q8_many_experts(sm):
    """As many experts as a config takes, most without tokens."""
    T, d, F, N = 300, 64, 128, 1024
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, 8.0, 3, dead=range(0, 1024, 3))
    xq, xs = ref.to_q8(x)
    w1q, w1s = ref.as_q8(*ref.quantize_weights(w1))
    w2q, w2s = ref.as_q8(*ref.quantize_weights(w2))
    cfg = sm.config(T, d, F, N, 8.0)
    ws = sm.workspace(cfg)
    y = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
    sm.switch_expert_ffn_q8(cfg, dev(xq), dev(xs), dev(slot), dev(counts), dev(w1q), dev(w1s),
                            dev(w2q), dev(w2s), y, ws)
    assert sm.switch_get_device_error(ws)[0] == 0
    xv, w1v, w2v = ref.rows(xq, xs), ref.weights(w1q, w1s), ref.weights(w2q, w2s)
    for e in range(N):
        n = int(kept[e])
        assert (y[e, n:] == -7).all()
        if n:
            want, tol = ffn_q8_want(xv[slot.view(N, C)[e, :n].long()], w1v[e], w2v[e])
            check(y[e, :n], want, tol, f"expert {e}")


# few tiles and long sums: the products go in parts (the second, the first, both, the second
# over many experts' few rows with most experts empty)
PARTS = [(300, 64, 4672, 1, 1.0), (300, 4672, 64, 1, 1.0), (20, 5632, 5696, 1, 1.0),
         (30, 128, 6016, 60, 4.0), (70, 192, 9472, 3, 2.0)]


@pytest.mark.parametrize("T,d,F,N,cf", PARTS)
@pytest.mark.parametrize("dispatched", [False, True])
def test_ffn_q8_in_parts(sm, T, d, F, N, cf, dispatched):
    test_ffn_q8(sm, T, d, F, N, cf, dispatched)


@pytest.mark.parametrize("T", [3, 400])
def test_ffn_q8_top2(sm, T):
    """Both routes of a token in slots of their experts: capacity over 2 T assignments, the
    same token's row twice."""
    from oracle.switch_oracle import capacity
    d, F, N, cf = 128, 320, 5, 1.0
    C = capacity(2 * T, N, cf)
    rng = np.random.default_rng(T)
    pairs = np.array([rng.permutation(N)[:2] for _ in range(T)])
    tok = [[t for t in range(T) if pairs[t, 0] == e] + [t for t in range(T) if pairs[t, 1] == e]
           for e in range(N)]
    counts = torch.tensor([len(t) for t in tok], dtype=torch.int32)
    slot = torch.full((N, C), -1, dtype=torch.int32)
    for e in range(N):
        slot[e, :min(len(tok[e]), C)] = torch.tensor(tok[e][:C], dtype=torch.int32)
    _, _, _, _, x, w1, w2 = ffn_inputs(T, d, F, N, cf, 17)
    xq, xs = ref.to_q8(x)
    w1q, w1s = ref.as_q8(*ref.quantize_weights(w1))
    w2q, w2s = ref.as_q8(*ref.quantize_weights(w2))
    cfg = sm.config(T, d, F, N, cf, flags=sm.FLAG_TOP2)
    ws = sm.workspace(cfg)
    y = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
    sm.switch_expert_ffn_q8(cfg, dev(xq), dev(xs), dev(slot.reshape(-1)), dev(counts), dev(w1q),
                            dev(w1s), dev(w2q), dev(w2s), y, ws)
    assert sm.switch_get_device_error(ws)[0] == 0
    xv, w1v, w2v = ref.rows(xq, xs), ref.weights(w1q, w1s), ref.weights(w2q, w2s)
    for e in range(N):
        n = min(len(tok[e]), C)
        assert (y[e, n:] == -7).all()
        if n:
            want, tol = ffn_q8_want(xv[slot[e, :n].long()], w1v[e], w2v[e])
            check(y[e, :n], want, tol, f"expert {e}")


def test_ffn_q8_more_rows_than_tokens(sm):
    """Rows dispatched by other means: a config of few tokens whose capacity holds more rows
    (the few-token path takes an expert's rows eight at a time)."""
    T, d, F, N, cf = 4, 192, 320, 2, 10.0
    C = sm.switch_capacity(T, N, cf)
    assert C == 20
    _, _, _, _, _, w1, w2 = ffn_inputs(T, d, F, N, cf, 23)
    x = torch.randn(N * C, d, generator=gen(2)).double()
    counts = torch.tensor([19, 8], dtype=torch.int32)
    xq, xs = ref.to_q8(x)
    w1q, w1s = ref.as_q8(*ref.quantize_weights(w1))
    w2q, w2s = ref.as_q8(*ref.quantize_weights(w2))
    cfg = sm.config(T, d, F, N, cf, flags=sm.FLAG_ROWS_DISPATCHED)
    ws = sm.workspace(cfg)
    y = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
    sm.switch_expert_ffn_q8(cfg, dev(xq), dev(xs), None, dev(counts), dev(w1q), dev(w1s), dev(w2q),
                            dev(w2s), y, ws)
    xv, w1v, w2v = ref.rows(xq, xs), ref.weights(w1q, w1s), ref.weights(w2q, w2s)
    for e, n in enumerate(counts.tolist()):
        assert (y[e, n:] == -7).all()
        want, tol = ffn_q8_want(xv.view(N, C, d)[e, :n], w1v[e], w2v[e])
        check(y[e, :n], want, tol, f"expert {e}")


@pytest.mark.parametrize("T", [7, 90])
def test_bad_slot_token_is_reported(sm, T):
    d, F, N = 64, 64, 2
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, 2.0, 9)
    slot[0] = T + 5
    xq, xs = ref.to_q8(x)
    w1q, w1s = ref.as_q8(*ref.quantize_weights(w1))
    w2q, w2s = ref.as_q8(*ref.quantize_weights(w2))
    cfg = sm.config(T, d, F, N, 2.0)
    ws = sm.workspace(cfg)
    y = torch.zeros(N, C, d, dtype=torch.bfloat16, device="cuda")
    sm.switch_expert_ffn_q8(cfg, dev(xq), dev(xs), dev(slot), dev(counts), dev(w1q), dev(w1s),
                            dev(w2q), dev(w2s), y, ws)
    assert sm.switch_get_device_error(ws)[0] == 6 and (y[0, 0] == 0).all()
    assert sm.switch_get_device_error(ws)[0] == 0


def test_ffn_q8_forced_timeout_reports_and_recovers(sm):
    """Rows so wide that a tile takes longer than the hardware's own suspended wait (20 us),
    which no limit of the call cuts short: a CTA's 128 weight rows are 4 MB, 68000 cycles at
    62 bytes each; and so many tiles that no sum goes in parts."""
    T, d, F, N = 32, 32768, 9728, 1
    C, counts, slot, kept = 32, *ref.routing(T, N, 32, 21)

    def codes(*shape):
        return torch.randint(0, 120, shape, dtype=torch.uint8, device="cuda")

    def scales(*shape):
        return torch.full(shape, 110, dtype=torch.uint8, device="cuda")

    torch.manual_seed(21)
    a = (codes(T, d), scales(T, d // 128), dev(slot), dev(counts), codes(N, F, d),
         scales(N, F // 128, d // 128), codes(N, d, F), scales(N, d // 128, F // 128))

    def run(spin):
        cfg = sm.config(T, d, F, N, 1.0, spin_limit=spin)
        ws = sm.workspace(cfg)
        y = torch.zeros(N, C, d, dtype=torch.bfloat16, device="cuda")
        sm.switch_expert_ffn_q8(cfg, *a, y, ws)
        return sm.switch_get_device_error(ws)[0], y

    assert run(1)[0] == 5
    (s1, y1), (s2, y2) = run(0), run(0)
    assert s1 == 0 and s2 == 0 and torch.equal(y1, y2)


def test_checkpoint_forced_timeouts_report_and_recover(sm):
    """The same for the products of the FFN with checkpoint and of its backward."""
    T, d, F, N = 64, 16384, 9728, 1
    C = sm.switch_capacity(T, N, 1.0)
    g = torch.Generator("cuda").manual_seed(5)
    flags = sm.FLAG_ROWS_DISPATCHED

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    x = rand(C, d)
    dy = rand(N, C, d)
    w1 = 0.01 * rand(N, F, d)
    w2 = 0.01 * rand(N, d, F)
    counts = torch.tensor([T - 3], dtype=torch.int32, device="cuda")

    def run(spin):
        cfg = sm.config(T, d, F, N, 1.0, flags=flags, spin_limit=spin)
        ws = sm.backward_workspace(cfg)
        q, s = sm.q8_rows(C, d)
        hq, hs = sm.q8_rows(C, F)
        y, dx = torch.zeros_like(dy), torch.zeros_like(dy)
        dw1, dw2 = torch.zeros_like(w1), torch.zeros_like(w2)
        sm.switch_expert_ffn_checkpoint(cfg, x, None, counts, w1, w2, y, q, s, hq, hs, ws)
        first = sm.switch_get_device_error(ws)[0]
        sm.switch_expert_ffn_backward_q8(cfg, q, s, hq, hs, counts, w1, w2, dy, dx, dw1, dw2, ws)
        return first, sm.switch_get_device_error(ws)[0], (y, dx, dw1, dw2)

    f, b, _ = run(1)
    assert f == 5 and b == 5
    (f1, b1, one), (f2, b2, two) = run(0), run(0)
    assert f1 == b1 == f2 == b2 == 0
    assert all(torch.equal(u, v) for u, v in zip(one, two))


# ------------------------------------------------------------ checkpoints

CKPT = [(1, 64, 64, 1, 1.0, ()), (300, 64, 128, 2, 1.0, ()), (700, 320, 832, 6, 1.25, (2,)),
        (513, 192, 320, 3, 2.0, ()), (1000, 512, 1024, 4, 0.5, (0,)), (129, 128, 256, 1, 1.0, ()),
        (200, 64, 64, 1000, 8.0, tuple(range(0, 1000, 3)))]


@pytest.mark.parametrize("T,d,F,N,cf,dead", CKPT)
@pytest.mark.parametrize("flags", [0, 32, 64, 128, 2048])
def test_ffn_checkpoint(sm, T, d, F, N, cf, dead, flags):
    check_ffn_checkpoint(sm, T, d, F, N, cf, dead, flags, True)


# sums in parts: hidden and da; out and dx; all four; dw1 and dw2, with an expert without rows
CKPT_PARTS = [(300, 2368, 64, 1, 1.0, ()), (300, 64, 4672, 1, 1.0, ()), (37, 2368, 2432, 1, 1.0, ()),
              (2500, 64, 192, 1, 1.0, ()), (8000, 128, 192, 3, 2.0, (1,)), (90, 128, 9472, 3, 4.0, (0,))]


@pytest.mark.parametrize("T,d,F,N,cf,dead", CKPT_PARTS)
@pytest.mark.parametrize("flags", [0, 32])
def test_ffn_checkpoint_in_parts(sm, T, d, F, N, cf, dead, flags):
    check_ffn_checkpoint(sm, T, d, F, N, cf, dead, flags, False)


def check_ffn_checkpoint(sm, T, d, F, N, cf, dead, flags, exact):
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, cf, T + d + F + 1, dead)
    x, w1, w2 = x.bfloat16(), w1.bfloat16(), w2.bfloat16()
    cfg = sm.config(T, d, F, N, cf, flags=flags)
    ws = sm.workspace(cfg)
    ws[256:] = 255
    y = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
    xq, xs = sm.q8_rows(N * C, d)
    hq, hs = sm.q8_rows(N * C, F)
    for t in (xq, xs, hq, hs):
        t.view(torch.uint8).fill_(85)
    src = x
    if flags & sm.FLAG_ROWS_DISPATCHED:
        src = x[slot.clamp(min=0).long()].clone()
        src[slot < 0] = float("nan")
    sm.switch_expert_ffn_checkpoint(cfg, dev(src), dev(slot), dev(counts), dev(w1), dev(w2), y, xq,
                                    xs, hq, hs, ws)
    assert sm.switch_get_device_error(ws)[0] == 0
    # the FFN itself is switch_expert_ffn's, bit for bit unless sums go in parts
    y2 = torch.full_like(y, -7.0)
    ws2 = sm.workspace(cfg)
    sm.switch_expert_ffn(cfg, dev(src), dev(slot), dev(counts), dev(w1), dev(w2), y2, ws2)
    assert torch.equal(y, y2) or not exact
    for e in range(N):
        n = int(kept[e])
        r = slice(e * C, e * C + n)
        for t in (xq, xs, hq, hs):
            assert (t.view(torch.uint8)[e * C + n:(e + 1) * C] == 85).all()
        if not n:
            continue
        xe = x[slot.view(N, C)[e, :n].long()].double()
        wq, wsc = ref.quantize(xe)
        assert torch.equal(ref.codes(xq[r]), wq) and torch.equal(ref.scales(xs[r]), wsc)
        pre = xe @ w1[e].double().T
        err = d * F32 * (xe.abs() @ w1[e].double().abs().T)
        h = pre.clamp(min=0)
        got, s = ref.rows(hq[r], hs[r]), ref.spread(ref.scales(hs[r]), F)
        mask = got > 0
        assert (mask[pre > err]).all() and not mask[pre < -err].any()
        # bf16's half step, then e4m3's (or its smallest value, taken for smaller ones)
        tol = 2.0 ** -8 * h + torch.maximum(2.0 ** -4 * (1 + 2.0 ** -8) * h, 2.0 ** -9 * s) + err
        check(got, h, tol, f"hidden rows of expert {e}")
        # y: the hidden rows' fp32 errors and bf16 rounding, its own sum and rounding
        b = w2[e].double()
        want = h @ b.T
        eh = err + 2.0 ** -8 * (h + err)
        tol = eh @ b.abs().T + F * F32 * ((h + eh) @ b.abs().T)
        check(y[e, :n], want, tol + 2.0 ** -8 * (want.abs() + tol), f"y of expert {e}")
        assert (y[e, n:] == -7).all()


@pytest.mark.parametrize("T,d,F,N,cf,dead", CKPT)
@pytest.mark.parametrize("flags", [0, 32])
def test_ffn_backward_q8(sm, T, d, F, N, cf, dead, flags):
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, cf, T + d + F + 2, dead)
    w1, w2 = w1.bfloat16(), w2.bfloat16()
    g = gen(T)
    rows = x[slot.clamp(min=0).long()]
    h = torch.stack([(rows.view(N, C, d)[e] @ w1[e].double().T) for e in range(N)]).clamp(min=0)
    xq, xs = ref.to_q8(rows)
    hq, hs = ref.to_q8(h.view(N * C, F), positive=True)
    xv, hv = ref.rows(xq, xs).view(N, C, d), ref.rows(hq, hs).view(N, C, F)
    dy = torch.randn(N, C, d, generator=g).bfloat16()
    empty = slot < 0
    for t in (xq, hq):
        t.view(torch.uint8)[empty] = 127             # NaN behind the last token
    for t in (xs, hs):
        t.view(torch.uint8)[empty] = 255
    dyv = dy.clone()
    dyv.view(N * C, d)[empty] = float("nan")
    cfg = sm.config(T, d, F, N, cf, flags=flags)
    ws = sm.backward_workspace(cfg)
    ws[256:] = 255
    dx = torch.full((N, C, d), -7.0, dtype=torch.bfloat16, device="cuda")
    dw1, dw2 = torch.empty_like(w1, device="cuda"), torch.empty_like(w2, device="cuda")
    sm.switch_expert_ffn_backward_q8(cfg, dev(xq), dev(xs), dev(hq), dev(hs), dev(counts), dev(w1),
                                     dev(w2), dev(dyv), dx, dw1, dw2, ws)
    assert sm.switch_get_device_error(ws)[0] == 0
    for e in range(N):
        n = int(kept[e])
        assert (dx[e, n:] == -7).all()
        if not n:
            assert (dw1[e] == 0).all() and (dw2[e] == 0).all()
            continue
        xe, he, ge = xv[e, :n], hv[e, :n], dy[e, :n].double()
        a, b = w1[e].double(), w2[e].double()
        da = (ge @ b) * (he > 0)
        # da: its sum's fp32 error, then half a bf16 step
        eda = (d * F32 * (ge.abs() @ b.abs()) + 2.0 ** -8 * da.abs()) * (he > 0)
        for name, got, want, size, more in (
                ("dx", dx[e, :n], da @ a, F * F32 * (da.abs() @ a.abs()), eda @ a.abs()),
                ("dw1", dw1[e], da.T @ xe, n * F32 * (da.abs().T @ xe.abs()), eda.T @ xe.abs()),
                ("dw2", dw2[e], ge.T @ he, n * F32 * (ge.abs().T @ he.abs()), 0.0)):
            check(got, want, 2.0 ** -8 * want.abs() + size + more, f"{name} of expert {e}")
            # independent roundings: half a step of the result and of da, in norm
            off = (got.cpu().double() - want).norm() / want.norm()
            assert off <= 2.0 ** -7, (name, e, off)


@pytest.mark.parametrize("T,d,F,N,cf,dead", CKPT_PARTS)
def test_ffn_backward_q8_in_parts(sm, T, d, F, N, cf, dead):
    test_ffn_backward_q8(sm, T, d, F, N, cf, dead, 0)


def test_ffn_backward_q8_by_differences(sm):
    """dx, dw1 and dw2 along random directions against differences of sum(dy y)."""
    T, d, F, N = 40, 64, 128, 2
    C, counts, slot, kept, x, w1, w2 = ffn_inputs(T, d, F, N, 2.0, 31)
    w1, w2 = w1.bfloat16(), w2.bfloat16()
    rows = x[slot.clamp(min=0).long()]
    xq, xs = ref.to_q8(rows)
    xv = ref.rows(xq, xs).view(N, C, d)
    valid = (slot >= 0).view(N, C, 1)
    dy = torch.randn(N, C, d, generator=gen(1)).bfloat16()

    def value(xx, a, b):
        hh = torch.einsum("ncd,nfd->ncf", xx, a).clamp(min=0)
        return (torch.einsum("ncf,ndf->ncd", hh, b) * dy.double() * valid).sum()

    h = torch.einsum("ncd,nfd->ncf", xv, w1.double()).clamp(min=0)
    hq, hs = ref.to_q8(h.view(N * C, F), positive=True)
    cfg = sm.config(T, d, F, N, 2.0)
    ws = sm.backward_workspace(cfg)
    dx = torch.zeros(N, C, d, dtype=torch.bfloat16, device="cuda")
    dw1, dw2 = torch.empty_like(w1, device="cuda"), torch.empty_like(w2, device="cuda")
    sm.switch_expert_ffn_backward_q8(cfg, dev(xq), dev(xs), dev(hq), dev(hs), dev(counts), dev(w1),
                                     dev(w2), dev(dy), dx, dw1, dw2, ws)
    for k, (got, at) in enumerate(((dx, xv), (dw1, w1.double()), (dw2, w2.double()))):
        u = torch.randn(at.shape, generator=gen(50 + k)).double()
        args = [xv, w1.double(), w2.double()]
        s = 1e-7
        hi, lo = list(args), list(args)
        hi[k], lo[k] = at + s * u, at - s * u
        num = ((value(*hi) - value(*lo)) / (2 * s)).item()
        grad = got.cpu().double() * (valid if k == 0 else 1.0)
        # dw2 is that of the rounded hidden rows: e4m3's half step in each h; the others
        # round da and themselves to bf16
        rel = 2.0 ** -4 if k == 2 else 2.0 ** -7
        assert abs((grad * u).sum().item() - num) <= rel * grad.norm().item() * u.norm().item() / 4


# ---------------------------------------------- the layer's kept state

@pytest.mark.parametrize("flags", [0, 512, 16, 8, 32])
def test_layer_checkpoint(sm, flags):
    """Two layers share one workspace: forward, forward, then both backward passes from their
    saved states.  Each equals the backward of the same state unpacked in place; only the
    hidden rows are rounded, so db_r, dW_r of the loss and the masks stay, and all gradients
    stay within the rounding of H."""
    T, d, F, N, cf = 900, 128, 320, 6, 1.0
    cfg = sm.config(T, d, F, N, cf, flags=flags | sm.FLAG_TRAINING)
    ws = sm.backward_workspace(cfg)
    g = gen(77)
    layers = []
    for _ in range(2):
        x = dev(torch.randn(T, d, generator=g).bfloat16())
        w_r = dev(torch.randn(N, d, generator=g) * 0.1)
        w1 = dev((torch.randn(N, F, d, generator=g) * 0.1).bfloat16())
        w2 = dev((torch.randn(N, d, F, generator=g) * 0.1).bfloat16())
        dout = dev(torch.randn(T, d, generator=g).bfloat16())
        layers.append((x, w_r, w1, w2, dout))

    def forward(p, w):
        out = torch.empty_like(p[0])
        sm.switch_layer_forward(cfg, p[0], p[1], None, p[2], p[3], out, None, None, None, None, w)
        return out

    def backward(p, w):
        o = [torch.empty_like(p[0]), torch.empty_like(p[1]), torch.empty(N, device="cuda"),
             torch.empty_like(p[2]), torch.empty_like(p[3])]
        sm.switch_layer_backward(cfg, p[0], p[1], None, p[2], p[3], p[4], 1.0, o[0], o[1], o[2],
                                 o[3], o[4], None, w)
        return o

    plain = []
    for p in layers:
        forward(p, ws)
        plain.append(backward(p, ws))
    saved = []
    for p in layers:
        forward(p, ws)
        c = sm.checkpoint(cfg)
        sm.switch_checkpoint_save(cfg, ws, c)
        saved.append(c)
    ws[256:] = 255                                   # the workspace served others meanwhile
    for p, c, want in reversed(list(zip(layers, saved, plain))):
        sm.switch_checkpoint_load(cfg, p[0], c, ws)
        got = backward(p, ws)
        assert sm.switch_get_device_error(ws)[0] == 0
        again = backward(p, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        # dW1 does not read H but through its mask: the same bits
        assert torch.equal(got[3], want[3])
        for name, a, b, tol in (("dx", got[0], want[0], 2.0 ** -4), ("dw_r", got[1], want[1], 2.0 ** -4),
                                ("db_r", got[2], want[2], 2.0 ** -4), ("dw2", got[4], want[4], 2.0 ** -4)):
            off = ((a.double() - b.double()).norm() / b.double().norm()).item()
            assert off <= tol, (name, off)           # H moves by at most e4m3's half step
    A = 2 * T if flags & 512 else T                  # top-2: the capacity is over 2 T assignments
    assert sm.switch_checkpoint_size(cfg) < 0.62 * N * sm.switch_capacity(A, N, cf) * F * 2 + \
        T * N * 4 + 64 * A + 20000


# ----------------------------------------- together, streams and graphs

def chain(sm, T, d, F, N, cf, seed):
    """Norm -> router -> dispatch -> 8-bit FFN -> combine, as a serving step runs them; returns
    the call, its buffers and its inputs."""
    g = gen(seed)
    cfg = sm.config(T, d, F, N, cf)
    C = sm.switch_capacity(T, N, cf)
    i = dict(x=dev(torch.randn(T, d, generator=g).bfloat16()),
             res=dev(torch.randn(T, d, generator=g).bfloat16()),
             gain=dev(1 + 0.1 * torch.randn(d, generator=g)),
             w_r=dev(torch.randn(N, d, generator=g) * 0.2))
    w1 = dev((torch.randn(N, F, d, generator=g) * 0.05).bfloat16())
    w2 = dev((torch.randn(N, d, F, generator=g) * 0.05).bfloat16())
    w1q, w2q = sm.q8_weights(N, F, d), sm.q8_weights(N, d, F)
    sm.switch_quantize_weights(cfg, w1, w2, *w1q, *w2q)
    b = dict(z=torch.empty_like(i["x"]), y=torch.empty_like(i["x"]), out=torch.empty_like(i["x"]),
             e=torch.zeros(N, C, d, dtype=torch.bfloat16, device="cuda"),
             idx=torch.empty(T, dtype=torch.int32, device="cuda"),
             gate=torch.empty(T, device="cuda"),
             rank=torch.empty(T, dtype=torch.int32, device="cuda"),
             drop=torch.empty(T, dtype=torch.uint8, device="cuda"),
             counts=torch.empty(N, dtype=torch.int32, device="cuda"),
             slot=torch.empty(N * C, dtype=torch.int32, device="cuda"), ws=sm.workspace(cfg))
    q = sm.q8_rows(T, d)

    def run():
        ws = b["ws"]
        sm.switch_residual_norm(cfg, i["x"], i["res"], i["gain"], 1e-6, b["z"], b["y"], *q, None)
        sm.switch_router(cfg, b["y"], i["w_r"], None, b["idx"], b["gate"], None, ws)
        sm.switch_dispatch(cfg, b["idx"], None, b["rank"], b["drop"], b["counts"], b["slot"], None,
                           None, ws)
        sm.switch_expert_ffn_q8(cfg, *q, b["slot"], b["counts"], *w1q, *w2q, b["e"], ws)
        sm.switch_combine(cfg, b["z"], b["idx"], b["rank"], b["drop"], b["gate"], b["e"], b["out"])
        return b["out"]
    return run, b, i, (w1q, w2q, q, C)


def test_serving_chain(sm):
    T, d, F, N, cf = 500, 256, 512, 8, 1.0
    run, b, i, (w1q, w2q, q, C) = chain(sm, T, d, F, N, cf, 1)
    out = run()
    assert sm.switch_get_device_error(b["ws"])[0] == 0
    xv, w1v, w2v = ref.rows(*q), ref.weights(*w1q), ref.weights(*w2q)
    idx, drop, gate = b["idx"].cpu(), b["drop"].cpu().bool(), b["gate"].cpu().double()
    z = b["z"].cpu().double()
    want, tol = z.clone(), 2.0 ** -8 * z.abs()
    for e in range(N):
        t = torch.nonzero((idx == e) & ~drop)[:, 0]
        if len(t):
            y, ty = ffn_q8_want(xv[t], w1v[e], w2v[e])
            v = z[t] + gate[t, None] * y
            want[t], tol[t] = v, gate[t, None] * ty + (2.0 ** -8 + 2.0 ** -20) * v.abs()
    check(out, want, tol, "chain")


def test_chain_on_a_side_stream_and_in_graphs(sm):
    """The same bits on another stream and from captured graphs; two graphs with their own
    workspaces replay side by side, with new inputs in the captured buffers."""
    a, ba, ia, _ = chain(sm, 333, 128, 256, 5, 1.0, 2)
    c, bc, ic, _ = chain(sm, 64, 192, 320, 3, 2.0, 3)
    want_a, want_c = a().clone(), c().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ba["out"].zero_()
        a()
    side.synchronize()
    assert torch.equal(ba["out"], want_a)
    ga, gc = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        a()
    with torch.cuda.graph(gc):
        c()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for s, g in ((s1, ga), (s2, gc)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ba["out"], want_a) and torch.equal(bc["out"], want_c)
    ia["x"].copy_(torch.randn(333, 128, generator=gen(9)).bfloat16())
    ga.replay()
    got = ba["out"].clone()
    assert torch.equal(got, a()) and not torch.equal(got, want_a)


def test_parts_repeat_and_replay(sm):
    """Sums in parts give the same bits each time: again, over scratch that holds NaN, on
    another stream, and from a captured graph; one workspace serves all the calls."""
    T, d, F, N, cf = 2600, 64, 4672, 1, 1.0
    C = sm.switch_capacity(T, N, cf)
    g = gen(77)
    x = dev(torch.randn(C, d, generator=g).bfloat16())
    dy = dev(torch.randn(N, C, d, generator=g).bfloat16())
    w1 = dev((torch.randn(N, F, d, generator=g) * d ** -0.5).bfloat16())
    w2 = dev((torch.randn(N, d, F, generator=g) * F ** -0.5).bfloat16())
    counts = torch.tensor([300], dtype=torch.int32, device="cuda")
    cfg = sm.config(T, d, F, N, cf, flags=sm.FLAG_ROWS_DISPATCHED)
    ws = sm.backward_workspace(cfg)
    (xq, xs), (hq, hs) = sm.q8_rows(C, d), sm.q8_rows(C, F)
    (w1q, w1s), (w2q, w2s) = sm.q8_weights(N, F, d), sm.q8_weights(N, d, F)
    sm.switch_quantize_weights(cfg, w1, w2, w1q, w1s, w2q, w2s)
    out = [torch.zeros_like(t) for t in (dy, dy, dy, w1, w2)]

    def run():
        sm.switch_expert_ffn_checkpoint(cfg, x, None, counts, w1, w2, out[0], xq, xs, hq, hs, ws)
        sm.switch_expert_ffn_q8(cfg, xq, xs, None, counts, w1q, w1s, w2q, w2s, out[1], ws)
        sm.switch_expert_ffn_backward_q8(cfg, xq, xs, hq, hs, counts, w1, w2, dy, *out[2:], ws)

    def same():
        torch.cuda.synchronize()
        ok = all(torch.equal(a, b) for a, b in zip(out, want))
        for t in out:
            t.zero_()
        return ok

    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    assert all(torch.isfinite(t).all() and t.abs().max() > 0 for t in want)
    ws[256:] = 255
    run()
    assert same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        graph.replay()
    assert same()
    assert sm.switch_get_device_error(ws)[0] == 0


def test_training_chain(sm):
    """Norm, FFN with 8-bit checkpoint, and both backward passes together: the gradients of
    sum(dy FFN(norm(x))) of a whole dispatched batch, against 64 bits."""
    T, d, F = 200, 128, 256
    g = gen(8)
    cfg = sm.config(T, d, F, 1, 1.0, flags=sm.FLAG_ROWS_DISPATCHED)
    x = torch.randn(T, d, generator=g).bfloat16()
    gain = 1 + 0.1 * torch.randn(d, generator=g)
    w1 = (torch.randn(1, F, d, generator=g) * 0.1).bfloat16()
    w2 = (torch.randn(1, d, F, generator=g) * 0.1).bfloat16()
    dy = torch.randn(1, T, d, generator=g).bfloat16()
    ws, wn = sm.backward_workspace(cfg), sm.norm_workspace(cfg)
    n, y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, T, d, dtype=torch.bfloat16, device="cuda")
    rstd = torch.empty(T, device="cuda")
    xq, xs = sm.q8_rows(T, d)
    hq, hs = sm.q8_rows(T, F)
    counts = torch.tensor([T], dtype=torch.int32, device="cuda")
    X, W1, W2, DY, G = dev(x), dev(w1), dev(w2), dev(dy), dev(gain)
    dn, dx = torch.empty_like(y), torch.empty_like(n)
    dw1, dw2, dg = torch.empty_like(W1), torch.empty_like(W2), torch.empty_like(G)

    def step():
        sm.switch_residual_norm(cfg, X, None, G, 1e-6, None, n, None, None, rstd)
        sm.switch_expert_ffn_checkpoint(cfg, n, None, counts, W1, W2, y, xq, xs, hq, hs, ws)
        sm.switch_expert_ffn_backward_q8(cfg, xq, xs, hq, hs, counts, W1, W2, DY, dn, dw1, dw2, ws)
        sm.switch_residual_norm_backward(cfg, X, G, rstd, dn, None, dx, dg, wn)

    step()
    assert sm.switch_get_device_error(ws)[0] == 0
    got = [t.clone() for t in (y, dx, dg, dw1, dw2)]
    p = [t.double().requires_grad_() for t in (x, gain, w1[0], w2[0])]
    nn = p[0] / torch.sqrt((p[0] ** 2).mean(1, keepdim=True) + 1e-6) * p[1]
    out = torch.relu(nn @ p[2].T) @ p[3].T
    (out * dy[0].double()).sum().backward()
    want = [out.detach(), p[0].grad, p[1].grad, p[2].grad, p[3].grad]
    for name, a, b in zip(("y", "dx", "dgain", "dw1", "dw2"), got, want):
        a = a.cpu().double().reshape(b.shape)
        # x and h in 8 bits reach dw1 and dw2 alone: e4m3's half step; the mask of a value
        # within bf16's rounding of zero may differ elsewhere
        assert ((a - b).norm() / b.norm()).item() <= 2.0 ** -4, name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (y, dx, dg, dw1, dw2):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, dx, dg, dw1, dw2), got))
