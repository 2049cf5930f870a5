"""Plain 64-bit forms of the norm and of the 8-bit block rows, for the tests.

Nothing here is shared with the library: the scale and the e4m3 rounding are
written from the format's definition (a block's scale is the smallest power of
two s >= 2^-100 with max |v| <= 448 s; e4m3 has 4 significant bits, exponents
-6 .. 8 and subnormals of 2^-9).
"""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative
E4M3_MIN = 2.0 ** -9


def e4m3(u):
    """Nearest e4m3 value, ties to even, of |u| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(u / step) * step


def scale_of(amax):
    s = torch.exp2(torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448)).clamp(min=-100))
    return torch.where(amax > 448 * s, 2 * s, s)       # log2 rounded down at a border


def spread(s, cols):
    return s.repeat_interleave(128, dim=-1)[..., :cols]


def quantize(v, positive=False):
    """[..., K] -> (codes' values, scales [..., ceil(K / 128)]), in 64 bits."""
    k = v.shape[-1]
    b = (k + 127) // 128
    p = torch.nn.functional.pad(v, (0, b * 128 - k))
    s = scale_of(p.reshape(*v.shape[:-1], b, 128).abs().amax(-1))
    u = v / spread(s, k)
    if positive:
        u = torch.where(v > 0, u.clamp(min=E4M3_MIN), u)
    return e4m3(u), s


def quantize_weights(w):
    """[N, R, K] -> (codes' values, scales [N, ceil(R / 128), ceil(K / 128)])."""
    n, r, k = w.shape
    br, bk = (r + 127) // 128, (k + 127) // 128
    p = torch.nn.functional.pad(w, (0, bk * 128 - k, 0, br * 128 - r))
    s = scale_of(p.reshape(n, br, 128, bk, 128).abs().amax((2, 4)))
    full = spread(s, k).repeat_interleave(128, dim=1)[:, :r]
    return e4m3(w / full), s


def codes(t):
    """The values of an e4m3 tensor, on the CPU in 64 bits."""
    return t.cpu().float().double()


def scales(t):
    return torch.exp2(t.cpu().view(torch.uint8).double() - 127)


def rows(q, s):
    """The values that 8-bit rows stand for."""
    return codes(q) * spread(scales(s), q.shape[-1])


def weights(q, s):
    full = spread(scales(s), q.shape[-1]).repeat_interleave(128, dim=1)[:, :q.shape[1]]
    return codes(q) * full


def to_q8(v, positive=False):
    """8-bit rows (tensors as the library takes them) of 64-bit values."""
    q, s = quantize(v, positive)
    return as_q8(q, s)


def as_q8(q, s):
    return (q.float().to(torch.float8_e4m3fn),
            (torch.log2(s) + 127).to(torch.uint8).view(torch.float8_e8m0fnu))


def routing(T, N, C, seed, dead=()):
    """Random skewed routing: counts, slot_token and each expert's tokens; experts in `dead`
    get none."""
    rng = np.random.default_rng(seed)
    p = rng.dirichlet(np.ones(N))
    p[list(dead)] = 0
    idx = rng.choice(N, size=T, p=p / p.sum())
    counts = np.bincount(idx, minlength=N)
    slot = np.full((N, C), -1, np.int32)
    for e in range(N):
        t = np.nonzero(idx == e)[0][:C]
        slot[e, :len(t)] = t
    return (torch.from_numpy(counts.astype(np.int32)), torch.from_numpy(slot.reshape(-1)),
            np.minimum(counts, C))
