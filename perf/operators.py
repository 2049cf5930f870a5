"""What the 8-bit block operators of the Switch-FFN layer are measured on.

Operators (public entry points of the binding `switch_moe`):

* ``norm``      switch_residual_norm: z = x + residual, y = z / rms(z) * gain, with y also as
                e4m3 rows that have one power-of-two scale (e8m0) for each 128 columns;
* ``norm_bwd``  switch_residual_norm_backward: the gradients of the sum and of the gain;
* ``ffn_q8``    switch_expert_ffn_q8: the experts' ReLU FFNs as 8-bit products, rows scaled
                for each 128 columns, weights for each 128 x 128 block, the hidden rows
                quantised in between;
* ``ckpt_fwd``  switch_expert_ffn_checkpoint: the bf16 expert FFNs, which also keep their
                input and hidden rows in 8 bits for the backward pass;
* ``ckpt_bwd``  switch_expert_ffn_backward_q8: the FFNs' gradients from those rows.

Nothing here is needed to use the library.  ``own`` chooses the plain form (elementary torch
operations in 32 bits) or the library's calls.
"""
import math

import torch

own = False

INIT_SCALE = 0.1        # of the experts' weights: std sqrt(0.1 / fan_in)
EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a serving step, the widest rows of the workloads: latency alone
        dict(name="norm_token", op="norm", T=1, d=4096, dtype="bf16", residual=True, q8=True),
        # a serving or training batch in front of the layer (Large's tokens and width)
        dict(name="norm_batch_q8", op="norm", T=32768, d=1024, dtype="bf16", residual=True, q8=True),
        # full precision, no residual, odd sizes: a last block of four columns
        dict(name="norm_f32_odd", op="norm", T=5003, d=772, dtype="f32", residual=False, q8=False),
        # the same norm's backward in a training step, the gradient of the sum added
        dict(name="norm_bwd_batch", op="norm_bwd", T=32768, d=1024, dtype="bf16", dsum=True),
        # few wide rows in full precision, no second gradient
        dict(name="norm_bwd_f32", op="norm_bwd", T=517, d=4096, dtype="f32", dsum=False),
        # one decoding step of a small batch: weights of the few experts that are hit
        dict(name="ffn_q8_decode", op="ffn_q8", T=8, d=1024, F=4096, N=128, cf=32.0),
        # Large, one prefill or evaluation batch: balanced between weights and products
        dict(name="ffn_q8_large", op="ffn_q8", T=32768, d=1024, F=4096, N=128, cf=1.0),
        # XXL's experts at its tokens for each expert, a quarter of its experts
        dict(name="ffn_q8_wide", op="ffn_q8", T=4096, d=4096, F=10240, N=16, cf=1.25),
        # a small model's training step, ragged sizes (rows that fill no block of 128)
        dict(name="ckpt_fwd_small", op="ckpt_fwd", T=700, d=320, F=832, N=6, cf=1.25),
        # Large's training forward
        dict(name="ckpt_fwd_large", op="ckpt_fwd", T=32768, d=1024, F=4096, N=128, cf=1.0),
        # the backward passes of the two
        dict(name="ckpt_bwd_small", op="ckpt_bwd", T=700, d=320, F=832, N=6, cf=1.25),
        dict(name="ckpt_bwd_large", op="ckpt_bwd", T=32768, d=1024, F=4096, N=128, cf=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "ffn_q8", "ffn_q8", "ckpt_fwd", "ckpt_bwd"])
    if op in ("norm", "norm_bwd"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = 64 * _log_int(rng, 1, 128) if dtype == "bf16" else 4 * _log_int(rng, 8, 2048)
        T = _log_int(rng, 1, max(2, min(65536, 2 ** 25 // (d * (1 if dtype == "bf16" else 2)))))
        if op == "norm":
            return dict(op=op, T=T, d=d, dtype=dtype, residual=rng.random() < 0.7,
                        q8=rng.random() < 0.6)
        return dict(op=op, T=T, d=d, dtype=dtype, dsum=rng.random() < 0.6)
    most = 0.5e12 if op == "ffn_q8" else 0.25e12
    while True:
        d = 64 * _log_int(rng, 1, 64)
        F = 64 * _log_int(rng, 1, 160)
        N = _log_int(rng, 1, 128)
        T = _log_int(rng, 1, 32768)
        cf = rng.choice([0.5, 1.0, 1.25, 2.0, 8.0])
        C = _capacity(T, N, cf)
        if N * d * F <= 2 ** 29 and 4.0 * N * C * d * F <= most and N * C <= 40000:
            return dict(op=op, T=T, d=d, F=F, N=N, cf=cf)


def _capacity(T, N, cf):
    return int(math.ceil(T * cf / N))      # the factors drawn here are exact in binary


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _blocks(cols):
    return (cols + 127) // 128


def _row_scales(v):
    """Exponents [R, blocks] of the smallest power of two s with amax(block) <= 448 s."""
    r, k = v.shape
    b = _blocks(k)
    a = torch.nn.functional.pad(v, (0, b * 128 - k)).view(r, b, 128).abs().amax(2)
    m, e = torch.frexp(a)                              # a = m 2^e, 1/2 <= m < 1
    e = torch.where(m > 0.875, e - 8, e - 9)           # 448 = 0.875 * 2^9
    return torch.where(a > 0, e, torch.full_like(e, -100)).clamp(min=-100)


def _spread(e, cols):
    return e.repeat_interleave(128, dim=-1)[..., :cols]


def _quantize_rows(v, keep_positive=False):
    """fp32 [R, K] -> e4m3 [R, K], e8m0 [R, blocks]; keep_positive: what is above zero does
    not round to zero (it takes the smallest value instead)."""
    e = _row_scales(v)
    u = torch.ldexp(v, -_spread(e, v.shape[1]))
    if keep_positive:
        u = torch.where(v > 0, u.clamp(min=2.0 ** -9), u)
    return u.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _rows_of(q, s):
    """The values that 8-bit rows stand for, in fp32."""
    e = s.view(torch.uint8).to(torch.int32) - 127
    return torch.ldexp(q.float(), _spread(e, q.shape[1]))


def _quantize_weights(w):
    """[N, R, K] -> e4m3 [N, R, K], e8m0 [N, ceil(R/128), ceil(K/128)]: a scale for each block
    of 128 x 128.  One expert at a time, to hold few copies."""
    n, r, k = w.shape
    br, bk = _blocks(r), _blocks(k)
    q = torch.empty(n, r, k, dtype=torch.float8_e4m3fn, device=w.device)
    s = torch.empty(n, br, bk, dtype=torch.uint8, device=w.device)
    for i in range(n):
        f = w[i].float()
        a = torch.nn.functional.pad(f, (0, bk * 128 - k, 0, br * 128 - r))
        a = a.view(br, 128, bk, 128).abs().amax((1, 3))
        e = _row_scales(a.reshape(-1, 1)).view(br, bk)
        full = _spread(e, k).repeat_interleave(128, dim=0)[:r]
        q[i] = torch.ldexp(f, -full).to(torch.float8_e4m3fn)
        s[i] = (e + 127).to(torch.uint8)
    return q, s.view(torch.float8_e8m0fnu)


def _weights_of(q, s):
    e = s.view(torch.uint8).to(torch.int32) - 127
    full = _spread(e, q.shape[2]).repeat_interleave(128, dim=1)[:, :q.shape[1]]
    return torch.ldexp(q.float(), full)


def _routing(case, g):
    """Expert of each token (skewed, as routers are), counts, and the token of each slot."""
    T, N = case["T"], case["N"]
    C = _capacity(T, N, case["cf"])
    lean = 0.5 * torch.randn(N, generator=g, device="cuda")
    idx = torch.multinomial(torch.softmax(lean, 0), T, replacement=True, generator=g)
    counts = torch.bincount(idx, minlength=N)
    order = torch.argsort(idx, stable=True)
    e = idx[order]
    rank = torch.arange(T, device="cuda") - (torch.cumsum(counts, 0) - counts)[e]
    slot_token = torch.full((N * C + 1,), -1, dtype=torch.int64, device="cuda")
    slot_token[torch.where(rank < C, e * C + rank, N * C)] = order
    return C, counts.int(), slot_token[:N * C].int().contiguous()


def _valid(counts, C):
    return torch.arange(C, device="cuda")[None, :] < counts[:, None]      # [N, C]


def _weight(n, r, k, g):
    w = torch.empty(n, r, k, dtype=torch.bfloat16, device="cuda")
    for i in range(n):
        w[i] = torch.randn(r, k, generator=g, device="cuda") * math.sqrt(INIT_SCALE / k)
    return w


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T, d = case["op"], case["T"], case["d"]
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    if op in ("norm", "norm_bwd"):
        gain = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        # a residual stream's rows differ in size
        size = torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
        s = dict(case=case, gain=gain, x=(size * torch.randn(T, d, generator=g, device="cuda")).to(dt))
        if op == "norm":
            s["residual"] = (size * torch.randn(T, d, generator=g, device="cuda")).to(dt) \
                if case["residual"] else None
            s["z"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["y"] = torch.empty_like(s["x"])
            s["rstd"] = torch.empty(T, device="cuda")
            s["yq"] = torch.empty(T, d, dtype=torch.float8_e4m3fn, device="cuda") if case["q8"] else None
            s["ys"] = torch.empty(T, _blocks(d), dtype=torch.uint8, device="cuda") \
                .view(torch.float8_e8m0fnu) if case["q8"] else None
        else:
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dy"] = normal(T, d)
            s["dsum"] = normal(T, d) if case["dsum"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dgain"] = torch.empty(d, device="cuda")
        s["handle"] = _handle(case) if own else None
        return s

    F, N = case["F"], case["N"]
    C, counts, slot_token = _routing(case, g)
    w1, w2 = _weight(N, F, d, g), _weight(N, d, F, g)
    s = dict(case=case, C=C, counts=counts, slot_token=slot_token)
    if op == "ffn_q8":
        s["xq"], s["xs"] = _quantize_rows(torch.randn(T, d, generator=g, device="cuda"))
        s["w1q"], s["w1s"] = _quantize_weights(w1)
        s["w2q"], s["w2s"] = _quantize_weights(w2)
        s["y"] = torch.zeros(N, C, d, dtype=torch.bfloat16, device="cuda")
    else:
        s["w1"], s["w2"] = w1, w2
        if op == "ckpt_fwd":
            s["x"] = normal(T, d)
            s["y"] = torch.zeros(N, C, d, dtype=torch.bfloat16, device="cuda")
            # rows behind an expert's last token are left as they are: zeros here
            for name, cols in (("x", d), ("h", F)):
                s[name + "q"] = torch.zeros(N * C, cols, dtype=torch.uint8, device="cuda") \
                    .view(torch.float8_e4m3fn)
                s[name + "s"] = torch.full((N * C, _blocks(cols)), 127, dtype=torch.uint8,
                                           device="cuda").view(torch.float8_e8m0fnu)
        else:
            x = torch.randn(N, C, d, generator=g, device="cuda") * _valid(counts, C)[:, :, None]
            h = torch.relu(torch.bmm(x, w1.float().transpose(1, 2)))
            s["xq"], s["xs"] = _quantize_rows(x.view(N * C, d))
            s["hq"], s["hs"] = _quantize_rows(h.view(N * C, F), keep_positive=True)
            s["dy"] = normal(N, C, d)
            s["dx"] = torch.zeros(N, C, d, dtype=torch.bfloat16, device="cuda")
            s["dw1"], s["dw2"] = torch.empty_like(w1), torch.empty_like(w2)
    s["handle"] = _handle(case) if own else None
    return s


def _handle(case):
    """The config and the workspace that a user's program keeps (only where `own` is true)."""
    from sparse_mixture_experts_switch_b200 import switch_moe as sm
    cfg = sm.config(case["T"], case["d"], case.get("F", case["d"]), case.get("N", 1),
                    case.get("cf", 1.0), dtype=case.get("dtype", "bf16"))
    size = sm.backward_workspace if case["op"] == "ckpt_bwd" else sm.workspace
    if case["op"] == "norm_bwd":
        ws = sm.norm_workspace(cfg)
    else:
        ws = None if case["op"] == "norm" else size(cfg)
    return sm, cfg, ws


# --------------------------------------------------------------------- run

def run(s):
    return _call(s) if own else _plain(s)


def _call(s):
    sm, cfg, ws = s["handle"]
    op = s["case"]["op"]
    if op == "norm":
        sm.switch_residual_norm(cfg, s["x"], s["residual"], s["gain"], EPS, s["z"], s["y"], s["yq"],
                                s["ys"], s["rstd"])
        return [s["z"], s["y"], s["yq"], s["ys"], s["rstd"]]
    if op == "norm_bwd":
        sm.switch_residual_norm_backward(cfg, s["x"], s["gain"], s["rstd"], s["dy"], s["dsum"],
                                         s["dx"], s["dgain"], ws)
        return [s["dx"], s["dgain"]]
    if op == "ffn_q8":
        sm.switch_expert_ffn_q8(cfg, s["xq"], s["xs"], s["slot_token"], s["counts"], s["w1q"],
                                s["w1s"], s["w2q"], s["w2s"], s["y"], ws)
        return s["y"]
    if op == "ckpt_fwd":
        sm.switch_expert_ffn_checkpoint(cfg, s["x"], s["slot_token"], s["counts"], s["w1"], s["w2"],
                                        s["y"], s["xq"], s["xs"], s["hq"], s["hs"], ws)
        return [s["y"], s["xq"], s["xs"], s["hq"], s["hs"]]
    sm.switch_expert_ffn_backward_q8(cfg, s["xq"], s["xs"], s["hq"], s["hs"], s["counts"], s["w1"],
                                     s["w2"], s["dy"], s["dx"], s["dw1"], s["dw2"], ws)
    return [s["dx"], s["dw1"], s["dw2"]]


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _dtype(case)
    if op == "norm":
        z = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
        f = z.float()
        rstd = torch.rsqrt((f * f).mean(1) + EPS)
        y = f * rstd[:, None] * s["gain"]
        yq, ys = _quantize_rows(y) if case["q8"] else (None, None)
        return [None if s["residual"] is None else z, y.to(dt), yq, ys, rstd]
    if op == "norm_bwd":
        z, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        t = dy * s["gain"]
        dz = t * rstd - z * (rstd ** 3 * (t * z).mean(1, keepdim=True))
        if s["dsum"] is not None:
            dz = dz + s["dsum"].float()
        # a sum over all rows: in 64 bits, as 32 would lose digits over tens of thousands
        return [dz.to(dt), (dy * z * rstd).double().sum(0).float()]
    N, C = case["N"], s["C"]
    valid = _valid(s["counts"], C)
    keep = valid[:, :, None]
    if op == "ffn_q8":
        x = _rows_of(s["xq"], s["xs"])[s["slot_token"].clamp(min=0).long()].view(N, C, -1) * keep
        h = torch.relu(torch.bmm(x, _weights_of(s["w1q"], s["w1s"]).transpose(1, 2)))
        h = _rows_of(*_quantize_rows(h.view(N * C, -1))).view(N, C, -1)
        return torch.bmm(h, _weights_of(s["w2q"], s["w2s"]).transpose(1, 2)).to(torch.bfloat16)
    w1, w2 = s["w1"].float(), s["w2"].float()
    if op == "ckpt_fwd":
        x = s["x"].float()[s["slot_token"].clamp(min=0).long()].view(N, C, -1) * keep
        h = torch.relu(torch.bmm(x, w1.transpose(1, 2))).to(torch.bfloat16).float()
        xq, xs = _quantize_rows(x.view(N * C, -1))
        hq, hs = _quantize_rows(h.view(N * C, -1), keep_positive=True)
        # rows without a token stay as they were
        row = valid.view(N * C, 1)
        one = torch.full_like(xs.view(torch.uint8)[:1, :1], 127)
        xs = torch.where(row, xs.view(torch.uint8), one).view(torch.float8_e8m0fnu)
        hs = torch.where(row, hs.view(torch.uint8), one).view(torch.float8_e8m0fnu)
        return [torch.bmm(h, w2.transpose(1, 2)).to(torch.bfloat16), xq, xs, hq, hs]
    x = _rows_of(s["xq"], s["xs"]).view(N, C, -1) * keep
    h = _rows_of(s["hq"], s["hs"]).view(N, C, -1) * keep
    dy = s["dy"].float() * keep
    da = torch.bmm(dy, w2) * (h > 0)
    return [torch.bmm(da, w1).to(torch.bfloat16),
            torch.bmm(da.transpose(1, 2), x).to(torch.bfloat16),
            torch.bmm(dy.transpose(1, 2), h).to(torch.bfloat16)]


# -------------------------------------------------------------------- work

def work(case):
    op, T, d = case["op"], case["T"], case["d"]
    e = 4 if case.get("dtype") == "f32" else 2
    if op == "norm":
        b = T * d * e * (4 if case["residual"] else 2) + 4 * d + 4 * T
        b += T * (d + _blocks(d)) if case["q8"] else 0
        return {"bytes": b, "flops": 4 * T * d}
    if op == "norm_bwd":
        return {"bytes": T * d * e * (4 if case["dsum"] else 3) + 8 * d + 4 * T, "flops": 9 * T * d}
    F, N = case["F"], case["N"]
    C = _capacity(T, N, case["cf"])
    rows = min(T, N * C)                    # most tokens that can have a slot
    hit = N * (1 - (1 - 1 / N) ** T)        # experts that some token takes
    if op == "ffn_q8":
        return {"bytes": hit * 2 * d * F * (1 + 1 / 16384) + rows * (d * (1 + 1 / 128) + 2 * d) + 4 * N * C,
                "flops": 4.0 * rows * d * F}
    if op == "ckpt_fwd":
        return {"bytes": hit * 4 * d * F + rows * (4 * d + (d + F) * (1 + 1 / 128)) + 4 * N * C,
                "flops": 4.0 * rows * d * F}
    return {"bytes": hit * 4 * d * F + N * 4 * d * F + rows * (4 * d + (d + F) * (1 + 1 / 128)),
            "flops": 8.0 * rows * d * F}


# ------------------------------------------------- 64 bits, from the formulas

def _e4m3_64(v):
    """The nearest e4m3 value (ties to even) of numbers of at most 448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _quantize_64(v, keep_positive=False):
    """64-bit rows -> (8-bit codes' values, scales), both in 64 bits."""
    r, k = v.shape
    q, s = torch.zeros_like(v), []
    for c in range(0, k, 128):
        b = v[:, c:c + 128]
        top = b.abs().amax(1, keepdim=True)
        sc = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-100))
        u = b / sc
        if keep_positive:
            u = torch.where(b > 0, u.clamp(min=2.0 ** -9), u)
        q[:, c:c + 128] = _e4m3_64(u)
        s.append(sc)
    return q, torch.cat(s, 1)


def _decode_64(q, s):
    """One matrix of 8-bit values with scales on 128 columns, or on 128 x 128 blocks."""
    r, k = q.shape
    sc = torch.exp2(s.view(torch.uint8).double() - 127)
    rows = torch.arange(r, device=q.device)
    if s.shape[0] != r:
        rows = rows // 128
    return q.double() * sc[rows][:, torch.arange(k, device=q.device) // 128]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        z = x if s["residual"] is None else x + s["residual"].double()
        held = z.to(_dtype(case)).double()
        rms = torch.sqrt(torch.sum(held ** 2, 1) / case["d"] + EPS)
        y = held / rms[:, None] * s["gain"].double()
        yq, ys = _quantize_64(y) if case["q8"] else (None, None)
        return [None if s["residual"] is None else z, y, yq, ys, 1 / rms]
    if op == "norm_bwd":
        z, dy, r = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        n = z * r
        t = dy * s["gain"].double()
        dz = r * (t - n * torch.sum(t * n, 1, keepdim=True) / case["d"])
        if s["dsum"] is not None:
            dz = dz + s["dsum"].double()
        return [dz, torch.sum(dy * n, 0)]
    N, C, d, F = case["N"], s["C"], case["d"], case["F"]
    counts, tokens = s["counts"].tolist(), s["slot_token"].view(N, C).long()
    dev = dict(dtype=torch.float64, device="cuda")
    if op == "ffn_q8":
        y = torch.zeros(N, C, d, **dev)
        for e in range(N):
            n = min(counts[e], C)
            if n:
                t = tokens[e, :n]
                x = _decode_64(s["xq"][t], s["xs"][t])
                h = (x @ _decode_64(s["w1q"][e], s["w1s"][e]).T).clamp(min=0)
                hq, hs = _quantize_64(h)
                h = hq * hs.repeat_interleave(128, 1)[:, :F]
                y[e, :n] = h @ _decode_64(s["w2q"][e], s["w2s"][e]).T
        return y
    if op == "ckpt_fwd":
        y = torch.zeros(N, C, d, **dev)
        q = [torch.zeros(N, C, d, **dev), torch.ones(N, C, _blocks(d), **dev),
             torch.zeros(N, C, F, **dev), torch.ones(N, C, _blocks(F), **dev)]
        for e in range(N):
            n = min(counts[e], C)
            if n:
                x = s["x"][tokens[e, :n]].double()
                h = (x @ s["w1"][e].double().T).clamp(min=0).bfloat16().double()
                q[0][e, :n], q[1][e, :n] = _quantize_64(x)
                q[2][e, :n], q[3][e, :n] = _quantize_64(h, keep_positive=True)
                y[e, :n] = h @ s["w2"][e].double().T
        return [y] + [v.view(N * C, -1) for v in q]
    dx = torch.zeros(N, C, d, **dev)
    dw1, dw2 = torch.zeros(N, F, d, **dev), torch.zeros(N, d, F, **dev)
    for e in range(N):
        n = min(counts[e], C)
        if n:
            r = slice(e * C, e * C + n)
            x, h = _decode_64(s["xq"][r], s["xs"][r]), _decode_64(s["hq"][r], s["hs"][r])
            dy = s["dy"][e, :n].double()
            da = (dy @ s["w2"][e].double()) * (h > 0)
            dx[e, :n] = da @ s["w1"][e].double()
            dw1[e], dw2[e] = da.T @ x, dy.T @ h
    return [dx, dw1, dw2]
