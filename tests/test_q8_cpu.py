"""Refusals of the norm's and the 8-bit rows' entry points, checked without a
GPU: every argument is examined before the device is, so none of these calls
reaches it.  And the plain 64-bit forms that the GPU tests compare with."""
import ctypes

import pytest
import torch

import q8_ref as ref

P = 4096          # an aligned address that is never read: every call below is refused


@pytest.fixture(scope="module")
def sm():
    from sparse_mixture_experts_switch_b200 import build
    build.build()
    from sparse_mixture_experts_switch_b200 import switch_moe
    return switch_moe


OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3

# (entry point, good arguments after cfg and before the workspace, indexes that must not be
# NULL, indexes that must be 16-byte aligned)
CALLS = {
    "switch_residual_norm": ([P, P, P, 1e-6, P, P, P, P, P], (0,), (0, 1, 2, 4, 5, 6)),
    "switch_residual_norm_backward": ([P, P, P, P, P, P, P], (0, 2, 3), (0, 1, 3, 4, 5)),
    "switch_quantize_weights": ([P] * 6, (2, 3, 4, 5), (0, 1, 2, 4)),
    "switch_expert_ffn_q8": ([P] * 9, tuple(range(9)), (0, 1, 4, 5, 6, 7, 8)),
    "switch_expert_ffn_checkpoint": ([P] * 10, tuple(range(10)), (0, 3, 4, 5, 6, 7, 8, 9)),
    "switch_expert_ffn_backward_q8": ([P] * 11, tuple(range(11)), (0, 1, 2, 3, 5, 6, 7, 8, 9, 10)),
}
NO_WS = ("switch_residual_norm", "switch_quantize_weights")


def call(sm, name, cfg, args, ws=P, ws_bytes=1 << 60):
    tail = [None] if name in NO_WS else [ws, ws_bytes, None]
    return getattr(sm._lib, name)(ctypes.byref(cfg), *args, *tail)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_arguments_are_refused(sm, name):
    good, needed, aligned = CALLS[name]
    cfg = sm.config(100, 128, 256, 4, 1.0)
    for i in needed:
        bad = list(good)
        bad[i] = None
        assert call(sm, name, cfg, bad) == INVALID, i
    for i in aligned:
        bad = list(good)
        bad[i] = P + 8
        assert call(sm, name, cfg, bad) == INVALID, i
    for T, d, F, N, cf, status in ((-1, 128, 256, 4, 1.0, INVALID), (8, 96, 256, 4, 1.0, UNSUPPORTED),
                                   (8, 128, 200, 4, 1.0, UNSUPPORTED), (8, 128, 256, 0, 1.0, INVALID)):
        assert call(sm, name, sm.config(T, d, F, N, cf), good) == status
    if "norm" not in name:
        assert call(sm, name, sm.config(8, 128, 256, 4, 1.0, dtype="f32"), good) == UNSUPPORTED
    if name != "switch_quantize_weights":
        assert call(sm, name, sm.config(0, 128, 256, 4, 1.0), good) == OK
    if name not in NO_WS:
        assert call(sm, name, cfg, good, ws=None) == INVALID
        assert call(sm, name, cfg, good, ws=P + 64) == INVALID
        assert call(sm, name, cfg, good, ws_bytes=1000) == SMALL


def test_norm_refusals(sm):
    cfg = sm.config(100, 128, 256, 4, 1.0)
    good = CALLS["switch_residual_norm"][0]

    def status(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return call(sm, "switch_residual_norm", cfg, a)

    assert status(_3=-1.0) == INVALID and status(_3=float("nan")) == INVALID
    assert status(_3=float("inf")) == INVALID
    assert status(_6=None) == INVALID and status(_7=None) == INVALID     # codes without scales
    assert status(_5=None, _6=None, _7=None) == INVALID                  # no output at all
    bwd = list(CALLS["switch_residual_norm_backward"][0])
    bwd[5] = bwd[6] = None
    assert call(sm, "switch_residual_norm_backward", cfg, bwd) == INVALID
    n = sm.switch_norm_workspace_size(cfg)
    assert call(sm, "switch_residual_norm_backward", cfg, CALLS["switch_residual_norm_backward"][0],
                ws_bytes=n - 1) == SMALL


def test_slot_token_only_without_dispatched_rows(sm):
    for name in ("switch_expert_ffn_q8", "switch_expert_ffn_checkpoint"):
        cfg = sm.config(100, 128, 256, 4, 1.0, flags=sm.FLAG_ROWS_DISPATCHED)
        a = list(CALLS[name][0])
        a[2 if name == "switch_expert_ffn_q8" else 1] = None
        assert call(sm, name, cfg, a, ws_bytes=1000) == SMALL            # not the missing pointer


def test_checkpoint_refusals(sm):
    train = sm.config(100, 128, 256, 4, 1.0, flags=sm.FLAG_TRAINING)
    n, w = sm.switch_checkpoint_size(train), sm.switch_backward_workspace_size(train)
    lib = sm._lib
    big = 1 << 60

    def save(cfg, ws=P, wsb=big, c=P, cb=big):
        return lib.switch_checkpoint_save(ctypes.byref(cfg), ws, wsb, c, cb, None)

    def load(cfg, x=P, c=P, cb=big, ws=P, wsb=big):
        return lib.switch_checkpoint_load(ctypes.byref(cfg), x, c, cb, ws, wsb, None)

    f32 = sm.config(100, 128, 256, 4, 1.0, dtype="f32", flags=sm.FLAG_TRAINING)
    for f in (save, load):
        assert f(sm.config(100, 128, 256, 4, 1.0)) == INVALID            # not a training config
        assert f(f32) == UNSUPPORTED
        assert f(sm.config(0, 128, 256, 4, 1.0, flags=sm.FLAG_TRAINING)) == OK
        assert f(train, c=None) == INVALID and f(train, c=P + 64) == INVALID
        assert f(train, ws=None) == INVALID and f(train, ws=P + 64) == INVALID
        assert f(train, cb=n - 1) == SMALL and f(train, wsb=w - 1) == SMALL
    assert load(train, x=None) == INVALID and load(train, x=P + 8) == INVALID
    with pytest.raises(sm.SwitchError):
        sm.switch_checkpoint_size(f32)
    with pytest.raises(ValueError):
        sm.switch_checkpoint_save(train, torch.zeros(8, dtype=torch.uint8), torch.zeros(8))


def test_checkpoint_is_smaller_than_the_state(sm):
    """Half of the hidden rows' bytes and the routing: at Large's shape 0.52 of the bf16 rows."""
    cfg = sm.config(32768, 1024, 4096, 128, 1.0, flags=sm.FLAG_TRAINING)
    rows = 128 * sm.switch_capacity(32768, 128, 1.0) * 4096 * 2
    routing = 4 * 32768 * 128 + 32 * 32768
    assert 0.5 * rows < sm.switch_checkpoint_size(cfg) < 0.505 * rows + routing


# ------------------------------------------------------- the plain forms

def test_reference_rounding_matches_the_type():
    """e4m3() against torch's own conversion over all magnitudes, ties and subnormals."""
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    v = v[torch.isfinite(v) & (v >= 0)].sort().values
    mid = (v[1:] + v[:-1]) / 2
    u = torch.cat([v, mid, mid * (1 + 1e-6), mid * (1 - 1e-6), torch.rand(4000).double() * 448])
    u = torch.cat([u, -u])
    assert torch.equal(ref.e4m3(u), u.float().to(torch.float8_e4m3fn).double())


def test_reference_scale():
    for a, s in ((448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (0.0, 2.0 ** -100),
                 (2.0 ** 127, 2.0 ** 119), (1e-40, 2.0 ** -100), (1.75 * 2.0 ** 20, 2.0 ** 12)):
        assert ref.scale_of(torch.tensor(a, dtype=torch.float64)).item() == s, a


def test_reference_keeps_positive_values():
    v = torch.tensor([[448.0, 1e-9, -1e-9, 0.0]], dtype=torch.float64)
    q, s = ref.quantize(v, positive=True)
    assert q.tolist() == [[448.0, 2.0 ** -9, 0.0, 0.0]] and s.item() == 1.0
