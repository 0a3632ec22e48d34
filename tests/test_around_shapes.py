"""Rows of another length than the call's are refused by the binding, not read
or written at the wrong places (no GPU: shapes are checked before places)."""

import pytest
import torch

import routed_expert_ffn_gemv_amd as moe

T, N, K = 4, 300, 256


def _codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _linear(x8=(T, K), xs=(T, 2), w8=(N, K), ws=(3, 2)):
    moe.moe_scaled_linear(_codes(*x8), torch.zeros(xs), T, _codes(*w8), torch.zeros(ws), N, K,
                          torch.zeros((T, N)))


def _norm(x8=(T, K), xs=(T, 2)):
    moe.moe_add_rmsnorm(T, K, None, torch.zeros((T, K)), torch.ones(K), 1e-6, x8=_codes(*x8),
                        x8_scale=torch.zeros(xs))


@pytest.mark.parametrize("call,what,kw", [
    (_linear, "x8", dict(x8=(T, K + 16))), (_linear, "x8", dict(x8=(2 * T, K // 2))),
    (_linear, "x_scale", dict(xs=(T, 3))), (_linear, "w8", dict(w8=(N, 2 * K))),
    (_linear, "w8", dict(w8=(N, 3, 128))), (_linear, "w_scale", dict(ws=(3, 4))),
    (_norm, "x8", dict(x8=(T, K + 1))), (_norm, "x8_scale", dict(xs=(T, 3))),
])
def test_longer_rows_are_refused(call, what, kw):
    with pytest.raises(ValueError, match=rf"^{what}: "):
        call(**kw)


@pytest.mark.parametrize("call,kw", [
    (_linear, {}), (_norm, {}),
    (_linear, dict(x8=(T + 3, K), xs=(T + 1, 2), w8=(N + 5, K), ws=(4, 2))),    # more rows
    (_linear, dict(x8=(T * K,), xs=(2 * T,), w8=(N * K,), ws=(6,))),            # flat
    (_linear, dict(x8=(2, 2, K), w8=(N, 2, 128), ws=(3, 1, 2))),                # in more dimensions
    (_norm, dict(x8=(1, T, K), xs=(T, 2, 1))),
])
def test_rows_of_the_right_length_pass_on_to_the_next_check(call, kw):
    with pytest.raises(ValueError, match="must be on one GPU"):
        call(**kw)


def test_one_row_may_lie_in_a_longer_one():
    with pytest.raises(ValueError, match="must be on one GPU"):
        moe.moe_scaled_linear(_codes(1, K + 16), torch.zeros((1, 3)), 1, _codes(N, K), torch.zeros((3, 2)),
                              N, K, torch.zeros((1, N)))


def test_sample_workspace_is_what_the_slices_need():
    """Rows that take a workgroup each use none; sizes grow with T and V, so
    that one workspace serves every smaller call."""
    size = moe.moe_sample_workspace_size
    row = size(1, 1000)
    assert 0 < row <= 256 * 1024
    assert size(256, 32000) == size(16384, 36000) == row
    assert size(16384, 151936) == size(256, 151936) < 256 * row
    assert size(4, 151936) <= 4 * row
    Ts = (0, 1, 2, 4, 53, 54, 55, 64, 76, 77, 78, 232, 233, 234, 300, 16384)
    Vs = (1, 4096, 36000, 36001, 50257, 50700, 151936, 1 << 26)
    for V in Vs:
        for a, b in zip(Ts, Ts[1:]):
            assert size(a, V) <= size(b, V)
    for T in Ts:
        for a, b in zip(Vs, Vs[1:]):
            assert size(T, a) <= size(T, b)


@pytest.mark.parametrize("off", [0, 4, -8, 12, -4])
def test_drafts_within_the_tokens_are_refused(off):
    """They are compared once the tokens are written.  (Addresses are never
    dereferenced: the call is refused before any launch.)"""
    at = 1 << 20
    assert moe.lib.moe_verify_sample(at, moe.MOE_W_F32, 4, 1000, 1000, None, at, at + 4096 + off, at + 4096,
                                     at, at, at, 1 << 30, None) == moe.MOE_ERR_INVALID
