"""Angles of the rotation near whole, half and quarter turns and very small ones."""
import numpy as np
import pytest
import torch

import context_causal_attention_tcgen05_gb300 as cpa
from gpu_common import _record, check_ok, need_gpu
from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
def test_cosine_and_sine_are_right_to_their_own_size(inter):
    """(1, 0) turns into (cos, sin), each right to 2 fp32 roundings of itself (2^-23: the function's and one of the angle
    inside its eighth of a turn, which moves neither function by more than itself) and the angle's fixed-point error, two
    units of 2^-64 of a turn a position: 2^-29 at 2^31."""
    rng = np.random.default_rng(0)
    S, pairs = 4096, 64
    pos = rng.integers(0, 131072, size=(1, S))
    pos[0, ::7] = rng.integers(-2**31, 2**31 - 1, size=len(pos[0, ::7]))
    # frequencies that put a position of a few thousands next to multiples of a quarter turn, and tiny ones
    inv = np.concatenate([np.pi / 2 * (np.arange(32) % 8 + 1) / 2 * (1 + rng.normal(size=32) * 1e-8),
                          500000.0 ** (-np.arange(32) / 32) * 1e-3])
    inv = torch.tensor(inv, dtype=torch.float32, device="cuda")
    x = torch.zeros(S, 1, 2 * pairs, device="cuda")
    x[..., 0::2] = 1 if inter else 0
    if not inter:
        x[..., :pairs] = 1
    for inverse in (False, True):
        y, _ = cpa.cp_rotary(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), inv, [pairs], inter, inverse)
        ref = serving.rotary(x.double().cpu().numpy(), pos, inv.double().cpu().numpy(), [pairs], inter, inverse)
        bound = 2 * 2.0**-23 * np.abs(ref) + 2.0**-29 * (np.abs(pos[0]) / 2**31)[:, None, None] + 1e-30
        r = float((np.abs(y.double().cpu().numpy() - ref) / bound).max())
        _record(f"angles {inverse}", r, 1.0)
        assert r <= 1, r
    check_ok()


def test_fp32_rotation_is_as_exact_as_fp32_allows():
    """Random pairs: the error against 64 bits is that of cos and sin rounded to fp32, of a product and of a sum."""
    S, D = 8192, 128
    x = torch.randn(S, 2, D, generator=torch.Generator().manual_seed(1)).cuda()
    pos = np.random.default_rng(1).integers(0, 131072, size=(1, S))
    inv = (500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    y, _ = cpa.cp_rotary(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), inv, [D // 2])
    ref = serving.rotary(x.double().cpu().numpy(), pos, inv.double().cpu().numpy(), [D // 2])
    e = np.linalg.norm(y.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    # a rounding to fp32 is off by 2^-24 / sqrt 3 of its binade's start, .425 * 2^-24 of values spread evenly over it.  The
    # variances of a c - b s, in units of the result's: cos and sin a half each, one product a half, the sum one.  A tenth
    # more for the functions' own error.
    bound = 1.1 * 2.5**0.5 * 0.425 * 2.0**-24
    _record("fp32 2-norm", e, bound)
    assert e <= bound, e
    check_ok()
