"""The 64-bit forms that the floating-point operators are tested against are
themselves pinned: hand-computed values, a brute-force nearest search, torch's
own group norm, and round trips of the storage layout."""
import pytest
import torch

from oracle import float_ref as F


def test_e2m1_rounding_by_hand():
    v = torch.tensor([0, 0.25, 0.26, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 3.49, 5, 5.01,
                      7.9], dtype=torch.float64)
    want = [0, 0, 1, 2, 1, 2, 3, 4, 4, 5, 6, 5, 6, 7, 7]
    assert F.round_e2m1(v).tolist() == want
    assert F.round_e2m1(-v).tolist() == want


def test_e2m1_rounding_is_nearest():
    g = torch.Generator().manual_seed(3)
    v = torch.rand(4000, generator=g, dtype=torch.float64) * 8
    grid = torch.tensor(F.E2M1, dtype=torch.float64)
    got = grid[F.round_e2m1(v)]
    best = (v.unsqueeze(1) - grid).abs().amin(1)
    assert torch.equal((v - got).abs(), best)


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (1.0, 125), (0.99, 124), (6.0, 127), (7.99, 127),
                                       (8.0, 128), (2.0 ** -140, 0), (3.3e38, 252),
                                       (float("inf"), 255), (float("nan"), 255)])
def test_scale_byte_by_hand(amax, byte):
    assert int(F.scale_byte(torch.tensor([amax], dtype=torch.float64))) == byte


@pytest.mark.parametrize("M,K", [(1, 32), (5, 96), (128, 128), (130, 160), (300, 512)])
def test_storage_round_trip(M, K):
    g = torch.Generator().manual_seed(M + K)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    codes, s = F.quantize_mx4(x)
    q, sf = F.pack_mx4(codes, s)
    c2, s2 = F.unpack_mx4(q, sf)
    assert torch.equal(codes, c2) and torch.equal(s, s2)
    assert sf.long().sum() == s.sum()  # padding is zero
    # one rounding: half the spacing at the block's top (2 * 2^(s-127)), or the saturation at 6
    v, top = F.values_mx4(codes, s), torch.exp2(s.double() - 127).repeat_interleave(32, 1)
    assert ((v - x.double()).abs() <= torch.maximum(top, x.double().abs() - 6 * top)).all()


def test_group_norm_matches_torch():
    g = torch.Generator().manual_seed(9)
    x = torch.randn(3, 5, 4, 12, generator=g, dtype=torch.float64) * 3 + 1
    gamma, beta = torch.randn(12, generator=g, dtype=torch.float64), torch.randn(12, generator=g, dtype=torch.float64)
    y, _ = F.group_norm(x, gamma, beta, 4, 1e-5)
    ref = torch.nn.functional.group_norm(x.permute(0, 3, 1, 2), 4, gamma, beta, 1e-5)
    assert torch.allclose(y, ref.permute(0, 2, 3, 1), rtol=1e-12, atol=1e-12)
