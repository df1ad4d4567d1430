"""Decode over caches some of whose V blocks are all zeros (padding, rows written for indices outside
the source): they have the scale 1, whatever the size of the other blocks, and must not take the other
blocks' weights their bits.

The bound, for one head of a unit with weights p and held rows v:

    |out - ref| <= 2^-8 |ref| + (2^-11 + 2^-15 S) W + sum_b TB 64 2^-26 448 max_{j in b} p_j scale_b + 2^-133

The first two terms are test_gpu_kv8.py's.  The third: a weight is held in three e4m3 terms a factor 16
apart, relative to the largest weight times scale of its tile, which stands at 256; the last term's step
is 2^-9 / 256 at that point, half of one 2^-18, which is 2^-26 of the largest.  A code is at most 448,
and a tile has TB blocks of 64 rows (2 for D = 128, 4 for D = 64), so a tile adds at most
TB 64 2^-26 448 max_{j in tile} p_j scale_j; tiles begin at any block, so the sum over tiles is taken as
the sum over blocks, each as if it were its tile's largest.  A block of zeros counts with
the least scale, 2^-126.  The last: below 2^-126 bf16's step is 2^-133, of which a rounding is off by half, and a sum in fp32 by a few
2^-149 (weights of e^-81 beside values of 1e-6 come to 1e-41)."""

import numpy as np
import pytest
import torch

from parity import f64
from test_gpu_kv8 import BF, dev, poison, rnd, unit_of

pytestmark = pytest.mark.gpu


def bound(q, k, vu, v, p):
    """The bound above and the weighted sum: q [G, D], held rows k and v, V's oracle unit vu."""
    D = k.shape[1]
    ref, W = p @ v, p @ np.abs(v)
    S = (np.abs(q) @ np.abs(k).T).max() / np.sqrt(D)
    extra = np.zeros((len(q), 1))
    for b, (codes, scale) in enumerate(zip(vu.codes, vu.scales)):
        scale = scale if np.nan_to_num(codes).any() else 2.0 ** -126
        extra[:, 0] += 256 // D * 64 * 2.0 ** -26 * 448 * p[:, 64 * b:64 * b + 64].max(1) * scale
    return ref, 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -15 * S) * W + extra + 2.0 ** -133


def weights(q, k):
    s = q @ k.T / np.sqrt(k.shape[1])
    p = np.exp(s - s.max(1, keepdims=True))
    return p / p.sum(1, keepdims=True)


def keys(D, n, zero, above, seed):
    """Queries' sign pattern, and keys whose logits are small but for `above` in the zero rows."""
    g = torch.Generator().manual_seed(seed)
    sign = torch.randint(0, 2, (D,), generator=g) * 2.0 - 1
    k = torch.randn((1, 1, 1, n, D), generator=g) * 0.3
    k[..., zero, :] = sign * (above / D ** 0.5) + k[..., zero, :] * 0.1
    return sign, k.to(BF)


@pytest.mark.parametrize("above", [0.0, 8.0, 60.0])
@pytest.mark.parametrize("size", [1.0, 1e-1, 1e-3, 1e-5, 1e-6])
@pytest.mark.parametrize("D,G", [(128, 1), (128, 4), (64, 2), (64, 8)])
def test_zero_blocks_beside_small_ones(kvc, D, G, size, above):
    n = 64 * 16 + 20
    zero = (torch.arange(n) // 64) % 2 == 0
    zero[64 * 16:] = False                             # the tail's rows count
    if above > 10:
        zero[64 * 8:64 * 12] = True                    # and whole tiles of zeros
    sign, k = keys(D, n, zero, above, 7)
    v = (rnd((1, 1, 1, n, D), 8, boost=False).float() * size).to(BF)
    v[..., zero, :] = 0
    v[..., 64 * 2:64 * 2 + 5, ::3] = -0.0
    q = (sign.expand(1, 1, G, D) * (1 + 0.05 * torch.arange(G)[:, None])).to(BF)
    cache = poison(kvc.KV8Cache(1, 1, 1, D, 64 * 17))
    kvc.kv8_write(*dev(k, v), cache)
    out = f64(kvc.kv8_decode_attn(q.cuda(), cache))[0, 0]
    ku, vu = unit_of(k[0, 0, 0]), unit_of(v[0, 0, 0])
    qh, rk, rv = f64(q)[0, 0], ku.read(), vu.read()
    ref, tol = bound(qh, rk, vu, rv, weights(qh, rk))
    assert (np.abs(out - ref) <= tol).all(), (np.abs(out - ref) / tol).max()
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_a_zero_block_with_a_nan_and_half_a_zero_block(kvc, D):
    """A block whose finite values are all zero, with a NaN in one column; a block of scale 1 whose
    first half is zero; columns without the NaN keep the small blocks' values."""
    n, G = 256, 2
    zero = torch.arange(n) < 64
    sign, k = keys(D, n, zero, 4.0, 17)
    v = (rnd((1, 1, 1, n, D), 18, boost=False).float() * 1e-4).to(BF)
    v[..., zero, :] = 0
    v[0, 0, 0, 11, 3] = float("nan")
    q = sign.expand(1, 1, G, D).to(BF)
    cache = poison(kvc.KV8Cache(1, 1, 1, D, n))
    for half in (False, True):
        if half:
            v[0, 0, 0, 64:96] = 0
            v[0, 0, 0, 100, :] = 300.0                 # scale 1
            k[0, 0, 0, 100] = -sign.to(BF) * 4         # at a small weight
        kvc.kv8_write(*dev(k, v), cache)
        out = f64(kvc.kv8_decode_attn(q.cuda(), cache))[0, 0]
        ku, vu = unit_of(k[0, 0, 0]), unit_of(v[0, 0, 0])
        if half:
            assert vu.scales[1] == 1.0
        qh, rk, rv = f64(q)[0, 0], ku.read(), vu.read()
        ref, tol = bound(qh, rk, vu, np.nan_to_num(rv), weights(qh, rk))
        assert np.isnan(out[:, 3]).all()
        rest = np.arange(D) != 3
        assert (np.abs(out - ref) <= tol)[:, rest].all(), half
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("D,G", [(128, 8), (64, 4)])
def test_zero_blocks_in_many_units(kvc, D, G):
    """Shared and whole units, zero blocks anywhere, rows written from indices outside the source
    among them (those are zeros, and are reported)."""
    Ly, B, H, L, cap = 1, 4, 24, 900, 960
    g = torch.Generator().manual_seed(27)
    k, v = rnd((Ly, B, H, L, D), 28, boost=False), rnd((Ly, B, H, L, D), 29, boost=False)
    v = (v.float() * torch.exp2(torch.randint(-14, 1, (Ly, B, H, 1, 1), generator=g).float())).to(BF)
    rows = torch.arange(L, dtype=torch.int32).expand(Ly, B, H, L).contiguous()
    out_of = torch.rand((Ly, B, H, L // 64 + 1), generator=g).repeat_interleave(64, -1)[..., :L] < 0.4
    rows[out_of] = -1
    n = torch.randint(1, L + 1, (Ly, B, H), generator=g, dtype=torch.int32)
    cache = poison(kvc.KV8Cache(Ly, B, H, D, cap))
    kvc.kv8_write(*dev(k, v), cache, rows=rows.cuda(), lengths=n.cuda())
    assert kvc.kvc_device_status() == kvc.DEV_BAD_STATE
    q = rnd((Ly, B, H * G, D), 30, boost=False)
    out = f64(kvc.kv8_decode_attn(q.cuda(), cache))
    for b in range(B):
        for h in range(H):
            m = int(n[0, b, h])
            kz, vz = k[0, b, h, :m].clone(), v[0, b, h, :m].clone()
            kz[out_of[0, b, h, :m]] = 0
            vz[out_of[0, b, h, :m]] = 0
            ku, vu = unit_of(kz), unit_of(vz)
            qh, rk, rv = f64(q)[0, b, h * G:h * G + G], ku.read(), vu.read()
            ref, tol = bound(qh, rk, vu, rv, weights(qh, rk))
            assert (np.abs(out[0, b, h * G:h * G + G] - ref) <= tol).all(), (b, h)
    assert kvc.kvc_device_status() == 0
