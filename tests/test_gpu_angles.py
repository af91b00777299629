"""Rotary angles against exact integer arithmetic, over all int32 positions and
frequencies up to 2^26.

A turn's fraction is off by at most (2^-49 |inv_freq| + 2^-61) |position|: of the
product with 1 / 2 pi in two fp32 numbers, the second is a sum below 2^-25.9
inv_freq and off by 2^-24 of that, its product with the constant's second part
(2^-27.2) by 2^-51.2 inv_freq, that part itself by 2^-52; two numbers are cut to 62
bits.  2^-32 turns are cut and pi 2^-25 radians lost in fp32.  Cosine and sine, the
products and their sum add the 20 u of the rest of the rotation (u = 2^-24), of the
row's largest value times sqrt 2: 2e-6."""
import math

import pytest
import torch

import gated_delta_rule_kaczmarz_gb300 as kla

pytestmark = pytest.mark.gpu
BITS = 512


def _arctan_inverse(n):
    """arctan(1 / n) 2^BITS."""
    total, power, k = 0, (1 << BITS) // n, 0
    while power:
        total += (-1) ** k * (power // (2 * k + 1))
        power, k = power // (n * n), k + 1
    return total


PI = 4 * (4 * _arctan_inverse(5) - _arctan_inverse(239))         # Machin
INV_2PI = (1 << 2 * BITS) // (2 * PI)                              # 2^BITS / 2 pi


def _angle(pos, freq):
    """pos freq modulo one turn, in radians."""
    a, b = float(freq).as_integer_ratio()
    turns = (pos * a * INV_2PI // b) & ((1 << BITS) - 1)
    return 2 * math.pi * ((turns >> (BITS - 64)) / 2.0 ** 64)


def _check(pos, freq, dtype=torch.float32):
    """One row a position: cosines and sines of every pair."""
    g = torch.Generator().manual_seed(7)
    q = torch.randn(len(pos), 1, 128, generator=g).to(dtype)
    p = torch.tensor(pos, dtype=torch.int64).int().cuda()
    got, _ = kla.kla_qk_norm_rope_fwd(q.cuda(), None, p, freq.cuda(), norm_q="none")
    ang = torch.tensor([[_angle(x, f) for f in freq.tolist()] for x in pos], dtype=torch.float64)[:, None]
    n = freq.numel()
    x = q.double()
    a, b = x[..., :n], x[..., n:2 * n]
    want = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin(), x[..., 2 * n:]], -1)
    size = freq.double().abs() * 2.0 ** -49 + 2.0 ** -61
    far = 2 * math.pi * (torch.tensor(pos).abs()[:, None] * size + 2.0 ** -32) + math.pi * 2.0 ** -25
    far = torch.cat([far, far, torch.zeros(len(pos), 128 - 2 * n)], -1)[:, None]
    tol = (2e-6 + math.sqrt(2) * far) * x.abs().amax(-1, keepdim=True)
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    off = (got.cpu().double() - want).abs() - tol
    assert float(off.max()) <= 0, float(off.max())


FAR = [2 ** 31 - 1, -2 ** 31, 0, 1, -1, 131072, 1000003, -1000003, 1 << 24, (1 << 24) + 1,
       123456789, -987654321, 2 ** 31 - 12345]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_positions_up_to_the_ends_of_int32(base, dtype):
    _check(FAR, (base ** (-torch.arange(64) / 64.0)).float(), dtype)


def test_frequencies_of_any_size_and_sign():
    g = torch.Generator().manual_seed(3)
    freq = (1 + torch.rand(64, generator=g)) * 2.0 ** torch.linspace(-126, 25, 64).double()
    freq = freq.float() * (1 - 2 * (torch.arange(64) % 2))
    freq[5], freq[9], freq[11], freq[12] = 0.0, -0.0, 2.0 ** 26, -torch.finfo(torch.float32).tiny
    assert float(freq.abs().max()) <= 2.0 ** 26
    _check(FAR, freq)


def test_many_tokens_at_far_positions():
    """The pipelined kernel: the same angles."""
    n, step = 9000, 238609
    pos = [i * step - 2 ** 30 for i in range(n)]
    assert pos[-1] < 2 ** 31
    freq = (10000.0 ** (-torch.arange(16) / 16.0)).float()
    _check(pos, freq)
