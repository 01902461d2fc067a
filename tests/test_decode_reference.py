"""The 64-bit forms that the GPU tests compare with, against cases worked out
by hand and torch on the CPU."""
import math

import pytest
import torch

import decode_reference as ref


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.isnan(codes), torch.isnan(ref.e4m3_values()))
    fine = ~torch.isnan(codes)
    assert torch.equal(codes[fine], ref.e4m3_values()[fine])


@pytest.mark.parametrize("top,scale", [(448.0, 1.0), (449.0, 2.0), (0.0, 1.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                       (1.7578125, 2.0 ** -7), (2.0 ** -133, 2.0 ** -127), (3.3895e38, 2.0 ** 120)])
def test_row_scale(top, scale):
    x = torch.tensor([top, -top / 2, 0.0, top / 64]).bfloat16()
    y, s = ref.quantise_row(x)
    if top == 449.0:  # rounds to 448 as bf16
        assert s == 1.0
        return
    assert s == scale
    assert torch.equal(torch.signbit(y), torch.signbit(x))
    err = (y * s - x.double()).abs()
    assert bool((err <= torch.maximum(x.double().abs() * 2.0 ** -4, torch.tensor(2.0 ** -10 * s, dtype=torch.float64))).all())


def test_row_codes_round_to_even_like_torch():
    x = torch.randn(4096, generator=torch.Generator().manual_seed(3)).bfloat16() * 100
    y, s = ref.quantise_row(x)
    assert torch.equal(y, (x.double() / s).float().to(torch.float8_e4m3fn).double())


def test_row_with_nan_or_infinity():
    for bad in (math.nan, math.inf, -math.inf):
        y, s = ref.quantise_row(torch.tensor([1.0, bad]).bfloat16())
        assert math.isnan(s) and bool(torch.isnan(y).all())


def test_attention_is_softmax_over_the_pages_rows():
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(5, 2, 4, 8, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(1, 4, 8, generator=g).bfloat16()
    table = torch.tensor([[3, 0, 4]], dtype=torch.int32)
    o, lse, _, _ = ref.attention(q, k, v, table, torch.tensor([9]), 0.5)
    kk = torch.cat([k[3], k[0], k[4, :, :1]], 1).double()
    vv = torch.cat([v[3], v[0], v[4, :, :1]], 1).double()
    t = torch.einsum("gud,gnd->gun", q[0].double().view(2, 2, 8), kk) * 0.5
    want = torch.einsum("gun,gnd->gud", torch.softmax(t, 2), vv).reshape(4, 8)
    assert torch.allclose(o[0], want, rtol=1e-12, atol=0)
    assert torch.allclose(lse[0], torch.logsumexp(t, 2).flatten(), rtol=1e-12)
    pos = torch.tensor([[[8, -1, 2, 2, 50, 9]]], dtype=torch.int32).expand(1, 2, 6)
    o, _, _, _ = ref.attention(q, k, v, table, torch.tensor([9]), 0.5, positions=pos)
    at = [8, 2, 2]
    want = torch.einsum("gun,gnd->gud", torch.softmax(t[:, :, at], 2), vv[:, at]).reshape(4, 8)
    assert torch.allclose(o[0], want, rtol=1e-12)


def test_beam_step_by_hand():
    x = torch.tensor([[0.0, 0.0, ref.NINF], [math.log(3.0), 0.0, 0.0]])
    got = ref.beam_step(x, torch.tensor([math.log(0.5), math.log(0.5)]), 4)
    # beam 0: 1/2 * (1/2, 1/2, -), beam 1: 1/2 * (3/5, 1/5, 1/5)
    assert [(i, t) for _, i, t in got] == [(1, 0), (0, 0), (0, 1), (1, 1)]
    assert got[0][0] == pytest.approx(math.log(0.3)) and got[3][0] == pytest.approx(math.log(0.1))
    assert ref.beam_step(x, torch.tensor([ref.NINF, ref.NINF]), 2) == []
    bad = ref.beam_step(torch.tensor([[0.0, 1.0], [math.inf, 0.0]]), torch.zeros(2), 3)
    assert [(i, t) for _, i, t in bad] == [(1, 0), (1, 1), (0, 1)] and math.isnan(bad[0][0])
