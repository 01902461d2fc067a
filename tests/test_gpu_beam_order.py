"""Order of continuations whose values are equal or nearly so, and how exactly
topk_beam knows a value.

A beam's log-sum-exp is a function of its logits alone, wherever the row lies:
beams of equal logits and scores tie exactly and rank by beam.

Bound on it, u = 2^-24, over n <= 2^18 tokens, p the softmax of the row: log2(e)
rounded to fp32 is off by 1.34e-8 relatively, of which E_p[max - x] <= ln n =
12.5 times as much stays: 1.7e-7; the exponent's rounding u * E_p[max - x] + u:
8.1e-7; the hardware's exp2 2^-22: 2.4e-7; a thread's sums are chains of at most
34 terms, joined over 2 + 5 steps: 41 u = 2.5e-6; the rest is 64-bit.  In all
3.7e-6, below 2^-18."""
import math

import pytest
import torch

import approximate_top_selection_b200 as atk

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
LSE = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA device")
    atk.load_library()
    torch.cuda.synchronize()
    atk.topk_device_status()
    yield


def row(n, dtype, seed, kind):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, generator=g) * 3
    if kind == "huge":
        x *= 1e7
    elif kind == "forbidden":
        x[torch.rand(n, generator=g) < 0.5] = -math.inf
    return x.to(dtype)


def best_of_equal_beams(x, beams, k):
    """(beam, token) of the k best of equal beams: by logit, then beam, then token."""
    live = torch.nonzero(x > -math.inf).flatten().tolist()
    xs = x.tolist()
    top = sorted(live, key=lambda t: (-xs[t], t))[:k]
    return sorted(((i, t) for i in range(beams) for t in top), key=lambda c: (-xs[c[1]], c[0], c[1]))[:k]


@pytest.mark.parametrize("copies", [1, 120])  # rows that CTAs hold, and rows that stream through them
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["normal", "huge", "forbidden"])
@pytest.mark.parametrize("n,beams,k", [(3001, 4, 8), (7, 5, 9), (50257, 4, 6), (8191, 8, 16), (70002, 3, 12), (1, 3, 3)])
def test_equal_beams_rank_by_beam(n, beams, k, kind, dtype, copies):
    for seed in range(3):
        x = row(n, dtype, n + seed, kind)
        logits = x.expand(copies, beams, n).contiguous().to(DEV)
        val, parent, token = (t.cpu() for t in atk.topk_beam(logits, torch.full((copies, beams), -1.0, device=DEV), k))
        want = best_of_equal_beams(x, beams, k)
        for b in range(copies):
            assert list(zip(parent[b].tolist(), token[b].tolist()))[: len(want)] == want, (seed, b)
        assert bool((val == val[:1]).all())


@pytest.mark.parametrize("copies", [1, 120])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [5, 16, 4096, 20001, 65537])
def test_the_place_of_the_logits_changes_nothing(n, dtype, copies):
    g = torch.Generator(device=DEV).manual_seed(n)
    x = (torch.randn(copies, 4, n, generator=g, device=DEV) * 3).to(dtype)
    s = torch.rand(copies, 4, generator=g, device=DEV) * -3
    want = atk.topk_beam(x, s, 8)
    room = torch.empty(x.numel() + 8, dtype=dtype, device=DEV)
    for off in range(1, 8):
        moved = room[off: off + x.numel()].view(x.shape)
        moved.copy_(x)
        got = atk.topk_beam(moved, s, 8)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), off


@pytest.mark.parametrize("copies", [1, 60])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,spread", [(1000, 1.0), (50257, 3.0), (131072, 3.0), (128255, 0.1), (262144, 2.0)])
def test_log_sum_exp(n, spread, dtype, copies):
    """Scores that bring the best values near zero, where fp32 outputs show the log-sum-exp's own error."""
    g = torch.Generator(device=DEV).manual_seed(n)
    rows = 6
    x = (torch.randn(rows, n, generator=g, device=DEV) * spread).to(dtype)
    lse = torch.logsumexp(x.double(), 1)
    top = x.double().amax(1)
    s = (lse - top).float()
    exact = s.double() + top - lse
    big = x.expand(copies, rows, n).reshape(-1, 1, n)
    val, _, token = atk.topk_beam(big, s.repeat(copies).view(-1, 1), 1)
    err = (val.double().view(copies, rows) - exact).abs()
    assert bool((err <= LSE + 2.0 ** -24 * exact.abs()).all()), float(err.max())
    first = torch.where(x.double() == top[:, None], torch.arange(n, device=DEV), n).amin(1)
    assert torch.equal(token.view(copies, rows).long(), first.expand(copies, rows))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beams_four_bounds_apart_keep_their_order(dtype):
    g = torch.Generator(device=DEV).manual_seed(9)
    batch, n = 64, 30011
    x = (torch.randn(batch, 2, n, generator=g, device=DEV) * 3).to(dtype)
    lse = torch.logsumexp(x.double(), 2)
    top = x.double().amax(2)
    ahead = torch.arange(batch, device=DEV) % 2  # the beam whose best value is 4 bounds larger
    s = lse - top
    s[torch.arange(batch, device=DEV), ahead] += 4 * LSE
    s = s.float()
    exact = s.double() + top - lse
    clear = (exact[:, 0] - exact[:, 1]).abs() > 2 * LSE  # what rounding s to fp32 left of it
    assert int(clear.sum()) > batch // 2
    _, parent, _ = atk.topk_beam(x, s, 2)
    assert torch.equal(parent[clear, 0].long(), exact.argmax(1)[clear])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("huge", [False, True])
def test_forbidden_stretches_before_the_first_token(dtype, huge):
    """Many pieces of a row without a token, before those that have some."""
    n, first = 262143, 170001
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.full((1, 1, n), -math.inf, device=DEV)
    x[..., first:] = torch.randn(n - first, generator=g, device=DEV)
    if huge:
        x[..., first + 50000:] -= 3e6  # pieces summed relative to their own maximum
    x = x.to(dtype)
    lse = torch.logsumexp(x.double().flatten(), 0)
    s = (lse - x.double().max()).float().view(1, 1)
    val, _, token = atk.topk_beam(x, s, 3)
    best = (x.double().flatten() + s.double().flatten() - lse).sort(descending=True, stable=True)
    assert bool(((val.double().flatten() - best.values[:3]).abs() <= LSE + 2.0 ** -24 * best.values[:3].abs()).all())
    assert torch.equal(token.flatten().long(), best.indices[:3])
