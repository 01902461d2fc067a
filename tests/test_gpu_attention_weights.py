"""Attention where the weights or the values span more than a float's bits.

The bound on an output is the one that test_gpu_paged_attention derives.  Beside
e4m3 codes a weight w_j = p_j * scale_j has 11 significant bits (2^-11 w_j), or lies
below 2^-24 of the head's largest, W, and is off by half a step at most, 2^-35 W;
products of scales near 2^-127 and weights are multiples of 2^-149.  Both times the
column's largest code."""
import math

import pytest
import torch

import approximate_top_selection_b200 as atk

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA device")
    atk.load_library()
    torch.cuda.synchronize()
    atk.topk_device_status()
    yield


def contiguous(batch, heads, kv_heads, d, lens, seed, page=16):
    """A bf16 case whose sequences own their pages in order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    width = -(-max(lens) // page)
    s = dict(q=torch.randn(batch, heads, d, generator=g, device=DEV).bfloat16(),
             table=torch.arange(batch * width, device=DEV, dtype=torch.int32).view(batch, width),
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV), k_scale=None, v_scale=None)
    for n in "kv":
        s[n] = torch.randn(batch * width, kv_heads, page, d, generator=g, device=DEV).bfloat16()
    return s


def call(s, **kw):
    return atk.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                               return_lse=True, **kw)


def rows(s, name, b):
    """Rows [kv_heads, n, d] of sequence b in 64 bits, and their scales (1 for bf16)."""
    n = int(s["lens"][b])
    x = s[name][s["table"][b].long()].double()
    w = s[name + "_scale"]
    w = torch.ones(x.shape[:3], dtype=torch.float64, device=DEV) if w is None else w[s["table"][b].long()].double()
    return x.transpose(0, 1).flatten(1, 2)[:, :n], w.transpose(0, 1).flatten(1, 2)[:, :n]


def reference(s, scale=None):
    """(out, tolerance, lse) in 64 bits."""
    outs, tols, lses = [], [], []
    batch, heads, d = s["q"].shape
    scale = d ** -0.5 if scale is None else scale
    e4m3 = s["k_scale"] is not None
    for b in range(batch):
        (k, ks), (v, vs) = rows(s, "k", b), rows(s, "v", b)
        kv_heads, n, _ = k.shape
        q = s["q"][b].double().view(kv_heads, -1, d)
        t = q @ (k * ks[..., None]).transpose(1, 2) * scale
        size = abs(scale) * q.norm(dim=2)[..., None] * (k * ks[..., None]).norm(dim=2).amax(1).view(-1, 1, 1)
        p = torch.softmax(t, 2)
        o, mass = p @ (v * vs[..., None]), p @ (v * vs[..., None]).abs()
        weights = (2.0 ** -11 if e4m3 else 2.0 ** -16)
        tol = 2.0 ** -8 * o.abs() + 2.0 ** -134 + (2 * size * (2 * d + 2) * U + 2.0 ** -20 + weights + 2 * U * (n + 64)) * mass
        if e4m3:
            largest = (p * vs[:, None]).abs().amax(2, keepdim=True)
            tol = tol + n * v.abs().amax(1, keepdim=True) * (2.0 ** -35 * largest + 2.0 ** -149)
        outs.append(o.reshape(heads, d))
        tols.append(tol.reshape(heads, d))
        lses.append(torch.logsumexp(t, 2).reshape(heads))
    return torch.stack(outs), torch.stack(tols), torch.stack(lses)


def check(s, got=None, **kw):
    out, lse = got or call(s, **kw)
    o, tol, l = reference(s, **kw)
    out = out.double()
    assert torch.equal(torch.isnan(out), torch.isnan(o))
    assert torch.equal(torch.isinf(out), torch.isinf(o)) and torch.equal(out[torch.isinf(o)], o[torch.isinf(o)])
    fine = torch.isfinite(o) & torch.isfinite(tol)
    assert int(fine.sum()) > 0
    assert bool(((out - o).abs() <= tol)[fine].all()), float(((out - o).abs() / tol)[fine].max())
    assert bool(((lse.double() - l).abs() <= 2.0 ** -10 + 2.0 ** -20 * l.abs()).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("batch,heads,kv_heads,longest", [(2, 4, 4, 40), (1, 8, 1, 3000), (3, 12, 1, 500), (40, 16, 16, 47),
                                                          (2, 40, 2, 333)])
def test_infinite_values(batch, heads, kv_heads, longest, d):
    """sum_j p_j V_j is infinite where one V_j is, and undefined only where they disagree."""
    lens = [max(2, longest - 7 * b) for b in range(batch)]
    s = contiguous(batch, heads, kv_heads, d, lens, longest + d)
    for b in range(batch):
        last = lens[b] - 1
        at = [(s["table"][b, t // 16].item(), t % 16) for t in (0, 1, last)]
        s["v"][at[0][0], :, at[0][1], 0:3] = math.inf
        s["v"][at[1][0], :, at[1][1], 3] = -math.inf
        s["v"][at[2][0], :, at[2][1], 5:9] = -math.inf
        s["v"][at[0][0], :, at[0][1], 7] = math.inf     # meets the -inf of the last token
        s["v"][at[0][0], :, at[0][1], d - 1] = math.nan
    check(s)


def test_infinite_values_of_listed_positions():
    s = contiguous(2, 8, 8, 128, [300, 200], 3)
    s["v"][:, :, ::3, ::5] = math.inf
    pos = torch.arange(200, device=DEV, dtype=torch.int32).expand(2, 8, 200).contiguous()
    got = call(s, positions=pos)
    s["lens"] = torch.tensor([200, 200], dtype=torch.int32, device=DEV)
    check(s, got)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 16])
def test_infinite_values_of_small_weights(heads, d):
    """Weights that are powers of two, of which a second part would be zero."""
    s = contiguous(1, heads, 1, d, [200], 7)
    s["q"][:] = 0
    s["q"][..., 0] = 1.0
    s["k"][..., 0] = 0.0
    for key, score, col in ((0, -1.0, 0), (70, -20.0, 1), (133, -60.0, 2), (199, -98.0, 3)):
        s["k"][key // 16, 0, key % 16, 0] = score
        s["v"][key // 16, 0, key % 16, col] = math.inf
    out, _ = call(s, scale=math.log(2.0))  # scores are powers of two's exponents
    assert bool((out[..., :4] == math.inf).all()) and bool(torch.isfinite(out[..., 4:]).all())


def quantised(s, k_exp=(-9, -5), v_exp=(-9, -5), seed=5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    for n, (lo, hi) in (("k", k_exp), ("v", v_exp)):
        s[n + "_scale"] = torch.exp2(torch.randint(lo, hi, s[n].shape[:3], generator=g, device=DEV).double()).float()
        s[n] = (s[n].float() * 100).clamp(-448, 448).to(E4M3)
    return s


@pytest.mark.parametrize("batch,heads,kv_heads,d,n", [(2, 4, 4, 64, 30), (1, 8, 2, 128, 3000), (60, 8, 8, 128, 40),
                                                      (2, 16, 1, 256, 600)])
@pytest.mark.parametrize("lowest,above", [(-127, 1), (-127, 30), (-120, 4), (110, 10)])
def test_smallest_and_largest_value_scales(batch, heads, kv_heads, d, n, lowest, above):
    """Scales as cache_write leaves them for rows of the smallest and the largest bf16 values."""
    check(quantised(contiguous(batch, heads, kv_heads, d, [n] * batch, n), v_exp=(lowest, lowest + above)))


def test_written_rows_of_tiny_values_come_back_through_attention():
    s = contiguous(1, 2, 2, 128, [64], 8)
    v = (s["v"].double() * 2.0 ** -119).bfloat16()
    kc, vc = (torch.zeros(4, 2, 16, 128, device=DEV).to(E4M3) for _ in range(2))
    ks, vs = (torch.ones(4, 2, 16, device=DEV) for _ in range(2))
    new = [x.transpose(1, 2).reshape(64, 2, 128).contiguous() for x in (s["k"], v)]
    atk.cache_write(*new, kc, vc, torch.arange(64, device=DEV), k_scale=ks, v_scale=vs)
    t = {**s, "k": kc, "v": vc, "k_scale": ks, "v_scale": vs}
    check(t)
    assert float(call(t)[0].abs().max()) > 2.0 ** -122


@pytest.mark.parametrize("batch,heads,kv_heads,d,n", [
    (450, 4, 1, 128, 1000),  # whole sequences by warps
    (400, 16, 1, 64, 500),
    (24, 8, 2, 128, 9000),   # sequences shared by CTAs
    (40, 1, 1, 256, 3000),
    (20, 16, 1, 256, 3000),
    (1, 4, 1, 128, 131072),
])
@pytest.mark.parametrize("ahead", [5.0, 8.3, 11.0, 16.2, 17.2, 19.0])
def test_a_key_that_outweighs_a_long_tail(batch, heads, kv_heads, d, n, ahead):
    """All scores are equal but one, `ahead` larger, whose values are zero in
    half of the columns: there the tail is all there is."""
    s = quantised(contiguous(batch, heads, kv_heads, d, [n] * batch, n))
    s["q"][:] = 0
    s["q"][..., 0] = 1.0
    s["k"].view(torch.uint8)[:] = 0
    s["v_scale"][:] = 2.0 ** -7
    s["v"].view(torch.uint8)[:] = 0x38  # 1.0
    width = s["table"].shape[1]
    for b in range(batch):
        key = (77 * b + n // 2) % n
        page, off = b * width + key // 16, key % 16
        s["k"].view(torch.uint8)[page, :, off, 0] = 0x38
        s["k_scale"][page, :, off] = 1.0
        s["v"].view(torch.uint8)[page, :, off, ::2] = 0
    check(s, scale=ahead)


def test_value_scales_far_apart():
    for heads, kv_heads, d, n in ((8, 2, 128, 5000), (3, 3, 64, 700), (16, 1, 128, 2000), (4, 4, 256, 3000)):
        check(quantised(contiguous(3, heads, kv_heads, d, [n, n // 3, 9], n), v_exp=(-30, -4)))
        check(quantised(contiguous(3, heads, kv_heads, d, [n, n // 3, 9], n), v_exp=(-100, 100)))


def test_scales_and_codes_of_the_values_against_each_other():
    """Half of the keys have scales 2^-20 of the others' and values where the others have none."""
    s = quantised(contiguous(2, 8, 2, 128, [900, 4000], 4))
    s["v"].view(torch.uint8)[:] = 0x40  # 2.0
    s["v_scale"][:] = 2.0 ** -6
    s["v_scale"][:, :, ::2] = 2.0 ** -26
    s["v"].view(torch.uint8)[:, :, 1::2, ::3] = 0
    check(s)
