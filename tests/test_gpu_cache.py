"""cache_write and cache_read on the GPU.  Nothing here has a tolerance: the
scales are powers of two, so every stored code is determined by its input, and
reading back is one exact product (scales that are no power of two: one
rounding to bf16)."""
import math

import pytest
import torch

import approximate_top_selection_b200 as atk
import decode_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA device")
    atk.load_library()
    torch.cuda.synchronize()
    atk.topk_device_status()
    yield


def empty_caches(pages, heads, page, d, kind):
    """Caches and scales filled with a pattern that a write must leave alone elsewhere."""
    if kind == "bf16":
        c = [torch.full((pages, heads, page, d), 7.0 + i, dtype=torch.bfloat16, device=DEV) for i in range(2)]
        return c, [None, None]
    c = [torch.full((pages, heads, page, d), 0x31 + i, dtype=torch.uint8, device=DEV).view(E4M3) for i in range(2)]
    return c, [torch.full((pages, heads, page), 3.0 + i, device=DEV) for i in range(2)]


def rows(tokens, heads, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, tokens, heads, d, generator=g)
    x *= torch.exp2(torch.randint(-20, 20, (2, tokens, heads, 1), generator=g).float())
    x *= torch.exp2(torch.randint(-9, 1, (2, tokens, heads, d), generator=g).float())
    return x.bfloat16()


def check_written(x, slots, before, caches, scales, page):
    """Caches hold `before` with the live tokens' rows replaced."""
    for i in range(2):
        want = before[0][i].cpu().clone()
        ws = before[1][i].cpu().clone() if scales[i] is not None else None
        raw = want.view(torch.uint8) if ws is not None else want
        for t, slot in enumerate(slots.tolist()):
            if not 0 <= slot < want.shape[0] * page:
                continue
            for h in range(want.shape[1]):
                if ws is None:
                    want[slot // page, h, slot % page] = x[i, t, h]
                else:
                    y, s = ref.quantise_row(x[i, t, h])
                    raw[slot // page, h, slot % page] = y.float().to(E4M3).view(torch.uint8)
                    ws[slot // page, h, slot % page] = s
        got = caches[i].cpu()
        if ws is None:
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        else:
            gs = scales[i].cpu()
            assert torch.equal(torch.isnan(gs), torch.isnan(ws))
            fine = ~torch.isnan(ws)
            assert torch.equal(gs[fine], ws[fine])
            assert torch.equal(got.view(torch.uint8)[fine], want.view(torch.uint8)[fine])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens,heads,d,page", [(1, 1, 64, 1), (3, 2, 128, 16), (37, 3, 256, 7), (130, 8, 64, 16),
                                                 (65, 1, 128, 1000)])
def test_write(kind, tokens, heads, d, page):
    x = rows(tokens, heads, d, tokens + d)
    if tokens > 2:
        x[0, 1] = 0.0                      # a row of zeros
        x[1, 2, 0, 5] = math.nan
        x[1, 1, 0, d - 1] = -math.inf
        x[0, 0, 0] = (x[0, 0, 0].float() * 2.0 ** -133).bfloat16()  # subnormal values
        x[0, 2, 0] = torch.linspace(-448, 448, d).bfloat16()
    pages = -(-tokens // page) + 2
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:tokens]
    slots[tokens // 2] = -1 if tokens > 1 else slots[0]
    caches, scales = empty_caches(pages, heads, page, d, kind)
    before = [c.clone() for c in caches], [s.clone() if s is not None else None for s in scales]
    xd = x.to(DEV)
    assert atk.cache_write(xd[0], xd[1], *caches, slots.to(DEV), k_scale=scales[0], v_scale=scales[1]) is None
    check_written(x, slots, before, caches, scales, page)
    assert atk.topk_device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_write_strided_sources_and_caches(kind):
    tokens, heads, d, page, pages = 20, 4, 128, 8, 5
    x = rows(tokens, heads, d, 3)
    proj = torch.zeros(tokens, 1000 * 2, dtype=torch.bfloat16, device=DEV)
    k = proj[:, 8:8 + heads * d].view(tokens, heads, d)
    v = proj[:, 1000:1000 + heads * d].view(tokens, heads, d)
    k.copy_(x[0])
    v.copy_(x[1])
    (kc, vc), scales = empty_caches(pages, heads, page, d, kind)
    both = torch.stack([kc.view(torch.uint8), vc.view(torch.uint8)], 1).transpose(2, 3).contiguous().view(kc.dtype)
    caches = [both[:, i].transpose(1, 2) for i in range(2)]   # [pages, heads, page, d], tokens first in memory
    if kind == "e4m3":
        sc = torch.stack(scales, 3)
        scales = [sc[..., 0], sc[..., 1]]
    before = [c.clone() for c in caches], [s.clone() if s is not None else None for s in scales]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2))[:tokens]
    atk.cache_write(k, v, *caches, slots.to(DEV), k_scale=scales[0], v_scale=scales[1])
    check_written(x, slots, before, caches, scales, page)
    out = atk.cache_read(caches[0], torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1),
                         torch.tensor([pages * page], dtype=torch.int32, device=DEV), 33, scale=scales[0])
    want = ref.decode_rows(caches[0].contiguous().cpu(), None if scales[0] is None else scales[0].contiguous().cpu())
    want = want.transpose(0, 1).reshape(heads, pages * page, d)[:, :33]
    assert torch.equal(out[0].cpu().double(), want)


def test_slots_out_of_range_are_skipped_and_flagged():
    x = rows(4, 2, 64, 4)
    caches, scales = empty_caches(2, 2, 16, 64, "e4m3")
    before = [c.clone() for c in caches], [s.clone() for s in scales]
    slots = torch.tensor([32, 5, 2 ** 40, -2 ** 40])
    atk.cache_write(*x.to(DEV), *caches, slots.to(DEV), k_scale=scales[0], v_scale=scales[1])
    check_written(x, slots, before, caches, scales, 16)
    assert atk.topk_device_status() == 2


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3 any scale"])
@pytest.mark.parametrize("heads,d,page,n", [(1, 64, 1, 5), (3, 128, 7, 40), (2, 256, 16, 33), (2, 128, 64, 1)])
def test_read(kind, heads, d, page, n):
    lens = [0, 1, n // 2, n, n + 9, -3]
    width = -(-(n + 9) // page)
    g = torch.Generator().manual_seed(n)
    pages = width * len(lens) + 2
    table = torch.randperm(pages, generator=g)[: width * len(lens)].view(len(lens), width).to(torch.int32)
    if kind == "bf16":
        cache, scale = torch.randn(pages, heads, page, d, generator=g).bfloat16(), None
    else:
        code = torch.randint(0, 256, (pages, heads, page, d), generator=g).to(torch.uint8)
        cache = torch.where(code & 0x7F == 0x7F, 3, code).to(torch.uint8).view(E4M3)
        scale = torch.exp2(torch.randint(-127, 100, (pages, heads, page), generator=g).float())
        if kind != "e4m3":
            scale = torch.rand(pages, heads, page, generator=g) + 0.5
    out = atk.cache_read(cache.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), n,
                         scale=None if scale is None else scale.to(DEV)).cpu()
    assert out.shape == (len(lens), heads, n, d) and out.dtype == torch.bfloat16
    for b, length in enumerate(lens):
        m = min(max(length, 0), n)
        for h in range(heads):
            want = torch.zeros(n, d, dtype=torch.float64)
            if m:
                want[:m] = ref.sequence_rows(cache, scale, table[b], range(m), h)
            # fp32 first (exact for powers of two above its subnormals), then bf16
            assert torch.equal(out[b, h].float(), want.float().bfloat16().float()), (b, h)
    assert atk.topk_device_status() == 0


def test_read_flags_bad_pages_and_lengths():
    cache = torch.randn(3, 1, 4, 64, device=DEV).bfloat16()
    table = torch.tensor([[0, -1, 2], [1, 3, -9]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([12, 4], dtype=torch.int32, device=DEV)
    out = atk.cache_read(cache, table, lens, 12)
    assert torch.equal(out[0, 0, :4], cache[0, 0]) and torch.equal(out[0, 0, 8:], cache[2, 0])
    assert bool((out[0, 0, 4:8] == 0).all()) and torch.equal(out[1, 0, :4], cache[1, 0])
    assert bool((out[1, 0, 4:] == 0).all())  # its other pages are behind its end and not looked at
    assert atk.topk_device_status() == 2
    out = atk.cache_read(cache, table[:1, ::2].contiguous(), torch.tensor([9], dtype=torch.int32, device=DEV), 10)
    assert torch.equal(out[0, 0, 4:8], cache[2, 0]) and bool((out[0, 0, 8:] == 0).all())
    assert atk.topk_device_status() == 2


def test_offsets_beyond_32_bits():
    pages = 18000  # of 8 heads x 64 tokens x 256 values: 2^31 elements lie on page 16384
    big = torch.empty(pages, 8, 64, 256, dtype=torch.bfloat16, device=DEV)
    other = torch.empty(4, 8, 64, 256, dtype=torch.bfloat16, device=DEV)
    x = rows(2, 8, 256, 6).to(DEV)
    slots = torch.tensor([17999 * 64 + 63, 16384 * 64])
    with pytest.raises(ValueError):
        atk.cache_write(x[0], x[1], big, other, slots.to(DEV))
    atk.cache_write(x[0], x[1], big, torch.empty_like(big), slots.to(DEV))
    assert torch.equal(big[17999, :, 63], x[0, 0]) and torch.equal(big[16384, :, 0], x[0, 1])
    table = torch.tensor([[16384], [17999]], dtype=torch.int32, device=DEV)
    out = atk.cache_read(big, table, torch.tensor([64, 64], dtype=torch.int32, device=DEV), 64)
    assert torch.equal(out[0, :, 0], x[0, 1]) and torch.equal(out[1, :, 63], x[0, 0])
    assert atk.topk_device_status() == 0


def test_in_a_graph_on_a_side_stream():
    tokens, heads, d, page = 16, 4, 128, 8
    caches, scales = empty_caches(4, heads, page, d, "e4m3")
    before = [c.clone() for c in caches], [s.clone() for s in scales]
    x = rows(tokens, heads, d, 8).to(DEV)
    slots = torch.arange(tokens, device=DEV)
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4)
    lens = torch.tensor([32], dtype=torch.int32, device=DEV)

    def step():
        atk.cache_write(x[0], x[1], *caches, slots, k_scale=scales[0], v_scale=scales[1])
        return atk.cache_read(caches[0], table, lens, 32, scale=scales[0])

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = step()
    new = rows(tokens, heads, d, 9)
    x.copy_(new)
    slots.copy_(torch.arange(tokens).flip(0) + 3)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    check_written(new, slots.cpu(), before, caches, scales, page)
    want = ref.decode_rows(caches[0].cpu(), scales[0].cpu()).transpose(0, 1).reshape(heads, 32, d)
    assert torch.equal(out[0].cpu().double(), want.float().bfloat16().double())
