"""paged_attention on the GPU against the 64-bit form.

Bound on an output o = sum_j p_j V_j, per element, with u = 2^-24 (fp32):
  - rounding to bf16: half a step, 2^-8 |o|;
  - a score's error e (absolute, in the exponent) moves every p_j by a factor
    within 1 +- 2e: its d products are summed in fp32, by tensor cores in an
    order and with a truncation of their own, d * 2u of the sum of magnitudes
    at most, which is at most scale |q||K_j|;
  - exp2 of the hardware is within 2^-21 relatively, the weights a product
    takes are rounded to 2^-11 at worst (f16 beside e4m3 codes; two bf16 parts
    beside bf16 values leave 2^-16);
  - the sum of n terms and of the joined parts: n * 2u;
all of these relative to sum_j p_j |V_j|.  The log-sum-exp has the score's
error, that of the sum and of exp2 and log2, and its own rounding.
"""
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


def make(batch, heads, kv_heads, d, page, lens, kind, seed, spare=3, poison=True):
    """CPU tensors of a call; pages no sequence uses and rows behind a
    sequence's end hold NaN and infinity."""
    g = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-n // page) for n in lens))
    pages = batch * width + spare
    table = torch.randperm(pages, generator=g)[: batch * width].view(batch, width).to(torch.int32)
    s = dict(q=torch.randn(batch, heads, d, generator=g).bfloat16(), table=table,
             lens=torch.tensor(lens, dtype=torch.int32), k_scale=None, v_scale=None)
    live = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            live[table[b, t // page], t % page] = True
    for n in "kv":
        x = torch.randn(pages, kv_heads, page, d, generator=g).bfloat16()
        dead = torch.where(torch.rand(x.shape, generator=g) < 0.5, math.nan, math.inf).bfloat16()
        mask = live[:, None, :, None]
        if kind == "bf16":
            s[n + "_cache"] = torch.where(mask, x, dead) if poison else x
        else:
            code = (x.float() * 100).clamp(-448, 448).to(E4M3)
            sc = torch.exp2(torch.randint(-9, -5, (pages, kv_heads, page), generator=g).float())
            sc = sc * (1 + torch.randint(0, 2, sc.shape, generator=g))
            if poison:
                code = torch.where(mask, code.view(torch.uint8), torch.tensor(0x7F, dtype=torch.uint8)).view(E4M3)
                sc = torch.where(mask[..., 0], sc, math.nan)
            s[n + "_cache"], s[n + "_scale"] = code, sc
    return s


def on_gpu(s):
    return {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in s.items()}


def call(s, **kw):
    return atk.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], k_scale=s["k_scale"],
                               v_scale=s["v_scale"], positions=s.get("positions"), return_lse=True, **kw)


def check(s, got, scale=None):
    out, lse = (t.cpu().double() for t in got)
    d = s["q"].shape[2]
    scale = d ** -0.5 if scale is None else scale
    o, l, mass, size = ref.attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], scale, s["k_scale"],
                                     s["v_scale"], s.get("positions"))
    n = s["positions"].shape[2] if s.get("positions") is not None else int(s["lens"].max())
    u = 2.0 ** -24
    score = (size * (d * 2 * u + 2 * u))[..., None]
    weights = 2.0 ** -11 if s["k_scale"] is not None else 2.0 ** -16
    tol = 2.0 ** -8 * o.abs() + (2 * score + 2.0 ** -20 + weights + 2 * u * (n + 64)) * mass
    assert torch.equal(torch.isnan(out), torch.isnan(o))
    fine = ~torch.isnan(o)
    assert bool(((out - o).abs() <= tol)[fine].all()), float(((out - o).abs() / tol)[fine].max())
    assert torch.equal(torch.isnan(lse), torch.isnan(l))
    assert torch.equal(lse == -math.inf, l == -math.inf)
    fine = torch.isfinite(l)
    tol = score[..., 0] + 2.0 ** -20 + 2 * u * (n + 64) + 4 * u * l.abs()
    assert bool(((lse - l).abs() <= tol)[fine].all()), float(((lse - l).abs() / tol)[fine].max())


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 300]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads,page", [(4, 4, 16), (8, 2, 7), (5, 1, 1), (16, 1, 64), (40, 2, 300)])
def test_whole_sequences(kind, d, heads, kv_heads, page):
    s = make(len(LENS), heads, kv_heads, d, page, LENS, kind, d + heads)
    check(s, call(on_gpu(s)))
    assert atk.topk_device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("batch,heads,kv_heads,d,page,longest", [
    (1, 8, 1, 128, 16, 5000),   # one row of work over many CTAs
    (1, 1, 1, 64, 16, 9001),
    (3, 6, 2, 256, 32, 2111),
    (2, 64, 2, 128, 24, 1500),  # 32 query heads to one of keys
    (37, 4, 2, 128, 16, 400),
])
def test_split_sequences(kind, batch, heads, kv_heads, d, page, longest):
    lens = [max(1, int(longest * (1 - (i * 0.618) % 1))) for i in range(batch)]
    s = make(batch, heads, kv_heads, d, page, lens, kind, longest)
    check(s, call(on_gpu(s)))
    assert atk.topk_device_status() == 0


def test_many_short_sequences():
    lens = [(i * 7) % 23 for i in range(700)]
    s = make(700, 2, 1, 64, 8, lens, "bf16", 11)
    check(s, call(on_gpu(s)))
    assert atk.topk_device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("batch,heads,kv_heads,d,page,longest", [
    (50, 16, 16, 64, 16, 47),
    (50, 16, 16, 128, 12, 47),
    (35, 36, 18, 256, 5, 40),
    (9, 40, 2, 128, 3, 11),      # three groups of a key head's 20 query heads
    (3, 700, 350, 64, 7, 33),
    (2, 512, 256, 256, 1, 30),
])
def test_many_short_units(kind, batch, heads, kv_heads, d, page, longest):
    lens = [(i * 13) % (longest + 1) for i in range(batch - 1)] + [longest]
    s = make(batch, heads, kv_heads, d, page, lens, kind, longest + d)
    got = call(on_gpu(s))
    check(s, got)
    again = call(on_gpu(s))
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    assert atk.topk_device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,kv_heads,lists,d,c,batch", [(250, 5, 250, 128, 70, 30), (256, 2, 128, 64, 150, 60),
                                                            (600, 3, 300, 256, 37, 17), (288, 2, 24, 128, 33, 200)])
def test_many_lists(kind, heads, kv_heads, lists, d, c, batch):
    g = torch.Generator().manual_seed(c)
    lens = [(i * 37) % 101 for i in range(batch)]
    s = make(batch, heads, kv_heads, d, 8, lens, kind, c + d)
    s["positions"] = torch.randint(-1, 104, (batch, lists, c), generator=g, dtype=torch.int32)
    check(s, call(on_gpu(s)))
    # positions behind a sequence's end are left out; those behind its table's end are also reported
    beyond = bool((s["positions"] >= s["table"].shape[1] * 8).any())
    assert atk.topk_device_status() == (2 if beyond else 0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,kv_heads,lists,d,c", [(8, 2, 2, 128, 50), (8, 2, 8, 128, 33), (8, 2, 4, 64, 1),
                                                      (4, 4, 4, 256, 200), (32, 1, 1, 128, 700)])
def test_listed_positions(kind, heads, kv_heads, lists, d, c):
    g = torch.Generator().manual_seed(c)
    lens = [0, 1, 40, 333]
    s = make(4, heads, kv_heads, d, 16, lens, kind, c + d)
    pos = torch.randint(-2, 333, (4, lists, c), generator=g).to(torch.int32)
    pos[3, 0] = -1              # a list that names nothing
    pos[2, -1, : c // 2] = 7    # a position named again and again
    s["positions"] = pos
    check(s, call(on_gpu(s)))
    assert atk.topk_device_status() == 0


def test_positions_in_any_order_and_alignment_agree_with_whole_sequences():
    s = make(2, 8, 4, 128, 16, [257, 100], "bf16", 5)
    whole = call(on_gpu(s))
    perm = torch.stack([torch.randperm(260, generator=torch.Generator().manual_seed(i)) for i in range(8)])
    s["positions"] = perm.view(2, 4, 260).to(torch.int32)
    check(s, call(on_gpu(s)))
    check({**s, "positions": None}, whole)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["interleaved", "tokens_first"])
def test_strided_caches_and_queries(kind, layout):
    s = make(5, 8, 2, 128, 16, [1, 16, 50, 200, 0], kind, 77)
    g = on_gpu(s)
    if layout == "interleaved":  # keys and values of a page side by side
        both = torch.stack([s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)], 1).to(DEV)
        both = both.view(s["k_cache"].dtype)
        g["k_cache"], g["v_cache"] = both[:, 0], both[:, 1]
        if kind == "e4m3":
            sc = torch.stack([s["k_scale"], s["v_scale"]], 1).to(DEV)
            g["k_scale"], g["v_scale"] = sc[:, 0], sc[:, 1]
    else:  # [pages, page, kv_heads, d] memory
        for n in "kv":
            x = g[n + "_cache"].view(torch.uint8).transpose(1, 2).contiguous().view(s["k_cache"].dtype)
            g[n + "_cache"] = x.transpose(1, 2)
            if kind == "e4m3":
                g[n + "_scale"] = g[n + "_scale"].transpose(1, 2).contiguous().transpose(1, 2)
    assert not g["k_cache"].is_contiguous()
    qkv = torch.zeros(5, 12, 128, dtype=torch.bfloat16, device=DEV)
    qkv[:, 2:10] = g["q"]
    g["q"] = qkv[:, 2:10]
    wide = torch.full((5, 40), -5, dtype=torch.int32, device=DEV)
    wide[:, : s["table"].shape[1]] = g["table"]
    g["table"] = wide[:, : s["table"].shape[1]]
    check(s, call(g))
    assert atk.topk_device_status() == 0


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_other_scales(scale):
    s = make(2, 4, 2, 64, 16, [40, 100], "bf16", 8)
    check(s, call(on_gpu(s), scale=scale), scale)


def test_large_scores_and_rows_of_infinity():
    s = make(4, 2, 1, 64, 16, [100, 100, 100, 3], "bf16", 9, poison=False)
    s["q"][0] *= 300                        # one key takes all the weight
    s["q"][1] = 0
    s["q"][2, 0, 0] = math.nan              # one head undefined, the other not
    at = s["table"][3, 0]
    s["q"][3] = 1.0
    s["k_cache"][at, 0, :3] = -math.inf     # every score -inf
    got = call(on_gpu(s))
    check(s, got)
    out, lse = got
    assert bool((out[3] == 0).all()) and bool((lse[3] == -math.inf).all())
    assert bool(torch.isnan(out[2, 0]).all()) and not bool(torch.isnan(out[2, 1]).any())


def test_small_and_large_e4m3_queries():
    """Queries far outside f16's range keep their precision beside e4m3 keys."""
    s = make(4, 4, 2, 64, 16, [70, 70, 70, 70], "e4m3", 10)
    s["q"][0] *= 2.0 ** 60
    s["q"][1] *= 2.0 ** -60
    s["q"][2, :, ::2] *= 2.0 ** -12
    s["k_scale"] = s["k_scale"].clone()
    got = call(on_gpu(s), scale=2.0 ** -63)
    check(s, got, 2.0 ** -63)
    check(s, call(on_gpu(s), scale=2.0 ** 57), 2.0 ** 57)


def test_bad_pages_lengths_and_positions_are_flagged():
    s = make(3, 4, 2, 128, 16, [40, 64, 5], "bf16", 12)
    s["table"][0, 1] = -1          # the middle page of a sequence
    s["table"][1, 3] = 10 ** 6
    check(s, call(on_gpu(s)))
    assert atk.topk_device_status() == 2
    s = make(2, 4, 2, 128, 16, [64, 30], "bf16", 13)
    full = dict(s, lens=torch.tensor([5000, -7], dtype=torch.int32))
    check(full, call(on_gpu(full)))
    assert atk.topk_device_status() == 2
    s["positions"] = torch.tensor([[[3, 64, 5]] * 2, [[29, 40, 30]] * 2], dtype=torch.int32)  # 64: behind the table
    check(s, call(on_gpu(s)))
    assert atk.topk_device_status() == 2
    s["positions"] = torch.tensor([[[3, -1, 5]] * 2, [[29, 40, 30]] * 2], dtype=torch.int32)  # 40: behind the sequence
    check(s, call(on_gpu(s)))
    assert atk.topk_device_status() == 0


def test_offsets_beyond_32_bits():
    pages, page, d = 18000, 64, 256  # 2^31 elements lie on page 16384 of 8 heads
    table = torch.tensor([[17999, 3, 16383], [16384, 17998, 0]], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    small = make(2, 8, 8, d, page, [150, 192], "bf16", 14)
    big = {}
    for n in "kv":
        big[n] = torch.empty(pages, 8, page, d, dtype=torch.bfloat16, device=DEV)
        for b in range(2):
            for i in range(3):
                big[n][table[b, i]] = small[n + "_cache"][small["table"][b, i]].to(DEV)
    out = atk.paged_attention(small["q"].to(DEV), big["k"], big["v"], table.to(DEV), small["lens"].to(DEV),
                              return_lse=True)
    check(small, out)
    assert atk.topk_device_status() == 0


def test_given_outputs_side_stream_and_workspace():
    s = make(3, 8, 2, 128, 16, [3000, 10, 700], "bf16", 15)
    g = on_gpu(s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(3, 8, device=DEV)
    need = atk.paged_attention_workspace_bytes(3, 8, 0, 128)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    got = call(g, out=out, out_lse=lse, workspace=ws, stream=side)
    side.synchronize()
    assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    check(s, got)
    got2 = call(g, stream=side)
    side.synchronize()
    assert torch.equal(got2[0], out) and torch.equal(got2[1], lse)
    if need:
        with pytest.raises(atk.TopkError) as e:
            call(g, workspace=ws[: need - 16])
        assert e.value.status == atk.TOPK_EWORKSPACE


def test_the_same_call_gives_the_same_bits():
    s = make(3, 8, 2, 128, 16, [3000, 10, 700], "e4m3", 16)
    g = on_gpu(s)
    first = call(g)
    for _ in range(5):
        again = call(g)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_two_graphs_replayed_side_by_side():
    """Graphs captured on one stream and replayed on two at once, with lengths
    that change between replays, agree with eager calls."""
    cases = [on_gpu(make(2, 8, 2, 128, 16, [4000, 900], "bf16", 20 + i)) for i in range(2)]
    stream = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(stream):
        for s in cases:
            call(s)
    torch.cuda.synchronize()
    for s in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append(call(s))
        graphs.append(g)
    sides = [torch.cuda.Stream() for _ in cases]
    for lens in ([4000, 900], [100, 3999], [1, 0], [2500, 700]):  # 3999 reaches poisoned rows: NaN on both sides
        for s in cases:
            s["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(20):
            for g, side in zip(graphs, sides):
                with torch.cuda.stream(side):
                    g.replay()
        torch.cuda.synchronize()
        for s, o in zip(cases, outs):
            want = call(s)
            assert torch.equal(o[0].view(torch.int16), want[0].view(torch.int16))
            assert torch.equal(o[1].view(torch.int32), want[1].view(torch.int32))
    assert atk.topk_device_status() == 0


@pytest.mark.parametrize("asked", [True, 1, False, 0])
def test_return_lse_by_truth(asked):
    s = on_gpu(make(1, 2, 1, 64, 8, [9], "bf16", 3))
    args = (s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"])
    for kw in ({}, {"stream": torch.cuda.current_stream()}):
        got = atk.paged_attention(*args, return_lse=asked, **kw)
        assert isinstance(got, tuple) == bool(asked)
