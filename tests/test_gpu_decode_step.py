"""The decoding step's operators together, as a decoding loop calls them: new
keys and values written into the paged cache, the cache read back for the
selector, attention over what the selector chose, and a beam step whose
parents reorder the beams' page tables, lengths and dense states."""
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


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_write_read_select_attend(kind):
    batch, heads, d, page, n, k = 2, 4, 128, 16, 1024, 128
    g = torch.Generator(device=DEV).manual_seed(1)
    width = n // page
    pages = batch * width + 1
    table = torch.randperm(pages, generator=g, device=DEV)[: batch * width].view(batch, width).to(torch.int32)
    lens = torch.full((batch,), n, dtype=torch.int32, device=DEV)
    dtype = torch.bfloat16 if kind == "bf16" else E4M3
    kc, vc = (torch.zeros(pages, heads, page, d, device=DEV).to(dtype) for _ in range(2))
    ks, vs = (torch.zeros(pages, heads, page, device=DEV) for _ in range(2)) if kind == "e4m3" else (None, None)
    new = torch.randn(2, batch * n, heads, d, generator=g, device=DEV).bfloat16()
    at = torch.arange(n, device=DEV)
    slots = (table[:, at // page].long() * page + at % page).flatten()
    for part in range(0, batch * n, 700):  # a prompt in pieces
        c = slice(part, part + 700)
        atk.cache_write(new[0, c], new[1, c], kc, vc, slots[c], k_scale=ks, v_scale=vs)
    keys = atk.cache_read(kc, table, lens, n, scale=ks).view(batch * heads, n, d)
    if kind == "bf16":
        assert torch.equal(keys.view(batch, heads, n, d), new[0].view(batch, n, heads, d).transpose(1, 2))
    q = torch.randn(batch, heads, d, generator=g, device=DEV).bfloat16()
    score, idx = atk.score_topk(q.view(batch * heads, d), keys, k, 64, 2)
    out, lse = atk.paged_attention(q, kc, vc, table, lens, k_scale=ks, v_scale=vs,
                                   positions=idx.view(batch, heads, k), return_lse=True)
    # the selector's scores are the attention's: the log-sum-exp over the selection follows from them
    want = torch.logsumexp(score.double() * d ** -0.5, 1).view(batch, heads)
    assert bool(((lse.double() - want).abs() <= 1e-4).all())  # sums of 128 products in two orders: 128 * 2^-23 * |q||k| d^-1/2
    s = dict(q=q.cpu(), k_cache=kc.cpu(), v_cache=vc.cpu(), table=table.cpu(), lens=lens.cpu())
    o, l, mass, size = ref.attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], d ** -0.5,
                                     None if ks is None else ks.cpu(), None if vs is None else vs.cpu(),
                                     idx.view(batch, heads, k).cpu())
    tol = 2.0 ** -8 * o.abs() + (4 * size[..., None] * d * 2.0 ** -24 + 2.0 ** -10) * mass
    assert bool(((out.cpu().double() - o).abs() <= tol).all())
    assert atk.topk_device_status() == 0


def _model(hidden, w):
    """A stand-in for a model: the same arithmetic for both loops below."""
    return torch.tanh(hidden @ w)


def test_beam_search_over_a_paged_cache_equals_recomputing():
    """Six steps of beam search.  One loop keeps a paged cache with pages of one
    token, whose tables are reordered; the other recomputes every beam from its
    tokens alone.  Both must follow the same beams."""
    batch, beams, heads, kv_heads, d, vocab, steps = 3, 4, 4, 2, 64, 401, 6
    g = torch.Generator(device=DEV).manual_seed(7)
    emb = torch.randn(vocab, heads * d, generator=g, device=DEV)
    wq, wk, wv = (torch.randn(heads * d, m * d, generator=g, device=DEV) / 16 for m in (heads, kv_heads, kv_heads))
    wo = torch.randn(heads * d, vocab, generator=g, device=DEV) / 4
    rows = batch * beams
    pages = rows * (steps + 1)
    kc, vc = (torch.zeros(pages, kv_heads, 1, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.zeros(batch, beams, steps + 1, dtype=torch.int32, device=DEV)
    history = torch.zeros(batch, beams, steps + 1, dtype=torch.int32, device=DEV)
    token = torch.arange(batch, device=DEV).view(batch, 1).expand(batch, beams).contiguous()
    scores = torch.full((batch, beams), -math.inf, device=DEV)
    scores[:, 0] = 0.0
    for step in range(steps):
        history[:, :, step] = token
        page = torch.arange(rows, device=DEV) + step * rows   # every beam's new token gets a page of its own
        table[:, :, step] = page.view(batch, beams)
        x = emb[token.view(rows)]
        q, k, v = ((x @ w).bfloat16().view(rows, -1, d) for w in (wq, wk, wv))
        atk.cache_write(k, v, kc, vc, page)
        lens = torch.full((rows,), step + 1, dtype=torch.int32, device=DEV)
        o = atk.paged_attention(q, kc, vc, table.view(rows, -1), lens)
        logits = _model(o.float().view(rows, -1), wo).view(batch, beams, vocab) * 4
        # the other loop: attention of the last token over the beam's own tokens
        hist = history[:, :, : step + 1].long().view(rows, step + 1)
        kk, vv = ((emb[hist] @ w).bfloat16().view(rows, step + 1, kv_heads, d).double() for w in (wk, wv))
        kk, vv = (t.repeat_interleave(heads // kv_heads, 2) for t in (kk, vv))
        p = torch.softmax(torch.einsum("rhd,rnhd->rhn", q.double(), kk) / math.sqrt(d), 2)
        want = torch.einsum("rhn,rnhd->rhd", p, vv)
        # half a bf16 step of |o| and the fp32 arithmetic of at most 6 weights of values below 16
        assert bool(((o.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12).all()), step
        new, parent, token = atk.topk_beam(logits, scores, beams)
        lp = torch.log_softmax(logits.double(), 2) + scores.double()[..., None]
        best = lp.flatten(1).topk(beams, dim=1).values
        assert bool(((new.double() - best).abs() <= 2.0 ** -14).all()), step
        for b in range(batch):
            for j in range(beams):
                i, t = int(parent[b, j]), int(token[b, j])
                assert abs(float(lp[b, i, t]) - float(new[b, j])) <= 2.0 ** -14
        table, history = atk.beam_reorder([table, history], parent)
        scores, token = new, token.long()
    assert atk.topk_device_status() == 0


def _attention_case(seed, lens):
    g = torch.Generator(device=DEV).manual_seed(seed)
    batch, page = len(lens), 16
    width = -(-max(lens) // page)
    q = torch.randn(batch, 8, 128, generator=g, device=DEV).bfloat16()
    k, v = (torch.randn(batch * width, 2, page, 128, generator=g, device=DEV).bfloat16() for _ in range(2))
    table = torch.randperm(batch * width, generator=g, device=DEV).view(batch, width).to(torch.int32)
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def test_eager_calls_side_by_side_on_two_streams():
    """Both split work over the GPU and use their stream's workspace at the same time."""
    cases = [_attention_case(i, [5000, 3000]) for i in range(2)]
    beams = [(torch.randn(2, 4, 50000, device=DEV), torch.zeros(2, 4, device=DEV)) for _ in range(2)]
    want = [(atk.paged_attention(*c), atk.topk_beam(*b, 8)) for c, b in zip(cases, beams)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(25):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((atk.paged_attention(*cases[i]), atk.topk_beam(*beams[i], 8)))
    torch.cuda.synchronize()
    for i in range(2):
        for o, b in got[i]:
            assert torch.equal(o, want[i][0])
            assert all(torch.equal(x, y) for x, y in zip(b, want[i][1]))


def test_one_workspace_for_attention_and_beam_search_in_turn():
    c = _attention_case(3, [4000, 17, 900])
    x, s = torch.randn(3, 4, 70000, device=DEV), torch.zeros(3, 4, device=DEV)
    need = max(atk.paged_attention_workspace_bytes(3, 8, 0, 128), atk.topk_beam_workspace_bytes(3, 4, 70000, 8))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    ws[16384:] = 0xFF  # only the first bytes have to be zero
    o, b = atk.paged_attention(*c), atk.topk_beam(x, s, 8)
    for _ in range(3):
        assert torch.equal(atk.paged_attention(*c, workspace=ws), o)
        assert all(torch.equal(p, w) for p, w in zip(atk.topk_beam(x, s, 8, workspace=ws), b))
        assert bool((ws[:16384] == 0).all())


def test_one_query_for_all_sequences_and_one_table():
    """Tensors broadcast over the batch: strides of zero."""
    q, k, v, table, lens = _attention_case(4, [700, 700, 700])
    lens.copy_(torch.tensor([700, 33, 0]))
    one, row = q[:1].expand(3, 8, 128), table[:1].expand(3, -1)
    got = atk.paged_attention(one, k, v, row, lens)
    want = atk.paged_attention(one.contiguous(), k, v, row.contiguous(), lens)
    assert torch.equal(got, want) and bool((got[2] == 0).all())


def test_calls_with_everything_given_equal_the_usual_ones():
    """The extension module's calls and the ones made step by step (a stream or an output given)."""
    c = _attention_case(5, [2000, 100])
    x, s = torch.randn(2, 4, 30001, device=DEV).bfloat16(), torch.zeros(2, 4, device=DEV)
    here = torch.cuda.current_stream()
    pos = torch.randint(-1, 2000, (2, 8, 77), device=DEV, dtype=torch.int32)
    a, b = (atk.paged_attention(*c, positions=pos, return_lse=True, **kw) for kw in ({}, {"stream": here}))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = (atk.paged_attention(*c, scale=kw.pop("scale"), **kw) for kw in ({"scale": 0.5}, {"scale": 0.5, "stream": here}))
    assert torch.equal(a, b) and torch.equal(a, atk.paged_attention(*c, scale=torch.tensor(0.5).item()))
    a, b = (atk.cache_read(c[1], c[3], c[4], 50, **kw) for kw in ({}, {"stream": here}))
    assert torch.equal(a, b)
    a, b = (atk.topk_beam(x, s, 8, **kw) for kw in ({}, {"stream": here}))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    par = a[1][:, :4].contiguous()
    a, b = (atk.beam_reorder([x, s], par, **kw) for kw in ({}, {"stream": here}))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    new = torch.randn(9, 2, 128, device=DEV).bfloat16()
    slots = torch.randperm(c[1].shape[0] * 16, device=DEV)[:9]
    k1, v1, k2, v2 = (t.clone() for t in (c[1], c[2], c[1], c[2]))
    atk.cache_write(new, new, k1, v1, slots)
    atk.cache_write(new, new, k2, v2, slots, stream=here)
    assert torch.equal(k1, k2) and torch.equal(v1, v2) and not torch.equal(k1, c[1])


def test_many_units_and_rows_captured_and_replayed():
    """Short sequences by whole warps and a streaming beam step in one graph;
    other lengths, queries and logits are in place at the second replay."""
    g = torch.Generator().manual_seed(21)
    batch, heads, page, width = 160, 8, 16, 3
    q = torch.randn(batch, heads, 128, generator=g).bfloat16().cuda()
    k, v = (torch.randn(batch * width, 8, page, 128, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.randperm(batch * width, generator=g).view(batch, width).to(torch.int32).cuda()
    lens = torch.randint(0, page * width + 1, (batch,), generator=g, dtype=torch.int32).cuda()
    logits, scores = torch.randn(160, 2, 5003, generator=g).cuda(), torch.randn(160, 2, generator=g).cuda()

    def step():
        return [*atk.paged_attention(q, k, v, table, lens, return_lse=True), *atk.topk_beam(logits, scores, 4)]

    first = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, first))
    q.copy_(q.roll(1, 0))
    lens.copy_(lens.flip(0))
    logits.copy_(logits.roll(7, 2))
    second = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, second))
    assert not torch.equal(first[0], second[0]) and not torch.equal(first[4], second[4])
    assert atk.topk_device_status() == 0
