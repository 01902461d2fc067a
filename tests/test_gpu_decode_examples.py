"""The README's examples of a decoding step, run as they stand on ragged
batches, and a beam search with pages of several tokens by its rule for pages
that beams share."""
import math
import os
import re

import pytest
import torch

import approximate_top_selection_b200 as atk
import decode_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA device")
    atk.load_library()
    torch.cuda.synchronize()
    atk.topk_device_status()
    yield


def example(call):
    """The README's Python block that makes `call`."""
    with open(README) as f:
        found = [b for b in re.findall(r"```python\n(.*?)```", f.read(), flags=re.S) if call in b]
    assert len(found) == 1
    return compile(found[0], "README.md", "exec")


def a_batch(lengths, heads, d=128, page_size=16, seed=1):
    """What the examples name: a filled e4m3 cache whose scores are mostly negative."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    batch, n = len(lengths), max(lengths)
    width = -(-n // page_size)
    pages = batch * width + 40
    e = dict(torch=torch, atk=atk, batch=batch, heads=heads, page_size=page_size, n=n, lengths=list(lengths), ks=None, vs=None)
    e["block_table"] = torch.randperm(pages - 40, generator=g, device=DEV)[: batch * width].view(batch, width).to(torch.int32)
    e["seq_lens"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    e["q"] = (torch.randn(batch, heads, d, generator=g, device=DEV) + 1).bfloat16()
    e["k_cache"], e["v_cache"] = (torch.zeros(pages, heads, page_size, d, device=DEV).to(E4M3) for _ in range(2))
    e["ks"], e["vs"] = (torch.ones(pages, heads, page_size, device=DEV) for _ in range(2))
    at = torch.cat([torch.arange(x, device=DEV) for x in lengths])
    of = torch.repeat_interleave(torch.arange(batch, device=DEV), torch.tensor(lengths, device=DEV))
    e["slots"] = e["block_table"][of, at // page_size].long() * page_size + at % page_size
    e["k_new"] = (torch.randn(len(at), heads, d, generator=g, device=DEV) - 1).bfloat16()
    e["v_new"] = torch.randn(len(at), heads, d, generator=g, device=DEV).bfloat16()
    atk.cache_write(e["k_new"], e["v_new"], e["k_cache"], e["v_cache"], e["slots"], k_scale=e["ks"], v_scale=e["vs"])
    beams, vocab = 4, 300
    e["beams"] = beams
    e["logits"] = torch.randn(batch, beams, vocab, generator=g, device=DEV)
    e["beam_scores"] = torch.zeros(batch, beams, device=DEV)
    return e


def test_selection_from_sequences_of_unlike_lengths(monkeypatch):
    lengths = [3000, 1200, 513, 512, 90, 1]
    e = a_batch(lengths, 4)
    called = []
    real = atk.paged_attention

    def recorded(*a, **kw):
        called.append((kw, real(*a, **kw)))
        return called[-1][1]

    monkeypatch.setattr(atk, "paged_attention", recorded)
    exec(example("atk.cache_read("), e)
    kw, out = [c for c in called if c[0].get("positions") is not None][-1]
    pos = kw["positions"]
    live = (pos >= 0) & (pos < e["seq_lens"].view(-1, 1, 1))
    assert torch.equal(live, pos >= 0), "padding was selected"
    want = torch.tensor([min(512, x) for x in lengths], device=DEV)
    assert torch.equal(live.sum(2), want.view(-1, 1).expand(-1, 4))
    o, _, mass, size = ref.attention(*(e[x].cpu() for x in ("q", "k_cache", "v_cache", "block_table", "seq_lens")), 128 ** -0.5,
                                     e["ks"].cpu(), e["vs"].cpu(), pos.cpu())
    # as in test_gpu_paged_attention: bf16's rounding, d products summed in fp32, weights of 11 bits
    tol = 2.0 ** -8 * o.abs() + (4 * size[..., None] * 128 * 2.0 ** -24 + 2.0 ** -10) * mass
    assert bool(((out.cpu().double() - o).abs() <= tol).all())
    assert atk.topk_device_status() == 0


def test_beam_step():
    e = a_batch([70] * 12, 4)  # three sentences of four beams
    e["batch"], beams = 3, e["beams"]
    e["n"], page = 70, e["page_size"]
    e["logits"], e["beam_scores"] = e["logits"][:3].contiguous(), e["beam_scores"][:3].contiguous()
    e["block_table"] = e["block_table"].view(3, beams, -1)
    e["history"] = torch.arange(3 * beams * 80, device=DEV).view(3, beams, 80)
    e["fresh"] = torch.arange(e["k_cache"].shape[0] - 40, e["k_cache"].shape[0] - 40 + 3 * beams, device=DEV)
    before = {x: e[x].clone() for x in ("block_table", "history")}

    def keys(table):
        return atk.cache_read(e["k_cache"], table.view(3 * beams, -1), e["seq_lens"], 70, scale=e["ks"]).view(3, beams, 4, 70, 128)

    old = keys(before["block_table"])
    exec(example("atk.beam_reorder("), e)
    p, b = e["parents"].long(), torch.arange(3, device=DEV).view(3, 1)
    assert torch.equal(e["history"], before["history"][b, p])
    assert torch.equal(keys(e["block_table"]), old[b, p])
    last = e["block_table"][:, :, 70 // page]
    assert last.unique().numel() == last.numel(), "two beams write into one page"
    assert atk.topk_device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_beam_search_with_pages_of_several_tokens_equals_recomputing(kind):
    batch, beams, heads, kv_heads, d, vocab, steps, page = 3, 4, 4, 2, 64, 401, 11, 4
    g = torch.Generator(device=DEV).manual_seed(11)
    emb = torch.randn(vocab, heads * d, generator=g, device=DEV)
    wq, wk, wv = (torch.randn(heads * d, m * d, generator=g, device=DEV) / 16 for m in (heads, kv_heads, kv_heads))
    wo = torch.randn(heads * d, vocab, generator=g, device=DEV) / 4
    rows = batch * beams
    pages = rows * (steps + 1)
    dtype = torch.bfloat16 if kind == "bf16" else E4M3
    kc, vc = (torch.zeros(pages, kv_heads, page, d, device=DEV).to(dtype) for _ in range(2))
    ks, vs = (torch.ones(pages, kv_heads, page, device=DEV) for _ in range(2)) if kind == "e4m3" else (None, None)
    table = torch.zeros(batch, beams, -(-steps // page), dtype=torch.int32, device=DEV)
    history = torch.zeros(batch, beams, steps, dtype=torch.int32, device=DEV)
    token = torch.arange(batch, device=DEV).view(batch, 1).expand(batch, beams).contiguous()
    scores = torch.full((batch, beams), -math.inf, device=DEV)
    scores[:, 0] = 0.0
    shared = 0
    for step in range(steps):
        history[:, :, step] = token
        fresh = torch.arange(rows, device=DEV) + step * rows
        if step % page:  # a page with room: beams that share it take copies
            last = table[:, :, step // page].flatten().long()
            shared += last.numel() - last.unique().numel()
            for t in (kc.view(torch.uint8), vc.view(torch.uint8)) + (() if ks is None else (ks, vs)):
                t[fresh] = t[last]
        table[:, :, step // page] = fresh.view(batch, beams)
        x = emb[token.view(rows)]
        q, k, v = ((x @ w).bfloat16().view(rows, -1, d) for w in (wq, wk, wv))
        atk.cache_write(k, v, kc, vc, fresh * page + step % page, k_scale=ks, v_scale=vs)
        lens = torch.full((rows,), step + 1, dtype=torch.int32, device=DEV)
        o = atk.paged_attention(q, kc, vc, table.view(rows, -1), lens, k_scale=ks, v_scale=vs)
        hist = history[:, :, : step + 1].long().view(rows, step + 1)
        kk, vv = ((emb[hist] @ w).bfloat16().view(rows, step + 1, kv_heads, d) for w in (wk, wv))
        if kind == "e4m3":  # as a cache of its own keeps them
            own = [torch.zeros(rows, kv_heads, step + 1, d, device=DEV).to(E4M3) for _ in range(2)]
            sc = [torch.ones(rows, kv_heads, step + 1, device=DEV) for _ in range(2)]
            flat = [t.reshape(rows * (step + 1), kv_heads, d) for t in (kk, vv)]
            atk.cache_write(*flat, *own, torch.arange(rows * (step + 1), device=DEV), k_scale=sc[0], v_scale=sc[1])
            kk, vv = ((c.float() * s[..., None]).transpose(1, 2) for c, s in zip(own, sc))
        kk, vv = (t.double().repeat_interleave(heads // kv_heads, 2) for t in (kk, vv))
        p = torch.softmax(torch.einsum("rhd,rnhd->rhn", q.double(), kk) / math.sqrt(d), 2)
        want = torch.einsum("rhn,rnhd->rhd", p, vv)
        mass = torch.einsum("rhn,rnhd->rhd", p, vv.abs())
        # half a bf16 step of |o|; weights of 11 bits beside codes; fp32 arithmetic of at most 11 values below 16
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -12 + (2.0 ** -11 * mass if kind == "e4m3" else 0.0)
        assert bool(((o.double() - want).abs() <= tol).all()), step
        logits = torch.tanh(o.float().view(rows, -1) @ wo).view(batch, beams, vocab) * 4
        scores, parent, token = atk.topk_beam(logits, scores, beams)
        token = token.long()
        table, history = atk.beam_reorder([table, history], parent)
    assert shared > 0  # beams did share pages
    assert atk.topk_device_status() == 0
