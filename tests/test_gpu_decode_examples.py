"""The README's examples of a decoding step, run as they stand."""
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
