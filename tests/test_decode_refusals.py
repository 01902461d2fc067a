"""What the decoding step's operators refuse, on the host, without a GPU: the
C entries return a status before they touch CUDA, and the binding raises."""
import ctypes

import pytest
import torch

import approximate_top_selection_b200 as atk
from approximate_top_selection_b200 import _binding, build

P = 4096  # never dereferenced: validation fails first
E, U = atk.TOPK_EINVAL, atk.TOPK_EUNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return atk.load_library()


def cache(**kw):
    a = dict(data=P, scale=None, pages=4, kv_heads=2, page_size=16, d=128, type=0, page_stride=4096, head_stride=2048,
             token_stride=128, scale_page_stride=32, scale_head_stride=16, scale_token_stride=1)
    a.update(kw)
    return ctypes.byref(_binding.TopkCache(*[a[n] for n, _ in _binding.TopkCache._fields_]))


BAD_CACHES = [
    (dict(data=None), E), (dict(data=P + 8), E), (dict(pages=0), E), (dict(pages=2 ** 31), U), (dict(kv_heads=0), E),
    (dict(page_size=0), E), (dict(d=0), E), (dict(d=96), U), (dict(d=512), U), (dict(type=2), E), (dict(type=-1), E),
    (dict(token_stride=129), E), (dict(head_stride=-128), E), (dict(page_stride=2 ** 51), E),
    (dict(type=1), E),                                # e4m3 without a scale
    (dict(type=1, scale=P + 2), E), (dict(type=1, scale=P, scale_token_stride=-1), E),
    (dict(type=1, scale=P, token_stride=136), E),     # 136 bytes: no multiple of 16
]


def attend(lib, k=None, v=None, **kw):
    a = dict(q=P, q_stride=1024, batch=2, heads=8, table=P, table_stride=4, width=4, lens=P, positions=None, lists=0,
             c=0, scale=0.1, out=P, lse=None, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.paged_attention(a["q"], a["q_stride"], a["batch"], a["heads"], k or cache(), v or cache(), a["table"],
                               a["table_stride"], a["width"], a["lens"], a["positions"], a["lists"], a["c"], a["scale"],
                               a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_caches(lib, bad, status):
    c = cache(**bad)
    assert attend(lib, k=c) == status
    assert attend(lib, v=c) == status
    assert lib.cache_write(P, 256, 128, P, 256, 128, 3, c, cache(), P, None) == status
    assert lib.cache_write(P, 256, 128, P, 256, 128, 3, cache(), c, P, None) == status
    assert lib.cache_read(c, P, 4, 4, P, 2, 10, P, None) == status


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), E), (dict(out=None), E), (dict(table=None), E), (dict(lens=None), E), (dict(batch=0), E),
    (dict(batch=2 ** 31), U), (dict(batch=2 ** 29), U), (dict(width=0), E), (dict(table_stride=-1), E), (dict(heads=0), E),
    (dict(heads=7), E), (dict(q=P + 2), E), (dict(out=P + 2), E), (dict(q_stride=1025), E), (dict(q_stride=-8), E),
    (dict(scale=float("nan")), E), (dict(scale=float("inf")), E), (dict(lists=2, c=4), E),
    (dict(positions=P, lists=0, c=4), E), (dict(positions=P, lists=2, c=0), E), (dict(positions=P, lists=3, c=4), E),
    (dict(positions=P, lists=16, c=4), E), (dict(positions=P, lists=1, c=4), E),
])
def test_attention(lib, bad, status):
    assert attend(lib, **bad) == status


@pytest.mark.parametrize("scale", [float("inf"), float("nan"), 3e38, -3e38])
def test_attention_refuses_a_scale_without_log2(lib, scale):
    assert attend(lib, scale=scale) == E


def test_attention_refuses_unlike_caches(lib):
    for other in (dict(pages=5), dict(kv_heads=4), dict(page_size=8), dict(d=64), dict(type=1, scale=P)):
        assert attend(lib, v=cache(**other)) == E
        assert lib.cache_write(P, 256, 128, P, 256, 128, 3, cache(), cache(**other), P, None) == E


def test_write_and_read(lib):
    c = cache()

    def write(k=P, ks=256, kh=128, v=P, vs=256, vh=128, tokens=3, slots=P):
        return lib.cache_write(k, ks, kh, v, vs, vh, tokens, c, c, slots, None)

    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(tokens=0), dict(tokens=-1), dict(k=P + 2),
                dict(v=P + 8), dict(ks=257), dict(kh=-8), dict(vs=4), dict(vh=2 ** 51)):
        assert write(**bad) == E, bad
    assert write(tokens=2 ** 50) == U

    def read(table=P, stride=4, width=4, lens=P, batch=2, n=10, out=P):
        return lib.cache_read(c, table, stride, width, lens, batch, n, out, None)

    for bad in (dict(table=None), dict(lens=None), dict(out=None), dict(n=0), dict(n=2 ** 31), dict(batch=0),
                dict(width=0), dict(stride=-4), dict(out=P + 4)):
        assert read(**bad) == E, bad
    assert read(batch=2 ** 30, n=2 ** 30) == U
    assert lib.cache_read(None, P, 4, 4, P, 2, 10, P, None) == E


def test_beam(lib):
    def beam(x=P, s=P, batch=2, beams=4, n=100, k=8, o=(P, P, P), fn=lib.topk_beam):
        return fn(x, s, batch, beams, n, k, *o, None, 0, None)

    for fn in (lib.topk_beam, lib.topk_beam_bf16):
        for bad in (dict(x=None), dict(s=None), dict(batch=0), dict(beams=0), dict(n=0), dict(k=0), dict(n=2 ** 31),
                    dict(o=(None, P, P)), dict(o=(P, None, P)), dict(o=(P, P, None))):
            assert beam(fn=fn, **bad) == E, bad
        for bad in (dict(beams=129), dict(k=129), dict(batch=2 ** 40), dict(batch=2 ** 31)):
            assert beam(fn=fn, **bad) == U, bad


def test_reorder(lib):
    def reorder(src=(P, 2 * P), dst=(3 * P, 4 * P), size=(64, 64), count=None, batch=2, beams=4, k=4, parents=P):
        m = len(src)
        a, b = (ctypes.c_void_p * m)(*src), (ctypes.c_void_p * m)(*dst)
        s = (ctypes.c_int64 * m)(*size)
        return lib.beam_reorder(a, b, s, m if count is None else count, batch, beams, k, parents, None)

    for bad in (dict(count=0), dict(batch=0), dict(beams=0), dict(k=0), dict(parents=None), dict(size=(64, 0)),
                dict(src=(P, None)), dict(dst=(None, P)), dict(dst=(P, 4 * P)), dict(dst=(P + 511, 4 * P)),
                dict(dst=(3 * P, 3 * P + 100)), dict(dst=(2 * P - 100, 4 * P)), dict(size=(2 * P, 64))):
        assert reorder(**bad) == E, bad
    many = tuple(P * (i + 1) for i in range(514))
    assert reorder(src=many[:257], dst=many[257:], size=(64,) * 257) == U
    assert reorder(batch=2 ** 31) == U and reorder(size=(2 ** 49, 64)) == U
    assert lib.beam_reorder(None, None, None, 1, 1, 1, 1, P, None) == E


def test_workspace_queries_of_bad_sizes(lib):
    assert lib.paged_attention_workspace_bytes(0, 8, 0, 128) == 0
    assert lib.paged_attention_workspace_bytes(2, 8, 0, 100) == 0
    assert lib.topk_beam_workspace_bytes(0, 4, 100, 8) == 0
    assert lib.topk_beam_workspace_bytes(2, 129, 100, 8) == 0


def test_binding_refuses_cpu_tensors(lib):
    c = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        atk.paged_attention(torch.zeros(1, 1, 64, dtype=torch.bfloat16), c, c, i, i[0, :1])
    with pytest.raises(TypeError):
        atk.cache_write(c[0], c[0], c, c, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(TypeError):
        atk.cache_read(c, i, i[0, :1], 4)
    with pytest.raises(TypeError):
        atk.topk_beam(torch.zeros(1, 2, 8), torch.zeros(1, 2), 2)
    with pytest.raises(TypeError):
        atk.beam_reorder(torch.zeros(1, 2, 8), i)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors():
    dev = "cuda:0"
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=dev)
    c = torch.zeros(3, 2, 4, 64, dtype=torch.bfloat16, device=dev)
    c8, sc = c.to(torch.float8_e4m3fn), torch.ones(3, 2, 4, device=dev)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=dev), torch.ones(2, dtype=torch.int32, device=dev)
    pos = torch.zeros(2, 2, 3, dtype=torch.int32, device=dev)

    def bad(kind, fn, *a, **kw):
        with pytest.raises(kind):
            fn(*a, **kw)

    att = atk.paged_attention
    bad(TypeError, att, q.float(), c, c, table, lens)
    bad(TypeError, att, q, c.half(), c, table, lens)
    bad(ValueError, att, q, c8, c8, table, lens)                    # no scales
    bad(ValueError, att, q, c, c, table, lens, k_scale=sc)
    bad(ValueError, att, q, c8, c8, table, lens, k_scale=sc, v_scale=sc[:2])
    bad(TypeError, att, q, c8, c8, table, lens, k_scale=sc, v_scale=sc.double())
    bad(ValueError, att, q, c8, c, table, lens, k_scale=sc)
    bad(ValueError, att, q, c, c[:2], table, lens)
    bad(ValueError, att, q[:, :3], c, c, table, lens)
    bad(ValueError, att, q[..., :32], c, c, table, lens)
    bad(ValueError, att, q.transpose(1, 2), c, c, table, lens)
    bad(ValueError, att, q, c.transpose(2, 3), c.transpose(2, 3), table, lens)
    bad(TypeError, att, q, c, c, table.long(), lens)
    bad(TypeError, att, q, c, c, table, lens.float())
    bad(ValueError, att, q, c, c, table[:1], lens)
    bad(ValueError, att, q, c, c, table, lens[:1])
    bad(ValueError, att, q, c, c, table, lens, positions=pos[:1])
    bad(ValueError, att, q, c, c, table, lens, positions=pos[:, :1].contiguous())
    bad(TypeError, att, q, c, c, table, lens, positions=pos.long())
    bad(ValueError, att, q, c, c, table, lens, out=q[:1])
    bad(ValueError, att, q, c, c, table, lens, out_lse=torch.zeros(3, device=dev))
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device=dev)
    slots = torch.arange(5, device=dev)
    bad(ValueError, atk.cache_write, k, k[:4], c, c, slots)
    bad(ValueError, atk.cache_write, k[:, :1], k[:, :1], c, c, slots)
    bad(TypeError, atk.cache_write, k, k, c, c, slots.int())
    bad(ValueError, atk.cache_write, k, k, c, c, slots[:4])
    bad(TypeError, atk.cache_write, k.float(), k, c, c, slots)
    bad(ValueError, atk.cache_read, c, table, lens, 4, out=torch.zeros(2, 2, 5, 64, dtype=torch.bfloat16, device=dev))
    bad(atk.TopkError, atk.cache_read, c, table, lens, 0)
    x, s = torch.zeros(2, 3, 10, device=dev), torch.zeros(2, 3, device=dev)
    bad(TypeError, atk.topk_beam, x.half(), s, 2)
    bad(ValueError, atk.topk_beam, x, s[:1], 2)
    bad(ValueError, atk.topk_beam, x.transpose(1, 2), s, 2)
    bad(TypeError, atk.topk_beam, x, s.double(), 2)
    bad(atk.TopkError, atk.topk_beam, x, s, 129)
    bad(ValueError, atk.topk_beam, x, s, 2, out_token=torch.zeros(2, 3, dtype=torch.int32, device=dev))
    par = torch.zeros(2, 3, dtype=torch.int32, device=dev)
    bad(ValueError, atk.beam_reorder, [], par)
    bad(ValueError, atk.beam_reorder, x[:, :, ::2], par)
    bad(ValueError, atk.beam_reorder, [x, x[:1]], par)
    bad(TypeError, atk.beam_reorder, x, par.long())
    bad(ValueError, atk.beam_reorder, x, par, out=torch.zeros(2, 3, 11, device=dev))
    bad(atk.TopkError, atk.beam_reorder, x, par, out=x)
    bad(ValueError, atk.beam_reorder, x[:, :, :0], par)


def test_sizes_beyond_32_bits_are_refused():
    from approximate_top_selection_b200 import _decode

    big = 2 ** 32 + 2

    def meta(*shape, dtype=torch.bfloat16):  # no memory; on device -1 as CPU tensors are
        return torch.empty(*shape, dtype=dtype, device="meta")

    for shape in ((1, big, 1, 64), (1, 1, big, 64), (1, 1, 1, big)):
        with pytest.raises(ValueError, match="32 bits"):
            _decode._cache(meta(*shape), None, "k_cache", -1)
    assert _decode._cache(meta(big, 1, 1, 64), None, "k_cache", -1)[0].pages == big  # pages are 64-bit
    with pytest.raises((TypeError, ValueError)):
        _decode._table(meta(1, big, dtype=torch.int32), meta(1, dtype=torch.int32), 1, -1)
    assert _decode._table(meta(1, 5, dtype=torch.int32), meta(1, dtype=torch.int32), 1, -1) == (5, 5)
    for name in ("heads", "lists", "c", "beams", "k"):
        _decode._int32(**{name: 2 ** 31 - 1})
        with pytest.raises(ValueError, match="32 bits"):
            _decode._int32(**{name: 2 ** 31})


@pytest.mark.gpu
def test_a_beam_of_more_than_32_bits_is_refused():
    x, s = torch.zeros(1, 3, 10, device="cuda:0"), torch.zeros(1, 3, device="cuda:0")
    with pytest.raises(ValueError):
        atk.topk_beam(x, s, 2 ** 32 + 2)
    with pytest.raises(ValueError):
        atk.topk_beam(x, s, 2 ** 32 + 2, stream=torch.cuda.current_stream())


def test_the_extension_module_leaves_unusual_calls_alone(lib):
    from approximate_top_selection_b200 import _decode

    calls = _decode._usual()
    c = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 2, dtype=torch.int32)
    assert calls.paged_attention(c[0], c, c, i, i[0], None, None, None, None, False) is None
    assert calls.cache_write(c[0], c[0], c, c, i[0], None, None) is None
    assert calls.cache_read(c, i, i[0], 4, None) is None
    assert calls.topk_beam(torch.zeros(1, 2, 8), torch.zeros(1, 2), 2) is None
    assert calls.beam_reorder([torch.zeros(1, 2, 8)], i) is None
    assert calls.cache_read("no", "tensor", 3, -1, None) is None
    assert calls.beam_reorder(None, None) is None
    with pytest.raises(TypeError):
        calls.topk_beam(c)
