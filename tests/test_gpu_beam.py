"""topk_beam and beam_reorder on the GPU.

A value s_i + x - lse_i: the sum of n exponentials is held in fp32 by chains of
at most 2^8 terms (2^8 * 2^-24 relatively), the hardware's exp2 is within
2^-21, so lse_i is within 2^-15 absolutely; the sum itself is 64-bit and
rounded once to fp32.  Tokens and beams must be the 64-bit form's wherever no
other continuation's value is within twice that bound (those of one beam are
ordered by their logits and must agree always)."""
import math

import pytest
import torch

import approximate_top_selection_b200 as atk
import decode_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NINF = -math.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA device")
    atk.load_library()
    torch.cuda.synchronize()
    atk.topk_device_status()
    yield


def check(logits, scores, k, got):
    val, parent, token = (t.cpu() for t in got)
    batch = logits.shape[0]
    assert val.shape == parent.shape == token.shape == (batch, k)
    assert val.dtype == torch.float32 and parent.dtype == token.dtype == torch.int32
    for b in range(batch):
        want = ref.beam_step(logits[b], scores[b], k + 8)
        m = min(k, len(want))
        assert bool((val[b, m:] == NINF).all()) and bool((parent[b, m:] == -1).all()), b
        assert bool((token[b, m:] == -1).all()), b
        for j in range(m):
            v, i, t = want[j]
            if math.isnan(v):
                assert math.isnan(float(val[b, j])) and (int(parent[b, j]), int(token[b, j])) == (i, t), (b, j)
                continue
            tol = 2.0 ** -24 * abs(v) + 2.0 ** -15
            assert abs(float(val[b, j]) - v) <= tol or v == float(val[b, j]), (b, j, float(val[b, j]), v)
            # continuations of other beams within the bound may take its place
            near = [w for w in want if w[1] != i and abs(w[0] - v) <= 2 * tol]
            if not near:
                assert (int(parent[b, j]), int(token[b, j])) == (i, t), (b, j, want[j])
            else:
                assert (int(parent[b, j]), int(token[b, j])) in [w[1:] for w in near] + [(i, t)], (b, j)
        # within a beam: the order of its logits, no token twice
        for i in range(logits.shape[1]):
            mine = [int(t) for p, t in zip(parent[b, :m], token[b, :m]) if int(p) == i]
            full = [t for _, p, t in want if p == i]
            assert mine == full[: len(mine)], (b, i)


def run(logits, scores, k, **kw):
    return atk.topk_beam(logits.to(DEV), scores.to(DEV), k, **kw)


def make(batch, beams, n, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    if kind == "ties":
        x = torch.randint(-3, 4, (batch, beams, n), generator=g).float()
    elif kind == "ascending":
        x = torch.arange(n).float().div(max(1, n)).expand(batch, beams, n).clone()
    elif kind == "descending":
        x = torch.arange(n).flip(0).float().div(max(1, n)).expand(batch, beams, n).clone()
    elif kind == "constant":
        x = torch.full((batch, beams, n), -1.25)
    elif kind == "one stripe":  # the largest values lie a fixed distance apart
        x = torch.randn(batch, beams, n, generator=g)
        x[..., ::1024] += 10
    else:
        x = torch.randn(batch, beams, n, generator=g) * 3
    return x.to(dtype), torch.rand(batch, beams, generator=g) * -5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,beams,n,k", [(1, 1, 1, 1), (2, 3, 1, 4), (1, 4, 7, 8), (3, 2, 100, 4), (2, 5, 1001, 10),
                                             (2, 4, 16384, 8), (1, 3, 50257, 6), (5, 8, 4099, 16), (1, 128, 300, 128),
                                             (2, 2, 40000, 128), (1, 2, 131072, 4)])
def test_step(dtype, batch, beams, n, k):
    x, s = make(batch, beams, n, dtype, n + k)
    check(x, s, k, run(x, s, k))
    assert atk.topk_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["ties", "ascending", "descending", "constant", "one stripe"])
@pytest.mark.parametrize("n,k", [(5000, 8), (70001, 100)])
def test_equal_and_ordered_logits(dtype, kind, n, k):
    x, s = make(2, 3, n, dtype, 7, kind)
    check(x, s, k, run(x, s, k))


def test_equal_beams_rank_by_beam():
    x, s = make(1, 4, 3000, torch.float32, 3)
    x[:] = x[:, :1]
    s[:] = -1.0
    val, parent, token = run(x, s, 8)
    assert parent[0].tolist() == [0, 1, 2, 3] * 2
    assert token[0, :4].unique().numel() == 1 and bool((val[0, :4] == val[0, 0]).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ended_beams_and_forbidden_tokens(dtype):
    x, s = make(4, 3, 20001, dtype, 5)
    s[0, 1:] = NINF            # the first step: one beam
    s[1] = NINF                # all ended
    x[2, 0] = NINF             # a beam with no token left
    x[2, 1, 3:] = NINF         # and one with three
    s[2, 2] = NINF
    x[2, 2, 5] = math.nan      # not looked at: the beam has ended
    x[3, :, ::2] = NINF
    got = run(x, s, 6)
    check(x, s, 6, got)
    assert got[1][1].tolist() == [-1] * 6 and got[1][2].tolist() == [1, 1, 1, -1, -1, -1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_undefined_logits(dtype):
    x, s = make(4, 3, 9000, dtype, 6)
    x[0, 1, 8999] = math.nan
    x[1, 2, 17] = math.inf
    x[2, 0, 5], x[2, 1, 4000] = math.nan, math.inf
    s[3, 1] = math.nan
    check(x, s, 5, run(x, s, 5))


def test_extreme_logits():
    x, s = make(5, 2, 5000, torch.float32, 8)
    x[0, 0, 77] = 3e38
    x[1] *= 1e36
    x[2] = -3.4e38
    x[2, 1, 9] = -3.3e38
    x[3, 0] -= 80000.0
    x[4] *= 1e-42
    x[4, 0, 3], x[4, 0, 5] = 0.0, -0.0
    check(x, s, 4, run(x, s, 4))


def check_many(x, s, k, rows=320):
    """As many copies of the sentences as make `rows` rows, the first and the last of them checked."""
    batch, beams, _ = x.shape
    copies = -(-rows // (batch * beams))
    got = run(x.repeat(copies, 1, 1), s.repeat(copies, 1), k)
    check(x, s, k, [t[:batch] for t in got])
    check(x, s, k, [t[-batch:] for t in got])
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("beams,n,k", [(3, 1, 4), (4, 7, 8), (2, 513, 16), (5, 5001, 10), (8, 33000, 16), (1, 128, 128),
                                       (3, 70001, 128), (1, 150000, 3)])
def test_many_rows(dtype, beams, n, k):
    x, s = make(2, beams, n, dtype, n + k)
    check_many(x, s, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["ties", "ascending", "descending", "constant", "one stripe"])
@pytest.mark.parametrize("n,k", [(5000, 8), (50001, 100)])
def test_many_rows_of_equal_and_ordered_logits(dtype, kind, n, k):
    x, s = make(1, 2, n, dtype, 7, kind)
    check_many(x, s, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_rows_with_ended_beams_and_undefined_logits(dtype):
    x, s = make(7, 3, 20001, dtype, 5)
    s[0, 1:] = NINF
    s[1] = NINF
    x[2, 0] = NINF
    x[2, 1, 3:] = NINF
    s[2, 2] = NINF
    x[2, 2, 5] = math.nan
    x[3, :, ::2] = NINF
    x[4, 1, 20000] = math.nan
    x[5, 2, 17] = math.inf
    x[6, 0, 5], x[6, 1, 4000] = math.nan, math.inf
    check_many(x, s, 6)


def test_many_rows_of_extreme_logits():
    x, s = make(7, 2, 25000, torch.float32, 8)
    x[0, 0, 77] = 3e38
    x[1] *= 1e36
    x[2] = -3.4e38
    x[2, 1, 9] = -3.3e38
    x[3, 0] -= 80000.0
    x[4] *= 1e-42
    x[4, 0, 3], x[4, 0, 5] = 0.0, -0.0
    x[5] = torch.arange(25000) * 0.01      # the running maximum rises all the time
    x[6, :, :20000] = -1e30                # and here at once, from far below
    check_many(x, s, 4)


def test_misaligned_logits_and_given_outputs():
    for dtype in (torch.float32, torch.bfloat16):
        x, s = make(2, 3, 5001, dtype, 9)
        flat = torch.full((x.numel() + 8,), math.nan, dtype=dtype, device=DEV)
        for off in (1, 3, 7):
            xd = flat[off: off + x.numel()].view(x.shape)
            xd.copy_(x)
            outs = dict(out_scores=torch.empty(2, 6, device=DEV),
                        out_parent=torch.empty(2, 6, dtype=torch.int32, device=DEV),
                        out_token=torch.empty(2, 6, dtype=torch.int32, device=DEV))
            got = atk.topk_beam(xd, s.to(DEV), 6, **outs)
            assert [a.data_ptr() for a in got] == [a.data_ptr() for a in outs.values()]
            check(x, s, 6, got)
            flat.fill_(math.nan)


def test_a_batch_of_many_sentences():
    x, s = make(5000, 2, 37, torch.float32, 10)
    val, parent, token = (t.cpu() for t in run(x, s, 4))
    lp = torch.log_softmax(x.double(), 2) + s.double()[..., None]
    best = lp.flatten(1).topk(5, dim=1)
    assert bool(((val.double() - best.values[:, :4]).abs() <= 2.0 ** -14).all())
    clear = (best.values[:, :-1] - best.values[:, 1:]).min(1).values > 2.0 ** -13
    assert int(clear.sum()) > 4500
    assert torch.equal((parent * 37 + token)[clear].long(), best.indices[clear][:, :4])


def test_side_stream_workspace_and_repeats():
    x, s = make(3, 4, 100000, torch.float32, 11)
    xd, sd = x.to(DEV), s.to(DEV)
    first = atk.topk_beam(xd, sd, 8)
    need = atk.topk_beam_workspace_bytes(3, 4, 100000, 8)
    ws = torch.zeros(max(16, need), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for kw in (dict(stream=side), dict(stream=side, workspace=ws), dict(stream=side, workspace=ws)):
        again = atk.topk_beam(xd, sd, 8, **kw)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    torch.cuda.synchronize()
    if need:
        with pytest.raises(atk.TopkError) as e:
            atk.topk_beam(xd, sd, 8, workspace=ws[: need - 16])
        assert e.value.status == atk.TOPK_EWORKSPACE


def test_two_graphs_replayed_side_by_side():
    stream = torch.cuda.Stream()
    cases = [tuple(t.to(DEV) for t in make(2, 4, 60000, torch.bfloat16, 30 + i)) for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, s in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append(atk.topk_beam(x, s, 8))
        graphs.append(g)
    sides = [torch.cuda.Stream() for _ in cases]
    for seed in (40, 50):
        for i, (x, s) in enumerate(cases):
            nx, ns = make(2, 4, 60000, torch.bfloat16, seed + i)
            x.copy_(nx)
            s.copy_(ns)
        torch.cuda.synchronize()
        for _ in range(20):
            for g, side in zip(graphs, sides):
                with torch.cuda.stream(side):
                    g.replay()
        torch.cuda.synchronize()
        for (x, s), o in zip(cases, outs):
            assert all(torch.equal(a, b) for a, b in zip(o, atk.topk_beam(x, s, 8)))


@pytest.mark.parametrize("shapes,dtype", [
    ([(1,)], torch.uint8), ([(3,), (5, 7)], torch.int16), ([(257,), (64, 33)], torch.int32),
    ([(2, 100, 64)] * 3, torch.bfloat16), ([(4097,)], torch.float8_e4m3fn), ([(100003,), (8,), (12,)], torch.uint8),
])
@pytest.mark.parametrize("batch,beams,k", [(1, 1, 1), (3, 4, 8), (2, 5, 3)])
def test_reorder(shapes, dtype, batch, beams, k):
    g = torch.Generator().manual_seed(k)
    raw = [torch.randint(0, 256, (batch, beams) + s[:-1] + (s[-1] * torch.empty(0, dtype=dtype).element_size(),),
                         generator=g).to(torch.uint8) for s in shapes]
    parents = torch.randint(-1, beams, (batch, k), generator=g).to(torch.int32)
    parents[0, 0] = -1
    states = [r.to(DEV).view(dtype) for r in raw]
    outs = atk.beam_reorder(states, parents.to(DEV))
    for r, o in zip(raw, outs):
        assert o.dtype == dtype and o.shape[:2] == (batch, k)
        want = torch.stack([torch.stack([r[b, p] if p >= 0 else torch.zeros_like(r[0, 0]) for p in parents[b].tolist()])
                            for b in range(batch)])
        assert torch.equal(o.cpu().view(torch.uint8), want)
    if len(states) == 1:
        one = atk.beam_reorder(states[0], parents.to(DEV))
        assert torch.equal(one.view(torch.uint8), outs[0].view(torch.uint8))
    assert atk.topk_device_status() == 0


def test_reorder_of_many_and_misaligned_tensors():
    flat = torch.randint(0, 256, (200, 4099), generator=torch.Generator().manual_seed(1)).to(torch.uint8).to(DEV)
    states = [flat[i, i % 16: i % 16 + 4 * (20 + i)].view(2, 2, 20 + i) for i in range(200)]
    parents = torch.tensor([[1, 0, 1], [0, 0, 7]], dtype=torch.int32, device=DEV)
    room = torch.full((200, 4099), 9, dtype=torch.uint8, device=DEV)
    outs = [room[i, i % 5: i % 5 + 6 * (20 + i)].view(2, 3, 20 + i) for i in range(200)]
    got = atk.beam_reorder(states, parents, out=outs)
    for i, (s, o) in enumerate(zip(states, got)):
        assert o.data_ptr() == outs[i].data_ptr()
        assert torch.equal(o[0], s[0][[1, 0, 1]]) and torch.equal(o[1, :2], s[1][[0, 0]]) and bool((o[1, 2] == 0).all())
        assert bool((room[i, : i % 5] == 9).all()) and bool((room[i, i % 5 + 6 * (20 + i):] == 9).all())
    assert atk.topk_device_status() == 2  # the parent 7


def test_reorder_beyond_32_bits():
    rows, width = 5, 600_000_000  # bytes: the last rows start behind 2^31
    x = torch.empty(1, rows, width, dtype=torch.uint8, device=DEV)
    for r in range(rows):
        x[0, r, :] = r + 1
        x[0, r, -5:] = 100 + r
    p = torch.tensor([[4, 0, 3, 3, 4]], dtype=torch.int32, device=DEV)
    o = atk.beam_reorder(x, p)
    for j, r in enumerate(p[0].tolist()):
        assert torch.equal(o[0, j], x[0, r])


def test_rows_beyond_32_bits():
    n = 1_200_000_001  # 2.4 GB of bf16; the row of the second beam starts off any boundary
    x = torch.zeros(1, 2, n, dtype=torch.bfloat16, device=DEV)
    x[0, 0, n - 1], x[0, 0, 5], x[0, 1, n - 2], x[0, 1, 1_073_741_824] = 30.0, 29.0, 31.0, 28.0
    s = torch.tensor([[0.0, -1.5]], device=DEV)
    val, parent, token = atk.topk_beam(x, s, 5)
    off = [math.log(math.exp(30.0) + math.exp(29.0) + n - 2), math.log(math.exp(31.0) + math.exp(28.0) + n - 2)]
    want = sorted([(30 - off[0], 0, n - 1), (29 - off[0], 0, 5), (29.5 - off[1], 1, n - 2), (26.5 - off[1], 1, 1_073_741_824)],
                  reverse=True) + [(-off[0], 0, 0)]
    assert list(zip(parent[0].tolist(), token[0].tolist())) == [w[1:] for w in want]
    assert all(abs(float(a) - w[0]) <= 2.0 ** -14 for a, w in zip(val[0], want))
