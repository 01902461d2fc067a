"""Unusual tensors given to the decoding step's operators."""
import pytest
import torch

import approximate_top_selection_b200 as atk

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA device")
    atk.load_library()
    torch.cuda.synchronize()
    atk.topk_device_status()
    yield


@pytest.mark.parametrize("path", ["usual", "step by step"])
def test_conjugate_and_negative_states(path):
    """Views whose bytes stand for other values are reordered as the values they are."""
    kw = {} if path == "usual" else {"stream": torch.cuda.current_stream()}
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.complex(*torch.randn(2, 2, 3, 7, generator=g, device=DEV))
    p = torch.tensor([[2, 0, 0], [1, 1, 2]], dtype=torch.int32, device=DEV)
    at = torch.arange(2, device=DEV).view(2, 1)
    states = [x, x.conj(), torch._neg_view(x.real.contiguous())]
    for s, o in zip(states, atk.beam_reorder(states, p, **kw)):
        assert torch.equal(o.resolve_conj().resolve_neg(), s.resolve_conj().resolve_neg()[at, p.long()])
    with pytest.raises(ValueError):
        atk.beam_reorder(x, p, out=torch.empty_like(x).conj(), **kw)


def test_workspaces():
    """A workspace of any type counts its bytes; a view of fewer, or one that is elsewhere, is refused."""
    x, s = torch.randn(3, 4, 70000, device=DEV), torch.zeros(3, 4, device=DEV)
    q = torch.randn(2, 4, 64, device=DEV).bfloat16()
    c = torch.randn(9, 2, 16, 64, device=DEV).bfloat16()
    table, lens = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4), torch.tensor([64, 3], dtype=torch.int32, device=DEV)
    calls = [(lambda **kw: atk.topk_beam(x, s, 8, **kw), atk.topk_beam_workspace_bytes(3, 4, 70000, 8)),
             (lambda **kw: (atk.paged_attention(q, c, c, table, lens, **kw),), atk.paged_attention_workspace_bytes(2, 4, 0, 64))]
    for call, need in calls:
        want = call()
        assert need % 4 == 0
        got = call(workspace=torch.zeros(need // 4, device=DEV))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        with pytest.raises(atk.TopkError) as e:
            call(workspace=torch.zeros(need // 4 - 4, device=DEV))
        assert e.value.status == atk.TOPK_EWORKSPACE
        with pytest.raises(ValueError):
            call(workspace=torch.zeros(1, dtype=torch.uint8, device=DEV).expand(need))
        with pytest.raises(ValueError):
            call(workspace=torch.zeros(2 * need, dtype=torch.uint8, device=DEV)[::2])
        for bad in (torch.zeros(need, dtype=torch.uint8), need):
            with pytest.raises(TypeError):
                call(workspace=bad)
