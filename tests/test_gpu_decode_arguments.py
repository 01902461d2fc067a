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
