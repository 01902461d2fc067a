"""Calls of several host threads on one stream: torch's threads share the
default stream, and a call of two launches must not find another's numbers
between them."""
import sys
import threading

import pytest
import torch

import approximate_top_selection_b200 as atk

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
CALLS = 400


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("these tests need a CUDA device")
    atk.load_library()
    torch.cuda.synchronize()
    atk.topk_device_status()
    yield


def _attention_case(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(2, 8, 128, generator=g, device=DEV).bfloat16()
    k, v = (torch.randn(256, 2, 16, 128, generator=g, device=DEV).bfloat16() for _ in range(2))
    table = torch.randperm(256, generator=g, device=DEV).view(2, 128).to(torch.int32)
    return q, k, v, table, torch.tensor([2000, 1999], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("path", ["usual", "step by step"])
def test_threads_on_one_stream_keep_their_results_apart(path):
    kw = {} if path == "usual" else {"stream": torch.cuda.current_stream()}
    g = torch.Generator(device=DEV).manual_seed(3)
    beams = [(torch.randn(2, 4, 40000, generator=g, device=DEV), torch.zeros(2, 4, device=DEV), 4),
             (torch.randn(1, 6, 30001, generator=g, device=DEV).bfloat16(), torch.zeros(1, 6, device=DEV), 12),
             (torch.randn(100, 4, 5000, generator=g, device=DEV), torch.zeros(100, 4, device=DEV), 8)]
    att = _attention_case(4)
    jobs = [lambda b=b: atk.topk_beam(*b, **kw) for b in beams] + [lambda: atk.paged_attention(*att, return_lse=True, **kw)]
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    wrong, errors = [0] * len(jobs), []
    start = threading.Barrier(len(jobs))

    def loop(i):
        try:
            start.wait()
            got = [jobs[i]() for _ in range(CALLS)]
            torch.cuda.synchronize()
            wrong[i] = sum(not all(torch.equal(x, y) for x, y in zip(o, want[i])) for o in got)
        except Exception as e:  # a thread's exception fails the test, not the thread alone
            errors.append(e)

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(jobs))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    assert not errors, errors
    assert wrong == [0] * len(jobs), wrong
    assert atk.topk_device_status() == 0
