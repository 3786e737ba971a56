"""GPU test of calls from several host threads: sorts of few and of many experts at once, which
share kernels and take different amounts of LDS."""
import threading

import pytest
import torch

import fp8_block_ref as ref
import skinny_gemm_projection_amd as sg
from gpu_common import DEV, announce

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]


@pytest.mark.parametrize("T", [20, 513, 9000])
def test_sorts_from_several_threads(T):
    announce(f"sorts from four threads T={T}")
    cases = []
    for i, E in enumerate((4096, 3, 1024, 4096)):
        ids = torch.randint(0, E, (T, 8), generator=ref.gen(i), dtype=torch.int32)
        cases.append((ids.to(DEV), E, ref.table(ids, E)))
    torch.cuda.synchronize()
    failures = []

    def work(ids, E, want):
        try:
            stream = torch.cuda.Stream()
            for _ in range(50):
                got = sg.skinny_moe_sort(ids, E, stream=stream)
            stream.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a.cpu(), b)
        except Exception as e:  # noqa: BLE001 - a thread's failure is the test's
            failures.append(f"E={E}: {e!r}")

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
