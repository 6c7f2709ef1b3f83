"""spec_logprobs holds no state: several threads may call it at once."""
import threading

import pytest
import torch

from _gpu_util import lib

pytestmark = pytest.mark.gpu


def test_calls_of_different_sizes_at_once():
    """Two threads, a stream each, with calls that need different amounts of shared memory."""
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    sizes, results = [(1 << 20, 32), (131072, 32)], {}

    def work(i):
        try:
            V, n = sizes[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                g = torch.Generator(device="cuda").manual_seed(i)
                x = torch.randn(1, V, generator=g, device="cuda")
                want = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :n].int()
                tok, lp = want[:, 0].contiguous(), torch.empty(1, device="cuda")
                ids, tlp = torch.empty(1, n, dtype=torch.int32, device="cuda"), torch.empty(1, n, device="cuda")
                torch.cuda.current_stream().synchronize()
                start.wait()
                for _ in range(20000):
                    spec.spec_logprobs(x, tok, lp, None, ids, tlp)
                torch.cuda.current_stream().synchronize()
                results[i] = torch.equal(ids, want)
        except Exception as e:
            results[i] = e

    start = threading.Barrier(2)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert results == {0: True, 1: True}
