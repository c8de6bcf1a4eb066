"""gmm_query_status while another stream's calls of the same handle report."""
import threading

import pytest

pytestmark = pytest.mark.gpu


def test_no_report_is_lost_between_reading_and_clearing():
    """A report that comes while a query runs is in that query's answer or in a later one's."""
    import torch
    from ragged_matmul_gb300 import binding
    h = binding.gmm_create(8, 0)
    bad = torch.full((1, 8), float("nan"), device="cuda")
    ids, w = torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.zeros((1, 2), device="cuda")
    reporting, asking = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    go, done = threading.Event(), threading.Event()
    rounds, failed = 3000, []

    def report():
        for _ in range(rounds):
            go.wait()
            go.clear()
            try:
                binding.gmm_route(h, ids, w, bad, stream=reporting)
                reporting.synchronize()
            except Exception as err:       # noqa: BLE001
                failed.append(err)
            done.set()

    t = threading.Thread(target=report)
    t.start()
    lost = 0
    for _ in range(rounds):
        seen = False
        go.set()
        while not done.is_set():
            seen |= binding.gmm_query_status(h, asking) == binding.GMM_ERR_BAD_INPUT
        done.clear()
        seen |= binding.gmm_query_status(h, asking) == binding.GMM_ERR_BAD_INPUT
        lost += not seen
    t.join()
    assert not failed and lost == 0
    assert binding.gmm_query_status(h, asking) == binding.GMM_OK
    binding.gmm_destroy(h)
