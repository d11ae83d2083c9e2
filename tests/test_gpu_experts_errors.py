"""What only the device sees is never dropped: calls without an error word use the module's own."""
import pytest
import torch

import combine_layout_02_gb300 as ep
from combine_layout_02_gb300 import experts

pytestmark = pytest.mark.gpu

E, H, F = 4, 128, 16


def zeros(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


@pytest.fixture(autouse=True)
def clean():
    experts.check_errors()
    yield
    assert experts.check_errors() == 0


def test_good_calls_leave_nothing():
    sort = experts.ExpertSort(torch.tensor([[0, 3], [-1, 2]], device="cuda"), E, H)
    rows = experts.sort_rows(zeros(2, H), sort)
    experts.unsort_rows(experts.expert_product(rows, zeros(E, H, H), sort.expert_prefix), sort)
    experts.adapter_projection(zeros(3, H), zeros(F, H), zeros(2, 8, H), zeros(2, F, 8), torch.ones(2, device="cuda"),
                               torch.tensor([0, 1, -1], device="cuda"))
    assert experts.check_errors() == 0


def test_each_kind_is_kept_until_it_is_read():
    sort = experts.ExpertSort(torch.tensor([[0, E], [1, 2]], device="cuda"), E, H)
    assert sort.rows == 3 and experts.check_errors() == ep.EP_DEVERR_BAD_EXPERT
    assert experts.check_errors() == 0
    experts.ExpertSort(torch.tensor([[0, 3], [1, 2]], device="cuda"), E, H, rows=3)
    assert experts.check_errors() == ep.EP_DEVERR_RECV_OVERFLOW
    experts.expert_product(zeros(4, H), zeros(E, F, H), torch.tensor([0, 1, 2, 3, 5], dtype=torch.int32, device="cuda"))
    assert experts.check_errors() == ep.EP_DEVERR_RECV_OVERFLOW
    experts.adapter_projection(zeros(3, H), zeros(F, H), zeros(2, 8, H), zeros(2, F, 8), torch.ones(2, device="cuda"),
                               torch.tensor([0, 2, -1], device="cuda"))
    experts.ExpertSort(torch.tensor([[-2]], device="cuda"), E, H)
    assert experts.check_errors() == ep.EP_DEVERR_BAD_ADAPTER | ep.EP_DEVERR_BAD_EXPERT


def test_backward_products_report_too():
    w = zeros(E, F, H).requires_grad_(True)
    prefix = torch.tensor([0, 1, 2, 3, 5], dtype=torch.int32, device="cuda")
    y = experts.expert_product(zeros(4, H).requires_grad_(True), w, prefix)
    assert experts.check_errors() == ep.EP_DEVERR_RECV_OVERFLOW
    y.sum().backward()
    assert experts.check_errors() == ep.EP_DEVERR_RECV_OVERFLOW


def test_a_word_of_ones_own_is_used_instead():
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    experts.ExpertSort(torch.tensor([[E]], device="cuda"), E, H, err=err)
    assert int(err.item()) == ep.EP_DEVERR_BAD_EXPERT and experts.check_errors() == 0


def test_a_replayed_graph_reports():
    ids = torch.zeros(5, dtype=torch.int64, device="cuda")
    args = zeros(5, H), zeros(F, H), zeros(2, 8, H), zeros(2, F, 8), torch.ones(2, device="cuda"), ids
    experts.adapter_projection(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        experts.adapter_projection(*args)
    graph.replay()
    assert experts.check_errors() == 0
    ids.fill_(7)
    graph.replay()
    assert experts.check_errors() == ep.EP_DEVERR_BAD_ADAPTER
