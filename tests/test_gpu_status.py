"""misa_check_device_status (GPU): no condition that a call left is lost."""

import pytest
import torch

from tests.test_gpu_paged import M, i32   # noqa: F401 (M is a fixture)

pytestmark = pytest.mark.gpu


def bad_position(M):
    q = torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, 64, 128), dtype=torch.bfloat16, device="cuda")
    M.dsa_score_topk(q, torch.zeros((1, 1, 4), device="cuda"), k, i32([[64]]), 4)


def out_of_pages(M):
    table = i32([[0, -1]])
    M.misa_pages_resize(table, i32([1]), i32([4]), i32([8]), 4)


def status(M, device):
    try:
        return M.misa_check_device_status(device)
    except M.MisaError as e:
        return e.status


@pytest.mark.parametrize("device", [None, 0, "cuda", "cuda:0", torch.device("cuda")])
def test_both_kinds_of_condition_are_reported(M, device):
    assert status(M, 0) == 0
    bad_position(M)
    out_of_pages(M)
    assert [status(M, device) for _ in range(3)] == [6, 8, 0]
    bad_position(M)
    assert [status(M, device) for _ in range(2)] == [6, 0]
    out_of_pages(M)
    assert [status(M, device) for _ in range(2)] == [8, 0]
