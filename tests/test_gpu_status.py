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


def fresh_workspace(M, monkeypatch):
    from long_context_block_b200 import _binding as b
    monkeypatch.setattr(b, "_WS", b._Workspace())
    return b._WS


def call(M, L, pos, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((8, 1, 8, 128), generator=g, device="cuda").bfloat16()
    k = torch.randn((8, L, 128), generator=g, device="cuda").bfloat16()
    w = torch.randn((8, 1, 8), generator=g, device="cuda")
    pos = torch.full((8, 1), pos, dtype=torch.int32, device="cuda")
    return q, w, k, pos, lambda: M.misa_indexer(q, w, k, pos, 64, 3, 100)


def test_a_condition_outlives_a_larger_workspace(M, monkeypatch):
    ws = fresh_workspace(M, monkeypatch)
    bad_position(M)
    small = ws.get(0, "cuda:0").numel()
    call(M, 120_000, 119_999)[-1]()
    assert ws.get(0, "cuda:0").numel() > small
    assert [status(M, 0) for _ in range(2)] == [6, 0]


def test_a_graph_keeps_its_workspace(M, monkeypatch):
    """A captured indexer step replayed after larger calls: its results stay, and so does memory
    that was allocated in between."""
    ws = fresh_workspace(M, monkeypatch)
    q, w, k, pos, f = call(M, 30_000, 29_999)
    want = [x.clone() for x in f()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = f()
    before = ws.get(0, "cuda:0")
    call(M, 200_000, 199_999)[-1]()
    assert ws.get(0, "cuda:0") is not before
    size = before.numel()
    del before
    others = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for x in got:
        x.fill_(0)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(bool((x == 7).all()) for x in others)
    assert status(M, 0) == 0
    pos.fill_(30_000)                       # what a replay reports shows
    g.replay()
    assert [status(M, 0) for _ in range(2)] == [6, 0]
    del g
