"""Paged-cache calls (GPU) whose outputs would lie over another of their buffers are refused before
anything is enqueued: every pair, over the C entry points."""

import array

import pytest
import torch

from tests.test_gpu_paged import M   # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

NSEQ, MP, NUM, PS, HKV, D, T, HQ, TOPK = 4, 4, 16, 16, 1, 64, 40, 64, 2048


class Buffers:
    """Named buffers of one allocation, 4096 bytes apart; `over` puts one where another ends."""

    def __init__(self, sizes):
        self.sizes = sizes
        step = -(-max(sizes.values()) // 4096) * 4096 + 4096
        self.mem = torch.zeros(step * (len(sizes) + 1), dtype=torch.uint8, device="cuda")
        base = -(-self.mem.data_ptr() // 4096) * 4096
        self.at = {n: base + i * step for i, n in enumerate(sizes)}

    def over(self, x, y):
        """x begins in the last bytes of y that its alignment allows, or at y where y is small."""
        at = dict(self.at)
        at[x] = self.at[y] + max(0, self.sizes[y] - 256) // 256 * 256
        return at


def attention(lib, at, ws):
    return lib.misa_paged_attention(
        at["q"], at["k"], at["v"], at["table"], at["pos"], at["idx"], 0, NSEQ, T, HQ, HKV, D, NUM,
        PS, MP, TOPK, 0.1, at["out"], at["lse"], at["status"], at["ws"], ws, None)


def append(lib, at, ws):
    return lib.misa_paged_append(at["kn"], at["vn"], at["pos"], at["table"], 0, NSEQ, T, HKV, D, NUM,
                                 PS, MP, at["k"], at["v"], at["status"], None)


def pool_lists(at):
    return array.array("Q", [at["k"], at["v"]]), array.array("q", [PS * HKV * D * 2] * 2)


def resize(lib, at, ws):
    p, s = pool_lists(at)
    return lib.misa_pages_resize(at["table"], at["refs"], at["old"], at["new"], NSEQ, MP, NUM, PS,
                                 p.buffer_info()[0], s.buffer_info()[0], 2, at["out_table"],
                                 at["out_refs"], at["status"], at["ws"], ws, None)


def fork(lib, at, ws):
    return lib.misa_pages_fork(at["table"], at["refs"], at["parent"], NSEQ, MP, NUM,
                               at["out_table"], at["out_refs"], at["status"], at["ws"], ws, None)


def compact(lib, at, ws):
    p, s = pool_lists(at)
    return lib.misa_pages_compact(at["table"], at["refs"], NSEQ, MP, NUM, p.buffer_info()[0],
                                  s.buffer_info()[0], 2, at["out_table"], at["out_refs"],
                                  at["n_live"], at["status"], at["ws"], ws, None)


POOL, TABLE, ROWS = NUM * PS * HKV * D * 2, NSEQ * MP * 4, NSEQ * T * HQ * D * 2
UPKEEP = dict(table=TABLE, refs=NUM * 4, out_table=TABLE, out_refs=NUM * 4, status=4)
# call, buffers, those that it writes, inputs that an output may take the place of
CALLS = {
    "attention": (attention, dict(q=ROWS, k=POOL, v=POOL, table=TABLE, pos=NSEQ * T * 4,
                                  idx=NSEQ * T * TOPK * 4, out=ROWS, lse=NSEQ * T * HQ * 4, status=4),
                  ["out", "lse", "status", "ws"], {"q": "out"}),
    "append": (append, dict(kn=NSEQ * T * HKV * D * 2, vn=NSEQ * T * HKV * D * 2, pos=NSEQ * T * 4,
                            table=TABLE, k=POOL, v=POOL, status=4), ["k", "v", "status"], {}),
    "resize": (resize, dict(UPKEEP, old=NSEQ * 4, new=NSEQ * 4, k=POOL, v=POOL),
               ["out_table", "out_refs", "status", "ws", "k", "v"],
               {"table": "out_table", "refs": "out_refs"}),
    "fork": (fork, dict(UPKEEP, parent=NSEQ * 4), ["out_table", "out_refs", "status"],
             {"table": "out_table", "refs": "out_refs"}),
    "compact": (compact, dict(UPKEEP, n_live=4, k=POOL, v=POOL),
                ["out_table", "out_refs", "n_live", "status", "ws", "k", "v"],
                {"table": "out_table", "refs": "out_refs"}),
}


def scratch_bytes(lib, name):
    if name == "attention":
        return lib.misa_paged_attention_workspace_size(NSEQ, T, HQ, HKV, D, PS, MP, TOPK)
    op = {"resize": 7, "fork": 8, "compact": 9}.get(name)
    return lib.misa_pages_workspace_size(op, NSEQ, MP, NUM) if op else 0


@pytest.mark.parametrize("name", list(CALLS))
def test_every_overlap_of_an_output_is_refused(M, name):
    call, sizes, written, in_place = CALLS[name]
    lib = M.library()
    nb = scratch_bytes(lib, name)
    assert (nb > 0) == ("ws" in written)
    b = Buffers(dict(sizes, ws=nb) if nb else dict(sizes))
    b.at.setdefault("ws", None)
    assert call(lib, b.at, nb) == 0
    torch.cuda.synchronize()
    refused = 0
    for x in written:
        for y in b.sizes:
            if x == y or x not in b.sizes or y in ("kn", "vn"):
                continue                                    # (rows of a cache may be appended)
            for at in (b.over(x, y), b.over(y, x)):
                if in_place.get(y) == x and at[x] == at[y]:
                    continue
                assert call(lib, at, nb) == 1, (x, y)
                refused += 1
    assert refused > 10
    for y, x in in_place.items():                           # in place: one buffer for both
        at = dict(b.at)
        at[x] = at[y]
        assert call(lib, at, nb) == 0, (x, y)
    torch.cuda.synchronize()
    if name == "append":
        at = dict(b.at, kn=b.at["k"], vn=b.at["v"])         # rows of the caches, none of them written
        assert call(lib, at, nb) == 0
        torch.cuda.synchronize()


def test_pools_that_overlap_are_refused(M):
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(10, dtype=torch.int32, device="cuda")
    buf = torch.zeros((31, 16), dtype=torch.int16, device="cuda")
    pools = [buf[20:30], buf[:10], buf[10:20]]
    M.misa_pages_compact(table, refs, pools)
    assert M.misa_check_device_status("cuda") == 0
    for bad in ([buf[:10], buf[9:19]], [buf[:10], buf[:10]], [buf[1:11], buf[20:30], buf[:10]]):
        with pytest.raises(M.MisaError) as e:
            M.misa_pages_compact(table, refs, bad)
        assert e.value.status == 1
