"""The paged-cache operators (GPU) against the fp64 / list oracle: attention over whole prefixes
and over selected tokens, appending, resize, fork, compact, their rows that see nothing, bad
device input, graphs and streams, and a run of them together."""

import math

import numpy as np
import pytest
import torch

import oracle.paged_oracle as po

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import long_context_block_b200 as M
    return M


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


class Case:
    """A cache, queries and positions from a seed.  What no query may see is filled with NaN."""

    def __init__(self, lens, T=1, Hq=8, Hkv=2, d=128, ps=16, dtype="bf16", topk=0, seed=0,
                 spare_slots=2, poison=True, scale=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        n = len(lens)
        self.lens, self.ps, self.T, self.topk = lens, ps, T, topk
        self.scale = d ** -0.5 if scale is None else scale
        pages = [max(0, -(-x // ps)) for x in lens]
        mp = max(1, max(pages)) + spare_slots
        num_pages = sum(pages) + 3
        perm = rng.permutation(num_pages)
        table = np.full((n, mp), -1, dtype=np.int32)
        at = 0
        for r, c in enumerate(pages):
            table[r, :c] = perm[at:at + c]
            at += c
        self.table = table
        self.k = torch.randn((num_pages, ps, Hkv, d), generator=g).to(DT[dtype])
        self.v = torch.randn((num_pages, ps, Hkv, d), generator=g).to(DT[dtype])
        self.q = (2 * torch.randn((n, T, Hq, d), generator=g)).to(DT[dtype])
        pos = np.array([[max(-1, x - T + t) for t in range(T)] for x in lens], dtype=np.int32)
        self.pos = pos
        self.idx = None
        if topk:
            idx = np.full((n, T, topk), -1, dtype=np.int32)
            for r in range(n):
                for t in range(T):
                    m = min(topk, pos[r, t] + 1)
                    if m > 0:
                        slots = rng.permutation(topk)[:m]      # empty slots anywhere
                        idx[r, t, slots] = rng.permutation(pos[r, t] + 1)[:m]
            self.idx = idx
        if poison:
            seen = torch.zeros((num_pages, ps), dtype=torch.bool)
            for r in range(n):
                for t in range(T):
                    for s in self.seen(r, t):
                        seen[table[r, s // ps], s % ps] = True
            self.k[~seen] = float("nan")
            self.v[~seen] = float("nan")

    def seen(self, n, t):
        if self.idx is None:
            return list(range(self.pos[n, t] + 1))
        return [int(s) for s in self.idx[n, t] if s >= 0]

    def run(self, M, **kw):
        a = [x.cuda() for x in (self.q, self.k, self.v)]
        idx = None if self.idx is None else torch.from_numpy(self.idx).cuda()
        return M.misa_paged_attention(*a, torch.from_numpy(self.table).cuda(),
                                      torch.from_numpy(self.pos).cuda(), idx=idx,
                                      scale=self.scale, return_lse=True, **kw)

    def check(self, out, lse, rows=None):
        """Bounds, with u half a step of the type and e = 2^-23 (two fp32 half steps):
          z (log2 domain): d products summed in fp32, the scale folded: |dz| <= (d + 8) e mag,
            mag = scale log2(e) max_s sum |q k|; a weight's relative error is then 2 ln2 |dz|
            (its own and its row maximum's) + 2^-22 (ex2) + u (rounded for the product with v);
          sums over S tokens in fp32: (S + 16) e relative to sum p |v|;
          the output is rounded once: u |out|.
        So |out - ref| <= u |ref| (1 + small) + w mean|v|, w = u + 2 ln2 (d + 8) e mag + 2^-22 +
        2 (S + 16) e (numerator and denominator).  lse: (d + 8) e mag ln2 + 2^-22 + (S + 16) e
        absolute, and 4 e |lse|."""
        q, k, v = f64(self.q), f64(self.k), f64(self.v)
        out, lse = f64(out), f64(lse)
        u = torch.finfo(self.q.dtype).eps / 2
        tiny = torch.finfo(self.q.dtype).tiny
        e, d = 2.0 ** -23, self.q.shape[-1]
        worst = 0.0
        for n in range(len(self.lens)):
            for t in range(self.T):
                if rows is not None and (n, t) not in rows:
                    continue
                seen = self.seen(n, t)
                ref, rl, mean, mag = po.attention_row(q[n, t], k, v, self.table[n], self.ps, seen,
                                                      self.scale)
                if not seen:
                    assert np.all(out[n, t] == 0) and np.all(np.isneginf(lse[n, t]))
                    continue
                dz = (d + 8) * e * mag * math.log2(math.e) * math.log(2)
                S = len(seen)
                w = u + 2 * dz + 2.0 ** -22 + 2 * (S + 16) * e
                bound = u * 1.02 * np.abs(ref) + w[:, None] * mean + tiny * u
                err = np.abs(out[n, t] - ref)
                assert np.all(err <= bound), (n, t, float((err / bound).max()))
                worst = max(worst, float((err / bound).max()))
                lb = dz + 2.0 ** -22 + (S + 16) * e + 4 * e * np.abs(rl)
                lerr = np.abs(lse[n, t] - rl)
                assert np.all(lerr <= lb), (n, t, float((lerr / lb).max()))
        return worst


CASES = {
    "one_token": dict(lens=[1]),
    "short": dict(lens=[5, 16, 17, 64, 65]),
    "ragged": dict(lens=[1000, 1, 333, 64, 0, 129], ps=16),
    "page1": dict(lens=[70, 3], ps=1),
    "page7": dict(lens=[200, 63, 64], ps=7),
    "page100_fp16": dict(lens=[777, 100, 101], ps=100, dtype="fp16"),
    "page256": dict(lens=[700, 255, 257], ps=256),
    "mha": dict(lens=[300, 20], Hq=3, Hkv=3),
    "group3": dict(lens=[400, 77], Hq=6, Hkv=2),
    "group16_mqa": dict(lens=[500, 31], Hq=16, Hkv=1),
    "group17": dict(lens=[500, 31], Hq=17, Hkv=1),
    "group32_fp16": dict(lens=[300, 15], Hq=64, Hkv=2, dtype="fp16"),
    "group40_two_blocks": dict(lens=[450, 31], Hq=40, Hkv=1),
    "group128": dict(lens=[130], Hq=128, Hkv=1, d=64),
    "d64": dict(lens=[1000, 127, 128, 129, 1], d=64),
    "d64_fp16_group5": dict(lens=[300, 32, 33], d=64, Hq=10, Hkv=2, dtype="fp16"),
    "draft4": dict(lens=[500, 4, 2, 130], T=4),            # the third has padded rows
    "draft16": dict(lens=[300, 64], T=16, Hq=8, Hkv=2),    # 64 rows per head: two blocks
    "draft7_d64": dict(lens=[300, 5], T=7, Hq=9, Hkv=3, d=64, dtype="fp16"),
    "chunk100": dict(lens=[150, 100], T=100, Hq=4, Hkv=2, d=64),
    "many_sequences": dict(lens=[(i * 37) % 200 for i in range(200)], Hq=2, Hkv=1, d=64),
    "ranges_long_one": dict(lens=[20000], Hq=4, Hkv=1, ps=64),
    "ranges_ragged": dict(lens=[(i * 977) % 2100 for i in range(37)] + [9000], Hq=4, Hkv=2),
    "ranges_group20_fp16": dict(lens=[3000, 1, 12000], Hq=20, Hkv=1, dtype="fp16", ps=48),
    "ranges_draft4_d64": dict(lens=[3000, 2, 30000], T=4, Hq=8, Hkv=2, d=64, ps=128),
    "ranges_sel": dict(lens=[1600] * 90, topk=1500, Hq=8, Hkv=4, d=64),
    "sel": dict(lens=[1000, 300, 40], topk=64),
    "sel_one": dict(lens=[50, 1], topk=1),
    "sel_more_than_tokens": dict(lens=[40, 0, 3], topk=128),
    "sel_draft": dict(lens=[400, 3], T=5, topk=33, Hq=6, Hkv=3, dtype="fp16"),
    "sel_group20": dict(lens=[600, 90], topk=100, Hq=20, Hkv=1, ps=48),
    "sel_group40_d64": dict(lens=[600, 90], topk=130, Hq=40, Hkv=1, d=64),
    "sel_long": dict(lens=[9000, 5000], topk=2048, Hq=8, Hkv=2, ps=64),
    # more than 32 query rows per key-value head, little work: clusters over several row blocks
    "rows33": dict(lens=[128, 129, 300, 1], Hq=33, Hkv=1),
    "rows127_fp16": dict(lens=[1000, 31], Hq=127, Hkv=1, dtype="fp16"),
    "rows_draft16_group8": dict(lens=[900, 16, 130, 9, 1], T=16, Hq=16, Hkv=2, ps=7),
    "rows_sel": dict(lens=[1500, 400, 0, 5], topk=700, Hq=64, Hkv=1, ps=48),
    "rows_negative_scale": dict(lens=[300], Hq=48, Hkv=1, scale=-0.15),
    # the same, the tensor-core form: one tile; an item per CTA; ranges that span items
    "tc_one_tile": dict(lens=[90, 1, 0, 33, 77], Hq=40, Hkv=1, ps=8),
    "tc_one_tile_d64_fp16": dict(lens=[90, 1, 0, 33, 77], T=9, Hq=8, Hkv=2, d=64, ps=8,
                                 dtype="fp16"),
    "tc_one_tile_sel": dict(lens=[3000, 100, 0], topk=128, Hq=80, Hkv=1, ps=48),
    "tc_whole_items": dict(lens=[400 - 9 * i for i in range(40)], Hq=100, Hkv=1, ps=7),
    "tc_whole_items_draft": dict(lens=[7 * i for i in range(60)], T=16, Hq=8, Hkv=1, d=64, ps=32,
                                 dtype="fp16"),
    "tc_whole_sel": dict(lens=[900 - 20 * i for i in range(40)], topk=300, Hq=128, Hkv=1, ps=64),
    "tc_ranges": dict(lens=[900 - 9 * i for i in range(60)], Hq=128, Hkv=1, ps=64),
    "tc_ranges_fp16_draft": dict(lens=[(i * 61) % 700 for i in range(90)], T=16, Hq=8, Hkv=2,
                                 ps=100, dtype="fp16"),
    "tc_ranges_d64": dict(lens=[1500 - 13 * i for i in range(70)], Hq=128, Hkv=1, d=64, ps=16),
    "tc_long_one": dict(lens=[70000], T=5, Hq=8, Hkv=1, ps=64),
    "tc_two_blocks_side_by_side": dict(lens=[2300 - 40 * i for i in range(20)], T=16, Hq=12,
                                       Hkv=1, d=64, ps=32),
    "tc_many_blocks": dict(lens=[700, 650, 0, 90], T=600, Hq=4, Hkv=1, d=64, ps=64),
    "tc_sel_ranges": dict(lens=[3000, 2000, 900, 2500, 1000, 2800], T=6, topk=900, Hq=128,
                          Hkv=1, ps=64),
    "tc_sel_ranges_d64_two_blocks": dict(lens=[2500] * 20, T=3, topk=1000, Hq=160, Hkv=1, d=64,
                                         dtype="fp16"),
    "tc_negative_scale": dict(lens=[100], spare_slots=0, Hq=48, Hkv=1, scale=-0.15),
    # several items to a CTA, some of no tokens
    "tc_many_items": dict(lens=[(i * 37) % 260 for i in range(500)], Hq=40, Hkv=1),
    "tc_many_items_negative_scale": dict(lens=[(i * 37) % 260 for i in range(500)], Hq=40, Hkv=1,
                                         d=64, scale=-0.15),
    "tc_many_items_zero_scale": dict(lens=[(i * 61) % 300 for i in range(400)], Hq=50, Hkv=1,
                                     dtype="fp16", scale=0.0),
    "tc_many_items_draft": dict(lens=[(i * 83) % 250 for i in range(430)], T=10, Hq=8, Hkv=2, d=64,
                                ps=7),
    "tc_many_items_chunk": dict(lens=[(i * 83) % 250 for i in range(430)], T=40, Hq=1, Hkv=1, d=64,
                                ps=7),
    "tc_many_items_sel": dict(lens=[100 + i for i in range(180)], topk=300, Hq=80, Hkv=2, d=64,
                              ps=32, scale=-0.1),
    "tc_zero_scale": dict(lens=[100], spare_slots=0, Hq=48, Hkv=1, scale=0.0),
    "negative_scale": dict(lens=[300], scale=-0.2),
    "zero_scale": dict(lens=[100], scale=0.0),
}


def form(M, c):
    """Which kernel a case takes, by the workspace that it asks for."""
    from long_context_block_b200 import _binding as b
    n, T, Hq, d = c.q.shape
    a256 = lambda x: (x + 255) // 256 * 256
    size = lambda ctas, rb: (a256(2 * ctas * rb * d * 4) + a256(2 * ctas * rb * 8)
                             + a256(ctas * 8))
    nb = b.library().misa_paged_attention_workspace_size(
        n, T, Hq, c.k.shape[2], d, c.ps, c.table.shape[1], c.topk)
    return {0: "cluster", size(148, 128): "tc", size(296, 16): "ranges",
            size(296, 32): "ranges"}[nb]


@pytest.mark.parametrize("name", list(CASES))
def test_attention(M, name):
    c = Case(**CASES[name])
    if name.startswith("tc_"):
        assert form(M, c) == "tc"
    elif name.startswith("ranges_"):
        assert form(M, c) == "ranges"
    elif name.startswith("rows"):
        assert form(M, c) == "cluster"
    out, lse = c.run(M)
    torch.cuda.synchronize()
    assert M.misa_check_device_status(out.device) == 0
    c.check(out, lse)
    again, lse2 = c.run(M)
    assert torch.equal(out, again) and torch.equal(lse, lse2)   # no order of atomics in results


def test_attention_without_lse_and_with_given_outputs(M):
    c = Case([300, 20], T=2)
    ref, lse = c.run(M)
    a = [x.cuda() for x in (c.q, c.k, c.v)] + [torch.from_numpy(x).cuda() for x in (c.table, c.pos)]
    assert torch.equal(M.misa_paged_attention(*a), ref)
    out, l2 = torch.full_like(ref, 7), torch.full_like(lse, 7)
    r = M.misa_paged_attention(*a, out=out, lse=l2, return_lse=True)
    assert r[0] is out and r[1] is l2 and torch.equal(out, ref) and torch.equal(l2, lse)


def test_padded_rows_and_empty_lists(M):
    c = Case([100, 60, 0], T=3, poison=False)
    c.pos[0, 1] = -1
    c.pos[1, :] = -1
    out, lse = c.run(M)
    c.check(out, lse)
    s = Case([100, 60], T=2, topk=40, poison=False)
    s.idx[0, 1] = -1
    s.pos[1, 0] = -1
    s.idx[1, 0] = -1
    out, lse = s.run(M)
    assert M.misa_check_device_status(out.device) == 0
    s.check(out, lse)


def test_infinite_scores_and_values(M):
    """A token of score -inf has weight 0, a row of nothing else counts as seeing nothing, and a
    NaN that is seen shows."""
    c = Case([40, 20, 30], Hq=2, Hkv=1, d=64, poison=False, T=1)
    c.q[:] = c.q.abs() + 0.5
    t = c.table
    c.k[t[0, 1], 3] = -float("inf")              # token 19 of sequence 0
    for s in range(20):
        c.k[t[1, s // 16], s % 16] = -float("inf")
    c.v[t[2, 0], 5, 0, 7] = float("nan")
    out, lse = c.run(M)
    keep = [s for s in range(40) if s != 19]
    c2 = Case([40, 20, 30], Hq=2, Hkv=1, d=64, poison=False)
    c2.q, c2.k, c2.v = c.q, c.k, c.v
    c2.seen = lambda n, t: keep if n == 0 else []
    c2.check(out, lse, rows={(0, 0), (1, 0)})
    bad = torch.isnan(out[2, 0]).cpu()
    assert bool(bad[:, 7].all()) and not bool(bad[:, :7].any()) and not bool(bad[:, 8:].any())


@pytest.mark.parametrize("name", [
    "draft4", "draft16", "draft7_d64", "ranges_draft4_d64", "rows_draft16_group8",
    "tc_one_tile_d64_fp16", "tc_whole_items_draft", "tc_ranges_fp16_draft", "tc_long_one",
    "tc_two_blocks_side_by_side", "tc_many_blocks", "tc_many_items_draft"])
def test_values_that_only_some_queries_see(M, name):
    """NaN and infinite values show in the queries that see them, and in no other of the same
    call: with each set to 0 the rest is the same to the bit."""
    c = Case(**CASES[name], poison=False)
    T, rng = c.T, np.random.default_rng(5)
    for n, x in enumerate(c.lens):      # some queries shorter by far than the rest, or padded
        if x > 200 and n % 2:
            c.pos[n, 0] = x // 3
            c.pos[n, 1] = -1
    H, d = c.k.shape[2:]
    special = [float("nan"), float("inf"), -float("inf")]
    marks = []
    for n, x in enumerate(c.lens):
        for _ in range(6):
            s = int(x - 1 - rng.integers(0, T))
            if s < 0:
                continue
            row = (c.table[n, s // c.ps], s % c.ps, int(rng.integers(H)), int(rng.integers(d)))
            marks.append((n, s, row, special[int(rng.integers(3))]))
    for _, _, row, _ in marks:
        c.v[row] = 0
    ref, lse = c.run(M)
    c.check(ref, lse)
    want = ref.float().cpu()
    last = {(n, row): x for n, s, row, x in marks}     # the value that a place ends with
    where = {(n, row): s for n, s, row, x in marks}
    G = c.q.shape[2] // H
    for (n, row), x in last.items():
        c.v[row] = x
        for t in range(T):
            if c.pos[n, t] >= where[n, row]:
                want[n, t, row[2] * G:(row[2] + 1) * G, row[3]] += x
    out, lse2 = c.run(M)
    assert M.misa_check_device_status(out.device) == 0
    assert torch.equal(lse, lse2)
    assert torch.equal(torch.nan_to_num(out.float().cpu(), 7.0, 8.0, 9.0),
                       torch.nan_to_num(want, 7.0, 8.0, 9.0))
    assert not torch.isfinite(want).all() and torch.isfinite(want).float().mean() > 0.5


def test_a_repeated_token_counts_twice(M):
    c = Case([50], topk=4, poison=False)
    c.idx[0, 0] = [7, 3, 7, 7]
    out, lse = c.run(M)
    c.check(out, lse)


def test_bad_device_input_is_reported_and_skipped(M):
    def status():
        with pytest.raises(M.MisaError) as e:
            M.misa_check_device_status("cuda")
        assert M.misa_check_device_status("cuda") == 0
        return e.value.status

    c = Case([100, 70], poison=False, spare_slots=0)
    good = c.table.copy()
    for entry in (-1, 10 ** 6, -7, 2 ** 31 - 1):
        c.table = good.copy()
        c.table[0, 2] = entry                     # tokens 32 .. 47 have no page
        out, lse = c.run(M)
        assert status() == 6
        c.seen = lambda n, t: [s for s in range(c.pos[n, t] + 1) if n or not 32 <= s < 48]
        c.check(out, lse)
    c = Case([100, 70], poison=False, spare_slots=0)
    cap = c.table.shape[1] * 16
    c.pos[0, 0] = cap + 5                         # clamped to the table's last token
    c.table[1] = c.table[0]
    out, lse = c.run(M)
    assert status() == 6
    c.pos[0, 0] = cap - 1
    c.check(out, lse)
    c.pos[0, 0] = -2                              # clamped to an empty row
    out, lse = c.run(M)
    assert status() == 6
    c.pos[0, 0] = -1
    c.check(out, lse)
    s = Case([100, 70], topk=8, poison=False)
    s.idx[0, 0] = [99, 100, -2, 5, 2 ** 31 - 1, -2 ** 31, 0, -1]
    out, lse = s.run(M)
    assert status() == 6
    s.seen = lambda n, t: [99, 5, 0] if n == 0 else [int(x) for x in s.idx[n, t] if x >= 0]
    s.check(out, lse)


def test_offsets_past_32_bits(M):
    """A pool of more than 2^32 bytes whose last pages hold the sequence."""
    ps, Hkv, d = 64, 8, 128
    num = (1 << 32) // (ps * Hkv * d * 2) + 40
    k = torch.empty((num, ps, Hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    small = Case([2000], Hq=16, Hkv=Hkv, d=d, ps=ps, poison=False)
    n = small.k.shape[0]
    M.misa_check_device_status("cuda")
    tail = i32(small.table + (small.table >= 0) * (num - n))
    pos = torch.arange(2000, device="cuda", dtype=torch.int32)[None]
    rows = [small.table[0, s // ps] * ps + s % ps for s in range(2000)]
    kn = small.k.view(-1, Hkv, d)[rows][None].cuda()
    vn = small.v.view(-1, Hkv, d)[rows][None].cuda()
    M.misa_paged_append(kn, vn, pos, tail, k, v)
    out, lse = M.misa_paged_attention(small.q.cuda(), k, v, tail,
                                      torch.from_numpy(small.pos).cuda(), return_lse=True)
    assert M.misa_check_device_status("cuda") == 0
    small.check(out, lse)


FORMS = {
    "cluster": dict(lens=[700, 10], Hq=16, Hkv=2, ps=64),
    "ranges": dict(lens=[6000, 10], Hq=16, Hkv=2, ps=64),
    "tc": dict(lens=[400 - 9 * i for i in range(40)], Hq=100, Hkv=1, d=64),
}


@pytest.mark.parametrize("name", list(FORMS))
def test_two_streams_and_two_graphs(M, name):
    """Eager calls on two streams at once, and two captured graphs replayed on both, share no
    scratch: each result equals the one computed alone."""
    cs = [Case(**FORMS[name], seed=s) for s in range(2)]
    assert all(form(M, c) == name for c in cs)
    args = []
    for c in cs:
        args.append([x.cuda() for x in (c.q, c.k, c.v)]
                    + [torch.from_numpy(x).cuda() for x in (c.table, c.pos)])
    ref = [M.misa_paged_attention(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(M.misa_paged_attention(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, ref[i]) for x in got[i])
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(M.misa_paged_attention(*args[i]))
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.fill_(7)
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], ref[i])
    # replays see new positions
    args[0][4][0, 0] = 57
    graphs[0].replay()
    cs[0].pos[0, 0] = 57
    out, lse = M.misa_paged_attention(*args[0], return_lse=True)
    assert torch.equal(outs[0], out)
    cs[0].check(out, lse, rows={(0, 0), (1, 0)})


@pytest.mark.parametrize("strided", ["q", "k", "table"])
def test_what_is_not_dense_is_refused(M, strided):
    c = Case([30], Hq=4)
    q, k, v = (x.cuda() for x in (c.q, c.k, c.v))
    table, pos = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.pos).cuda()
    if strided == "q":
        q = torch.cat([q, q], -1)[..., :128]
    elif strided == "k":
        k = k.transpose(1, 2).contiguous().transpose(1, 2)
    else:
        table = table.t().contiguous().t() if table.shape[0] > 1 else torch.cat([table, table])[::2]
        table = torch.stack([table, table], -1)[..., 0]
    with pytest.raises(ValueError):
        M.misa_paged_attention(q, k, v, table, pos)


def test_misaligned_and_short_buffers_are_refused(M):
    c = Case([30], Hq=4)
    q, k, v = (x.cuda() for x in (c.q, c.k, c.v))
    table, pos = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.pos).cuda()
    odd = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
    with pytest.raises(M.MisaError) as e:
        M.misa_paged_attention(odd, k, v, table, pos)
    assert e.value.status == 1
    from long_context_block_b200 import _binding as b
    nb = b.library().misa_paged_attention_workspace_size(1, 1, 4, 2, 128, 16, 4096, 0)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    wide = torch.full((1, 4096), -1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    rc = b.library().misa_paged_attention(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), wide.data_ptr(), pos.data_ptr(), None, 0, 1, 1,
        4, 2, 128, k.shape[0], 16, 4096, 0, 0.1, out.data_ptr(), None, None, ws.data_ptr(), nb - 1,
        None)
    assert rc == 5


@pytest.mark.parametrize("name", ["draft4", "rows33", "ranges_draft4_d64", "ranges_sel",
                                  "tc_whole_items_draft", "tc_ranges", "tc_sel_ranges",
                                  "tc_two_blocks_side_by_side"])
def test_output_over_the_queries(M, name):
    c = Case(**CASES[name])
    ref, lse = c.run(M)
    q, k, v = (x.cuda() for x in (c.q, c.k, c.v))
    idx = None if c.idx is None else torch.from_numpy(c.idx).cuda()
    out, l2 = M.misa_paged_attention(q, k, v, torch.from_numpy(c.table).cuda(),
                                     torch.from_numpy(c.pos).cuda(), idx=idx, scale=c.scale,
                                     return_lse=True, out=q)
    assert out is q and torch.equal(out, ref) and torch.equal(l2, lse)


def test_overlapping_buffers_are_refused(M):
    c = Case([40], Hq=4)
    buf = torch.zeros(3, c.k.shape[0] // 2, *c.k.shape[1:], dtype=c.k.dtype, device="cuda")
    half = buf.shape[1] * buf[0, 0].numel()
    k, v = buf[:2].view(c.k.shape), buf[1:].view(c.k.shape)     # v starts in the middle of k
    q = c.q.cuda()
    table, pos = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.pos).cuda()
    new = torch.zeros(1, 1, *c.k.shape[2:], dtype=c.k.dtype, device="cuda")
    assert half and c.k.shape[0] % 2 == 0

    def refused(call):
        with pytest.raises(M.MisaError) as e:
            call()
        assert e.value.status == 1

    refused(lambda: M.misa_paged_append(new, new, pos, table, k, v))
    refused(lambda: M.misa_paged_append(new, new, pos, table, k, k))
    inside = buf.view(-1)[:q.numel()].view(q.shape)
    refused(lambda: M.misa_paged_attention(q, k, v, table, pos, out=inside))
    two = torch.zeros(2 * q.numel(), dtype=q.dtype, device="cuda")
    shifted = two[8:8 + q.numel()].view(q.shape)
    refused(lambda: M.misa_paged_attention(two[:q.numel()].view(q.shape), k, v, table, pos,
                                           out=shifted))
    lse = two.view(torch.float32)[:4].view(1, 1, 4)
    refused(lambda: M.misa_paged_attention(q, k, v, table, pos, out=two[:q.numel()].view(q.shape),
                                           lse=lse))
    M.misa_paged_attention(q, k, v, table, pos)                # two readings may overlap


# ------------------------------------------------------------------------------------- append

APPENDS = {
    "one": dict(nseq=1, T=1, Hkv=1, d=64, ps=16),
    "step": dict(nseq=7, T=1, Hkv=8, d=128, ps=64),
    "odd_heads": dict(nseq=3, T=5, Hkv=3, d=64, ps=7),
    "page1": dict(nseq=2, T=33, Hkv=2, d=128, ps=1),
    "prompt": dict(nseq=3, T=700, Hkv=4, d=128, ps=48),
    "prompt_odd": dict(nseq=2, T=1000, Hkv=3, d=64, ps=100),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(APPENDS))
def test_append(M, name, dtype):
    c = APPENDS[name]
    nseq, T, Hkv, d, ps = c["nseq"], c["T"], c["Hkv"], c["d"], c["ps"]
    rng = np.random.default_rng(3)
    mp = -(-(T + 40) // ps)
    num = nseq * mp + 2
    table = rng.permutation(num)[:nseq * mp].reshape(nseq, mp).astype(np.int32)
    first = rng.integers(0, 41, nseq)
    pos = (first[:, None] + np.arange(T)).astype(np.int32)
    pos[rng.random((nseq, T)) < 0.2] = -1
    bits = lambda *s: torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, s).astype(np.int16))
    kn, vn = bits(nseq, T, Hkv, d), bits(nseq, T, Hkv, d)      # any bit pattern, NaNs too
    k0, v0 = bits(num, ps, Hkv, d), bits(num, ps, Hkv, d)
    rk, rv = k0.clone(), v0.clone()
    for n in range(nseq):
        for t in range(T):
            p = pos[n, t]
            if p >= 0:
                rk[table[n, p // ps], p % ps] = kn[n, t]
                rv[table[n, p // ps], p % ps] = vn[n, t]
    dev = [x.cuda().view(DT[dtype]) for x in (kn, vn, k0, v0)]
    M.misa_paged_append(dev[0], dev[1], i32(pos), i32(table), dev[2], dev[3])
    assert M.misa_check_device_status("cuda") == 0
    assert torch.equal(dev[2].view(torch.int16).cpu(), rk)
    assert torch.equal(dev[3].view(torch.int16).cpu(), rv)


def test_append_bad_positions_and_pages_are_skipped(M):
    k = torch.zeros((6, 16, 2, 64), dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    new = torch.ones((1, 5, 2, 64), dtype=torch.float16, device="cuda")
    table = i32([[2, 99, -1, 5]])
    M.misa_paged_append(new, 2 * new, i32([[3, 20, 40, 64, -2]]), table, k, v)
    with pytest.raises(M.MisaError) as e:
        M.misa_check_device_status("cuda")
    assert e.value.status == 6
    assert k.sum().item() == 128 and v.sum().item() == 256
    assert bool((k[2, 3] == 1).all()) and bool((v[2, 3] == 2).all())


# ------------------------------------------------------------------------------------- upkeep

def _state(rng, nseq, mp, ps, spare, share):
    """A random valid state: lengths, a table whose rows may share leading pages, and refs."""
    lens = [int(x) for x in rng.integers(0, mp * ps + 1, nseq)]
    held = [-(-x // ps) for x in lens]
    num = sum(held) + spare + 1
    perm = [int(x) for x in rng.permutation(num)]
    table = []
    for n in range(nseq):
        row = [perm.pop() for _ in range(held[n])]
        if share and n and rng.random() < share:      # follow an earlier row, whole or in part
            m = int(rng.integers(0, n))
            lens[n] = lens[m]
            row = [e for e in table[m] if e >= 0]
        table.append(row + [-1] * (mp - len(row)))
    refs = [0] * num
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    return lens, table, refs


def _pools(num, rng):
    """Pools of different page sizes and types, every page with contents of its own."""
    a = torch.from_numpy(rng.integers(0, 1 << 30, (num, 3, 4), dtype=np.int32)).cuda()
    b = torch.from_numpy(rng.integers(0, 1 << 30, (num, 16400), dtype=np.int32)).cuda()
    c = torch.from_numpy(rng.integers(0, 255, (num, 1, 16), dtype=np.uint8)).cuda()
    return [a, b, c]


def _check_pools(pools, before, copies):
    for p, x in zip(pools, before):
        ref = x.clone()
        for a, b in copies:
            ref[b] = x[a]
        assert torch.equal(p, ref)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed", range(12))
def test_resize(M, seed, in_place):
    rng = np.random.default_rng(seed)
    nseq, mp, ps = [(1, 1, 1), (5, 4, 4), (40, 9, 16), (300, 6, 7)][seed % 4]
    lens, table, refs = _state(rng, nseq, mp, ps, spare=nseq * mp, share=[0, 0.6, 0.9][seed % 3])
    new = [int(np.clip(x + rng.integers(-2 * ps, 3 * ps), 0, mp * ps)) if rng.random() < 0.8
           else int(rng.choice([0, x, mp * ps])) for x in lens]
    rt, rr, copies = po.resize(table, refs, lens, new, ps)
    pools = _pools(len(refs), rng)
    before = [p.clone() for p in pools]
    t, r = i32(table), i32(refs)
    kw = dict(out_table=t, out_refs=r) if in_place else {}
    ot, orf = M.misa_pages_resize(t, r, i32(lens), i32(new), ps, pools, **kw)
    assert M.misa_check_device_status("cuda") == 0
    assert ot.cpu().tolist() == rt and orf.cpu().tolist() == rr
    _check_pools(pools, before, copies)
    if not in_place:
        assert t.cpu().tolist() == table and r.cpu().tolist() == refs


@pytest.mark.parametrize("in_place", [False, True])
def test_resize_without_enough_pages_changes_nothing(M, in_place):
    table, refs = [[0, -1, -1], [1, -1, -1], [2, 3, -1]], [1, 1, 1, 1, 0, 0]
    pools = _pools(6, np.random.default_rng(0))
    before = [p.clone() for p in pools]
    t, r = i32(table), i32(refs)
    kw = dict(out_table=t, out_refs=r) if in_place else {}
    # rows 0 and 1 want three pages, two are free; row 2 would let go of one only afterwards
    ot, orf = M.misa_pages_resize(t, r, i32([4, 4, 8]), i32([12, 8, 4]), 4, pools, **kw)
    with pytest.raises(M.MisaError) as e:
        M.misa_check_device_status("cuda")
    assert e.value.status == 8
    assert ot.cpu().tolist() == table and orf.cpu().tolist() == refs
    _check_pools(pools, before, [])
    # exactly enough
    ot, orf = M.misa_pages_resize(i32(table), i32(refs), i32([4, 4, 8]), i32([8, 8, 4]), 4, pools)
    assert M.misa_check_device_status("cuda") == 0
    assert ot.cpu().tolist() == [[0, 4, -1], [1, 5, -1], [2, -1, -1]]
    assert orf.cpu().tolist() == [1, 1, 1, 0, 1, 1]


def test_resize_bad_lengths_and_entries_are_reported(M):
    table, refs = [[0, -1], [1, -1], [2, 77], [99, -1]], [1, 1, 1, 0, 0, 0]
    ot, orf = M.misa_pages_resize(i32(table), i32(refs), i32([4, -1, 8, 2]), i32([9, 4, 2, 6]), 4)
    with pytest.raises(M.MisaError) as e:
        M.misa_check_device_status("cuda")
    assert e.value.status == 6
    # rows 0 and 1: lengths out of range; row 2: lets go of a page that is none; row 3: its last
    # page is none, the new slot is filled
    assert ot.cpu().tolist() == [[0, -1], [1, -1], [2, -1], [99, 3]]
    assert orf.cpu().tolist() == [1, 1, 1, 1, 0, 0]


def test_resize_a_large_pool(M):
    """Free pages spread over a large pool and more sequences than one pass of the plan holds."""
    rng = np.random.default_rng(5)
    nseq, mp, ps, num = 2500, 40, 16, 300_000
    held = rng.integers(0, 20, nseq)
    lens = np.maximum(0, held * ps - rng.integers(0, ps, nseq))
    held = -(-lens // ps)
    perm = rng.permutation(num)
    table = np.full((nseq, mp), -1, dtype=np.int32)
    at = 0
    for n in range(nseq):
        table[n, :held[n]] = perm[at:at + held[n]]
        at += held[n]
    refs = np.zeros(num, dtype=np.int32)
    refs[table[table >= 0]] = 1
    refs[perm[at:]] = (rng.random(num - at) < 0.8)       # pages that others hold
    new = np.minimum(mp * ps, lens + rng.integers(-100, 300, nseq)).clip(0)
    rt, rr, copies = po.resize(table.tolist(), refs.tolist(), lens.tolist(), new.tolist(), ps)
    ot, orf = M.misa_pages_resize(i32(table), i32(refs), i32(lens), i32(new), ps)
    assert M.misa_check_device_status("cuda") == 0 and not copies
    assert np.array_equal(ot.cpu().numpy(), np.array(rt)) and orf.cpu().tolist() == rr


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("nseq, mp, seed", [(1, 1, 0), (4, 3, 1), (32, 17, 2), (300, 65, 3)])
def test_fork(M, nseq, mp, seed, in_place):
    rng = np.random.default_rng(seed)
    _, table, refs = _state(rng, nseq, mp, 4, spare=3, share=0.5)
    parent = [int(x) for x in rng.integers(-1, nseq, nseq)]
    rt, rr = po.fork(table, refs, parent)
    t, r = i32(table), i32(refs)
    kw = dict(out_table=t, out_refs=r) if in_place else {}
    ot, orf = M.misa_pages_fork(t, r, i32(parent), **kw)
    assert M.misa_check_device_status("cuda") == 0
    assert ot.cpu().tolist() == rt and orf.cpu().tolist() == rr
    parent = [nseq, -2, 0, 1][:nseq]
    if nseq >= 4:
        parent += list(range(4, nseq))
        ot, orf = M.misa_pages_fork(i32(table), i32(refs), i32(parent))
        with pytest.raises(M.MisaError) as e:
            M.misa_check_device_status("cuda")
        assert e.value.status == 6
        rt, rr = po.fork(table, refs, parent)
        assert ot.cpu().tolist() == rt and orf.cpu().tolist() == rr


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("nseq, mp, spare, seed", [(1, 1, 0, 0), (4, 3, 9, 1), (32, 17, 300, 2),
                                                   (300, 30, 9000, 3), (8, 4, 0, 4)])
def test_compact(M, nseq, mp, spare, seed, in_place):
    rng = np.random.default_rng(seed)
    _, table, refs = _state(rng, nseq, mp, 4, spare=spare, share=0.3)
    rt, rr, n, copies = po.compact(table, refs)
    pools = _pools(len(refs), rng)[:: (1 if len(refs) < 2000 else 2)]
    before = [p.clone() for p in pools]
    t, r = i32(table), i32(refs)
    kw = dict(out_table=t, out_refs=r) if in_place else {}
    ot, orf, live = M.misa_pages_compact(t, r, pools, **kw)
    assert M.misa_check_device_status("cuda") == 0
    assert live.item() == n and ot.cpu().tolist() == rt and orf.cpu().tolist() == rr
    _check_pools(pools, before, copies)
    ot2, orf2, _ = M.misa_pages_compact(ot, orf, pools)      # nothing left to move
    assert torch.equal(ot2, ot) and torch.equal(orf2, orf)


def test_compact_inconsistent_entries_are_reported(M):
    # entry 5 is free by refs, 9 is no page
    ot, orf, n = M.misa_pages_compact(i32([[3, 5], [9, -1]]), i32([0, 0, 0, 1, 0, 0]))
    with pytest.raises(M.MisaError) as e:
        M.misa_check_device_status("cuda")
    assert e.value.status == 6
    assert ot.cpu().tolist() == [[0, 5], [9, -1]] and n.item() == 1
    assert orf.cpu().tolist() == [1, 0, 0, 0, 0, 0]


def test_upkeep_refuses_overlap_and_bad_pools(M):
    buf = torch.zeros(64, dtype=torch.int32, device="cuda")
    table, out = buf[:32].view(4, 8), buf[16:48].view(4, 8)
    refs = torch.zeros(10, dtype=torch.int32, device="cuda")
    parent = i32([0, 1, 2, 3])
    with pytest.raises(M.MisaError) as e:
        M.misa_pages_fork(table, refs, parent, out_table=out)
    assert e.value.status == 1
    with pytest.raises(M.MisaError) as e:
        M.misa_pages_compact(table, refs, [torch.zeros((10, 6), dtype=torch.int16, device="cuda")])
    assert e.value.status == 1
    with pytest.raises(ValueError):
        M.misa_pages_compact(table, refs, [torch.zeros((9, 8), device="cuda")])
    many = [torch.zeros((10, 4), device="cuda")] * 257
    with pytest.raises(M.MisaError) as e:
        M.misa_pages_compact(table, refs, many)
    assert e.value.status == 2


def test_upkeep_in_a_graph(M):
    """A speculative step captured once: room for a draft, then back; replays keep the state."""
    rng = np.random.default_rng(2)
    lens, table, refs = _state(rng, 16, 8, 16, spare=100, share=0)
    lens = [min(x, 100) for x in lens]
    table = [[e if c < -(-lens[n] // 16) else -1 for c, e in enumerate(row)]
             for n, row in enumerate(table)]
    refs = [0] * len(refs)
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    t, r, old = i32(table), i32(refs), i32(lens)
    new = old + 20
    mid_t, mid_r = torch.empty_like(t), torch.empty_like(r)
    M.misa_pages_fork(t, r, torch.arange(16, dtype=torch.int32, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.misa_pages_resize(t, r, old, new, 16, out_table=t, out_refs=r)
        mid_t.copy_(t)
        mid_r.copy_(r)
        M.misa_pages_resize(t, r, new, old, 16, out_table=t, out_refs=r)
    want = po.resize(table, refs, lens, [x + 20 for x in lens], 16)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert mid_t.cpu().tolist() == want[0] and mid_r.cpu().tolist() == want[1]
        assert t.cpu().tolist() == table and r.cpu().tolist() == refs
    assert M.misa_check_device_status("cuda") == 0


# ------------------------------------------------------------------------------------- together

def test_sparse_decode_with_beams_and_drafts(M):
    """The operators as a decoder uses them: prompts into fresh pages, beams forked from them,
    drafts of three tokens with copy on write, selection by the indexer, attention over the
    selection, rejected tokens given back, beams reordered, the pool compacted.  The reference
    keeps every row's keys and values in plain arrays."""
    rng = np.random.default_rng(11)
    ps, Hkv, Hq, d, H, T, R = 16, 2, 8, 128, 8, 3, 4
    num, mp, Lmax, topk, B, h = 80, 12, 192, 24, 16, 3
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16()
    k_cache = torch.full((num, ps, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v_cache = k_cache.clone()
    table = torch.full((R, mp), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    ki = bf(R, Lmax, 128).cuda() * 0.1
    rows = [[] for _ in range(R)]                     # (key, value) of every token, fp64
    lens = [0] * R

    def resize(new):
        M.misa_pages_resize(table, refs, i32(lens), i32(new), ps, [k_cache, v_cache],
                            out_table=table, out_refs=refs)
        lens[:] = new

    def append(kn, vn, pos):
        M.misa_paged_append(kn.cuda(), vn.cuda(), i32(pos), table, k_cache, v_cache)
        for n in range(R):
            for t in range(pos.shape[1]):
                if pos[n, t] >= 0:
                    assert len(rows[n]) == pos[n, t]
                    rows[n].append((f64(kn[n, t]), f64(vn[n, t])))

    def fork(parent):
        nonlocal ki
        M.misa_pages_fork(table, refs, i32(parent), out_table=table, out_refs=refs)
        rows[:] = [list(rows[p]) if p >= 0 else [] for p in parent]
        lens[:] = [lens[p] if p >= 0 else 0 for p in parent]
        ki = ki[torch.tensor([max(p, 0) for p in parent]).cuda()].contiguous()

    def step():
        start = list(lens)
        resize([x + T for x in lens])
        pos = np.array([[x + t for t in range(T)] for x in start], dtype=np.int32)
        kn, vn, q = bf(R, T, Hkv, d), bf(R, T, Hkv, d), 2 * bf(R, T, Hq, d)
        qi, w = bf(R, T, H, 128) * 0.1, torch.from_numpy(rng.standard_normal((R, T, H))).float()
        for n in range(R):
            ki[n, start[n]:start[n] + T] = bf(T, 128).cuda() * 0.1
        out, idx, heads = M.misa_sparse_attention(
            qi.cuda(), w.cuda(), ki, i32(pos), B, h, topk, q.cuda(), k_cache, v_cache, table,
            k_new=kn.cuda(), v_new=vn.cuda())
        for n in range(R):
            rows[n] += [(f64(kn[n, t]), f64(vn[n, t])) for t in range(T)]
        full, lse = M.misa_paged_attention(q.cuda(), k_cache, v_cache, table, i32(pos),
                                           return_lse=True)
        assert M.misa_check_device_status("cuda") == 0
        want, _ = M.misa_score_topk(qi.cuda(), w.cuda(), ki, heads, i32(pos), topk)
        assert torch.equal(idx, want)
        u, e = torch.finfo(torch.bfloat16).eps / 2, 2.0 ** -23
        for n in range(R):
            K = np.stack([x[0] for x in rows[n]])[:, None]
            V = np.stack([x[1] for x in rows[n]])[:, None]
            for t in range(T):
                for got, seen in ((out, [s for s in idx[n, t].tolist() if s >= 0]),
                                  (full, list(range(pos[n, t] + 1)))):
                    assert len(seen) == min(pos[n, t] + 1, topk if got is out else 10 ** 6)
                    ref, _, mean, mag = po.attention_row(f64(q[n, t]), K, V, range(len(rows[n])),
                                                         1, seen, d ** -0.5)
                    w_ = u + 2 * (d + 8) * e * mag + 2.0 ** -22 + 2 * (len(seen) + 16) * e
                    err = np.abs(f64(got[n, t]) - ref)
                    assert np.all(err <= 1.02 * u * np.abs(ref) + w_[:, None] * mean)

    # prompts of 53 and 40 tokens into rows 0 and 2, padded to one batch
    first = [53, 0, 40, 0]
    resize(first)
    pos = np.full((R, 53), -1, dtype=np.int32)
    for n, x in enumerate(first):
        pos[n, :x] = np.arange(x)
    append(bf(R, 53, Hkv, d), bf(R, 53, Hkv, d), pos)
    fork([0, 0, 2, 2])
    assert int((refs > 0).sum()) == 4 + 3 and int(refs.max()) == 2
    step()
    resize([x - 2 for x in lens])                     # one drafted token accepted
    for n in range(R):
        del rows[n][-2:]
    fork([1, 0, 3, 3])                                # beams change places, one is dropped
    step()
    t, r, live = M.misa_pages_compact(table, refs, [k_cache, v_cache], out_table=table,
                                      out_refs=refs)
    n_live = live.item()
    assert bool((refs[:n_live] > 0).all()) and int(refs[n_live:].abs().sum()) == 0
    held = torch.bincount(table[table >= 0].long(), minlength=num)
    assert torch.equal(held.int(), refs)              # every count is the holders' number
    k_cache[n_live:] = float("nan")
    v_cache[n_live:] = float("nan")
    step()
    fork([0, -1, -1, 2])
    resize([lens[0], 0, 0, 0])
    assert int((refs > 0).sum()) == -(-lens[0] // ps)


def test_sparse_attention_with_the_dagger_rerank(M):
    rng = np.random.default_rng(3)
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().cuda()
    qi, ki = f(2, 1, 8, 128), f(2, 500, 128)
    w = torch.from_numpy(rng.standard_normal((2, 1, 8))).float().cuda()
    pos = i32([[499], [300]])
    table = i32(rng.permutation(16).reshape(2, 8))
    k, v, q = f(16, 64, 1, 64), f(16, 64, 1, 64), f(2, 1, 4, 64)
    out, idx, heads = M.misa_sparse_attention(qi, w, ki, pos, 64, 2, 32, q, k, v, table, kprime=64)
    want, _, _, h2 = M.misa_dagger(qi, w, ki, pos, 64, 2, 32, 64)
    assert torch.equal(idx, want) and torch.equal(heads, h2)
    assert torch.equal(out, M.misa_paged_attention(q, k, v, table, pos, idx=idx))
    with pytest.raises(ValueError):
        M.misa_sparse_attention(qi, w, ki, pos, 64, 2, 32, q, k, v, table, k_new=k)


def test_a_wait_that_runs_out_is_reported(M):
    """The tensor-core form with short waits and one key tile never loaded: the call reports the
    timeout, and the next ones on the same context are right."""
    c = Case([400 - 9 * i for i in range(40)], Hq=100, Hkv=1, ps=7)
    assert form(M, c) == "tc"
    a = [x.cuda() for x in (c.q, c.k, c.v)] + [torch.from_numpy(x).cuda() for x in (c.table, c.pos)]
    ref = M.misa_paged_attention(*a)
    assert M.misa_check_device_status("cuda") == 0
    same = M.misa_testing_paged_attention_wait_expiry(*a, wait_cycles=2_000_000, skip_tile=-1)
    assert M.misa_check_device_status("cuda") == 0 and torch.equal(same, ref)
    for tile in (0, 1):
        M.misa_testing_paged_attention_wait_expiry(*a, wait_cycles=2_000_000, skip_tile=tile)
        with pytest.raises(M.MisaError) as e:
            M.misa_check_device_status("cuda")
        assert e.value.status == 4
        assert torch.equal(M.misa_paged_attention(*a), ref)
        assert M.misa_check_device_status("cuda") == 0


def test_output_aligned_to_16_bytes_only(M):
    c = Case([90, 60], Hq=40, Hkv=1, d=64)
    ref, _ = c.run(M)
    buf = torch.zeros(ref.numel() + 8, dtype=ref.dtype, device="cuda")
    out = buf[8:].view(ref.shape)
    assert out.data_ptr() % 32 == 16
    c.run(M, out=out)
    assert torch.equal(out, ref) and bool((buf[:8] == 0).all())


def test_compact_a_large_pool(M):
    """More pages than the plan holds at once per CTA."""
    rng = np.random.default_rng(9)
    num, nseq, mp = 400_000, 500, 200
    perm = rng.permutation(num)[:nseq * mp].reshape(nseq, mp)
    refs = np.zeros(num, dtype=np.int32)
    refs[perm] = 1
    table = perm.astype(np.int32)
    table[:, 150:] = -1
    rt, rr, n, _ = po.compact(table.tolist(), refs.tolist())
    ot, orf, live = M.misa_pages_compact(i32(table), i32(refs))
    assert M.misa_check_device_status("cuda") == 0 and live.item() == n
    assert np.array_equal(ot.cpu().numpy(), np.array(rt)) and orf.cpu().tolist() == rr
