"""The paged attention (GPU) at scores and weights far from the ordinary.  Cases and oracle as in
test_gpu_paged.py."""

import math

import numpy as np
import pytest
import torch

import oracle.paged_oracle as po
from tests.test_gpu_paged import M, Case, f64, form   # noqa: F401 (M is a fixture)

pytestmark = pytest.mark.gpu

EVERY_FORM = {
    "cluster": dict(lens=[1000, 300], Hq=8, Hkv=2),
    "cluster_draft4_d64": dict(lens=[900, 130], T=4, Hq=8, Hkv=2, d=64, ps=48),
    "cluster_sel": dict(lens=[3000, 900], topk=800, Hq=8, Hkv=2),
    "ranges": dict(lens=[9000, 700], Hq=20, Hkv=2, ps=64),
    "tc_one_tile": dict(lens=[90, 33, 77], T=9, Hq=8, Hkv=2, d=64, ps=8),
    "tc_whole": dict(lens=[400 - 9 * i for i in range(40)], Hq=100, Hkv=1, ps=7),
    "tc_ranges_d64": dict(lens=[1500 - 13 * i for i in range(70)], Hq=128, Hkv=1, d=64),
    "tc_ranges_draft": dict(lens=[6000, 2500], T=10, Hq=8, Hkv=2, ps=100),
    "tc_sel": dict(lens=[3000, 2000, 900, 2500, 1000, 2800], T=6, topk=900, Hq=128, Hkv=1),
}


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("scale", [1, -1, 0.1, 1e-3])
@pytest.mark.parametrize("name", list(EVERY_FORM))
def test_large_scores(M, name, scale, dtype):
    """Scores of up to 5e8 (fp16: 5e7), whose neighbours in fp32 are tens apart.  The outputs are
    means of the values still: a weight's rounding (u up, u down in the sum of all) and the output's
    own leave 3 u, fp32 sums of 9000 terms 2 (9000 + 16) 2^-23 < 5 u in fp16.  A row whose best
    score leads by more than the scores' own errors, 2 (d + 8) 2^-23 sum |q k|, and 40 nats, has its
    value (the rest weighs less than 9000 e^-40)."""
    scale *= 0.01 if dtype == "fp16" else 0.1
    c = Case(**EVERY_FORM[name], dtype=dtype, poison=False, seed=3, scale=scale)
    assert form(M, c) == name.split("_")[0]
    c.q.mul_(4000)
    c.k.mul_(8000)
    assert torch.isfinite(c.q).all() and torch.isfinite(c.k).all()
    out, lse = c.run(M)
    assert M.misa_check_device_status(out.device) == 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    u, d = torch.finfo(c.q.dtype).eps / 2, c.q.shape[-1]
    assert float(out.float().abs().max()) <= float(c.v.float().abs().max()) * (1 + 8 * u)
    q, k, v, got, lse = f64(c.q), f64(c.k), f64(c.v), f64(out), f64(lse)
    G, clear = q.shape[2] // k.shape[2], 0
    for n in (0, 1, len(c.lens) - 1):
        t = c.T - 1
        seen = c.seen(n, t)
        pages, offs = [c.table[n, s // c.ps] for s in seen], [s % c.ps for s in seen]
        for j in range(q.shape[2]):
            kk = k[pages, offs, j // G]
            z = scale * (kk @ q[n, t, j])
            err = 2 * (d + 8) * 2.0 ** -23 * abs(scale) * (np.abs(kk) @ np.abs(q[n, t, j])).max()
            top = int(z.argmax())
            assert abs(lse[n, t, j] - z[top]) <= err + np.log(len(seen)) + 2.0 ** -20 * abs(z[top])
            if z[top] - np.partition(z, -2)[-2] > err + 40:
                clear += 1
                want = v[pages[top], offs[top], j // G]
                assert np.all(np.abs(got[n, t, j] - want) <= 4 * u * np.abs(want) + 1e-7)
    assert clear > 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("name", list(EVERY_FORM))
def test_scores_beyond_the_largest_show(M, name, sign, dtype):
    """Scores of 1e9 and more, in every row, are NaN, not a row that sees nothing."""
    c = Case(**EVERY_FORM[name], dtype=dtype, poison=False, scale=2.0)
    c.q.zero_()
    c.q[..., 0] = 30000
    c.k[..., 0] = sign * (20000 + 10000 * c.k[..., 0].abs())
    out, lse = c.run(M)
    assert M.misa_check_device_status(out.device) == 0
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("where", ["first", "last", "spread"])
@pytest.mark.parametrize("name", list(EVERY_FORM))
def test_scores_far_below_the_largest_weigh_nothing(M, name, where, dtype):
    """Tokens whose scores are -1.8e9, beyond what a row's largest may be: the outputs are those of
    the other tokens (Case.check's bound over them), wherever in the sequence they stand."""
    c = Case(**EVERY_FORM[name], dtype=dtype, poison=False, seed=6, scale=2.0)
    assert form(M, c) == name.split("_")[0]
    d = c.q.shape[-1]
    c.q[..., 0] = 30000
    c.k.mul_(0.05)
    c.k[..., 0] = 0
    low = [set(range(min(x, 70))) if where == "first" else set(range(x - 3, x)) if where == "last"
           else set(range(0, x, 3)) for x in c.lens]
    for n, tokens in enumerate(low):
        for s in tokens:
            c.k[c.table[n, s // c.ps], s % c.ps, :, 0] = -30000
    out, lse = c.run(M)
    assert M.misa_check_device_status(out.device) == 0
    q, k, v, got, lse = f64(c.q), f64(c.k), f64(c.v), f64(out), f64(lse)
    u, e, rows = torch.finfo(c.q.dtype).eps / 2, 2.0 ** -23, 0
    q0 = q.copy()
    q0[..., 0] = 0                    # adds nothing to the other tokens' scores, nor their errors
    for n in (0, 1, len(c.lens) - 1):
        for t in {0, c.T - 1}:
            seen = [s for s in c.seen(n, t) if s not in low[n]]
            if not seen:
                assert not c.seen(n, t) or np.isnan(got[n, t]).all()
                continue
            rows += 1
            ref, rl, mean, mag = po.attention_row(q0[n, t], k, v, c.table[n], c.ps, seen, c.scale)
            S, dz = len(seen), (d + 8) * e * mag
            w = u + 2 * dz + 2.0 ** -22 + 2 * (S + 16) * e
            bound = u * 1.02 * np.abs(ref) + w[:, None] * mean + torch.finfo(c.q.dtype).tiny * u
            if dtype == "fp16":       # small weights: see below
                bound += S * 2.0 ** -36 * np.abs(v).max()
            assert np.all(np.abs(got[n, t] - ref) <= bound), (n, t)
            assert np.all(np.abs(lse[n, t] - rl)
                          <= dz + 2.0 ** -22 + (S + 16) * e + 4 * e * np.abs(rl)), (n, t)
    assert rows > 0


@pytest.mark.parametrize("name", ["cluster", "ranges", "tc_one_tile", "tc_whole"])
def test_scores_beyond_fp32_show(M, name):
    """A finite product q k whose scale times it is none: NaN, not a row that sees nothing."""
    c = Case(**EVERY_FORM[name], poison=False, scale=4.0)
    c.q.zero_()
    c.q[..., 0] = 2.0 ** 63
    c.k[..., 0] = 2.0 ** 63
    out, lse = c.run(M)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [11, 14, 17, 18])
@pytest.mark.parametrize("name", list(EVERY_FORM))
def test_an_attention_sink_over_a_long_tail(M, name, gap, dtype):
    """A token with a zero value scores `gap` nats above all others, whose small weights make the
    whole output.  The bound is Case.check's, and for fp16, whose steps below 2^-14 are 2^-24: a
    weight is off by half a step, 2^-25, where the largest weight of its part is 2^11 at least, and
    no part's largest score exceeds the row's.  So the sum over S tokens is off by S 2^-36 max|v|
    more, over a sum of weights of 1 at least (both relative to the row's largest weight)."""
    c = Case(**EVERY_FORM[name], dtype=dtype, poison=False, seed=gap)
    assert form(M, c) == name.split("_")[0]
    d = c.q.shape[-1]
    c.q[..., 0] = 8
    c.k.mul_(0.05)
    c.k[..., 0] = 0
    c.v = (100 + 10 * c.v.float()).to(c.v.dtype)
    for n in range(len(c.lens)):
        at = 0 if n % 2 == 0 else c.lens[n] // 3         # first, or in the middle
        page, off = c.table[n, at // c.ps], at % c.ps
        c.k[page, off] = 0
        c.k[page, off, :, 0] = gap / (8 * c.scale)
        c.v[page, off] = 0
        if c.topk:
            for t in range(c.T):
                if at not in c.idx[n, t]:
                    c.idx[n, t, c.topk // 2] = at
    out, lse = c.run(M)
    assert M.misa_check_device_status(out.device) == 0
    q, k, v, got, lse = f64(c.q), f64(c.k), f64(c.v), f64(out), f64(lse)
    u, e = torch.finfo(c.q.dtype).eps / 2, 2.0 ** -23
    least = torch.finfo(c.q.dtype).tiny * u
    for n in (0, 1, len(c.lens) - 1):
        for t in {0, c.T - 1}:
            seen = c.seen(n, t)
            ref, rl, mean, mag = po.attention_row(q[n, t], k, v, c.table[n], c.ps, seen, c.scale)
            S, dz = len(seen), (d + 8) * e * mag
            w = u + 2 * dz + 2.0 ** -22 + 2 * (S + 16) * e
            bound = u * 1.02 * np.abs(ref) + w[:, None] * mean + least
            if dtype == "fp16":
                bound += S * 2.0 ** -36 * np.abs(v).max()
            err = np.abs(got[n, t] - ref)
            assert np.all(err <= bound), (n, t, float((err / bound).max()))
            assert np.all(np.abs(lse[n, t] - rl)
                          <= dz + 2.0 ** -22 + (S + 16) * e + 4 * e * np.abs(rl)), (n, t)
            assert 0 < ref.mean() < 60 and math.isfinite(rl.sum())


# ------------------------------------------------------- values that only some queries see

DRAFTS = {
    "cluster_draft4": dict(lens=[900, 40, 2, 130], T=4),
    "cluster_draft16_d64": dict(lens=[700, 64], T=16, Hq=4, Hkv=2, d=64, dtype="fp16", ps=48),
    "ranges_draft4_d64": dict(lens=[3000, 2, 30000], T=4, Hq=8, Hkv=2, d=64, ps=128),
    "ranges_draft8": dict(lens=[9000, 20000], T=8, Hq=8, Hkv=2, ps=64),
    "tc_one_tile": dict(lens=[90, 33, 77], T=9, Hq=8, Hkv=2, d=64, ps=8, dtype="fp16"),
    "tc_whole_draft": dict(lens=[7 * i for i in range(60)], T=16, Hq=8, Hkv=1, d=64, ps=32),
    "tc_ranges_draft": dict(lens=[(i * 61) % 700 for i in range(90)], T=16, Hq=8, Hkv=2, ps=100),
    "tc_long_one": dict(lens=[70000], T=5, Hq=8, Hkv=1, ps=64),
    "tc_two_blocks": dict(lens=[2300 - 40 * i for i in range(20)], T=16, Hq=12, Hkv=1, d=64, ps=32),
}


def classes(t):
    """Finite values as they are, one number for each kind of the others."""
    return torch.nan_to_num(t.float().cpu(), 7e7, 8e7, 9e7)


@pytest.mark.parametrize("name", list(DRAFTS))
def test_values_between_positions_far_apart(M, name):
    """Queries anywhere in their sequence, and NaN and infinite values anywhere between them: they
    show in the queries that see them and in no other; the rest is the same to the bit."""
    c = Case(**DRAFTS[name], poison=False, seed=2)
    assert form(M, c) == name.split("_")[0]
    rng = np.random.default_rng(7)
    for n, x in enumerate(c.lens):
        if x > 1:
            c.pos[n] = rng.integers(0, x, c.T)
            c.pos[n, -1], c.pos[n, 0] = x - 1, x // 9
    H, d = c.k.shape[2:]
    special = [float("nan"), float("inf"), -float("inf")]
    marks = {}
    for n, x in enumerate(c.lens):
        for _ in range(40 if len(c.lens) < 5 else 4):
            s = int(rng.integers(x // 9 + 1, x)) if x // 9 + 1 < x else x - 1
            if s >= 0:
                row = (c.table[n, s // c.ps], s % c.ps, int(rng.integers(H)), int(rng.integers(d)))
                marks[row] = (n, s, special[int(rng.integers(3))])
    for row in marks:
        c.v[row] = 0
    ref, lse = c.run(M)
    want, G = ref.float().cpu(), c.q.shape[2] // H
    for row, (n, s, x) in marks.items():
        c.v[row] = x
        for t in range(c.T):
            if c.pos[n, t] >= s:
                want[n, t, row[2] * G:(row[2] + 1) * G, row[3]] += x
    out, lse2 = c.run(M)
    assert M.misa_check_device_status(out.device) == 0
    assert torch.equal(lse, lse2) and torch.equal(classes(out), classes(want))
    assert not torch.isfinite(want).all() and torch.isfinite(want).float().mean() > 0.5


@pytest.mark.parametrize("name", list(DRAFTS))
def test_scores_of_minus_infinity_below_infinite_values(M, name):
    """A query whose scores are all -inf sees nothing, also where its tokens' values are infinite and
    shorter queries of its block do not see them.  The other columns and queries have what each
    query has in a call of its own, and infinite values of a finite score show."""
    c = Case(**DRAFTS[name], poison=False, seed=4)
    c.q.abs_().add_(0.5)
    for n, x in enumerate(c.lens):
        if x <= 20:
            continue
        c.pos[n, 0], c.pos[n, 1] = 1, 9
        for s in range(10):
            c.k[c.table[n, s // c.ps], s % c.ps, :, 7] = -float("inf")
        c.v[c.table[n, 5 // c.ps], 5 % c.ps, :, 9] = float("inf")
        at = (c.table[n, (x - 2) // c.ps], (x - 2) % c.ps)
        c.v[at][:, 3] = float("inf")
        c.v[at][:, 5] = -float("inf")
    out, lse = c.run(M)
    a = [x.cuda() for x in (c.q, c.k, c.v)]
    table, pos = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.pos).cuda()
    alone = torch.stack([M.misa_paged_attention(a[0][:, t].unsqueeze(1).contiguous(), a[1], a[2],
                                                table, pos[:, t:t + 1].contiguous(),
                                                scale=c.scale)[:, 0] for t in range(c.T)], 1)
    assert M.misa_check_device_status(out.device) == 0
    for n, x in enumerate(c.lens):
        if x > 20:
            assert bool((out[n, :2] == 0).all()) and torch.isneginf(lse[n, :2]).all()
            assert bool((alone[n, :2] == 0).all())
            assert torch.isposinf(out[n, -2:, :, 3]).all() and torch.isneginf(out[n, -2:, :, 5]).all()
    out[..., 9] = alone[..., 9] = 0              # an infinite value of weight 0: not defined
    for f in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(f(out), f(alone))


def test_one_infinite_value_does_not_hold_up_a_long_call(M):
    """Drafts whose queries lie 32767 tokens apart, one infinite value between them: only its
    neighbours are read again, so that no bounded wait of a millisecond runs out."""
    n, L, T, Hq, d, ps = 320, 32768, 8, 8, 64, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    k, v, q = r(L // ps, ps, 1, d), r(L // ps, ps, 1, d), r(n, T, Hq, d)
    table = torch.arange(L // ps, dtype=torch.int32, device="cuda").repeat(n, 1)
    pos = torch.full((n, T), L - 1, dtype=torch.int32, device="cuda")
    pos[:, 0] = 0
    v[300, 5, 0, 11] = 0
    ref = M.misa_paged_attention(q, k, v, table, pos)
    same = M.misa_testing_paged_attention_wait_expiry(q, k, v, table, pos, wait_cycles=2_000_000,
                                                      skip_tile=-1)
    assert M.misa_check_device_status("cuda") == 0 and torch.equal(same, ref)
    v[300, 5, 0, 11] = float("inf")
    out = M.misa_testing_paged_attention_wait_expiry(q, k, v, table, pos, wait_cycles=2_000_000,
                                                     skip_tile=-1)
    assert M.misa_check_device_status("cuda") == 0
    ref[:, 1:, :, 11] = float("inf")
    assert torch.equal(out, ref)


@pytest.mark.parametrize("kw", [dict(Hq=8, Hkv=2), dict(Hq=40, Hkv=1, d=64, dtype="fp16")])
def test_a_prompt_over_its_selected_tokens(M, kw):
    """Thousands of queries of one sequence, each with tokens of its own and the first ones with
    fewer than the list holds."""
    c = Case([3000], T=3000, topk=200, ps=64, poison=False, **kw)
    out, lse = c.run(M)
    assert M.misa_check_device_status(out.device) == 0
    c.check(out, lse, rows={(0, t) for t in (0, 1, 63, 199, 200, 1511, 2048, 2998, 2999)})
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
