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
