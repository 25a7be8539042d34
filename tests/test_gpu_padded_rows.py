"""Padded rows (pos = -1, GPU): the indexer's entry points select nothing for them, report nothing,
and give the other rows what they get without them; misa_sparse_attention over a ragged batch."""

import numpy as np
import pytest
import torch

import oracle.paged_oracle as po
from tests.test_gpu_paged import M, f64, i32   # noqa: F401 (M is a fixture)

pytestmark = pytest.mark.gpu


def inputs(nseq, T, H, L, seed=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((nseq, T, H, 128), generator=g).bfloat16().cuda()
    k = torch.randn((nseq, L, 128), generator=g).bfloat16().cuda()
    w = torch.randn((nseq, T, H), generator=g).cuda()
    last = torch.randint(L // 3, L - T + 1, (nseq, 1), generator=g)
    pos = (last + torch.arange(T)).int()
    pad = torch.rand((nseq, T), generator=g) < 0.4
    pad[0, 0], pad[-1, -1] = True, False
    return q, w, k, pos.cuda(), pad.cuda()


# nseq, T, H, L, B, h, topk: rows in one CTA's memory, of a given histogram, longer ones in groups
# (with and without the exact pass of its own), clusters, many queries (tensor-core router, blocks
# of queries that hold padded rows only)
SHAPES = {
    "short": (5, 1, 8, 300, 64, 3, 40),
    "few_queries": (4, 3, 16, 1000, 64, 4, 128),
    "decode_hist": (6, 1, 64, 20000, 128, 8, 2048),
    "decode_groups": (3, 1, 16, 60000, 128, 4, 2048),
    "decode_groups_large_k": (3, 1, 16, 60000, 128, 4, 8192),
    "rows_hist": (2, 5, 16, 50000, 128, 4, 1024),
    "large_k": (2, 2, 8, 30000, 128, 4, 12000),
    "prefill": (2, 600, 16, 2000, 64, 4, 256),
    "prefill_long": (1, 300, 16, 20000, 128, 4, 1024),
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_the_indexer_leaves_padded_rows_empty(M, name):
    nseq, T, H, L, B, h, topk = SHAPES[name]
    q, w, k, pos, pad = inputs(nseq, T, H, L)
    if T >= 300:
        pad[0, :290] = True          # whole blocks of queries
    padded = torch.where(pad, -1, pos).int()
    kp = M.misa_pool_keys(k, B)
    kprime = min(2 * topk, 16384)
    calls = {
        "misa": lambda p: M.misa_indexer(q, w, k, p, B, h, topk),
        "dsa": lambda p: M.dsa_score_topk(q, w, k, p, topk),
        "dagger": lambda p: M.misa_dagger(q, w, k, p, B, h, topk, kprime),
        "hisa": lambda p: M.hisa_block_filter_topk(q, w, k, kp, p, B, 8, topk, return_blocks=True),
    }
    if nseq * T * L <= 4194304 and topk <= 4096:
        heads = M.misa_route_heads(q, w, k, kp, pos, B, h)
        calls["noalloc"] = lambda p: M.misa_score_topk_noalloc(q, w, k, heads, p, topk)
    for call, f in calls.items():
        want, got = f(pos), f(padded)
        assert M.misa_check_device_status("cuda") == 0, call
        for x, y in zip(want, got):
            assert torch.equal(x[~pad], y[~pad]), call
        idx, vals = got[0], got[1]
        assert bool((idx[pad] == -1).all()) and bool(torch.isneginf(vals[pad]).all()), call
        if call in ("dagger", "hisa"):
            assert bool((got[2][pad] == -1).all()), call      # candidates, blocks
    # positions below -1 are reported still
    bad = padded.clone()
    bad[0, 0] = -2
    M.dsa_score_topk(q, w, k, bad, topk)
    with pytest.raises(M.MisaError) as e:
        M.misa_check_device_status("cuda")
    assert e.value.status == 6


def test_candidates_of_a_padded_row_are_reported(M):
    q, w, k, pos, _ = inputs(2, 2, 8, 300)
    pos[0, 1] = -1
    cand = torch.full((2, 2, 32), -1, dtype=torch.int32, device="cuda")
    cand[..., 3] = 5
    idx, vals = M.misa_dagger_rerank(q, w, k, pos, cand, 16)
    with pytest.raises(M.MisaError) as e:
        M.misa_check_device_status("cuda")
    assert e.value.status == 6
    assert bool((idx[0, 1] == -1).all()) and idx[0, 0, 0].item() == 5
    assert idx[1, 1].tolist() == [5] + [-1] * 15


@pytest.mark.parametrize("kprime", [None, 96])
def test_sparse_attention_over_a_ragged_batch(M, kprime):
    """Sequences with 0 to 4 new tokens each, padded to one batch: every row is what its oracle
    says, padded ones are empty, nothing is reported."""
    rng = np.random.default_rng(4)
    nseq, T, H, L, B, h, topk, ps, Hkv, Hq, d = 5, 4, 8, 400, 32, 3, 48, 16, 2, 8, 64
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().cuda()
    old, new = [390, 17, 0, 200, 63], [4, 1, 3, 0, 2]
    pos = np.full((nseq, T), -1, dtype=np.int32)
    for n in range(nseq):
        at = 0 if n % 2 else T - new[n]          # padding behind or in front
        pos[n, at:at + new[n]] = old[n] + np.arange(new[n])
    mp = L // ps
    table = rng.permutation(nseq * mp).reshape(nseq, mp).astype(np.int32)
    kc, vc = f(nseq * mp, ps, Hkv, d), f(nseq * mp, ps, Hkv, d)
    kn, vn, q = f(nseq, T, Hkv, d), f(nseq, T, Hkv, d), f(nseq, T, Hq, d)
    qi, ki, w = f(nseq, T, H, 128), f(nseq, L, 128), f(nseq, T, H).float()
    k0, v0 = kc.clone(), vc.clone()
    out, idx, heads = M.misa_sparse_attention(qi, w, ki, i32(pos), B, h, topk, q, kc, vc,
                                              i32(table), k_new=kn, v_new=vn, kprime=kprime)
    assert M.misa_check_device_status("cuda") == 0
    for n in range(nseq):
        for t in range(T):
            if pos[n, t] >= 0:
                k0[table[n, pos[n, t] // ps], pos[n, t] % ps] = kn[n, t]
                v0[table[n, pos[n, t] // ps], pos[n, t] % ps] = vn[n, t]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    u, e = torch.finfo(torch.bfloat16).eps / 2, 2.0 ** -23
    for n in range(nseq):
        for t in range(T):
            seen = [s for s in idx[n, t].tolist() if s >= 0]
            if pos[n, t] < 0:
                assert not seen and bool((out[n, t] == 0).all())
                continue
            assert len(seen) == min(topk, pos[n, t] + 1) and max(seen) <= pos[n, t]
            one = M.misa_indexer if kprime is None else M.misa_dagger
            more = () if kprime is None else (kprime,)
            alone = one(qi[n:n + 1, t:t + 1], w[n:n + 1, t:t + 1], ki[n:n + 1],
                        i32([[pos[n, t]]]), B, h, topk, *more)[0]
            assert set(alone[0, 0].tolist()) == set(idx[n, t].tolist())
            ref, _, mean, mag = po.attention_row(f64(q[n, t]), f64(kc), f64(vc), table[n], ps, seen,
                                                 d ** -0.5)
            w_ = u + 2 * (d + 8) * e * mag + 2.0 ** -22 + 2 * (len(seen) + 16) * e
            err = np.abs(f64(out[n, t]) - ref)
            assert np.all(err <= 1.02 * u * np.abs(ref) + w_[:, None] * mean)
