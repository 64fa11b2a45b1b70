"""Windowed and paged attention at the edges of its number formats: norms far
apart at tokens that a query sees and tokens that it does not."""

import numpy as np
import pytest
import torch

from online_kv_cache_quantize_gb300 import binding as B
from online_kv_cache_quantize_gb300 import workloads as W
from test_gpu_view import (D, OUT_TOL, Pool, _built, _check_prefill, _decode, _paged_table, _prefill,  # noqa: F401
                           _seen)

pytestmark = pytest.mark.gpu

MAX_F16 = 0x7BFF  # 65504


def _scaled_values(pool, by):
    """The pool's value norms times `by`, rounded to fp16 on both sides."""
    n = (pool.vq["norm16"].astype(np.float64) * by).astype(np.float16)
    pool.vq["norm16"] = n
    pool.v.norm.copy_(torch.from_numpy(n.view(np.int16)).reshape(pool.v.norm.shape))


@pytest.mark.parametrize("path", ["decode", "mma", "tcgen05"])
@pytest.mark.parametrize("by", [1.0, 2.0**-18])
@pytest.mark.parametrize("window,sinks", [(20, 0), (20, 3), (150, 8)])
def test_large_norms_at_unseen_tokens(path, by, window, sinks):
    """The largest finite norms at tokens that a query does not see, before its window and behind its position in
    tiles that it reads: the output does not change in a bit, whatever the size of the norms that it sees."""
    hkv, page, n, c = 2, 64, 384, 8
    pool = Pool(6 * hkv, page)
    _scaled_values(pool, by)
    table = np.random.default_rng(1).permutation(6).astype(np.int32)[None]

    def slots(tokens):
        t = np.asarray(tokens)
        return torch.from_numpy(np.concatenate([(table[0][t // page] * hkv + h) * page + t % page for h in range(hkv)])).cuda()

    def run():
        if path == "decode":
            return _decode(pool, W.query_vectors((1, 8, D), dtype="bf16", seed=8), [n - 3], hkv, window, sinks, table)[0]
        B.load().tq_prefill_force_mma_sync(1 if path == "mma" else 0)
        try:
            return _prefill(pool, W.query_vectors((1, c, 8, D), dtype="bf16", seed=9), [n - c], hkv, window, sinks, table)
        finally:
            B.load().tq_prefill_force_mma_sync(0)

    clean = run()
    if path == "decode":
        seen = set(_seen(n - 4, n - 3, window, sinks).tolist())
        pool.v.norm[slots([t for t in range(n) if t not in seen])] = MAX_F16
        assert np.array_equal(run(), clean)
        return
    # what the oracle gives for the first and the last query (before anything is planted)
    lim = OUT_TOL * by * float(pool.vq["norm16"].astype(np.float64).max() / by / np.sqrt(D))
    if path == "tcgen05":
        q = W.query_vectors((1, c, 8, D), dtype="bf16", seed=9)
        for i in (0, c - 1):
            t = _seen(n - c + i, n, window, sinks)
            for h in range(8):
                kv = h // 4
                want = pool.oracle(q[0, i, h], (table[0][t // page] * hkv + kv) * page + t % page)
                assert np.abs(clean[0, i, h] - want).max() <= lim, (i, h)
    seen = set().union(*(_seen(n - c + i, n, window, sinks).tolist() for i in range(c)))
    pool.v.norm[slots([t for t in range(n) if t not in seen])] = MAX_F16
    assert np.array_equal(run(), clean)
    pool.v.norm[slots([n - 1])] = MAX_F16  # the last query's own token
    assert np.array_equal(run()[0, :-1], clean[0, :-1])


@pytest.mark.parametrize("path", ["tcgen05", "mma"])
@pytest.mark.parametrize("hq", [2, 8])
def test_prefill_keeps_the_bits_of_an_fp32_output(path, hq):
    """An fp32 output is as exact as the unwindowed call's. With 2-bit key and value codes the centroid tables are
    exact to about 2^-22; queries, sign queries and weights in two fp16 limbs drop 2^-22 of themselves, u from three
    bf16 limbs 2^-24. What remains is the fp32 accumulation of a logit: 32 (tcgen05, 256 products in steps of 16, two
    limbs) to 64 additions, each dropping at most 2^-23 of a partial sum below 8 (a logit is about normal): rms
    sqrt(64) 2^-23 8 / sqrt(3) = 4.4e-6. An output is a mean of values of rms 1 over the 8 tokens that are seen,
    weights about 1/8: rms 4.4e-6 sqrt(8) / 8 sqrt(2) < 3e-6, and four times that is the limit. With weights in one
    limb (2^-11 / sqrt(3) off) it would be 8e-5."""
    hkv, page, n, c, window = 1, 64, 256, 64, 8
    pool = Pool(4 * hkv, page, 3, 2, seed=3)
    table = np.array([[2, 0, 3, 1]], dtype=np.int32)
    q = W.query_vectors((1, c, hq, D), dtype="bf16", seed=31)
    B.load().tq_prefill_force_mma_sync(1 if path == "mma" else 0)
    try:
        got = _prefill(pool, q, [n - c], hkv, window, 0, table)
    finally:
        B.load().tq_prefill_force_mma_sync(0)
    want = np.empty_like(got, dtype=np.float64)
    for i in range(c):
        t = _seen(n - c + i, n, window, 0)
        for h in range(hq):
            want[0, i, h] = pool.oracle(q[0, i, h], table[0][t // page] * page + t % page)
    rms = float(np.sqrt(((got - want) ** 2).mean()))
    assert rms <= 1.2e-5, rms


@pytest.mark.parametrize("path", ["decode", "tcgen05", "tcgen05 f32", "mma"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("what", ["query", "value norm", "key norm"])
def test_nan_reaches_the_rows_that_see_it(path, many, what):
    """A NaN in a query, or in a norm of every token that a query sees, gives NaN in that query's output, not a
    silent zero, and leaves the others as they were; few rows and many, which the partials are merged for
    differently, in one split and in several."""
    hkv, page, c, window = 1, 64, 6, 90
    bsz = 20 if many else 1
    n = 320
    pool = Pool(5 * bsz * hkv, page)
    table = np.arange(5 * bsz, dtype=np.int32).reshape(bsz, 5)
    dtype = torch.float32 if path == "tcgen05 f32" else torch.bfloat16
    shape = (bsz, 8, D) if path == "decode" else (bsz, c, 8, D)
    q = W.query_vectors(shape, dtype="bf16", seed=5)

    def run(q, splits):
        if path == "decode":
            return _decode(pool, q, [n] * bsz, hkv, window, 0, table, out_dtype=dtype, n_splits=splits)[0]
        B.load().tq_prefill_force_mma_sync(1 if path == "mma" else 0)
        try:
            return _prefill(pool, q, [n - c] * bsz, hkv, window, 0, table, out_dtype=dtype, n_splits=splits)
        finally:
            B.load().tq_prefill_force_mma_sync(0)

    for splits in (1, 2, 0):
        clean = run(q, splits)
        assert np.isfinite(clean).all()
        hit = np.zeros(shape[:-1], dtype=bool)
        if what == "query":
            bad = q.copy()
            at = (0, 3) if path == "decode" else (0, 2, 3)
            bad[at][17] = np.nan
            hit[at] = True
            got = run(bad, splits)
        else:
            plane = pool.v.norm if what == "value norm" else pool.k.norm
            keep = plane.clone()
            plane[:5 * page] = 0x7E00  # every token of the first sequence
            hit[0] = True
            got = run(q, splits)
            plane.copy_(keep)
        assert np.isnan(got[hit]).all(), splits
        assert np.array_equal(got[~hit], clean[~hit]), splits


@pytest.mark.parametrize("path", ["decode", "tcgen05", "tcgen05 f32", "mma"])
def test_value_norms_of_zero(path):
    """Tokens of zero values take their weight and add nothing, be it all of a sequence's tokens or the ones that
    most of the weight goes to; a row that sees nothing else is 0 to far below any other output (2^-60)."""
    hkv, page, c, n = 1, 64, 6, 128
    pool = Pool(4 * hkv, page)
    table = np.arange(4, dtype=np.int32).reshape(2, 2)
    dtype = torch.float32 if path == "tcgen05 f32" else torch.bfloat16
    shape = (2, 8, D) if path == "decode" else (2, c, 8, D)
    q = W.query_vectors(shape, dtype="bf16", seed=5)
    nv = pool.vq["norm16"].copy()
    nv[:2 * page] = 0  # the first sequence
    r = np.random.default_rng(2)
    some = 2 * page + r.permutation(2 * page)[:100]
    nv[some] = 0  # most of the second one
    pool.vq["norm16"] = nv
    pool.v.norm.copy_(torch.from_numpy(nv.astype(np.float16).view(np.int16)).reshape(pool.v.norm.shape))
    if path == "decode":
        got = _decode(pool, q, [n, n], hkv, 0, 0, table, out_dtype=dtype)[0]
        pos = [n - 1]
        got = got[:, None]
    else:
        B.load().tq_prefill_force_mma_sync(1 if path == "mma" else 0)
        try:
            got = _prefill(pool, q, [n - c] * 2, hkv, 0, 0, table, out_dtype=dtype)
        finally:
            B.load().tq_prefill_force_mma_sync(0)
        pos = list(range(n - c, n))
    assert np.abs(got[0]).max() <= 2.0**-60
    qq = q[:, None] if path == "decode" else q
    for i, at in enumerate(pos):
        t = np.arange(at + 1)
        for h in range(8):
            want = pool.oracle(qq[1, i, h], 2 * page + t)
            lim = OUT_TOL + (2.0**-8 * np.abs(want) if dtype == torch.bfloat16 else 0)
            assert (np.abs(got[1, i, h] - want) <= lim).all(), (i, h)


# --------------------------------------------- the prefill of a bf16 output ---
@pytest.mark.parametrize("kbits,vbits,bits2", [(2, 1, None), (2, 2, None), (2, 3, None), (2, 4, None), (3, 1, None), (3, 2, None),
                                               (3, 3, None), (3, 4, None), (3, 2, (2, 1)), (3, 3, (2, 2)), (3, 4, (2, 3))])
@pytest.mark.parametrize("kind", ["rht", "dense"])
def test_bf16_prefill_widths(kbits, vbits, bits2, kind):
    """Every width of the tcgen05 scan with the output type that holds its weights in one limb, over several tiles,
    missing pages among them."""
    r = np.random.default_rng(kbits * 10 + vbits)
    hkv, page, start, c = 2, 80, 300, 70
    need = -(-(start + c) // page) + 1
    pool = Pool(need * hkv, page, kbits, vbits, kind, bits2=bits2)
    table = _paged_table(r, [start + c], page, need)
    table[0, 1] = -1
    q = W.query_vectors((1, c, 2 * hkv, D), dtype="bf16", seed=14)
    got = _prefill(pool, q, [start], hkv, 200, 9, table, torch.bfloat16, torch.bfloat16)
    _check_prefill(pool, q, [start], hkv, 200, 9, table, got, bf16=True, every=23)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 4), (130, 17), (300, 200), (10**9, 10**9)])
@pytest.mark.parametrize("page", [None, 16, 48, 128])
def test_bf16_prefill_masks(window, sinks, page):
    r = np.random.default_rng(window % 1000 + sinks % 1000 + (page or 0))
    hkv, starts, c = 2, [600, 0, 131], 21
    lens = [s + c for s in starts]
    if page is None:
        pool, table = Pool(len(lens) * hkv, 640), None
    else:
        need = sum(-(-n // page) for n in lens) + 2
        pool = Pool(need * hkv, page)
        table = _paged_table(r, lens, page, need)
    q = W.query_vectors((3, c, 4 * hkv, D), dtype="bf16", seed=12)
    got = _prefill(pool, q, starts, hkv, window, sinks, table, torch.bfloat16, torch.bfloat16)
    _check_prefill(pool, q, starts, hkv, window, sinks, table, got, bf16=True, every=4)


@pytest.mark.parametrize("n_splits", [0, 1, 3, 8, 9])
def test_bf16_prefill_splits(n_splits):
    """Units in several splits, CTAs that go through several units."""
    r = np.random.default_rng(n_splits)
    hkv, page, c, group = 2, 64, 270, 4
    start = 128 * 9 - 20
    need = -(-(start + c) // page)
    pool = Pool(need * hkv, page)
    table = _paged_table(r, [start + c], page, need, holes=0.1)
    q = W.query_vectors((1, c, group * hkv, D), dtype="bf16", seed=13)
    got = _prefill(pool, q, [start], hkv, 0, 0, table, torch.bfloat16, torch.bfloat16, n_splits)
    _check_prefill(pool, q, [start], hkv, 0, 0, table, got, bf16=True, every=45)
