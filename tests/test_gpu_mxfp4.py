"""The 4-bit (MXFP4) cache on the GPU: rows into and out of it, decode and
multi-token attention over it, against the format and the formulas in 64 bits
(mxfp4_ref)."""
import math

import numpy as np
import pytest
import torch

import mxfp4_ref as mx
import paged_kv_cache_448_b200 as pk
from gpu_helpers import Guarded, guarded_workspace, i32
from paged_kv_cache_448_b200 import _native

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- rows in and out

def odd_rows(rng, shape, dtype):
    """Rows with what a block can hold: ordinary values, zeros, ties, the type's largest and
    smallest values, infinities and NaN."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-8, 8, shape[:-1] + (1,))
    flat = x.reshape(-1, 32)
    n = len(flat)
    pick = rng.permutation(n)
    info = torch.finfo(mx.TORCH[dtype])
    flat[pick[:n // 8]] = 0.0
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, -0.25, -5.0, 4.0] * 3)[:32]
    flat[pick[n // 8:n // 4]] = ties * 2.0 ** rng.integers(-6, 6, (n // 4 - n // 8, 1))
    k = n // 4
    flat[pick[k], 3] = np.inf
    flat[pick[k + 1], 31] = np.nan
    flat[pick[k + 2], 0] = -np.inf
    flat[pick[k + 3]] = info.max
    flat[pick[k + 4]] = info.tiny
    flat[pick[k + 5]] = info.smallest_normal / 64
    flat[pick[k + 6], 1:] = 0.0
    flat[pick[k + 7]] = -0.0
    return torch.from_numpy(x).to(mx.TORCH[dtype])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hkv,D,bs,pad", [(37, 3, 64, 16, 0), (130, 1, 128, 32, 7),
                                            (9, 8, 128, 16, 2), (5, 5, 64, 32, 3)])
def test_rows_in_and_out(dtype, T, Hkv, D, bs, pad):
    rng = np.random.default_rng(T)
    nb = -(-T // bs) + 2
    key, value = odd_rows(rng, (T, Hkv, D), dtype), odd_rows(rng, (T, Hkv, D), dtype)
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    if pad:
        slots[pad - 1::pad] = -1
        slots[0] = nb * bs                                # outside the pool: not written
    sizes = (D // 2, D // 2, D // 32, D // 32)
    g = [Guarded((nb, Hkv, bs, w), torch.uint8, fill=0x5A) for w in sizes]
    pk.reshape_and_cache_mxfp4(key.cuda(), value.cuda(), *[p.t for p in g], i32(slots))
    want = [np.full((nb, Hkv, bs, w), 0x5A, np.uint8) for w in sizes]
    real = (slots >= 0) & (slots < nb * bs)
    blk, off = slots[real] // bs, slots[real] % bs
    for i, x in enumerate((key, value)):
        c, s = mx.encode(x.double().numpy()[real])
        want[i][blk, :, off], want[2 + i][blk, :, off] = c, s
    for p, w in zip(g, want):
        p.check("cache plane")
        assert np.array_equal(p.t.cpu().numpy(), w)
    # and back: other rows of the output stay as they were
    rows = [Guarded((T, Hkv, D), mx.TORCH[dtype], fill=3.0) for _ in range(2)]
    pk.gather_cache_mxfp4(rows[0].t, rows[1].t, *[p.t for p in g], i32(slots))
    for i, r in enumerate(rows):
        r.check("gathered rows")
        got = r.t.cpu()
        assert (got[torch.from_numpy(~real)] == 3.0).all()
        v = mx.values(want[i][blk, :, off], want[2 + i][blk, :, off])
        exact = torch.from_numpy(v).to(mx.TORCH[dtype])
        assert torch.equal(got[torch.from_numpy(real)].nan_to_num(-77), exact.nan_to_num(-77))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gather_every_code_and_scale(dtype):
    # 256 rows, one a scale byte, holding all 16 codes
    D, bs = 64, 16
    kc, vc, ks, vs = [p.cpu().numpy() for p in pk.mxfp4_cache(16, 1, bs, D)]
    codes = np.arange(16) * 17                            # both halves of a byte
    kc[:] = np.tile(codes, 2)
    vc[:] = np.tile(codes[::-1], 2)
    ks[:] = np.arange(256).reshape(16, 1, 16, 1)
    vs[:] = ks[:, :, ::-1]
    slots = i32(np.concatenate([np.arange(256), [5, 5]]))  # a slot read several times
    key = torch.zeros(258, 1, D, dtype=mx.TORCH[dtype], device="cuda")
    value = torch.zeros_like(key)
    pk.gather_cache_mxfp4(key, value, *[mx.to_dev(p) for p in (kc, vc, ks, vs)], slots)
    for got, c, s in ((key, kc, ks), (value, vc, vs)):
        v = mx.values(c, s).reshape(256, 1, D)
        # beyond fp32's largest number and below its smallest normal one: as fp32 has them
        v = torch.from_numpy(v).float().to(mx.TORCH[dtype])
        assert torch.equal(got[:256].cpu().nan_to_num(-77), v.nan_to_num(-77))
        assert torch.equal(got[256], got[5]) or torch.isnan(got[5]).any()


def test_rows_empty_and_one():
    planes = pk.mxfp4_cache(2, 2, 16, 64)
    empty = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    pk.reshape_and_cache_mxfp4(empty, empty, *planes, i32(np.zeros(0)))
    pk.gather_cache_mxfp4(empty, empty.clone(), *planes, i32(np.zeros(0)))
    one = torch.full((1, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    pk.reshape_and_cache_mxfp4(one, -one, *planes, i32([17]))
    k, v = torch.zeros_like(one), torch.zeros_like(one)
    pk.gather_cache_mxfp4(k, v, *planes, i32([17]))
    assert torch.equal(k, one) and torch.equal(v, -one)


# ------------------------------------------------------------- decode

def run_decode(q, cache, scale, partition=0, table=None, ctxs=None, max_ctx=None, ok=True):
    S, H, D = q.shape
    table = cache.table if table is None else table
    ctxs = cache.ctxs if ctxs is None else ctxs
    max_ctx = max(1, int(np.max(ctxs))) if max_ctx is None else max_ctx
    out = Guarded(tuple(q.shape), q.dtype, fill=float("nan"))
    ws = guarded_workspace(pk.decode_workspace_size(S, H, cache.shape[1], D, cache.bs, max_ctx,
                                                    partition, pk.PA_MXFP4))
    pk.decode_mxfp4(out.t, q, *[mx.to_dev(p) for p in cache.planes], i32(table), i32(ctxs),
                    max_ctx, scale, partition_tokens=partition, workspace=ws.t)
    torch.cuda.synchronize()
    out.check("decode output")
    ws.check("decode workspace")
    if ok:
        pk.decode_check(ws.t)
    return out.t, ws.t


CTXS = [1, 15, 16, 17, 0, 31, 32, 33, 100, 129, 300, 700]


@pytest.mark.parametrize("partition", [0, 32, 256])
@pytest.mark.parametrize("Hkv,group,D,bs,dtype", [
    (1, 1, 64, 16, "f16"), (3, 2, 64, 32, "bf16"), (2, 4, 128, 16, "bf16"),
    (2, 8, 128, 32, "f16"), (5, 1, 128, 16, "f16"), (1, 8, 64, 16, "bf16")])
def test_decode(Hkv, group, D, bs, dtype, partition):
    rng = np.random.default_rng(Hkv * 100 + group)
    cache = mx.Cache(CTXS, Hkv, D, bs, rng)
    q, qx = mx.query(rng, len(CTXS), Hkv * group, D, dtype)
    scale = 1 / math.sqrt(D)
    out, _ = run_decode(q, cache, scale, partition)
    ref, bound = mx.attention(qx, cache, [1] * len(CTXS), scale, dtype)
    mx.check(out, ref, bound, "decode")
    assert not out[CTXS.index(0)].any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_peaked_and_growing_logits(dtype, D):
    # logits that rise and fall by hundreds along the context
    rng = np.random.default_rng(8)
    ctxs = [900, 450, 33]
    cache = mx.Cache(ctxs, 2, D, 16, rng, k_rows=lambda s: rng.standard_normal(s) * 4 *
                     np.exp2(rng.integers(-4, 5, s[:3] + (1,))))
    q, qx = mx.query(rng, 3, 4, D, dtype, amp=3.0)
    scale = 0.05
    out, _ = run_decode(q, cache, scale)
    ref, bound = mx.attention(qx, cache, [1] * 3, scale, dtype)
    # a logit is a sum of |q||k| scale < 2^10 in all, off by 2^-22 of that: weights by a factor
    # of 1 +- 2^-12, the output by 2^-11 of the largest value
    top = np.abs(mx.values(cache.vc, np.where(cache.vs == 255, 0, cache.vs))).max()
    mx.check(out, ref, bound + 2.0 ** -11 * top, "decode, peaked")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", ["falling", "rising", "sink", "mixed"])
def test_decode_values_of_very_different_scales(dtype, D, order):
    """A token with a huge value and next to no weight must not cost the others theirs."""
    rng = np.random.default_rng(9)
    ctx = 200

    def v_rows(shape):
        n = shape[0] * shape[2]
        if order == "sink":
            e = np.zeros(n)
        elif order == "mixed":
            e = rng.integers(-50, 10, n).astype(float)
        else:
            e = np.linspace(9, -40, n) if order == "falling" else np.linspace(-40, 9, n)
        return rng.standard_normal(shape) * np.exp2(e.reshape(shape[0], 1, shape[2], 1))
    cache = mx.Cache([ctx], 1, D, 16, rng, spare=0, v_rows=v_rows)
    if order == "sink":      # one value of 2^30, with a logit 60 below the others
        cache.vs[cache.table[0, 1], 0, 3] = 157
        kx = np.zeros((1, 1, D))
        kx[...] = -4.0
        c, s = mx.encode(kx)
        cache.kc[cache.table[0, 1], 0, 3], cache.ks[cache.table[0, 1], 0, 3] = c[0, 0], s[0, 0]
    q = torch.ones(1, 2, D, dtype=mx.TORCH[dtype], device="cuda")
    qx = np.ones((1, 2, D))
    scale = 60.0 / (4 * D)
    out, _ = run_decode(q, cache, scale)
    ref, bound = mx.attention(qx, cache, [1], scale, dtype)
    if order == "sink":
        # its probability, some e^-60, is rounded like the others, relatively
        vals = cache.rows(0)[1][0]
        others = np.abs(np.delete(vals, 16 + 3, 0)).max(0)
        w = np.exp(-50.0) * np.abs(vals[16 + 3])
        bound = (mx.HALF_STEP[dtype] * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * others +
                 ctx * 2.0 ** -24 * others + w + 2.0 ** -25)
    mx.check(out, ref, bound, f"decode, {order} scales")


def test_decode_range_of_keys_and_queries():
    # tiny queries on huge keys and the reverse, bf16: logits of ordinary size
    rng = np.random.default_rng(10)
    for e in (-100, -40, 40, 90):
        cache = mx.Cache([75, 40], 2, 128, 16, rng, k_rows=lambda s: rng.standard_normal(s) *
                         2.0 ** -e, v_rows=lambda s: rng.standard_normal(s) * 2.0 ** 60)
        q, qx = mx.query(rng, 2, 8, 128, "bf16", amp=2.0 ** e)
        out, _ = run_decode(q, cache, 0.1)
        ref, bound = mx.attention(qx, cache, [1, 1], 0.1, "bf16")
        mx.check(out, ref, bound, f"query 2^{e}")


@pytest.mark.parametrize("partition", [0, 32])
def test_decode_nan_blocks(partition):
    rng = np.random.default_rng(11)
    ctxs = [90, 90, 90, 60]
    cache = mx.Cache(ctxs, 2, 128, 16, rng)
    q, qx = mx.query(rng, 4, 8, 128, "f16")
    clean, _ = run_decode(q, cache, 0.1, partition)
    cache.ks[cache.table[0, 2], 1, 5, 2] = 255        # K: every output row of kv-head 1
    cache.vs[cache.table[1, 0], 0, 0, 3] = 255        # V: dims 96..127 of kv-head 0
    cache.vs[cache.table[2, 5], 1, 9, 0] = 255        # V, the last token: dims 0..31
    out, _ = run_decode(q, cache, 0.1, partition)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 4:] = True
    bad[1, :4, 96:] = True
    bad[2, 4:, :32] = True
    assert torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], clean[~bad])


def test_decode_zero_scale_byte_reads_as_zero():
    rng = np.random.default_rng(12)
    cache = mx.Cache([50], 1, 64, 16, rng)
    cache.vs[:] = np.where(cache.vs == 255, 255, 0)
    q, _ = mx.query(rng, 1, 1, 64, "bf16")
    out, _ = run_decode(q, cache, 0.1)
    assert not out.any()
    # beside scales of 2^-126 and 2^-120
    cache.vs[cache.table[0, 0], 0, 3:7] = [[1, 1], [7, 7], [1, 1], [7, 1]]
    q0 = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    out, _ = run_decode(q0, cache, 0.1)
    ref, bound = mx.attention(np.zeros((1, 1, 64)), cache, [1], 0.1, "bf16")
    # fp32 and bf16 hold multiples of 2^-149 and 2^-133 there
    mx.check(out, ref, bound + 2.0 ** -133 + 50 * 2.0 ** -149, "tiny scales")


def test_decode_reports_bad_tables():
    rng = np.random.default_rng(13)
    cache = mx.Cache([40, 40], 1, 64, 16, rng)
    q, qx = mx.query(rng, 2, 1, 64, "f16")
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):
        table = cache.table.copy()
        table[0, 1] = bad
        out, ws = run_decode(q, cache, 0.1, table=table, ok=False)
        with pytest.raises(pk.PagedError) as e:
            pk.decode_check(ws)
        assert e.value.status == _native.PA_ERR_BAD_TABLE
        ref, bound = mx.attention(qx, cache, [1, 1], 0.1, "f16")
        mx.check(out[1:], ref[1:], bound[1:], "the other sequence")
        assert torch.isfinite(out).all()
    # a context longer than the call's limit is clipped and reported
    out, ws = run_decode(q, cache, 0.1, max_ctx=33, ok=False)
    with pytest.raises(pk.PagedError):
        pk.decode_check(ws)
    short = mx.Cache([33, 33], 1, 64, 16, np.random.default_rng(0))
    short.__dict__.update(cache.__dict__)
    short.ctxs = np.array([33, 33], np.int32)
    ref, bound = mx.attention(qx, short, [1, 1], 0.1, "f16")
    mx.check(out, ref, bound, "clipped")


def test_decode_uses_up_an_injection():
    """Decode over a 4-bit cache has no wait that could run out."""
    rng = np.random.default_rng(14)
    cache = mx.Cache([300, 100], 2, 128, 16, rng)
    q, qx = mx.query(rng, 2, 4, 128, "f16")
    ref, bound = mx.attention(qx, cache, [1, 1], 0.1, "f16")
    pk.inject_wait_timeout(5, 20_000_000)
    mx.check(run_decode(q, cache, 0.1)[0], ref, bound, "decode")
    mx.check(run_chunk(q, cache, [1, 1], 0.1)[0], ref, bound, "the next call")


# ------------------------------------------------------------- several tokens

def run_chunk(q, cache, qlens, scale, ctxs=None, table=None, max_ctx=None, ok=True):
    ctxs = cache.ctxs if ctxs is None else ctxs
    table = cache.table if table is None else table
    T, H, D = q.shape
    max_ctx = max(1, int(np.max(ctxs))) if max_ctx is None else max_ctx
    cu = np.concatenate([[0], np.cumsum(qlens)])
    out = Guarded(tuple(q.shape), q.dtype, fill=float("nan"))
    ws = guarded_workspace(pk.chunked_prefill_workspace_size(
        len(qlens), T, H, cache.shape[1], D, max(qlens), max_ctx, pk.PA_MXFP4))
    pk.chunked_prefill_mxfp4(out.t, q, i32(cu), max(qlens), *[mx.to_dev(p) for p in cache.planes],
                             i32(table), i32(ctxs), max_ctx, scale, workspace=ws.t)
    torch.cuda.synchronize()
    out.check("multi-token output")
    ws.check("multi-token workspace")
    if ok:
        pk.decode_check(ws.t)
    return out.t, ws.t


@pytest.mark.parametrize("qlens,ctxs", [
    ([1, 1, 1], [1, 16, 47]),                         # single tokens
    ([3, 0, 8, 1], [3, 20, 300, 65]),                 # drafts; a sequence without queries
    ([40, 17, 64], [40, 200, 64]),                    # one row group
    ([150, 1, 130, 33], [150, 700, 385, 33]),         # long ragged chunks
    ([300], [1100])])                                 # one sequence, split key range
@pytest.mark.parametrize("Hkv,group,D,bs,dtype", [
    (2, 1, 128, 16, "f16"), (1, 8, 128, 32, "bf16"), (2, 4, 64, 16, "bf16"),
    (3, 2, 64, 32, "f16"), (1, 2, 128, 16, "bf16")])
def test_chunks(qlens, ctxs, Hkv, group, D, bs, dtype):
    rng = np.random.default_rng(len(qlens) * 10 + group)
    cache = mx.Cache(ctxs, Hkv, D, bs, rng)
    q, qx = mx.query(rng, sum(qlens), Hkv * group, D, dtype)
    scale = 1 / math.sqrt(D)
    out, _ = run_chunk(q, cache, qlens, scale)
    ref, bound = mx.attention(qx, cache, qlens, scale, dtype)
    mx.check(out, ref, bound, "chunks")


def test_chunks_of_one_token_are_decode():
    rng = np.random.default_rng(21)
    ctxs = [33, 700, 1, 64]
    cache = mx.Cache(ctxs, 2, 128, 16, rng)
    q, qx = mx.query(rng, 4, 8, 128, "bf16")
    ref, bound = mx.attention(qx, cache, [1] * 4, 0.09, "bf16")
    mx.check(run_chunk(q, cache, [1] * 4, 0.09)[0], ref, bound, "chunks of one token")
    mx.check(run_decode(q, cache, 0.09)[0], ref, bound, "decode")


def test_chunks_many_short_units():
    # enough units of a few draft tokens to fill the GPU without a split
    rng = np.random.default_rng(22)
    n = 160
    ctxs = [int(c) for c in rng.integers(8, 260, n)]
    qlens = [int(x) for x in rng.integers(1, 9, n)]
    cache = mx.Cache(ctxs, 2, 64, 16, rng)
    q, qx = mx.query(rng, sum(qlens), 8, 64, "f16")
    out, _ = run_chunk(q, cache, qlens, 0.125)
    ref, bound = mx.attention(qx, cache, qlens, 0.125, "f16")
    mx.check(out, ref, bound, "short units")


@pytest.mark.parametrize("Hkv,group,D,dtype,n,qlen", [
    (2, 8, 128, "bf16", 80, 8), (1, 1, 128, "f16", 3, 100), (1, 2, 64, "bf16", 2, 200)])
def test_chunks_whose_rows_maxima_grow_apart(Hkv, group, D, dtype, n, qlen):
    """Keys that grow along the context with a few large channels: the running maxima of a
    warp's rows move at different steps."""
    rng = np.random.default_rng(27)
    ctxs = [int(c) for c in rng.integers(500, 700, n)]

    def k_rows(shape):
        return (rng.standard_normal(shape) * (1 + 3 * (rng.random(D) < 0.06)) *
                np.exp2(rng.uniform(-2, 2, shape[:1] + (1, 1, 1))))
    cache = mx.Cache(ctxs, Hkv, D, 16, rng, k_rows=k_rows)
    q, qx = mx.query(rng, n * qlen, Hkv * group, D, dtype, amp=2.0)
    scale = 1 / math.sqrt(D)
    out, _ = run_chunk(q, cache, [qlen] * n, scale)
    ref, bound = mx.attention(qx, cache, [qlen] * n, scale, dtype)
    # a logit is a sum of |q||k| scale < 2^10 in all, off by 2^-22 of that: weights by a factor
    # of 1 +- 2^-12, the output by 2^-11 of the largest value
    top = np.abs(mx.values(cache.vc, np.where(cache.vs == 255, 0, cache.vs))).max()
    mx.check(out, ref, bound + 2.0 ** -11 * top, "growing maxima")


def test_chunks_bf16_full_range():
    """A bf16 query takes every scale the format has, and values down to 2^-36 of the largest."""
    rng = np.random.default_rng(23)
    for e in (-110, -30, 30, 100):
        cache = mx.Cache([60, 130], 1, 128, 16, rng,
                         k_rows=lambda s: rng.standard_normal(s) * 2.0 ** -e,
                         v_rows=lambda s: rng.standard_normal(s) * 2.0 ** e)
        q, qx = mx.query(rng, 90, 2, 128, "bf16", amp=2.0 ** e)
        out, _ = run_chunk(q, cache, [30, 60], 0.1)
        ref, bound = mx.attention(qx, cache, [30, 60], 0.1, "bf16")
        mx.check(out, ref, bound, f"query 2^{e}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("qlen", [3, 100, 300])
def test_chunks_bf16_large_value_with_no_weight(D, qlen):
    """One value 2^20 times the others whose weight is next to nothing: the others' sum keeps its
    accuracy (2^-17 of them: f16's 2^-11, its exponent's 36 powers of two less the 20)."""
    rng = np.random.default_rng(28)
    cache = mx.Cache([400], 1, D, 16, rng, spare=0)
    at = (int(cache.table[0, 3]), 0, 7)
    cache.vs[at] = 147
    c, sc = mx.encode(np.full((1, D), -4.0))
    cache.kc[at], cache.ks[at] = c[0], sc[0]
    q = torch.ones(qlen, 1, D, dtype=torch.bfloat16, device="cuda")
    scale = 40.0 / (4 * D)
    out, _ = run_chunk(q, cache, [qlen], scale)
    ref, bound = mx.attention(np.ones((qlen, 1, D)), cache, [qlen], scale, "bf16")
    others = np.abs(np.delete(cache.rows(0)[1][0], 3 * 16 + 7, 0)).max(0)
    # the large value's weight is below e^-38 / 100; the rest as for the others alone
    bound = (mx.HALF_STEP["bf16"] * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * others +
             400 * 2.0 ** -24 * others + math.exp(-38) * 2.0 ** 23)
    mx.check(out, ref, bound, "large value")


def test_chunks_f16_range():
    """An f16 query reads the cache as f16: exact for what f16 rows give, larger scales as
    2^13."""
    rng = np.random.default_rng(24)
    v = torch.from_numpy(rng.standard_normal((6, 1, 16, 128)) *
                         2.0 ** rng.integers(-14, 13, (6, 1, 16, 1))).half().double().numpy()
    cache = mx.Cache([90], 1, 128, 16, rng, spare=0, v_rows=lambda s: v)
    q, qx = mx.query(rng, 20, 2, 128, "f16")
    ref, bound = mx.attention(qx, cache, [20], 0.1, "f16")
    mx.check(run_chunk(q, cache, [20], 0.1)[0], ref, bound + 2.0 ** -24, "f16 rows")
    cache.vs[cache.vs < 255] = 200
    big, _ = run_chunk(q, cache, [20], 0.1)
    cache.vs[cache.vs < 255] = 140
    assert torch.equal(big, run_chunk(q, cache, [20], 0.1)[0])


def test_chunk_longer_than_its_context_and_bad_tables():
    rng = np.random.default_rng(25)
    cache = mx.Cache([10, 50], 1, 64, 16, rng)
    q, qx = mx.query(rng, 40, 2, 64, "f16")
    ref, bound = mx.attention(qx, cache, [20, 20], 0.1, "f16")
    out, ws = run_chunk(q, cache, [20, 20], 0.1, ok=False)
    with pytest.raises(pk.PagedError, match="longer"):
        pk.decode_check(ws)
    mx.check(out, ref, bound, "zeros, and the other sequence")
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):
        table = cache.table.copy()
        table[0, 0] = bad
        out, ws = run_chunk(q, cache, [5, 35], 0.1, table=table, ok=False)
        with pytest.raises(pk.PagedError) as e:
            pk.decode_check(ws)
        assert e.value.status == _native.PA_ERR_BAD_TABLE
        ref, bound = mx.attention(qx, cache, [5, 35], 0.1, "f16")
        mx.check(out[5:], ref[5:], bound[5:], "the other sequence")
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("qlens,ctxs", [([100, 30], [300, 90]), ([4, 2], [300, 90])])
def test_chunk_wait_that_runs_out(qlens, ctxs):
    rng = np.random.default_rng(26)
    cache = mx.Cache(ctxs, 1, 128, 16, rng)
    q, qx = mx.query(rng, sum(qlens), 1, 128, "bf16")
    ref, bound = mx.attention(qx, cache, qlens, 0.1, "bf16")
    pk.inject_wait_timeout(2, 20_000_000)
    out, ws = run_chunk(q, cache, qlens, 0.1, ok=False)
    with pytest.raises(pk.PagedError, match="timed out"):
        pk.decode_check(ws)
    assert torch.isfinite(out).all()
    mx.check(out[qlens[0]:], ref[qlens[0]:], bound[qlens[0]:], "the other sequence")
    out, _ = run_chunk(q, cache, qlens, 0.1)
    mx.check(out, ref, bound, "the next call")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [-0.4, 0.0])
def test_scales_of_any_sign(dtype, scale):
    """A negative softmax scale (maxima are then the smallest products), and none at all."""
    rng = np.random.default_rng(31)
    ctxs = [300, 33, 120]
    cache = mx.Cache(ctxs, 2, 128, 16, rng)
    for qlens in ([1, 1, 1], [5, 3, 2], [150, 33, 100]):
        q, qx = mx.query(rng, sum(qlens), 4, 128, dtype, amp=2.0)
        ref, bound = mx.attention(qx, cache, qlens, scale, dtype)
        # a logit is a sum of |q||k| scale < 2^9 in all, off by 2^-22 of that (see above)
        bound = bound + 2.0 ** -11 * 6
        mx.check(run_chunk(q, cache, qlens, scale)[0], ref, bound, "chunks")
        if sum(qlens) == 3:
            mx.check(run_decode(q, cache, scale)[0], ref, bound, "decode")


def test_query_with_nan_stays_in_its_row():
    rng = np.random.default_rng(32)
    cache = mx.Cache([80, 40], 2, 128, 16, rng)
    q, _ = mx.query(rng, 20, 4, 128, "bf16")
    clean = run_chunk(q, cache, [15, 5], 0.1)[0].clone()
    one = run_decode(q[:2].contiguous(), cache, 0.1)[0].clone()
    q[1, 2, 5] = float("nan")
    q[7, 0, 127] = float("inf")
    out = run_chunk(q, cache, [15, 5], 0.1)[0]
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, 2] = bad[7, 0] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])
    out = run_decode(q[:2].contiguous(), cache, 0.1)[0]
    bad = bad[:2]
    bad[1, 2] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], one[~bad])


def test_output_over_the_query():
    rng = np.random.default_rng(33)
    cache = mx.Cache([700, 40], 2, 64, 16, rng)
    q, qx = mx.query(rng, 2, 8, 64, "f16")
    planes = [mx.to_dev(p) for p in cache.planes]
    want = run_decode(q, cache, 0.1, 256)[0]
    x = q.clone()
    pk.decode_mxfp4(x, x, *planes, i32(cache.table), i32(cache.ctxs), 700, 0.1,
                    partition_tokens=256)
    assert torch.equal(x, want)
    want = run_chunk(q, cache, [1, 1], 0.1)[0]
    x = q.clone()
    pk.chunked_prefill_mxfp4(x, x, i32([0, 1, 2]), 1, *planes, i32(cache.table), i32(cache.ctxs),
                             700, 0.1)
    assert torch.equal(x, want)


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(34)
    ctxs = [int(c) for c in rng.integers(1, 3000, 24)]
    cache = mx.Cache(ctxs, 2, 128, 16, rng)
    q, _ = mx.query(rng, 24, 16, 128, "bf16")
    a = [run_decode(q, cache, 0.1)[0].clone() for _ in range(3)]
    b = [run_chunk(q, cache, [1] * 24, 0.1)[0].clone() for _ in range(3)]
    assert all(torch.equal(x, a[0]) for x in a) and all(torch.equal(x, b[0]) for x in b)


@pytest.mark.parametrize("D", [64, 128])
def test_chunks_of_long_contexts(D):
    """Contexts beyond 4096 tokens with enough rows for two groups a CTA, bf16 and f16."""
    rng = np.random.default_rng(35)
    ctxs, qlens = [4150, 300], [260, 130]
    cache = mx.Cache(ctxs, 40, D, 32, rng)
    for dtype in ("f16", "bf16"):
        q, qx = mx.query(rng, sum(qlens), 40, D, dtype)
        out, _ = run_chunk(q, cache, qlens, 1 / math.sqrt(D))
        heads = [0, 17, 39]
        sub = mx.Cache.__new__(mx.Cache)
        sub.__dict__.update(cache.__dict__)
        for name in ("kc", "vc", "ks", "vs"):
            setattr(sub, name, getattr(cache, name)[:, heads])
        ref, bound = mx.attention(qx[:, heads], sub, qlens, 1 / math.sqrt(D), dtype)
        mx.check(out[:, heads], ref, bound, f"long contexts, {dtype}")
