"""Attention over a 4-bit (MXFP4) cache at the ends of the format: keys that are all zero,
caches never written, scale bytes at both ends of their range."""
import math

import numpy as np
import pytest
import torch

import mxfp4_ref as mx
import paged_kv_cache_448_b200 as pk
from gpu_helpers import Guarded, guarded_workspace, i32

pytestmark = pytest.mark.gpu


def chunk(q, planes, table, ctxs, qlens, scale):
    T, H, D = q.shape
    Hkv = planes[0].shape[1]
    out = Guarded(tuple(q.shape), q.dtype, fill=5.0)
    ws = guarded_workspace(pk.chunked_prefill_workspace_size(
        len(qlens), T, H, Hkv, D, max(qlens), max(ctxs), pk.PA_MXFP4))
    cu = i32(np.concatenate([[0], np.cumsum(qlens)]))
    pk.chunked_prefill_mxfp4(out.t, q, cu, max(qlens), *planes, i32(table), i32(ctxs), max(ctxs),
                             scale, workspace=ws.t)
    torch.cuda.synchronize()
    out.check("output"), ws.check("workspace")
    pk.decode_check(ws.t)
    return out.t


def decode(q, planes, table, ctxs, scale, partition=0):
    S, H, D = q.shape
    Hkv, bs = planes[0].shape[1:3]
    out = Guarded(tuple(q.shape), q.dtype, fill=5.0)
    ws = guarded_workspace(pk.decode_workspace_size(S, H, Hkv, D, bs, max(ctxs), partition,
                                                    pk.PA_MXFP4))
    pk.decode_mxfp4(out.t, q, *planes, i32(table), i32(ctxs), max(ctxs), scale,
                    partition_tokens=partition, workspace=ws.t)
    torch.cuda.synchronize()
    out.check("output"), ws.check("workspace")
    pk.decode_check(ws.t)
    return out.t


# ------------------------------------------------------------- keys of zero

UNITS = {  # query lengths, contexts, query heads on one kv-head
    "doubled": ([8, 3], [300, 40], 8), "one group": ([100, 60], [300, 160], 1),
    "split": ([100], [1100], 1), "split, doubled": ([6], [900], 2)}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("byte", [0, 1])
@pytest.mark.parametrize("units", list(UNITS))
@pytest.mark.parametrize("D", [64, 128])
def test_keys_of_zero_give_the_mean(dtype, byte, units, D):
    """Keys of zero (rows of zeros are written with scale byte 1, a new cache has byte 0): every
    visible token weighs the same, whatever the query, down to its type's smallest number."""
    qlens, ctxs, group = UNITS[units]
    rng = np.random.default_rng(41)
    cache = mx.Cache(ctxs, 1, D, 16, rng)
    cache.kc[:] = 0
    cache.ks[:] = np.where(cache.ks == 255, 255, byte)
    planes = [mx.to_dev(p) for p in cache.planes]
    tiny = torch.finfo(mx.TORCH[dtype]).smallest_normal
    for amp in (1.0, 2.0 ** -12, tiny, tiny * torch.finfo(mx.TORCH[dtype]).eps, 0.0):
        for scale in (1 / math.sqrt(D), -1e-3):
            q, qx = mx.query(rng, sum(qlens), group, D, dtype, amp)
            ref, bound = mx.attention(qx, cache, qlens, scale, dtype)
            mx.check(chunk(q, planes, cache.table, ctxs, qlens, scale), ref, bound,
                     f"chunks, query {amp}")
            one = q[:len(ctxs)].contiguous()
            ref, bound = mx.attention(qx[:len(ctxs)], cache, [1] * len(ctxs), scale, dtype)
            mx.check(decode(one, planes, cache.table, ctxs, scale), ref, bound,
                     f"decode, query {amp}")


def test_two_row_groups_over_keys_of_zero():
    Hkv, qlens, ctxs = 40, [260, 130], [4150, 300]
    planes = pk.mxfp4_cache(300, Hkv, 16, 64)
    v = torch.randn(4800, Hkv, 64, device="cuda").to(torch.bfloat16)
    pk.reshape_and_cache_mxfp4(torch.zeros_like(v), v, *planes, i32(np.arange(4800)))
    back, value = torch.empty_like(v), torch.empty_like(v)
    pk.gather_cache_mxfp4(back, value, *planes, i32(np.arange(4800)))
    table = np.full((2, 260), -1, np.int32)
    table[0], table[1, :19] = np.arange(260), np.arange(260, 279)
    q = torch.full((390, Hkv, 64), 2.0 ** -12, device="cuda", dtype=torch.bfloat16)
    out = chunk(q, planes, table, ctxs, qlens, 0.125)
    at = 0
    for s, n in enumerate(qlens):
        x = value[4160 * s:4160 * s + ctxs[s]].double()
        count = torch.arange(1, ctxs[s] + 1, device="cuda", dtype=torch.float64)[:, None, None]
        mean, size = (y.cumsum(0) / count for y in (x, x.abs()))
        ref = mean[ctxs[s] - n:]
        # the output's rounding; 2^-11 a probability in f16; 2^-13 sums in fp32 (as in mxfp4_ref)
        bound = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -13) * size[ctxs[s] - n:] + \
            ctxs[s] * 2.0 ** -24 * x.abs().amax(0)
        assert ((out[at:at + n].double() - ref).abs() <= bound).all()
        at += n


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_cache_never_written(dtype):
    planes = pk.mxfp4_cache(80, 2, 16, 128)
    for qlens, ctxs in (([8, 3], [300, 40]), ([100, 60], [300, 160]), ([100], [1100])):
        table = np.arange(len(ctxs) * 69).reshape(len(ctxs), 69) % 80
        q = torch.randn(sum(qlens), 4, 128, device="cuda").mul(2.0 ** -9).to(mx.TORCH[dtype])
        assert not chunk(q, planes, table, ctxs, qlens, 0.09).any()
        assert not decode(q[:len(ctxs)].contiguous(), planes, table, ctxs, 0.09).any()


# ------------------------------------------------------------- values of zero, then a far scale

@pytest.mark.parametrize("Hkv,group,D,dtype", [
    (1, 8, 128, "bf16"), (2, 4, 128, "f16"), (1, 8, 64, "bf16"), (2, 2, 128, "bf16"),
    (1, 1, 64, "f16")])
@pytest.mark.parametrize("zero", [0, 1, 6])
def test_far_value_scales_after_values_of_zero(Hkv, group, D, dtype, zero):
    """All logits alike, so that no maximum moves; values of zero (scale bytes as a new cache and
    the writer leave them, and a larger one), and in a later step of the same warp a block of NaN
    or one of the largest scales."""
    rng = np.random.default_rng(42)
    ctxs = [300, 70]
    for far in (255, 254, 250, 248 + zero, 247):
        for at in (130, 159, 261, 299):
            cache = mx.Cache(ctxs, Hkv, D, 16, rng)
            cache.kc[:] = 0
            cache.vc[:] = 0
            for plane in (cache.ks, cache.vs):
                plane[:] = np.where(plane == 255, 255, zero)
            blk = at % (D // 32)
            where = (int(cache.table[0, at // 16]), Hkv - 1, at % 16)
            cache.vs[where + (blk,)] = far
            cache.vc[where + (slice(16 * blk, 16 * blk + 16),)] = 0x21        # 0.5 and 1
            planes = [mx.to_dev(p) for p in cache.planes]
            q, qx = mx.query(rng, 2, Hkv * group, D, dtype)
            out = decode(q, planes, cache.table, ctxs, 0.1, partition=512)
            mine = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
            mine[0, -group:, 32 * blk:32 * blk + 32] = True
            assert not out[~mine].any()
            if far == 255:
                assert torch.isnan(out[mine]).all()
            elif dtype == "f16":
                assert torch.isinf(out[mine]).all()
            else:
                ref, bound = mx.attention(qx, cache, [1, 1], 0.1, dtype)
                mx.check(out, ref, bound, f"scale byte {far}")


# ------------------------------------------------------------- the smallest and largest values

@pytest.mark.parametrize("units", list(UNITS))
@pytest.mark.parametrize("e", [-125, -122, -118, -115, -112, -60, 100])
def test_values_of_every_size(units, e):
    """Values around 2^e, bf16 (its normal numbers go down to 2^-126)."""
    qlens, ctxs, group = UNITS[units]
    rng = np.random.default_rng(43)
    cache = mx.Cache(ctxs, 1, 128, 16, rng, v_rows=lambda s: rng.standard_normal(s) * 2.0 ** e)
    planes = [mx.to_dev(p) for p in cache.planes]
    q, qx = mx.query(rng, sum(qlens), group, 128, "bf16")
    # the output and the sums are off by half a step of bf16's and fp32's smallest numbers as well
    extra = 2.0 ** -134 + max(ctxs) * 2.0 ** -149
    ref, bound = mx.attention(qx, cache, qlens, 0.1, "bf16")
    mx.check(chunk(q, planes, cache.table, ctxs, qlens, 0.1), ref, bound + extra, "chunks")
    ref, bound = mx.attention(qx[:len(ctxs)], cache, [1] * len(ctxs), 0.1, "bf16")
    mx.check(decode(q[:len(ctxs)].contiguous(), planes, cache.table, ctxs, 0.1), ref,
             bound + extra, "decode")


@pytest.mark.parametrize("units", list(UNITS))
@pytest.mark.parametrize("k,v", [(-60, 0), (-24, -20), (0, -23), (20, -10), (60, 8), (14, 13)])
def test_f16_query_over_scales_that_f16_rows_do_not_have(units, k, v):
    """Keys around 2^k (the softmax scale makes up for it) and values around 2^v, as bf16 rows
    write them: both calls read the same cache."""
    qlens, ctxs, group = UNITS[units]
    rng = np.random.default_rng(44)
    cache = mx.Cache(ctxs, 1, 64, 32, rng, k_rows=lambda s: rng.standard_normal(s) * 2.0 ** k,
                     v_rows=lambda s: np.clip(rng.standard_normal(s), -3.9, 3.9) * 2.0 ** v)
    assert cache.vs[cache.vs < 255].max() <= 140
    planes = [mx.to_dev(p) for p in cache.planes]
    q, qx = mx.query(rng, sum(qlens), group, 64, "f16", amp=3.0)
    scale = 0.1 * 2.0 ** -k
    extra = 2.0 ** -25                                   # half of f16's smallest step
    ref, bound = mx.attention(qx, cache, qlens, scale, "f16")
    mx.check(chunk(q, planes, cache.table, ctxs, qlens, scale), ref, bound + extra, "chunks")
    ref, bound = mx.attention(qx[:len(ctxs)], cache, [1] * len(ctxs), scale, "f16")
    mx.check(decode(q[:len(ctxs)].contiguous(), planes, cache.table, ctxs, scale), ref,
             bound + extra, "decode")


def test_blocks_of_f16s_smallest_numbers():
    """Values of a few times 2^-24 (scale bytes 101 and 102) are f16 numbers and read as such."""
    D = 64
    v = torch.full((16, 1, D), 2.0 ** -24, device="cuda").half()
    v[:, :, 32:] = 3 * 2.0 ** -24
    planes = pk.mxfp4_cache(1, 1, 16, D)
    pk.reshape_and_cache_mxfp4(v, v, *planes, i32(np.arange(16)))
    assert set(planes[3].flatten().tolist()) == {101, 102}
    q = torch.randn(12, 1, D, device="cuda").half()
    out = chunk(q, planes, [[0]], [16], [12], 0.1)
    assert torch.equal(out, v[:12])
    assert torch.equal(decode(q[:1].contiguous(), planes, [[0]], [16], 0.1), v[:1])


# ------------------------------------------------------------- NaN values without weight

@pytest.mark.parametrize("Hkv,group,D,dtype", [(1, 8, 128, "bf16"), (2, 1, 128, "f16"),
                                               (1, 4, 64, "bf16"), (1, 2, 64, "f16")])
@pytest.mark.parametrize("partition", [32, 512])
def test_a_nan_value_whose_weight_underflows(Hkv, group, D, dtype, partition):
    """Logits hundreds below the largest have the weight 0 in fp32; a NaN value among them, in any
    warp, partition or tile, makes its 32 outputs NaN as the formula has it (0 times NaN)."""
    rng = np.random.default_rng(45)
    ctxs = [400]
    cache = mx.Cache(ctxs, Hkv, D, 16, rng, k_rows=lambda s: np.ones(s))
    top = (int(cache.table[0, 5]), slice(None), 3)             # token 83: the largest logit by far
    c, sc = mx.encode(np.full((1, D), 6.0))
    cache.kc[top], cache.ks[top] = c[0], sc[0]
    q = torch.ones(1, Hkv * group, D, device="cuda").to(mx.TORCH[dtype])
    scale = 500.0 / (5 * D)                                    # e^-500 for the others
    clean = [mx.to_dev(p) for p in cache.planes]
    want = decode(q, clean, cache.table, ctxs, scale, partition)
    want_chunk = chunk(q, clean, cache.table, ctxs, [1], scale)
    for t in (0, 40, 70, 82, 84, 200, 399):
        spoilt = cache.vs.copy()
        spoilt[int(cache.table[0, t // 16]), 0, t % 16, 1] = 255
        planes = clean[:3] + [mx.to_dev(spoilt)]
        bad = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
        bad[:, :group, 32:64] = True
        out = decode(q, planes, cache.table, ctxs, scale, partition)
        assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], want[~bad]), t
        out = chunk(q, planes, cache.table, ctxs, [1], scale)
        assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], want_chunk[~bad]), t


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("qlens,ctxs,Hkv,group,D", [
    ([8, 3], [300, 40], 2, 8, 128), ([8], [900], 1, 4, 64), ([30, 32], [32, 64], 2, 2, 64),  # doubled
    ([100, 60], [300, 160], 2, 1, 128), ([100], [1100], 1, 1, 64),                   # one group
    ([260, 130], [4150, 300], 40, 1, 64)])                                           # two groups
def test_a_masked_nan_value_leaves_the_row_alone(qlens, ctxs, Hkv, group, D, dtype):
    """A NaN value among the call's own tokens: the rows before it do not attend to it."""
    bs = 16
    nb = [-(-c // bs) for c in ctxs]
    table = np.full((len(ctxs), max(nb)), -1, np.int32)
    for s, n in enumerate(nb):
        table[s, :n] = sum(nb[:s]) + np.arange(n)
    planes = pk.mxfp4_cache(sum(nb), Hkv, bs, D)
    rows = [torch.randn(sum(nb) * bs, Hkv, D, device="cuda").to(mx.TORCH[dtype]) for _ in range(2)]
    pk.reshape_and_cache_mxfp4(*rows, *planes, i32(np.arange(sum(nb) * bs)))
    q = torch.randn(sum(qlens), Hkv * group, D, device="cuda").to(mx.TORCH[dtype])
    clean = chunk(q, planes, table, ctxs, qlens, 0.1)
    for s, n in enumerate(qlens):
        for back in {1, 2, n // 2 + 1, n}:                     # the token of the back-th last query
            t = ctxs[s] - back
            at = (int(table[s, t // bs]), Hkv - 1, t % bs, 1)
            old = planes[3][at].clone()
            planes[3][at] = 255
            bad = torch.zeros_like(clean, dtype=torch.bool)
            end = sum(qlens[:s + 1])
            bad[end - back:end, -group:, 32:64] = True
            out = chunk(q, planes, table, ctxs, qlens, 0.1)
            assert torch.isnan(out[bad]).all(), (s, t)
            assert torch.equal(out[~bad], clean[~bad]), (s, t)
            planes[3][at] = old
