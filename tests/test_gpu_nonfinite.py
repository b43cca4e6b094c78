"""NaN keys, values and queries in multi-token attention: what a NaN belongs to is NaN
whichever way the launch shares out rows and keys, and nothing else changes by a bit."""
import math

import numpy as np
import pytest
import torch

import mxfp4_ref as mx
import paged_kv_cache_448_b200 as pk
from gpu_helpers import Guarded, guarded_workspace, i32

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


class Call:
    """A multi-token call over a cache of any type: its tensors, and what may be made NaN in them."""

    def __init__(self, cache, qdt, qlens, ctxs, Hkv, group, D, bs, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.kind, self.qlens, self.ctxs, self.group = cache, qlens, ctxs, group
        self.Hkv, self.D, self.bs = Hkv, D, bs
        need = [-(-c // bs) for c in ctxs]
        nb = sum(need) + 2
        ids = rng.permutation(nb)
        self.table = np.full((len(ctxs), max(need)), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda")
        self.q = randn(sum(qlens), Hkv * group, D).to(TORCH[qdt])
        if cache == "mxfp4":
            k, v = (randn(nb * bs, Hkv, D).to(TORCH[qdt]) for _ in range(2))
            self.planes = pk.mxfp4_cache(nb, Hkv, bs, D)
            pk.reshape_and_cache_mxfp4(k, v, *self.planes, i32(np.arange(nb * bs)))
            self.code = pk.PA_MXFP4
        else:
            self.planes = [randn(nb, bs, Hkv, D).to(TORCH[cache]) for _ in range(2)]
            self.code = {"f16": pk.PA_F16, "bf16": pk.PA_BF16, "e4m3": pk.PA_FP8_E4M3}[cache]

    def sizes(self):
        return (len(self.ctxs), sum(self.qlens), self.Hkv * self.group, self.Hkv, self.D,
                max(self.qlens), max(self.ctxs), self.code)

    def split(self):
        """The launch cuts the key range into parts (they need room in the workspace)."""
        return pk.chunked_prefill_workspace_size(*self.sizes()) > 256

    def run(self):
        out = Guarded(tuple(self.q.shape), self.q.dtype, fill=5.0)
        ws = guarded_workspace(pk.chunked_prefill_workspace_size(*self.sizes()))
        cu = i32(np.concatenate([[0], np.cumsum(self.qlens)]))
        args = (i32(self.table), i32(self.ctxs), max(self.ctxs), 1 / math.sqrt(self.D))
        if self.kind == "mxfp4":
            pk.chunked_prefill_mxfp4(out.t, self.q, cu, max(self.qlens), *self.planes, *args,
                                     workspace=ws.t)
        else:
            one = torch.ones(self.Hkv, device="cuda") if self.kind == "e4m3" else None
            pk.chunked_prefill(out.t, self.q, cu, max(self.qlens), *self.planes, *args,
                               k_scale=one, v_scale=one, workspace=ws.t)
        torch.cuda.synchronize()
        out.check("output")
        ws.check("workspace")
        pk.decode_check(ws.t)
        return out.t

    def spoil(self, which, s, t, h, dim):
        """Make dimension dim (its block of 32, for an MXFP4 cache) of token t's key or value NaN."""
        b, r = int(self.table[s, t // self.bs]), t % self.bs
        i = 0 if which == "k" else 1
        if self.kind == "mxfp4":
            self.planes[2 + i][b, h, r, dim // 32] = 255
        else:
            p = self.planes[i][b, r, h]
            p[dim:dim + 1] = torch.full((1,), float("nan"), device="cuda").to(p.dtype)

    def rows(self, s, h, t=0):
        """Output rows of sequence s that see token t, as a mask of [T, H]."""
        m = torch.zeros(self.q.shape[:2], dtype=torch.bool, device="cuda")
        q0, n = sum(self.qlens[:s]), self.qlens[s]
        first = max(0, t - (self.ctxs[s] - n))
        m[q0 + first:q0 + n, h * self.group:(h + 1) * self.group] = True
        return m

    def dims(self, dim):
        m = torch.zeros(self.D, dtype=torch.bool, device="cuda")
        if self.kind == "mxfp4":
            m[dim // 32 * 32:dim // 32 * 32 + 32] = True
        else:
            m[dim] = True
        return m


def check_nan_keys_values_queries(call, seqs, keys):
    """NaN keys (tokens `keys` of sequences `seqs`), a NaN value that every row sees, a NaN query:
    NaN exactly where the formula has it, the bits of the clean call elsewhere."""
    clean = call.run().clone()
    assert torch.isfinite(clean).all()
    q0, planes = call.q.clone(), [p.clone() for p in call.planes]

    def against(bad, what):
        out = call.run()
        assert torch.isnan(out[bad]).all(), f"{what}: a NaN was lost"
        same = torch.where(bad, clean, out).view(torch.int16) == clean.view(torch.int16)
        assert same.all(), f"{what}: other outputs changed"
        call.q.copy_(q0)
        for p, x in zip(call.planes, planes):
            p.copy_(x)

    for s in seqs:
        h, dim = s % call.Hkv, 37 % call.D
        for t in keys:
            call.spoil("k", s, t, h, dim)
            against(call.rows(s, h, t)[..., None].expand_as(clean), f"key {t} of sequence {s}")
        t = keys[0]
        call.spoil("v", s, t, h, dim)
        bad = call.rows(s, h)[..., None] & call.dims(dim)
        against(bad, f"value {t} of sequence {s}")
        row, head = sum(call.qlens[:s]) + call.qlens[s] // 2, call.group * call.Hkv - 1
        call.q[row, head, 3] = float("nan")
        bad = torch.zeros_like(clean, dtype=torch.bool)
        bad[row, head] = True
        against(bad, f"query {row}")


# ------------------------------------------------------------- split key ranges

@pytest.mark.parametrize("cache,qdt,group,D,qlen", [
    ("mxfp4", "f16", 1, 128, 100), ("mxfp4", "bf16", 2, 64, 90), ("mxfp4", "bf16", 1, 128, 300),
    ("f16", "f16", 1, 128, 40), ("bf16", "bf16", 4, 64, 12),           # mma.sync kernel
    ("bf16", "bf16", 1, 128, 150), ("f16", "f16", 2, 64, 75),          # tcgen05, one row group
    ("f16", "f16", 2, 128, 200), ("bf16", "bf16", 8, 128, 40),         # two row groups
    ("e4m3", "f16", 1, 64, 40), ("e4m3", "bf16", 1, 128, 150), ("e4m3", "bf16", 8, 128, 40)])
def test_split_key_range_keeps_nan(cache, qdt, group, D, qlen):
    call = Call(cache, qdt, [qlen, 7], [1300, 600], 2, group, D, 16, seed=qlen)
    assert call.split()
    # keys in the first, a middle and the last part, the last ones masked from some rows
    check_nan_keys_values_queries(call, [0], [3, 650, 1299 - qlen // 2, 1299])
    check_nan_keys_values_queries(call, [1], [40, 599])


# ------------------------------------------------------------- rows held twice

@pytest.mark.parametrize("cache,qdt,group,D,n,qlen", [
    ("mxfp4", "f16", 1, 128, 3, 8), ("mxfp4", "bf16", 8, 128, 80, 8), ("mxfp4", "bf16", 4, 64, 2, 1),
    ("mxfp4", "f16", 2, 64, 3, 32), ("f16", "f16", 8, 128, 150, 8), ("bf16", "bf16", 4, 64, 150, 16),
    ("e4m3", "bf16", 8, 128, 150, 8)])
@pytest.mark.parametrize("ctx", [90, 700])
def test_rows_held_twice_keep_nan(cache, qdt, group, D, n, qlen, ctx):
    """Units of at most 64 rows: each row is in two lanes, for the lower and the upper 32 tokens
    of every step. NaN keys in either, in the first step, a later one and the last."""
    call = Call(cache, qdt, [qlen] * n, [ctx] * n, 2, group, D, 16, seed=ctx + n)
    assert qlen * group <= 64
    if n > 3:
        assert not call.split()
    check_nan_keys_values_queries(call, [n - 1], [5, 40, ctx - 33, ctx - 1])


@pytest.mark.parametrize("cache,qdt,Hkv,D,qlens,ctxs", [
    ("mxfp4", "f16", 2, 128, [100, 70], [300, 160]),                   # one row group
    ("mxfp4", "bf16", 2, 64, [100, 300], [120, 400]),
    ("mxfp4", "f16", 40, 64, [260, 130], [4150, 300]),                 # two row groups
    ("mxfp4", "bf16", 40, 128, [260, 130], [4150, 300]),
    ("f16", "f16", 2, 128, [300, 270], [400, 300]), ("bf16", "bf16", 2, 64, [130, 70], [300, 90]),
    ("e4m3", "bf16", 2, 128, [300, 270], [400, 300]), ("bf16", "bf16", 2, 128, [9, 3], [300, 90])])
def test_whole_key_range_keeps_nan(cache, qdt, Hkv, D, qlens, ctxs):
    call = Call(cache, qdt, qlens, ctxs, Hkv, 1, D, 16, seed=ctxs[0])
    assert not call.split()
    check_nan_keys_values_queries(call, [0], [5, ctxs[0] - 40, ctxs[0] - 1])
    check_nan_keys_values_queries(call, [1], [2, ctxs[1] - 1])
