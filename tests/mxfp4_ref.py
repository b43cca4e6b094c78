"""The 4-bit cache format and attention over it in 64 bits (numpy), written from
the definitions: OCP Microscaling v1.0 MXFP4 (32 elements share a power of two,
each an E2M1 code), and softmax(scale q.K^T) V with the causal rule."""
from __future__ import annotations

import numpy as np
import torch

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
# half a step of the output type, relative
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def encode(x: np.ndarray):
    """float64 rows [..., D] -> (codes uint8 [..., D / 2], scale bytes uint8 [..., D / 32])."""
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(blocks).max(-1)
    bad = ~np.isfinite(blocks).all(-1)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    e = np.clip(np.floor(np.log2(safe)) - 2, -126, 125)
    e = np.where(amax == 0, -126, e)
    y = np.abs(np.where(bad[..., None], 0.0, blocks)) * 2.0 ** -e[..., None]
    dist = np.abs(y[..., None] - MAGNITUDES)
    near = dist.min(-1, keepdims=True)
    hit = dist == near
    tie = hit.sum(-1, keepdims=True) > 1
    code = np.where(tie, hit & (np.arange(8) % 2 == 0), hit).argmax(-1)
    code = code + 8 * np.signbit(blocks)
    code = np.where(bad[..., None], 0, code).reshape(*x.shape[:-1], -1, 2)
    byte = np.where(bad, 255, e + 127)
    return (code[..., 0] + 16 * code[..., 1]).astype(np.uint8), byte.astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of codes [..., D / 2] with scale bytes [..., D / 32]."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 0, 0.0, 2.0 ** (scales.astype(np.float64) - 127))
    s = np.where(scales == 255, np.nan, s)
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(v.shape)


class Cache:
    """Planes of a small pool on the host, and block tables for given context lengths."""

    def __init__(self, ctxs, Hkv, D, bs, rng, amp=1.0, spare=3, k_rows=None, v_rows=None):
        need = [-(-c // bs) for c in ctxs]
        nb = sum(need) + spare
        self.shape = (nb, Hkv, bs, D)
        k = rng.standard_normal(self.shape) * amp if k_rows is None else k_rows(self.shape)
        v = rng.standard_normal(self.shape) * amp if v_rows is None else v_rows(self.shape)
        self.kc, self.ks = encode(k)
        self.vc, self.vs = encode(v)
        ids = rng.permutation(nb)
        self.table = np.full((len(ctxs), max(1, max(need))), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.ctxs = np.array(ctxs, np.int32)
        self.bs = bs
        # rows that belong to no sequence read as NaN
        used = np.zeros((nb, bs), bool)
        for s, c in enumerate(ctxs):
            for t in range(c):
                used[self.table[s, t // bs], t % bs] = True
        for plane in (self.ks, self.vs):
            plane[np.broadcast_to(~used[:, None, :, None], plane.shape)] = 255

    @property
    def planes(self):
        return [self.kc, self.vc, self.ks, self.vs]

    def rows(self, s):
        """(K, V) float64 [Hkv, ctx, D] of sequence s."""
        c = int(self.ctxs[s])
        ids = self.table[s, :-(-c // self.bs)]
        out = []
        for codes, scales in ((self.kc, self.ks), (self.vc, self.vs)):
            v = values(codes[ids], scales[ids])                   # [n, Hkv, bs, D]
            out.append(v.transpose(1, 0, 2, 3).reshape(v.shape[1], -1, v.shape[3])[:, :c])
        return out


def attention(q, cache, qlens, scale, dtype):
    """q float64 [T, H, D] -> (out, bound): the 64-bit result and, per element, how far a
    result may be off that rounds each probability to f16 and the output to dtype.

    bound = h |out| + (2^-11 + 2^-13) sum_t w_t |v_t| + ctx 2^-24 max_t |v_t|:
      h       the output's rounding;
      2^-11   a probability rounded to f16;
      2^-13   logits, exponentials and sums in fp32 (logits below 2^6 carry an
              absolute error below 2^-17; a sum of n terms n 2^-24 at most);
      2^-24   f16's absolute step (a probability below 2^-14, before and after
              the product with a power of two), each at most 2^-25 of the largest
              value, the largest probability being at least 1.
    """
    out = np.zeros_like(q)
    bound = np.zeros_like(q)
    H, D = q.shape[1:]
    at = 0
    for s, n in enumerate(qlens):
        c = int(cache.ctxs[s])
        if n and c >= n:
            k, v = cache.rows(s)
            g = H // k.shape[0]
            k, v = k.repeat(g, 0), v.repeat(g, 0)                 # [H, c, D]
            x = np.einsum("qhd,htd->hqt", q[at:at + n], k) * scale
            late = np.arange(c)[None] > c - n + np.arange(n)[:, None]
            x[:, late] = -np.inf
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            o = np.einsum("hqt,htd->qhd", w, v)
            a = np.einsum("hqt,htd->qhd", w, np.abs(v))
            out[at:at + n] = o
            bound[at:at + n] = (HALF_STEP[dtype] * np.abs(o) + (2.0 ** -11 + 2.0 ** -13) * a +
                                c * 2.0 ** -24 * np.abs(v).max(1)[None])
        at += n
    return out, bound


def to_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def query(rng, T, H, D, dtype, amp=1.0):
    """A query on the device and its exact values."""
    t = torch.from_numpy(rng.standard_normal((T, H, D)) * amp).to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


def check(got, ref, bound, what=""):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err = np.abs(got - ref)
    worst = (err - bound).max(initial=0.0)
    if not (err <= bound).all():
        i = tuple(np.argwhere(err > bound)[0])
        raise AssertionError(f"{what}: {int((err > bound).sum())} elements beyond the bound; first "
                             f"{i}: got {got[i]!r} ref {ref[i]!r} bound {bound[i]!r} ({worst:.3g})")
