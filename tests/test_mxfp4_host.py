"""The 4-bit cache and the page operators on the host: the format's reference
against its definition, the allocator's fork and compact against a plain model,
and every refusal before a launch (no GPU)."""
import numpy as np
import pytest
import torch

import mxfp4_ref as mx
import paged_kv_cache_448_b200 as pk
from paged_kv_cache_448_b200 import _native

BAD, UNSUP, OK = _native.PA_ERR_INVALID_ARG, _native.PA_ERR_UNSUPPORTED, _native.PA_OK
P = 1 << 20                     # any aligned address; never touched


def test_reference_format():
    x = np.zeros((3, 64))
    x[0, :8] = [6, 5, -5, 2.5, 0.25, -0.75, 1.25, 7.9]      # scale 1: amax in [4, 8)
    x[0, 32] = 2.0 ** 100
    x[1, 0] = np.inf
    x[1, 32:] = -3 * 2.0 ** -140                            # below the smallest scale
    x[2, 5] = np.nan
    codes, scales = mx.encode(x)
    assert scales.tolist() == [[127, 225], [255, 1], [255, 1]]
    v = mx.values(codes, scales)
    # nearest of the eight magnitudes; ties to the even code; saturating at 6
    assert v[0, :8].tolist() == [6, 4, -4, 2, 0, -1, 1, 6]
    assert v[0, 32] == 2.0 ** 100 and not v[0, 33:].any()
    assert np.isnan(v[1, :32]).all() and (v[1, 32:] == 0).all() and np.isnan(v[2, :32]).all()
    # every code value times every power of two is itself
    for b in (1, 64, 127, 200, 252):
        y = np.tile(mx.MAGNITUDES, 4) * 2.0 ** (b - 127.0)
        c, s = mx.encode(y[None])
        assert s[0, 0] == b and (mx.values(c, s)[0] == y).all()


def state(a):
    return a.free_list(), [a.refcount(i) for i in range(a.num_blocks)]


@pytest.mark.parametrize("partial", [True, False])
def test_allocator_fork(partial):
    a = pk.BlockAllocator(12)
    ids = a.allocate(4)
    fresh = a.fork(ids, partial, 3)
    assert fresh == ([4, 5, 6] if partial else [-1, -1, -1])
    want = [4, 4, 4, 1 if partial else 4] + ([1, 1, 1] if partial else [0, 0, 0]) + [0] * 5
    assert [a.refcount(i) for i in range(12)] == want
    # every child and the parent can be freed once
    for f in fresh:
        a.free(ids[:-1] + [f if partial else ids[-1]])
    a.free(ids)
    assert a.num_free == 12


def test_allocator_fork_all_or_nothing():
    a = pk.BlockAllocator(6)
    ids = a.allocate(4)
    before = state(a)
    with pytest.raises(pk.PagedError) as e:
        a.fork(ids, True, 3)
    assert e.value.status == _native.PA_ERR_OOM and state(a) == before
    for bad in ([0, 5], [0, -1], [0, 6], []):
        with pytest.raises(pk.PagedError) as e:
            a.fork(bad, True, 1)
        assert e.value.status == BAD and state(a) == before
    assert a.fork(ids, False, 0) == [] and state(a) == before
    assert a.fork([], False, 2) == [-1, -1] and state(a) == before


def test_allocator_compact_against_model():
    rng = np.random.default_rng(3)
    for trial in range(60):
        n = int(rng.integers(1, 60))
        a = pk.BlockAllocator(n)
        held = a.allocate(int(rng.integers(0, n + 1)))
        for b in held:
            if rng.random() < 0.3:
                a.share(b)
        rng.shuffle(held)
        gone, kept = held[:len(held) // 2], held[len(held) // 2:]
        for b in gone:
            while a.refcount(b):
                a.free([b])
        hashes = {}
        for b in kept[::2]:
            h = bytes(rng.integers(0, 256, 32).astype(np.uint8))
            a.register_hash(b, h)
            hashes[h] = b
        refs = {b: a.refcount(b) for b in kept}
        moves = a.compact()
        L = len(kept)
        assert moves.dtype == np.int32 and moves.shape == (sum(b >= L for b in kept), 2)
        assert (np.diff(moves[:, 0]) > 0).all() and (np.diff(moves[:, 1]) > 0).all()
        to = {int(s): int(d) for s, d in moves}
        assert set(to) == {b for b in kept if b >= L}
        assert set(to.values()) == set(range(L)) - set(kept)
        for b in kept:
            assert a.refcount(to.get(b, b)) == refs[b]
        assert sorted(a.free_list()) == list(range(L, n))
        for h, b in hashes.items():
            assert a.lookup(h) == to.get(b, b)
        assert len(a.compact()) == 0
        assert sorted(a.allocate(n - L)) == list(range(L, n))


def test_allocator_compact_evicts_cached_blocks_it_lands_on():
    a = pk.BlockAllocator(4)
    ids = a.allocate(4)
    h = bytes(range(32))
    a.register_hash(ids[1], h)
    a.free([ids[1], ids[0]])
    assert a.lookup(h) == ids[1]
    assert a.compact().tolist() == [[2, 0], [3, 1]]
    assert a.lookup(h) < 0


def test_allocator_compact_needs_room():
    a = pk.BlockAllocator(6)
    ids = a.allocate(6)
    a.free(ids[:2])
    before = state(a)
    import ctypes
    n = ctypes.c_int32()
    out = np.zeros((1, 2), np.int32)
    assert _native.lib().pa_alloc_compact(a._h, out.ctypes.data, 1, ctypes.byref(n)) == BAD
    assert n.value == 2 and state(a) == before
    assert _native.lib().pa_alloc_compact(a._h, None, 4, ctypes.byref(n)) == BAD
    assert _native.lib().pa_alloc_compact(None, None, 0, ctypes.byref(n)) == BAD


@pytest.mark.parametrize("name", ["pa_reshape_and_cache_mxfp4", "pa_gather_cache_mxfp4"])
def test_rows_refusals(name):
    fn = getattr(_native.lib(), name)

    def call(key=P, value=P, kc=P, vc=P, ks=P, vs=P, slots=P, T=4, Hkv=2, D=128, bs=16, nb=8,
             dt=_native.PA_F16):
        return fn(key, value, kc, vc, ks, vs, slots, T, Hkv, D, bs, nb, dt, None)
    assert call(T=0) == OK
    assert call(T=-1) == call(Hkv=0) == call(nb=0) == BAD
    assert call(D=96) == call(bs=8) == UNSUP
    assert call(dt=_native.PA_FP8_E4M3) == call(dt=_native.PA_MXFP4) == UNSUP
    for arg in ("key", "value", "kc", "vc", "ks", "vs", "slots"):
        assert call(**{arg: None}) == BAD, arg
        assert call(**{arg: P + 2}) == BAD, arg
    assert call(Hkv=65537) == UNSUP


def test_decode_refusals():
    lib = _native.lib()

    def call(out=P, q=P, kc=P, vc=P, ks=P, vs=P, bt=P, mb=8, cl=P, mctx=100, S=2, H=8, Hkv=2,
             D=128, bs=16, nb=64, scale=0.1, qd=_native.PA_F16, part=0, ws=P, wsb=1 << 30):
        return lib.pa_decode_mxfp4(out, q, kc, vc, ks, vs, bt, mb, cl, mctx, S, H, Hkv, D, bs,
                                   nb, scale, qd, part, ws, wsb, None)
    assert call(S=0) == OK
    assert call(S=-1) == call(H=0) == call(mb=0) == call(nb=0) == call(mctx=-1) == BAD
    assert call(part=-1) == call(H=7) == call(scale=float("inf")) == BAD
    assert call(H=12) == call(D=96) == call(bs=8) == call(qd=_native.PA_FP8_E4M3) == UNSUP
    assert call(ws=None) == call(ws=P + 16) == call(wsb=128) == BAD
    for arg in ("out", "q", "kc", "vc", "ks", "vs", "bt", "cl"):
        assert call(**{arg: None}) == BAD, arg
        assert call(**{arg: P + 2}) == BAD, arg
    need = pk.decode_workspace_size(2, 8, 2, 128, 16, 4096, cache_dtype=pk.PA_MXFP4)
    assert need > 256 and call(mctx=4096, mb=256, wsb=need - 16) == BAD
    assert call(S=65536) == UNSUP
    # the 4-bit type belongs to the calls of its own
    assert lib.pa_decode(P, P, P, P, P, 8, P, 100, 2, 8, 2, 128, 16, 64, 0.1, _native.PA_F16,
                         _native.PA_MXFP4, None, None, 0, P, 1 << 30, None) == UNSUP


def test_chunked_prefill_refusals():
    lib = _native.lib()

    def call(out=P, q=P, cu=P, T=8, mql=8, kc=P, vc=P, ks=P, vs=P, bt=P, mb=64, cl=P, mctx=64,
             S=1, H=8, Hkv=2, D=128, bs=16, nb=64, scale=0.1, qd=_native.PA_BF16, ws=P, wsb=256):
        return lib.pa_chunked_prefill_mxfp4(out, q, cu, T, mql, kc, vc, ks, vs, bt, mb, cl, mctx,
                                            S, H, Hkv, D, bs, nb, scale, qd, ws, wsb, None)
    assert call(T=0) == call(S=0) == call(mql=0) == OK
    assert call(T=-1) == call(mql=-1) == call(Hkv=0) == call(mb=0) == call(nb=0) == BAD
    assert call(H=7) == call(scale=float("nan")) == BAD
    assert call(H=12) == call(D=96) == call(bs=8) == call(qd=_native.PA_MXFP4) == UNSUP
    assert call(ws=None) == call(ws=P + 16) == call(wsb=128) == BAD
    for arg in ("out", "q", "cu", "kc", "vc", "ks", "vs", "bt", "cl"):
        assert call(**{arg: None}) == BAD, arg
        assert call(**{arg: P + 2}) == BAD, arg
    need = pk.chunked_prefill_workspace_size(1, 8, 8, 2, 128, 8, 1024, pk.PA_MXFP4)
    assert need > 256 and call(mctx=1024, wsb=need - 16) == BAD
    assert call(S=65536) == UNSUP


def planes(*specs):
    return (_native.Plane * max(1, len(specs)))(*[_native.Plane(b, n) for b, n in specs])


def test_fork_refusals():
    lib = _native.lib()

    def call(pl=((P, 4096),), np_=None, nb=8, bs=16, bt=P, S=2, mb=4, cl=P, par=P, fr=P, n=3,
             nbt=2 * P, ncl=3 * P, err=None):
        return lib.pa_fork_sequences(planes(*pl), len(pl) if np_ is None else np_, nb, bs, bt, S,
                                     mb, cl, par, fr, n, nbt, ncl, err, None)
    assert call(n=0) == OK
    assert call(np_=-1) == call(nb=0) == call(bs=0) == call(S=0) == call(mb=0) == call(n=-1) == BAD
    assert call(pl=((None, 4096),)) == call(pl=((P + 8, 4096),)) == BAD
    assert call(pl=((P, 0),)) == call(pl=((P, 24),)) == call(pl=((P, -16),)) == BAD
    assert call(pl=((P, 2 ** 31),)) == UNSUP
    assert call(mb=2 ** 30) == UNSUP
    for arg in ("bt", "cl", "par", "fr", "nbt", "ncl"):
        assert call(**{arg: None}) == BAD, arg
        assert call(**{arg: P + 2}) == BAD, arg
    assert call(err=P + 2) == BAD
    # the new tables may not lie over the old ones
    assert call(nbt=P) == call(nbt=P + 16) == call(ncl=P) == call(ncl=P + 4) == BAD


def test_compact_refusals():
    lib = _native.lib()

    def call(pl=((P, 4096),), np_=None, nb=8, moves=P, n=2, bt=2 * P, entries=8, err=None):
        return lib.pa_compact_blocks(planes(*pl), len(pl) if np_ is None else np_, nb, moves, n,
                                     bt, entries, err, None)
    assert call(n=0) == OK
    assert call(np_=-1) == call(nb=0) == call(n=-1) == call(entries=-1) == BAD
    assert call(pl=((None, 4096),)) == call(pl=((P, 24),)) == BAD
    assert call(moves=None) == call(bt=None) == BAD
    assert call(moves=P + 4) == call(bt=P + 2) == call(err=P + 2) == BAD


def test_binding_refusals_without_a_gpu():
    D, bs = 64, 16
    kc, vc, ks, vs = pk.mxfp4_cache(5, 2, bs, D, device="cpu")
    assert kc.shape == (5, 2, 16, 32) and ks.shape == (5, 2, 16, 2) and not kc.any()
    q = torch.zeros(3, 4, D, dtype=torch.float16)
    key = torch.zeros(3, 2, D, dtype=torch.float16)
    slots = torch.zeros(3, dtype=torch.int32)
    bt, cl = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)

    def write(**kw):
        a = dict(key=key, value=key, kc=kc, vc=vc, ks=ks, vs=vs, slots=slots)
        a.update(kw)
        pk.reshape_and_cache_mxfp4(*a.values())
    for bad in (dict(key=key.float()), dict(value=key[:2]), dict(value=key.bfloat16()),
                dict(key=key.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(ks=kc), dict(kc=kc[:, :, :8]), dict(vs=vs.float()),
                dict(slots=slots.long()), dict(slots=slots[:2]),
                dict(key=torch.zeros(3, 1, D, dtype=torch.float16),
                     value=torch.zeros(3, 1, D, dtype=torch.float16))):
        with pytest.raises((ValueError, TypeError)):
            write(**bad)
    with pytest.raises(ValueError, match="CUDA"):
        write()
    ws = torch.zeros(256, dtype=torch.uint8)

    def dec(**kw):
        a = dict(out=q, query=q, kc=kc, vc=vc, ks=ks, vs=vs, bt=bt, cl=cl)
        a.update(kw)
        pk.decode_mxfp4(*a.values(), 32, 0.1, workspace=ws)
    for bad in (dict(out=q[:2]), dict(out=q.bfloat16()), dict(bt=bt.long()), dict(bt=bt[:2]),
                dict(bt=bt.t()), dict(cl=cl[:2]), dict(ks=ks[:4])):
        with pytest.raises(ValueError):
            dec(**bad)
    with pytest.raises(ValueError, match="CUDA"):
        dec()
    with pytest.raises(ValueError, match="cu_query_lens"):
        pk.chunked_prefill_mxfp4(q, q, cl, 1, kc, vc, ks, vs, bt, cl, 32, 0.1, workspace=ws)
    for bad in ([], [kc, kc[:2]], [kc.transpose(1, 2)], [kc]):
        with pytest.raises(ValueError):
            pk.CachePool(bad, 16)


def test_workspace_sizes_of_empty_calls():
    for dt in (pk.PA_F16, pk.PA_FP8_E4M3, pk.PA_MXFP4):
        assert pk.chunked_prefill_workspace_size(0, 0, 8, 2, 128, 0, 4096, dt) == 256
        assert pk.chunked_prefill_workspace_size(4, 0, 8, 2, 128, 0, 4096, dt) == 256
        assert pk.decode_workspace_size(0, 8, 2, 128, 16, 4096, cache_dtype=dt) >= 256
