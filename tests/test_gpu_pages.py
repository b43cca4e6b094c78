"""Forking sequences and compacting the pool on the GPU, and a run of the new
operators together: writing, forking, decoding and compacting a 4-bit cache."""
import numpy as np
import pytest
import torch

import mxfp4_ref as mx
import paged_kv_cache_448_b200 as pk
from gpu_helpers import Guarded, i32

pytestmark = pytest.mark.gpu


def pool(rng, nb, shapes):
    """Guarded planes [nb, ...] of random bytes, and their host copies."""
    gs = []
    for shape, dt in shapes:
        g = Guarded((nb,) + shape, dt)
        g.raw[4096:4096 + g.n] = torch.from_numpy(rng.integers(0, 256, g.n).astype(np.uint8)).cuda()
        gs.append(g)
    return gs, [raw(g) for g in gs]


def raw(g):
    nb = g.t.shape[0]
    return g.raw[4096:4096 + g.n].cpu().numpy().reshape(nb, -1).copy()


def fork_model(host, table, ctx, parents, fresh, bs):
    n, width = len(parents), table.shape[1]
    rows, lens = np.full((n, width), -1, np.int32), np.zeros(n, np.int32)
    host = [h.copy() for h in host]
    for i, (p, f) in enumerate(zip(parents, fresh)):
        if not 0 <= p < len(table):
            continue
        c = min(max(int(ctx[p]), 0), width * bs)
        k = -(-c // bs)
        rows[i, :k], lens[i] = table[p, :k], c
        if c % bs and f >= 0:
            src = table[p, k - 1]
            rows[i, k - 1] = f if f < len(host[0]) else -1
            if 0 <= src < len(host[0]) and f < len(host[0]):
                for h in host:
                    h[f] = h[src]
    return rows, lens, host


SHAPES = {
    "one": [((16, 8, 128), torch.bfloat16)],
    "mxfp4": [((3, 16, 32), torch.uint8)] * 2 + [((3, 16, 2), torch.uint8)] * 2,
    "many": [((16, 1, 64), torch.float16)] * 300,          # more planes than one launch takes
    "odd": [((16,), torch.uint8), ((4112,), torch.uint8), ((1, 12304), torch.uint8),
            ((40, 8), torch.float32)],
}


@pytest.mark.parametrize("kind", list(SHAPES))
@pytest.mark.parametrize("bs", [16, 32])
def test_fork(kind, bs):
    rng = np.random.default_rng(bs)
    ctx = np.array([0, 1, bs, bs + 1, 3 * bs, 4 * bs - 1, 2 * bs + 5], np.int32)
    nb, width = 60, 5
    ids = rng.permutation(nb)
    table, at = np.full((len(ctx), width), -1, np.int32), 0
    for s, c in enumerate(ctx):
        k = -(-int(c) // bs)
        table[s, :k] = ids[at:at + k]
        at += k
    parents = rng.integers(0, len(ctx), 17).astype(np.int32)
    fresh = ids[at:at + 17].astype(np.int32)
    fresh[::5] = -1
    gs, host = pool(rng, nb, SHAPES[kind])
    nt, nc = Guarded((17, width), torch.int32, fill=-9), Guarded((17,), torch.int32, fill=-9)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = pk.CachePool([g.t for g in gs], bs)
    p.fork(i32(table), i32(ctx), i32(parents), i32(fresh), nt.t, nc.t, error_word=err)
    rows, lens, want = fork_model(host, table, ctx, parents, fresh, bs)
    assert np.array_equal(nt.t.cpu().numpy(), rows) and np.array_equal(nc.t.cpu().numpy(), lens)
    for g, h in zip(gs, want):
        assert np.array_equal(raw(g), h)
        g.check("plane")
    nt.check("tables"), nc.check("lengths")
    assert int(err) == 0


def test_fork_reports():
    bs, nb = 16, 10
    rng = np.random.default_rng(1)
    ctx = np.array([20, -3, 99, 20], np.int32)             # 99: more than the row has
    table = np.array([[0, 1], [2, -1], [3, 4], [-1, 77]], np.int32)
    cases = [([0, 4], [5, 6], 32), ([-1, 0], [5, 6], 32), ([1], [5], 2), ([2], [5], 2),
             ([3], [5], 1), ([0], [10], 1), ([0, 3, 4, 1], [2 ** 31 - 1, 7, 8, 9], 35)]
    for parents, fresh, word in cases:
        gs, host = pool(rng, nb, SHAPES["mxfp4"])
        nt = torch.full((len(parents), 2), -9, dtype=torch.int32, device="cuda")
        nc = torch.zeros(len(parents), dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        p = pk.CachePool([g.t for g in gs], bs)
        p.fork(i32(table), i32(ctx), i32(parents), i32(fresh), nt, nc, error_word=err)
        rows, lens, want = fork_model(host, table, ctx, parents, fresh, bs)
        assert np.array_equal(nt.cpu().numpy(), rows) and np.array_equal(nc.cpu().numpy(), lens)
        assert all(np.array_equal(raw(g), h) for g, h in zip(gs, want))
        assert int(err) == word
        p.fork(i32(table), i32(ctx), i32(parents), i32(fresh), nt, nc)     # without a word


@pytest.mark.parametrize("kind", list(SHAPES))
@pytest.mark.parametrize("n", [1, 40])
def test_compact(kind, n):
    rng = np.random.default_rng(n)
    nb = 100
    ids = rng.permutation(nb)
    src, dst = np.sort(ids[:n]), ids[n:2 * n]
    moves = np.stack([src, dst], 1).astype(np.int32)
    table = rng.integers(-1, nb, (9, 7)).astype(np.int32)
    table[0, :2] = -1, src[0]
    gs, host = pool(rng, nb, SHAPES[kind])
    tg = Guarded((9, 7), torch.int32)
    tg.t.copy_(i32(table))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.CachePool([g.t for g in gs], 16).compact(i32(moves), tg.t, error_word=err)
    to = {int(a): int(b) for a, b in moves}
    assert np.array_equal(tg.t.cpu().numpy(), np.vectorize(lambda b: to.get(int(b), int(b)))(table))
    for g, h in zip(gs, host):
        h[dst] = h[src]
        assert np.array_equal(raw(g), h)
        g.check("plane")
    tg.check("table")
    assert int(err) == 0


def test_compact_reports():
    rng = np.random.default_rng(5)
    for moves, word, kept in (([[3, 20], [4, 1]], 1, [1]), ([[-1, 2], [4, 1]], 1, [1]),
                              ([[4, 1], [3, 2]], 64, None), ([[3, 4], [4, 1]], 64, None),
                              ([[3, 1], [3, 2]], 64, None)):
        gs, host = pool(rng, 10, SHAPES["mxfp4"])
        table = i32(np.arange(-1, 10).reshape(1, 11))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pk.CachePool([g.t for g in gs], 16).compact(i32(moves), table, error_word=err)
        assert int(err) == word
        for g in gs:
            g.check("plane")
        if kept is not None:                              # the good moves are made
            want = list(range(-1, 10))
            for i in kept:
                want[moves[i][0] + 1] = moves[i][1]
            assert table.flatten().tolist() == want
            for g, h in zip(gs, host):
                for i in kept:
                    h[moves[i][1]] = h[moves[i][0]]
                assert np.array_equal(raw(g), h)


def test_empty_calls():
    planes = pk.mxfp4_cache(4, 1, 16, 64)
    p = pk.CachePool(planes, 16)
    none = i32(np.zeros(0))
    nt = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    p.fork(i32(np.zeros((2, 3))), i32([1, 2]), none, none, nt, none.clone())
    p.compact(i32(np.zeros((0, 2))), i32(np.zeros((2, 3))))
    table = i32([[3, -1]])
    p.compact(i32([[3, 0]]), table)
    assert table.tolist() == [[0, -1]]
    p.compact(i32([[3, 0]]))                              # pages alone


# ------------------------------------------------------------- together

class Serving:
    """A small serving loop over a two-layer 4-bit cache: its allocator, tables and pool."""

    def __init__(self, nb=64, Hkv=2, D=128, bs=16):
        self.bs, self.D, self.Hkv = bs, D, Hkv
        self.layers = [pk.mxfp4_cache(nb, Hkv, bs, D) for _ in range(2)]
        self.pool = pk.CachePool([p for layer in self.layers for p in layer], bs)
        self.alloc = pk.BlockAllocator(nb)
        self.seqs, self.lens = [], []

    def table(self, width=8):
        return pk.build_block_table(self.seqs, width)

    def append(self, gen, new):
        """new tokens for every sequence, the same rows for all layers."""
        slots, rows = [], []
        for i, n in enumerate(new):
            need = -(-(self.lens[i] + n) // self.bs) - len(self.seqs[i])
            if need > 0:
                self.seqs[i] = self.seqs[i] + self.alloc.allocate(need)
            slots += [self.seqs[i][t // self.bs] * self.bs + t % self.bs
                      for t in range(self.lens[i], self.lens[i] + n)]
            self.lens[i] += n
        k = torch.randn(sum(new), self.Hkv, self.D, generator=gen, device="cuda").half()
        v = torch.randn(sum(new), self.Hkv, self.D, generator=gen, device="cuda").half()
        for layer in self.layers:
            pk.reshape_and_cache_mxfp4(k, v, *layer, i32(slots))

    def decode(self, q, layer=0):
        out = torch.empty_like(q)
        return pk.decode_mxfp4(out, q, *self.layers[layer], i32(self.table()), i32(self.lens),
                               max(self.lens), 0.1)


def test_fork_decode_append_compact():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    sv = Serving()
    sv.seqs, sv.lens = [[], [], []], [0, 0, 0]
    sv.append(gen, [37, 16, 5])
    q = torch.randn(3, 8, sv.D, generator=gen, device="cuda").half()
    base = sv.decode(q)
    # three children of sequence 0, one of 1 (a full last block), two of 2
    parents = [0, 0, 0, 1, 2, 2]
    fresh = []
    for p, n in ((0, 3), (1, 1), (2, 2)):
        fresh += sv.alloc.fork(sv.seqs[p], sv.lens[p] % sv.bs != 0, n)
    nt = torch.empty(6, 8, dtype=torch.int32, device="cuda")
    nc = torch.empty(6, dtype=torch.int32, device="cuda")
    sv.pool.fork(i32(sv.table()), i32(sv.lens), i32(parents), i32(fresh), nt, nc)
    for row, c in zip(nt.cpu().tolist(), nc.cpu().tolist()):
        sv.seqs.append(row[:-(-c // sv.bs)])
        sv.lens.append(c)
    q9 = torch.cat([q, q[parents]])
    for layer in range(2):
        out = sv.decode(q9, layer)
        assert torch.equal(out[:3], base) and torch.equal(out[3:], base[parents])
    # they part ways: writing to one leaves the others
    sv.append(gen, [0, 0, 0, 1, 2, 20, 1, 1, 12])
    out = sv.decode(q9)
    assert torch.equal(out[:3], base)
    assert not torch.equal(out[3], out[4])
    # the parents end; the pages left behind move together
    for i in range(3):
        sv.alloc.free(sv.seqs[i])
    sv.seqs, sv.lens = sv.seqs[3:], sv.lens[3:]
    before = [sv.decode(q9[3:], layer) for layer in range(2)]
    moves = sv.alloc.compact()
    assert len(moves)
    live = sv.alloc.num_blocks - sv.alloc.num_free
    table = i32(sv.table())
    sv.pool.compact(i32(moves), table)
    for layer in sv.layers:                               # nothing behind them is read
        for plane in layer:
            plane[live:] = 255
    sv.seqs = [r[:len(s)] for r, s in zip(table.cpu().tolist(), sv.seqs)]
    assert max(max(s) for s in sv.seqs) < live
    for layer in range(2):
        assert torch.equal(sv.decode(q9[3:], layer), before[layer])
    for s in sv.seqs:
        sv.alloc.free(s)
    assert sv.alloc.num_free == 64


def test_captured_step_replays():
    """A step (write, decode, verify, fork, compact) in a graph, replayed on new inputs, and a
    second graph of the same calls with a workspace of its own."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    Hkv, D, bs, nb, S = 2, 64, 16, 48, 3
    width = 6
    tables = torch.randperm(nb, generator=gen, device="cuda")[:S * width].int().reshape(S, width)
    spare = [b for b in range(nb) if b not in set(tables.flatten().tolist())]
    ctx = i32([33, 80, 17])

    def make():
        planes = pk.mxfp4_cache(nb, Hkv, bs, D)
        st = dict(planes=planes, pool=pk.CachePool(planes, bs), tables=tables.clone(),
                  key=torch.zeros(S, Hkv, D, device="cuda").bfloat16(),
                  q=torch.zeros(S, 4, D, device="cuda").bfloat16(),
                  nt=torch.zeros(S, width, dtype=torch.int32, device="cuda"),
                  nc=torch.zeros(S, dtype=torch.int32, device="cuda"),
                  fresh=i32(spare[:S]), parents=i32([0, 0, 2]),
                  slots=(tables[torch.arange(S), ((ctx - 1) // bs).cpu().tolist()] * bs +
                         (ctx - 1) % bs).int().contiguous(),
                  moves=i32(sorted([[spare[4], spare[5]], [spare[6], spare[7]]])),
                  cu=i32([0, 1, 2, 3]))
        st["out"], st["out2"] = torch.zeros_like(st["q"]), torch.zeros_like(st["q"])
        st["ws"] = pk.decode_workspace(S, 4, Hkv, D, bs, 96, 32, cache_dtype=pk.PA_MXFP4)
        st["ws2"] = pk.chunked_prefill_workspace(S, S, 4, Hkv, D, 1, 96, pk.PA_MXFP4)
        return st

    def step(st):
        pk.reshape_and_cache_mxfp4(st["key"], st["key"], *st["planes"], st["slots"])
        pk.decode_mxfp4(st["out"], st["q"], *st["planes"], st["tables"], ctx, 96, 0.1,
                        partition_tokens=32, workspace=st["ws"])
        st["pool"].fork(st["tables"], ctx, st["parents"], st["fresh"], st["nt"], st["nc"])
        pk.chunked_prefill_mxfp4(st["out2"], st["q"], st["cu"], 1, *st["planes"], st["nt"],
                                 st["nc"], 96, 0.1, workspace=st["ws2"])
        st["pool"].compact(st["moves"], st["nt"])

    states = [make() for _ in range(3)]
    graphs = []
    for st in states[:2]:
        step(st)                                          # first calls outside a capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(st)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for r in range(3):
        for st in states:
            g2 = torch.Generator(device="cuda")
            g2.manual_seed(100 + r)
            st["key"].copy_(torch.randn(st["key"].shape, generator=g2, device="cuda"))
            st["q"].copy_(torch.randn(st["q"].shape, generator=g2, device="cuda"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):                 # both at once
            with torch.cuda.stream(s):
                g.replay()
        step(states[2])
        torch.cuda.synchronize()
        for st in states[:2]:
            for k in ("out", "out2", "nt", "nc"):
                assert torch.equal(st[k], states[2][k]), k
            for a, b in zip(st["planes"], states[2]["planes"]):
                assert torch.equal(a, b)
        assert states[2]["out"].any() and states[2]["out2"].any()


def test_on_another_stream_without_a_workspace():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    sv = Serving()
    sv.seqs, sv.lens = [[], []], [0, 0]
    sv.append(gen, [50, 40])
    q = torch.randn(2, 4, sv.D, generator=gen, device="cuda").half()
    table, lens = i32(sv.table()), i32(sv.lens)
    want = sv.decode(q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(q)
    pk.decode_mxfp4(out, q, *sv.layers[0], table, lens, 50, 0.1, stream=s)
    junk = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")   # reuses freed memory
    out2 = torch.empty_like(q)
    pk.chunked_prefill_mxfp4(out2, q, i32([0, 1, 2]), 1, *sv.layers[0], table, lens, 50, 0.1,
                             stream=s)
    s.synchronize()
    assert torch.equal(out, want) and junk.all()
    assert (out2.float() - want.float()).abs().max() < 2e-3


def test_pages_far_into_a_large_pool():
    """Codes that begin beyond 4 GiB of a plane: offsets of more than 32 bits."""
    Hkv, D, bs = 8, 128, 16
    nb = (1 << 32) // (Hkv * bs * D // 2) + 40            # 8 KiB of codes a block
    planes = pk.mxfp4_cache(nb, Hkv, bs, D)
    small = pk.mxfp4_cache(40, Hkv, bs, D)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    T = 150
    k = torch.randn(T, Hkv, D, generator=gen, device="cuda").bfloat16()
    v = torch.randn(T, Hkv, D, generator=gen, device="cuda").bfloat16()
    pos = torch.randperm(20 * bs, generator=gen, device="cuda")[:T].int()
    base = nb - 40
    pk.reshape_and_cache_mxfp4(k, v, *small, pos)
    for big, little in zip(planes, small):
        big[base:] = little
    far = (pos + base * bs).int()
    kk, vv, k2, v2 = (torch.zeros_like(k) for _ in range(4))
    pk.gather_cache_mxfp4(kk, vv, *small, pos)
    pk.gather_cache_mxfp4(k2, v2, *planes, far)
    assert torch.equal(kk, k2) and torch.equal(vv, v2)
    pk.reshape_and_cache_mxfp4(v, k, *small, pos)
    pk.reshape_and_cache_mxfp4(v, k, *planes, far)
    for big, little in zip(planes, small):
        assert torch.equal(big[base:], little)
    table = torch.randperm(20, generator=gen, device="cuda").int().reshape(2, 10)
    ctx = i32([155, 90])
    q = torch.randn(40, 16, D, generator=gen, device="cuda").bfloat16()
    outs = []
    for p, at in ((small, 0), (planes, base)):
        t = (table + at).int()
        o1, o2 = torch.empty_like(q[:2]), torch.empty_like(q)
        pk.decode_mxfp4(o1, q[:2], *p, t, ctx, 155, 0.1)
        pk.chunked_prefill_mxfp4(o2, q, i32([0, 25, 40]), 25, *p, t, ctx, 155, 0.1)
        pool = pk.CachePool(p, bs)
        nt = torch.empty(2, 10, dtype=torch.int32, device="cuda")
        nc = torch.empty(2, dtype=torch.int32, device="cuda")
        pool.fork(t, ctx, i32([0, 1]), i32([at + 30, at + 31]), nt, nc)
        pool.compact(i32([[at + 30, at + 22], [at + 31, at + 23]]), nt)
        o3 = torch.empty_like(o1)
        pk.decode_mxfp4(o3, q[:2], *p, nt, nc, 155, 0.1)
        assert torch.equal(o1, o3)
        outs.append((o1, o2, nt - at * (nt >= 0)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
