"""The cases of the 4-bit cache and of the page operators: what a pass of each takes and gives.

``run`` makes the library's calls where ``own`` is true; elsewhere it computes
the same operator from elementary torch operations in 32 bits.

A cache held in 4 bits (OCP Microscaling MXFP4): 32 consecutive elements of a
row share one byte b, the power of two 2^(b - 127), and each is an E2M1 code
of 4 bits; codes are uint8 [num_blocks, num_kv_heads, block_size, D / 2] with
element 2i in the low half of byte i, scales uint8 [num_blocks, num_kv_heads,
block_size, D / 32].
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    def store(name, tokens, kv_heads, head_dim, block_size, dtype, pad):
        return dict(name=name, op="store", tokens=tokens, kv_heads=kv_heads, head_dim=head_dim,
                    block_size=block_size, dtype=dtype, pad=pad)

    def decode(name, seqs, heads, kv_heads, head_dim, block_size, dtype, lo, hi, empty=0):
        return dict(name=name, op="decode", seqs=seqs, heads=heads, kv_heads=kv_heads,
                    head_dim=head_dim, block_size=block_size, dtype=dtype, lo=lo, hi=hi,
                    empty=empty)

    def chunk(name, seqs, qlo, qhi, heads, kv_heads, head_dim, block_size, dtype, lo, hi):
        return dict(name=name, op="chunk", seqs=seqs, qlo=qlo, qhi=qhi, heads=heads,
                    kv_heads=kv_heads, head_dim=head_dim, block_size=block_size, dtype=dtype,
                    lo=lo, hi=hi)

    def pages(name, op, layers, kind, kv_heads, head_dim, block_size, seqs, lo, hi, count):
        return dict(name=name, op=op, layers=layers, kind=kind, kv_heads=kv_heads,
                    head_dim=head_dim, block_size=block_size, seqs=seqs, lo=lo, hi=hi,
                    count=count)

    return [
        # the new tokens of one decode step of 64 sequences, 8 kv-heads
        store("store step", 64, 8, 128, 16, "bf16", 0),
        # a prompt chunk written at once, an odd number of tokens, every 7th padding
        store("store prompt", 8191, 32, 128, 16, "f16", 7),
        # the smallest decode: a handful of short sequences, where latency counts
        decode("decode tiny", 4, 4, 4, 64, 16, "f16", 1, 100),
        # the headline decode step: 32 sequences of about 2048 tokens, 32 heads
        decode("decode mha", 32, 32, 32, 128, 16, "f16", 2011, 2048),
        # a batch of grouped-query sequences of very different lengths, one not begun
        decode("decode gqa long", 24, 64, 8, 128, 32, "bf16", 1024, 32768, empty=1),
        # verification of 8 draft tokens for 64 sequences
        chunk("verify gqa", 64, 8, 8, 64, 8, 128, 16, "bf16", 1024, 4096),
        # chunked prefill of 16 prompts, 32 heads
        chunk("chunk mha", 16, 512, 512, 32, 32, 128, 16, "f16", 0, 3584),
        # short ragged chunks of a small model (head_dim 64), odd lengths from one token
        chunk("chunk ragged", 5, 1, 301, 16, 4, 64, 16, "bf16", 0, 777),
        # one sequence forked into a few samples, one layer, 16-bit cache
        pages("fork one", "fork", 1, "bf16", 8, 128, 16, 1, 100, 100, 4),
        # a beam step: 32 sequences into 128 beams over the layers of a model, 4-bit cache
        pages("fork beams", "fork", 32, "mxfp4", 8, 128, 16, 32, 300, 1500, 128),
        # a few pages moved in a small pool
        pages("compact few", "compact", 2, "mxfp4", 8, 128, 16, 8, 100, 400, 9),
        # a pool emptied by half and moved together, 16-bit cache
        pages("compact half", "compact", 4, "f16", 32, 128, 16, 16, 500, 2000, 700),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["store", "decode", "decode", "chunk", "chunk", "fork", "compact"])
    head_dim = rng.choice([64, 128, 128])
    block_size = rng.choice([16, 32])
    dtype = rng.choice(["f16", "bf16"])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32])
    if op == "store":
        return dict(op=op, tokens=log_int(1, 8000), kv_heads=kv_heads, head_dim=head_dim,
                    block_size=block_size, dtype=dtype, pad=rng.choice([0, 0, 2, 5]))
    group = rng.choice([1, 2, 4, 8])
    heads = kv_heads * group
    if op == "decode":
        # sequences x longest context x kv-heads within the largest listed case
        hi = log_int(1, 32000)
        seqs = log_int(1, max(1, min(200, 32 * 2048 * 32 // (hi * kv_heads))))
        lo = log_int(1, hi)
        return dict(op=op, seqs=seqs, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                    block_size=block_size, dtype=dtype, lo=lo, hi=hi,
                    empty=rng.choice([0, 0, 1]))
    if op == "chunk":
        qhi = log_int(1, 600)
        hi = log_int(1, 6000)
        most = 16 * 512 * 32 * 2048        # query rows x heads x keys of the largest listed case
        most = min(most // (qhi * heads), 32 * 2048 * 32 // kv_heads)
        seqs = log_int(1, max(1, min(64, most // (hi + qhi))))
        return dict(op=op, seqs=seqs, qlo=rng.choice([1, qhi, max(1, qhi // 3)]), qhi=qhi,
                    heads=heads, kv_heads=kv_heads, head_dim=head_dim, block_size=block_size,
                    dtype=dtype, lo=rng.choice([0, hi // 2]), hi=hi)
    layers = log_int(1, 16)
    kind = rng.choice(["f16", "bf16", "mxfp4"])
    seqs = log_int(1, 16)
    hi = log_int(20, 1000)
    lo = rng.randint(1, hi)
    kv_heads = min(kv_heads, 16)
    count = log_int(1, 96)
    return dict(op=op, layers=layers, kind=kind, kv_heads=kv_heads, head_dim=head_dim,
                block_size=block_size, seqs=seqs, lo=lo, hi=hi, count=count)


# ------------------------------------------------------------------ the shape of a case

def spread(n, lo, hi):
    """n lengths between lo and hi, even over their logarithm, hi the last, in a mixed order."""
    if n == 1:
        return [hi]
    a, b = math.log(lo + 1), math.log(hi + 1)
    v = [int(round(math.exp(a + (b - a) * i / (n - 1)))) - 1 for i in range(n)]
    random.Random(n * 1000003 + lo * 1009 + hi).shuffle(v)
    return v


def lengths(case):
    """(query lengths, context lengths) of the sequences of a case."""
    n = case["seqs"]
    if case["op"] == "chunk":
        q = spread(n, case["qlo"], case["qhi"])
        return q, [p + x for p, x in zip(spread(n, case["lo"], case["hi"]), q)]
    ctx = spread(n, case["lo"], case["hi"])
    if case.get("empty") and n > 1:
        ctx[n // 2] = 0
        ctx[0] = max(ctx[0], case["hi"])
    return [1] * n, ctx


def blocks_of(ctx, bs):
    return [-(-c // bs) for c in ctx]


def pool_shapes(case, num_blocks):
    """Shape and dtype of a pool's tensors over all layers: keys and values, or their codes and scales."""
    hkv, d, bs, n = case["kv_heads"], case["head_dim"], case["block_size"], case["layers"]
    if case["kind"] == "mxfp4":
        return [((n, num_blocks, hkv, bs, d // 2), torch.uint8)] * 2 + \
               [((n, num_blocks, hkv, bs, d // 32), torch.uint8)] * 2
    return [((n, num_blocks, bs, hkv, d), DTYPES[case["kind"]])] * 2


def copies_of(case):
    """Pages that a pass copies: forks of a page that is not full, or moves."""
    ctx = lengths(case)[1]
    if case["op"] == "compact":
        return min(case["count"], sum(blocks_of(ctx, case["block_size"])))
    n, count = len(ctx), case["count"]
    made = [len(range(s, count, n)) for s in range(n)]      # children of each parent
    kept = 1 if count >= 8 else 0
    return sum(max(0, m - kept) for m, c in zip(made, ctx) if c % case["block_size"])


# ------------------------------------------------------------------ the inputs

def quantised(x):
    """Codes and scales of 32-bit values [..., D]: the format's own rule."""
    shape = x.shape
    x = x.reshape(*shape[:-1], shape[-1] // 32, 32)
    amax = x.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(amax)
    e = (torch.frexp(torch.where(bad, torch.ones_like(amax), amax))[1] - 3).clamp(-126, 125)
    e = torch.where(amax == 0, torch.full_like(e, -126), e)
    y = x.abs() * ((127 - e) << 23).view(torch.float32)      # times 2^-e, exactly
    # nearest of the eight magnitudes, ties to the even code
    code = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int() +
            (y > 2.5).int() + (y >= 3.5).int() + (y > 5.0).int())
    code = torch.where(bad, torch.zeros_like(code), code + 8 * torch.signbit(x).int())
    byte = torch.where(bad, torch.full_like(e, 255), e + 127)
    code = code.reshape(*shape[:-1], shape[-1] // 2, 2)
    packed = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
    return packed, byte.reshape(*shape[:-1], shape[-1] // 32).to(torch.uint8)


def values_of(codes, scales):
    """The 32-bit values that codes [..., D / 2] and scales [..., D / 32] stand for."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    c = codes.int()
    v = table[torch.stack((c & 15, c >> 4), -1)]
    v = v.reshape(*codes.shape[:-1], scales.shape[-1], 32)
    s = (scales.int() << 23).view(torch.float32)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return (v * s.unsqueeze(-1)).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    rng = random.Random(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def kv_rows(*shape):
        """Keys or values as projections give them: some channels of a head much larger."""
        x = randn(*shape)
        return x * (1 + 3 * (torch.rand((shape[-1],), generator=g, device=dev) < 0.06).float())

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if case["op"] == "store":
        t, hkv, d, bs = case["tokens"], case["kv_heads"], case["head_dim"], case["block_size"]
        nb = -(-t // bs) + 3
        dt = DTYPES[case["dtype"]]
        slots = torch.randperm(nb * bs, generator=g, device=dev)[:t].to(torch.int32)
        if case["pad"]:
            slots[case["pad"] - 1::case["pad"]] = -1
        planes = [torch.zeros(s, dtype=torch.uint8, device=dev)
                  for s in ((nb, hkv, bs, d // 2),) * 2 + ((nb, hkv, bs, d // 32),) * 2]
        return dict(case=case, key=kv_rows(t, hkv, d).to(dt), value=kv_rows(t, hkv, d).to(dt),
                    planes=planes, slots=slots, rows=(torch.zeros((t, hkv, d), dtype=dt, device=dev),
                                                      torch.zeros((t, hkv, d), dtype=dt, device=dev)))

    qlens, ctx = lengths(case)
    bs, hkv, d, n = case["block_size"], case["kv_heads"], case["head_dim"], case["seqs"]
    need = blocks_of(ctx, bs)
    width = max(1, max(need))
    if case["op"] in ("fork", "compact"):
        live, count = sum(need), case["count"]
        if case["op"] == "fork":
            nb = live + count + 5
            ids = rng.sample(range(nb), live + count)
        else:
            # `moved` pages lie behind the first `live` places of the pool, the rest among them
            nb = live + max(count + 5, live // 2)
            moved = copies_of(case)
            tops = sorted(rng.sample(range(live, nb), moved))
            ids = tops + rng.sample(range(live), live - moved)
            holes = sorted(set(range(live)) - set(ids))
            rng.shuffle(ids)
        table, at = [], 0
        for k in need:
            table.append(ids[at:at + k] + [-1] * (width - k))
            at += k
        pools = [torch.randint(0, 256, shape, generator=g, device=dev, dtype=torch.uint8)
                 if dt is torch.uint8 else randn(*shape).to(dt) for shape, dt in pool_shapes(case, nb)]
        st = dict(case=case, pools=pools, tables=i32(table), ctx=i32(ctx))
        if case["op"] == "fork":
            parents = [i % n for i in range(count)]
            rng.shuffle(parents)
            # of many children of one parent the first keeps the parent's last page
            seen, fresh = set(), []
            for p, f in zip(parents, ids[at:]):
                fresh.append(f if p in seen or count < 8 else -1)
                seen.add(p)
            st.update(parents=i32(parents), fresh=i32(fresh),
                      new_tables=torch.full((count, width), -7, dtype=torch.int32, device=dev),
                      new_ctx=torch.zeros((count,), dtype=torch.int32, device=dev))
        else:
            st["moves"] = i32([list(m) for m in zip(tops, holes)])
        if own:
            import paged_kv_cache_448_b200 as pk
            st["pool"] = pk.CachePool([layer for pool in pools for layer in pool], bs)
        return st

    nb = sum(need) + 3
    order = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = order[at:at + k]
        at += k
    planes = [torch.empty(s, dtype=torch.uint8, device=dev)
              for s in ((nb, hkv, bs, d // 2),) * 2 + ((nb, hkv, bs, d // 32),) * 2]
    step = max(1, (1 << 26) // (hkv * bs * d))
    for kv in range(2):
        for b in range(0, nb, step):
            e = min(nb, b + step)
            planes[kv][b:e], planes[2 + kv][b:e] = quantised(kv_rows(e - b, hkv, bs, d))
    dt = DTYPES[case["dtype"]]
    t = sum(qlens)
    cu = [0]
    for q in qlens:
        cu.append(cu[-1] + q)
    query = randn(t, case["heads"], d).to(dt)
    st = dict(case=case, planes=planes, tables=table, ctx=i32(ctx), cu=i32(cu), query=query,
              out=torch.zeros_like(query), max_q=max(qlens), max_ctx=max(max(ctx), 1),
              scale=1.0 / math.sqrt(d))
    if own:
        import paged_kv_cache_448_b200 as pk
        if case["op"] == "decode":
            st["workspace"] = pk.decode_workspace(n, case["heads"], hkv, d, bs, st["max_ctx"],
                                                  cache_dtype=pk.PA_MXFP4)
        else:
            st["workspace"] = pk.chunked_prefill_workspace(n, t, case["heads"], hkv, d, st["max_q"],
                                                           st["max_ctx"], pk.PA_MXFP4)
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return run_own(state, op)
    if op == "store":
        return plain_store(state)
    if op in ("decode", "chunk"):
        return plain_attention(state)
    return plain_fork(state) if op == "fork" else plain_compact(state)


def run_own(st, op):
    import paged_kv_cache_448_b200 as pk
    if op == "store":
        pk.reshape_and_cache_mxfp4(st["key"], st["value"], *st["planes"], st["slots"])
        pk.gather_cache_mxfp4(*st["rows"], *st["planes"], st["slots"])
        return st["rows"], st["planes"]
    if op == "decode":
        return pk.decode_mxfp4(st["out"], st["query"], *st["planes"], st["tables"], st["ctx"],
                               st["max_ctx"], st["scale"], workspace=st["workspace"])
    if op == "chunk":
        return pk.chunked_prefill_mxfp4(st["out"], st["query"], st["cu"], st["max_q"],
                                        *st["planes"], st["tables"], st["ctx"], st["max_ctx"],
                                        st["scale"], workspace=st["workspace"])
    if op == "fork":
        st["pool"].fork(st["tables"], st["ctx"], st["parents"], st["fresh"], st["new_tables"],
                        st["new_ctx"])
        return st["new_tables"], st["new_ctx"], st["pools"]
    st["pool"].compact(st["moves"], st["tables"])
    return st["tables"], st["pools"]


def plain_store(st):
    """Write the rows, then read them back; padding rows and other slots stay as they were."""
    slots, bs = st["slots"].long(), st["case"]["block_size"]
    real = slots >= 0
    blk, off = slots[real] // bs, slots[real] % bs
    for x, c, s, r in zip((st["key"], st["value"]), st["planes"][:2], st["planes"][2:], st["rows"]):
        codes, scales = quantised(x[real].float())
        c[blk, :, off] = codes
        s[blk, :, off] = scales
        r[real] = values_of(c[blk, :, off], s[blk, :, off]).to(r.dtype)
    return st["rows"], st["planes"]


def plain_attention(st):
    """Attention of the last query positions of each sequence over its pages, in 32 bits."""
    c, dev = st["case"], st["query"].device
    hkv, bs, d = c["kv_heads"], c["block_size"], c["head_dim"]
    n, group, width = c["seqs"], c["heads"] // c["kv_heads"], st["tables"].shape[1]
    ctx, cu, max_q = st["ctx"].long(), st["cu"].long(), st["max_q"]
    qlen = cu[1:] - cu[:-1]
    pages = st["tables"].long().clamp(min=0)
    k, v = (values_of(st["planes"][i][pages], st["planes"][2 + i][pages])
            .transpose(1, 2).reshape(n, hkv, width * bs, d) for i in range(2))
    # queries padded to [sequence, position]
    i = torch.arange(max_q, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=st["query"].shape[0] - 1)
    q = st["query"][rows].float().reshape(n, max_q, hkv, group, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(n, hkv, group * max_q, d)
    x = (q @ k.transpose(-1, -2)).mul_(st["scale"]).reshape(n, hkv, group, max_q, width * bs)
    pos = ctx[:, None] - qlen[:, None] + i                      # position of each query row
    sees = torch.arange(width * bs, device=dev) <= pos[..., None]
    sees &= (torch.arange(width * bs, device=dev) < ctx[:, None])[:, None]
    x.masked_fill_(~sees[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    # a page that no row of its sequence sees may hold anything
    v = torch.where((torch.arange(width * bs, device=dev) < ctx[:, None])[:, None, :, None], v,
                    torch.zeros_like(v))
    o = x.reshape(n, hkv, group * max_q, -1) @ v
    o = o / total.reshape(n, hkv, group * max_q, 1).clamp(min=1e-30)
    o = o.reshape(n, hkv, group, max_q, d).permute(0, 3, 1, 2, 4).reshape(n, max_q, c["heads"], d)
    st["out"].copy_(o[i[None] < qlen[:, None]].to(st["out"].dtype))
    return st["out"]


def plain_fork(st):
    bs, parents, fresh = st["case"]["block_size"], st["parents"].long(), st["fresh"].long()
    rows = st["tables"][parents].clone()
    ctx = st["ctx"][parents]
    last = ((ctx.long() + bs - 1) // bs - 1).clamp(min=0)
    copies = (ctx % bs != 0) & (fresh >= 0)
    at = torch.arange(rows.shape[0], device=rows.device)
    src, dst = rows[at, last][copies].long(), fresh[copies]
    for p in st["pools"]:
        p[:, dst] = p[:, src]
    rows[at[copies], last[copies]] = dst.int()
    used = torch.arange(rows.shape[1], device=rows.device) < ((ctx + bs - 1) // bs)[:, None]
    st["new_tables"].copy_(torch.where(used, rows, torch.full_like(rows, -1)))
    st["new_ctx"].copy_(ctx)
    return st["new_tables"], st["new_ctx"], st["pools"]


def plain_compact(st):
    src, dst = st["moves"][:, 0].long(), st["moves"][:, 1].long()
    for p in st["pools"]:
        p[:, dst] = p[:, src]
    to = torch.arange(st["pools"][0].shape[1] + 1, dtype=torch.int32, device=src.device)
    to[-1] = -1                                     # the entry of a place that holds no page
    to[src] = dst.int()
    st["tables"].copy_(to[st["tables"].long()])
    return st["tables"], st["pools"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "store":
        real = case["tokens"] - (case["tokens"] // case["pad"] if case["pad"] else 0)
        elems = 2 * real * case["kv_heads"] * case["head_dim"]
        # rows in, codes and scales out; the same back for the reading
        return dict(bytes=int(elems * 2 * (2 + 17 / 32)) + 8 * case["tokens"], flops=elems * 4)
    qlens, ctx = lengths(case)
    bs = case["block_size"]
    if case["op"] in ("decode", "chunk"):
        kv = sum(ctx) * case["kv_heads"] * case["head_dim"] * 2 * 17 // 32
        rows = sum(qlens) * case["heads"] * case["head_dim"]
        pairs = sum(c * q - q * (q - 1) // 2 for c, q in zip(ctx, qlens) if c >= q)
        return dict(bytes=kv + 4 * rows + 4 * sum(blocks_of(ctx, bs)) + 4 * len(ctx),
                    flops=4 * pairs * case["heads"] * case["head_dim"])
    elem = 17 / 32 if case["kind"] == "mxfp4" else 2
    page = int(2 * case["layers"] * bs * case["kv_heads"] * case["head_dim"] * elem)
    width = max(1, max(blocks_of(ctx, bs)))
    rows = case["count"] if case["op"] == "fork" else len(ctx)
    return dict(bytes=2 * page * copies_of(case) + 8 * width * rows, flops=0)


# ------------------------------------------------------------------ the same in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("fork", "compact"):
        return None
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def power(e):
        """2^e in 64 bits, by the bits of its exponent."""
        return ((e + 1023) << 52).view(torch.float64)

    def read(codes, scales):
        lo, hi = codes % 16, codes // 16
        c = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.int64, device="cuda")
        c[..., 0::2], c[..., 1::2] = lo, hi
        v = grid[c % 8] * (1 - 2 * (c // 8)).double()
        return v * power(scales.long() - 127).repeat_interleave(32, -1)

    if case["op"] == "store":
        outs = []
        for x in (st["key"], st["value"]):
            y = x.double().reshape(-1, 32)
            top = y.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -124)
            e = torch.round(torch.log2(top)).long()
            e = e - (power(e) > top).long() - 2       # the largest power of two below, over four
            z = y.abs() / power(e)
            dist = (z.unsqueeze(-1) - grid).abs()
            near = dist.amin(-1, keepdim=True)
            hit = dist == near                       # two of them at a tie: the even code
            even = torch.arange(8, device="cuda") % 2 == 0
            code = torch.where((hit.sum(-1, keepdim=True) > 1), hit & even, hit).int().argmax(-1)
            val = (grid[code] * power(e) * torch.sign(y)).reshape(x.shape)
            val[st["slots"] < 0] = 0
            outs.append(val)
        return (outs[0], outs[1]), [None] * 4
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device="cuda")
    group, hkv, bs = case["heads"] // case["kv_heads"], case["kv_heads"], case["block_size"]
    qlens, ctx = lengths(case)
    at = 0
    for s, (q, c) in enumerate(zip(qlens, ctx)):
        if c:
            ids = st["tables"][s, :-(-c // bs)].long()
            for h in range(hkv):
                k, v = (read(st["planes"][i][ids, h], st["planes"][2 + i][ids, h])
                        .reshape(-1, case["head_dim"])[:c] for i in range(2))
                qs = st["query"][at:at + q, h * group:(h + 1) * group].double()
                x = torch.einsum("qgd,td->gqt", qs, k) * st["scale"]
                late = torch.arange(c, device="cuda") > (c - q + torch.arange(q, device="cuda"))[:, None]
                x[:, late] = float("-inf")
                p = torch.softmax(x, -1)
                out[at:at + q, h * group:(h + 1) * group] = torch.einsum("gqt,td->qgd", p, v)
        at += q
    return out
