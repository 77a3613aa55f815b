"""The serving step's operators around the packed latent cache, as measured work.

Step maps from request lengths, the cache write (norm, rotary, quantisation,
scatter), the gather back to bf16, sparse decode over the 4-bit cache and
sliding-window decode with sinks over either cache.  ``own`` selects the
library's calls; otherwise ``run`` is their plain form in torch.

Cache rows: fp8 656 bytes = 512 e4m3 codes | 4 fp32 scales | 64 bf16;
fp4 416 bytes = 256 bytes of e2m1 codes (low nibble = even dim) | 32 e4m3
scales, one per 16 dims | 64 bf16.
"""
import math

import torch

own = False

ROW = {"fp8": 656, "fp4": 416}
SCALE = 1.0 / math.sqrt(192.0)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6
KV_STRIDE = 1536 + 576  # the latent is the tail of a fused down-projection's output
NEG_INF = float("-inf")


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one rank's maps of a decode step: every request brings one token
        dict(name="maps_decode", op="maps", B=64, T=64, q_hi=1, ctx_lo=4096, ctx_hi=65536,
             D=4, rank=1, bs=64, I=1),
        # a mixed step of many requests: decodes beside ragged prefill chunks,
        # padded to a captured row count
        dict(name="maps_mixed", op="maps", B=509, T=66000, q_hi=256, ctx_lo=1, ctx_hi=8192,
             D=2, rank=0, bs=16, I=4),
        # the decode step's own rows going into the 8-bit cache
        dict(name="write_decode_fp8", op="write", fmt="fp8", T=64, D=1, slots=65536, pairs=True),
        # a long prefill chunk written by one of four ranks into the 4-bit cache
        dict(name="write_prefill_fp4", op="write", fmt="fp4", T=16384, D=4, slots=65536,
             pairs=False),
        # a chunk's cached context read back for prefill attention
        dict(name="gather_chunk_fp8", op="gather", fmt="fp8", N=4001, slots=65536, dtype="bf16"),
        dict(name="gather_context_fp4", op="gather", fmt="fp4", N=131072, slots=262144,
             dtype="bf16"),
        # one shard's sparse decode of a small batch: latency
        dict(name="sparse4_small", op="sparse4", T=2, H=16, K=64, D=1, bs=16, ctx_lo=37,
             ctx_hi=200, neg=0.1),
        # one pool, half the heads, the usual top-k
        dict(name="sparse4_rank", op="sparse4", T=32, H=64, K=2048, D=1, bs=64, ctx_lo=4096,
             ctx_hi=4096, neg=0.0),
        # the long-context serving batch over four pools, fused
        dict(name="sparse4_dcp4", op="sparse4", T=64, H=128, K=2048, D=4, bs=64, ctx_lo=2,
             ctx_hi=65536, neg=0.0),
        # one request's window: latency
        dict(name="window_small_fp4", op="window", fmt="fp4", B=1, S=1, H=16, window=128, sinks=4,
             D=2, rank=-1, bs=16, I=1, ctx_lo=300, ctx_hi=300),
        # a serving batch over eight pools in 4 bits
        dict(name="window_dcp8_fp4", op="window", fmt="fp4", B=128, S=1, H=128, window=1024,
             sinks=64, D=8, rank=-1, bs=64, I=1, ctx_lo=1024, ctx_hi=65536),
        # two speculative tokens a request and a wide window, 8 bits
        dict(name="window_mtp2_fp8", op="window", fmt="fp8", B=32, S=2, H=128, window=4096,
             sinks=16, D=2, rank=-1, bs=64, I=1, ctx_lo=8192, ctx_hi=32768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["maps", "write", "gather", "sparse4", "window"])
    fmt = rng.choice(["fp8", "fp4"])
    D = rng.choice([1, 2, 3, 4, 8])
    bs = rng.choice([1, 16, 48, 64, 128])
    if op == "maps":
        B = _log(rng, 1, 600)
        q_hi = _log(rng, 1, 256)
        hi = _log(rng, 4 * q_hi, 16384)
        return dict(op=op, B=B, T=min(66000, B * (q_hi + 1) // 2 + rng.randrange(0, 65)), q_hi=q_hi,
                    ctx_lo=1, ctx_hi=hi, D=D, rank=rng.randrange(D), bs=bs, I=rng.choice([1, 1, 4, 64]))
    if op == "write":
        return dict(op=op, fmt=fmt, T=_log(rng, 1, 8192), D=D, slots=65536,
                    pairs=rng.random() < 0.5)
    if op == "gather":
        return dict(op=op, fmt=fmt, N=_log(rng, 1, 60000), slots=_log(rng, 1000, 262144),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "sparse4":
        return dict(op=op, T=_log(rng, 1, 64), H=rng.choice([1, 16, 37, 64, 128]),
                    K=_log(rng, 1, 2048), D=D, bs=bs, ctx_lo=1, ctx_hi=_log(rng, 64, 32768),
                    neg=rng.choice([0.0, 0.05, 0.3]))
    if fmt == "fp8":  # wide windows of long contexts, merged: the 8-bit cache's use
        ctx = _log(rng, 2048, 16384)
        return dict(op=op, fmt=fmt, B=_log(rng, 1, 32), S=rng.choice([1, 2, 3]),
                    H=rng.choice([1, 16, 37, 64, 128]), window=_log(rng, 700, 4000),
                    sinks=rng.choice([0, 1, 4, 64, 130]), D=D, rank=-1, bs=bs,
                    I=rng.choice([1, 1, 4]), ctx_lo=ctx // 2, ctx_hi=ctx)
    W = _log(rng, 1, 2048)
    ctx = _log(rng, 64, 16384)
    S = rng.choice([1, 2, 3])
    return dict(op=op, fmt=fmt, B=_log(rng, 1, 32), S=S, H=rng.choice([1, 16, 37, 64, 128]),
                window=W, sinks=rng.choice([0, 1, 4, 64, 130]), D=D,
                rank=rng.choice([-1, -1, rng.randrange(D)]), bs=bs, I=rng.choice([1, 1, 4]),
                ctx_lo=max(S, ctx // 64), ctx_hi=ctx)


# --------------------------------------------------------------------------
# sizes that follow from a case
# --------------------------------------------------------------------------
def _ladder(lo, hi, n):
    """n lengths from lo to hi, evenly spaced in their logarithm."""
    if n == 1:
        return [hi]
    return [min(hi, max(lo, int(lo * (hi / lo) ** (i / (n - 1))))) for i in range(n)]


def _rows(c, D, r, I):
    """Of the first c positions, how many rank r holds."""
    full, rem = divmod(c, I * D)
    return full * I + min(max(rem - r * I, 0), I)


def _map_lengths(case):
    """(ctx, q) of every request: q cycles through 0..q_hi (all q_hi where
    that is 1), cut so that the rows fit T."""
    B, q_hi = case["B"], case["q_hi"]
    ctx = _ladder(max(1, case["ctx_lo"]), case["ctx_hi"], B)
    q, left = [], case["T"]
    for b in range(B):
        want = 1 if q_hi == 1 else (b * 97 + 13) % (q_hi + 1)
        n = min(want, left, ctx[b])
        q.append(n)
        left -= n
    return ctx, q


def _sparse_ctx(case):
    return _ladder(case["ctx_lo"], case["ctx_hi"], case["T"])


def _window_keys(case, p):
    """Keys the token at position p attends, on the case's rank or all."""
    D, I, r = case["D"], case["I"], case["rank"]
    w0 = max(p + 1 - case["window"], 0)
    s1 = min(case["sinks"], w0)
    if r < 0:
        return s1 + p + 1 - w0
    return _rows(s1, D, r, I) + _rows(p + 1, D, r, I) - _rows(w0, D, r, I)


def work(case):
    op = case["op"]
    if op == "maps":
        ctx, q = _map_lengths(case)
        D, r, I, bs = case["D"], case["rank"], case["I"], case["bs"]
        new = sum(-(-_rows(c, D, r, I) // bs) - -(-_rows(c - n, D, r, I) // bs)
                  for c, n in zip(ctx, q))
        # lengths in; rows (request, position, slot), starts, counts and new blocks out
        return {"bytes": 8 * case["B"] + 12 * case["T"] + 8 * case["B"] + 4 + 8 * new,
                "flops": 10 * case["T"]}
    if op == "write":
        T, held = case["T"], -(-case["T"] // case["D"])
        # latent, slot, position and angles of the rows this rank holds in, its
        # rows out, and once more through the gather that hands back their values
        return {"bytes": 8 * T + held * (1152 + 256 + 2 * ROW[case["fmt"]]) + T * (4 + 1152),
                "flops": held * 512 * 8}
    if op == "gather":
        return {"bytes": case["N"] * (4 + ROW[case["fmt"]] + (1152 if case["dtype"] == "bf16" else 2304)),
                "flops": case["N"] * 512}
    H = case["H"]
    if op == "sparse4":
        keys = sum(int(min(case["K"], c) * (1 - case["neg"])) for c in _sparse_ctx(case))
        T = case["T"]
        return {"bytes": keys * ROW["fp4"] + T * H * (1152 + 1024 + 4) + T * case["K"] * 4,
                "flops": keys * 2 * H * (576 + 512)}
    T = case["B"] * case["S"]
    keys = read = 0
    for c in _ladder(case["ctx_lo"], case["ctx_hi"], case["B"]):
        per = [_window_keys(case, c - case["S"] + s) for s in range(case["S"])]
        keys += sum(per)
        read += max(per)  # the tokens of a request share their keys' rows
    return {"bytes": read * ROW[case["fmt"]] + T * H * (1152 + 1024 + 4),
            "flops": keys * 2 * H * (576 + 512)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _e2m1_codes(v):
    """Nearest e2m1 code (ties to the even code) of v, |v| <= 6."""
    a = v.abs()
    c = torch.zeros_like(a, dtype=torch.uint8)
    for i, (b, even_below) in enumerate([(0.25, True), (0.75, False), (1.25, True), (1.75, False),
                                         (2.5, True), (3.5, False), (5.0, True)]):
        c += (a > b) if even_below else (a >= b)
    return c + (torch.signbit(v)).to(torch.uint8) * 8


def _quantised_rows(n, fmt, g, dev):
    """n rows of normalised latents N(0, 1) and rope values N(0, 1)."""
    out = torch.empty((n, ROW[fmt]), dtype=torch.uint8, device=dev)
    for s in range(0, n, 1 << 17):
        m = min(1 << 17, n - s)
        y = torch.randn((m, 512), generator=g, device=dev)
        rope = torch.randn((m, 64), generator=g, device=dev).to(torch.bfloat16)
        o = out[s:s + m]
        if fmt == "fp8":
            y = y.view(m, 4, 128)
            sc = y.abs().amax(2, keepdim=True) / 448.0
            o[:, :512] = (y / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(m, 512)
            o[:, 512:528] = sc.reshape(m, 4).contiguous().view(torch.uint8)
        else:
            y = y.view(m, 32, 16)
            sc = (y.abs().amax(2, keepdim=True) / 6.0).to(torch.float8_e4m3fn)
            c = _e2m1_codes((y / sc.float()).clamp(-6, 6)).view(m, 256, 2)
            o[:, :256] = c[:, :, 0] | (c[:, :, 1] << 4)
            o[:, 256:288] = sc.view(torch.uint8).view(m, 32)
        o[:, -128:] = rope.view(torch.uint8).view(m, 128)
    return out


def _paged_pools(ctx, D, bs, I, fmt, seed, g, dev):
    """D pools of one tensor and their block tables: request b's blocks are a
    random choice of its pool's; ~10% of the blocks belong to nobody."""
    cg = torch.Generator().manual_seed(seed)
    c = torch.tensor(ctx, dtype=torch.int64)
    tables, counts = [], []
    for d in range(D):
        n = (c // (I * D)) * I + (c % (I * D) - d * I).clamp(0, I)
        nb = (n + bs - 1) // bs
        total = int(nb.sum()) + max(1, int(nb.sum()) // 10)
        perm = torch.randperm(total, generator=cg).to(torch.int32)
        W = max(1, int(nb.max()))
        col = torch.arange(W)[None]
        at = (torch.cumsum(nb, 0) - nb)[:, None] + col
        tables.append(torch.where(col < nb[:, None], perm[at.clamp(max=total - 1)],
                                  torch.tensor(-1, dtype=torch.int32)))
        counts.append(total * bs)
    W = max(t.shape[1] for t in tables)
    bt = torch.full((D, len(ctx), W), -1, dtype=torch.int32)
    for d, t in enumerate(tables):
        bt[d, :, :t.shape[1]] = t
    pool = _quantised_rows(sum(counts), fmt, g, dev)
    base = [0]
    for n in counts:
        base.append(base[-1] + n)
    bt = bt.to(dev)
    return dict(pool=pool, bt=bt, base=torch.tensor(base[:-1], device=dev),
                pools=[pool[base[d]:base[d + 1]] for d in range(D)], tables=[bt[d] for d in range(D)])


def _shuffled(values, seed):
    p = torch.randperm(len(values), generator=torch.Generator().manual_seed(seed)).tolist()
    return [values[i] for i in p]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "maps":
        ctx, q = _map_lengths(case)
        p = torch.randperm(case["B"], generator=torch.Generator().manual_seed(seed))
        ctx, q = torch.tensor(ctx)[p], torch.tensor(q)[p]
        D, r, I, bs = case["D"], case["rank"], case["I"], case["bs"]
        rows = lambda c: (c // (I * D)) * I + (c % (I * D) - r * I).clamp(0, I)  # noqa: E731
        nb0, nb1 = (rows(ctx - q) + bs - 1) // bs, (rows(ctx) + bs - 1) // bs
        total = int(nb1.sum()) + 7
        perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed + 1)).to(torch.int32)
        W = max(1, int(nb1.max())) + 3
        col = torch.arange(W)[None]
        at = (torch.cumsum(nb0, 0) - nb0)[:, None] + col
        bt = torch.where(col < nb0[:, None], perm[at.clamp(max=total - 1)],
                         torch.tensor(-1, dtype=torch.int32))
        free = perm[int(nb0.sum()):]
        s.update(ctx=ctx.to(torch.int32).to(dev), q=q.to(torch.int32).to(dev), bt=bt.to(dev),
                 free=free.contiguous().to(dev))
    elif op == "write":
        T, D, fmt = case["T"], case["D"], case["fmt"]
        cg = torch.Generator().manual_seed(seed)
        fused = torch.randn((T, KV_STRIDE), generator=g, device=dev) * 2.0
        s["kv"] = fused.to(torch.bfloat16)[:, -576:]
        s["gamma"] = (1.0 + 0.2 * torch.randn(512, generator=g, device=dev)).to(torch.bfloat16)
        start = int(torch.randint(0, 65536 - 20000, (1,), generator=cg))
        pos = torch.arange(T) + start
        slots = torch.randperm(case["slots"], generator=cg)[:T].to(torch.int32)
        slots[pos % D != seed % D] = -1  # another rank's tokens
        s["pos"], s["slots"] = pos.to(torch.int32).to(dev), slots.to(dev)
        f = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device=dev) / 32)
        a = torch.arange(65536, dtype=torch.float64, device=dev)[:, None] * f
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        s["pool"] = torch.zeros((case["slots"], ROW[fmt]), dtype=torch.uint8, device=dev)
    elif op == "gather":
        s["pool"] = _quantised_rows(case["slots"], case["fmt"], g, dev)
        sl = torch.randint(0, case["slots"], (case["N"],), generator=g, device=dev, dtype=torch.int32)
        sl[torch.rand(case["N"], generator=g, device=dev) < 0.01] = -1
        s["slots"] = sl
    elif op == "sparse4":
        T, H, K, D = case["T"], case["H"], case["K"], case["D"]
        ctx = _shuffled(_sparse_ctx(case), seed)
        s.update(_paged_pools(ctx, D, case["bs"], 1, "fp4", seed, g, dev))
        s["q"] = torch.randn((T, H, 576), generator=g, device=dev).to(torch.bfloat16)
        s["req"] = torch.arange(T, dtype=torch.int32, device=dev)
        # min(K, ctx) distinct positions, one from each of as many equal runs
        c = torch.tensor(ctx, device=dev, dtype=torch.float64)[:, None]
        n = c.clamp(max=K)
        j = torch.arange(K, device=dev, dtype=torch.float64)[None]
        u = torch.rand((T, K), generator=g, device=dev, dtype=torch.float64)
        lo, hi = torch.floor(j * c / n), torch.floor((j + 1) * c / n)
        ids = torch.where(j < n, lo + torch.floor(u * (hi - lo)), -1.0).to(torch.int32)
        order = torch.rand((T, K), generator=g, device=dev).argsort(1)
        ids = ids.gather(1, order)
        n_neg = int(case["neg"] * K)
        if n_neg:
            drop = torch.rand((T, K), generator=g, device=dev).argsort(1)[:, :n_neg]
            ids.scatter_(1, drop, -1)
        s["topk"] = ids.contiguous()
        if D == 1:  # the per-rank form takes slots
            t = torch.arange(T, device=dev)[:, None]
            v = ids.clamp(min=0).long()
            bs = case["bs"]
            sl = s["bt"][0][t, v // bs].long() * bs + v % bs
            s["slots"] = torch.where(ids >= 0, sl, -1).to(torch.int32).contiguous()
    else:
        B, S, H, D = case["B"], case["S"], case["H"], case["D"]
        ctx = _shuffled(_ladder(case["ctx_lo"], case["ctx_hi"], B), seed)
        s.update(_paged_pools(ctx, D, case["bs"], case["I"], case["fmt"], seed, g, dev))
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s["q"] = torch.randn((B * S, H, 576), generator=g, device=dev).to(torch.bfloat16)
    return s


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------
def _run_own(s):
    from sparse_mla_decode_dcp_gb300 import capi
    c, op, b = s["case"], s["op"], s.setdefault("buffers", {})
    if op == "maps":
        b["out"] = capi.dcp_step_maps(s["ctx"], s["q"], s["free"], s["bt"], c["T"], c["D"], c["rank"],
                                      c["bs"], interleave=c["I"], out=b.get("out"))
        return list(b["out"]) + [s["bt"]]
    if op == "write":
        capi.mla_cache_write(s["kv"], s["slots"], s["pool"], gamma=s["gamma"], eps=EPS,
                             positions=s["pos"], cos_sin=s["cos_sin"], rope_pairs=c["pairs"])
        b["out"] = capi.mla_cache_gather(s["pool"], s["slots"], out=b.get("out"))
        return b["out"]
    if op == "gather":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        b["out"] = capi.mla_cache_gather(s["pool"], s["slots"], dtype=dt, out=b.get("out"))
        return b["out"]
    T, H = s["q"].shape[:2]
    if not b:  # what a serving loop allocates once for its batch shape
        b["out"] = torch.empty((T, H, 512), dtype=torch.bfloat16, device=s["q"].device)
        b["lse"] = torch.empty((T, H), dtype=torch.float32, device=s["q"].device)
        if op == "sparse4":
            b["workspace"] = capi.alloc_fp4_decode_workspace(T, H, c["K"], s["q"].device)
        else:
            b["workspace"] = capi.alloc_window_decode_workspace(
                T, H, c["ctx_hi"], c["window"], c["sinks"], c["D"], c["I"], c["rank"], s["q"].device)
    if op == "sparse4" and c["D"] == 1:
        return capi.sparse_mla_decode_fp4(s["q"], s["pool"], s["slots"], SCALE, **b)
    if op == "sparse4":
        return capi.dcp_sparse_mla_decode_fused_fp4(s["q"], s["req"], s["topk"], s["pools"], s["tables"],
                                                    c["bs"], SCALE, **b)
    return capi.dcp_window_mla_decode(s["q"], s["ctx"], c["ctx_hi"], c["S"], c["window"], c["sinks"],
                                      s["pools"], s["tables"], c["bs"], SCALE, rank=c["rank"],
                                      interleave=c["I"], **b)


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _plain_maps(s):
    c = s["case"]
    D, r, I, bs, T, B = c["D"], c["rank"], c["I"], c["bs"], c["T"], c["B"]
    dev = s["bt"].device
    ctx, q = s["ctx"].long(), s["q"].long()
    before = ctx - q
    rows = lambda n: (n // (I * D)) * I + (n % (I * D) - r * I).clamp(0, I)  # noqa: E731
    nb0, nb1 = (rows(before) + bs - 1) // bs, (rows(ctx) + bs - 1) // bs
    need = nb1 - nb0
    col = torch.arange(s["bt"].shape[1], device=dev)[None]
    at = (torch.cumsum(need, 0) - need)[:, None] + col - nb0[:, None]
    new = (col >= nb0[:, None]) & (col < nb1[:, None])
    s["bt"].copy_(torch.where(new, s["free"][at.clamp(0, s["free"].numel() - 1)], s["bt"]))
    ends = torch.cumsum(q, 0)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), ends])
    t = torch.arange(T, device=dev)
    live = t < ends[-1]
    b = torch.where(live, torch.searchsorted(ends, t, right=True), 0)
    p = torch.where(live, before[b] + t - starts[b], 0)
    lp = (p // (I * D)) * I + p % I
    mine = live & ((p // I) % D == r)
    blk = s["bt"][b, torch.where(mine, lp // bs, 0)].long()
    slot = torch.where(mine, blk * bs + lp % bs, -1)
    i32 = torch.int32
    return [starts.to(i32), b.to(i32), p.to(i32), slot.to(i32), rows(ctx).to(i32),
            need.sum().reshape(1).to(i32), s["bt"]]


def _values(rows, fmt):
    """fp32 [..., 576] of packed rows."""
    shape = rows.shape[:-1]
    rope = rows[..., -128:].contiguous().view(torch.bfloat16).float()
    if fmt == "fp8":
        v = rows[..., :512].contiguous().view(torch.float8_e4m3fn).float().view(*shape, 4, 128)
        sc = rows[..., 512:528].contiguous().view(torch.float32)
    else:
        lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=rows.device)
        codes = rows[..., :256].int()
        v = lut[torch.stack([codes & 15, codes >> 4], -1)].view(*shape, 32, 16)
        sc = rows[..., 256:288].contiguous().view(torch.float8_e4m3fn).float()
    return torch.cat([(v * sc[..., None]).view(*shape, 512), rope], -1)


def _plain_gather(pool, slots, fmt, dtype):
    v = _values(pool[slots.clamp(min=0).long()], fmt)
    return torch.where((slots >= 0)[:, None], v, 0.0).to(dtype)


def _plain_write(s):
    c = s["case"]
    fmt = c["fmt"]
    live = (s["slots"] >= 0).nonzero()[:, 0]
    # codes sit next to rounding borders: 64 bits up to the quantisation
    x = s["kv"][live].double()
    lat = x[:, :512]
    y = lat * torch.rsqrt(lat.square().mean(1, keepdim=True) + EPS) * s["gamma"].double()
    cs = s["cos_sin"][s["pos"][live].long()].double()
    co, si = cs[:, :32], cs[:, 32:]
    r = x[:, 512:]
    if c["pairs"]:
        a, b = r[:, 0::2], r[:, 1::2]
        rope = torch.stack([a * co - b * si, a * si + b * co], 2).reshape(-1, 64)
    else:
        a, b = r[:, :32], r[:, 32:]
        rope = torch.cat([a * co - b * si, a * si + b * co], 1)
    n = x.shape[0]
    rows = torch.empty((n, ROW[fmt]), dtype=torch.uint8, device=x.device)
    if fmt == "fp8":
        y = y.view(n, 4, 128)
        sc = (y.abs().amax(2, keepdim=True) / 448.0).float()
        v = (y / torch.where(sc > 0, sc, 1.0).double()).clamp(-448, 448)
        # one step of e4m3 at v's magnitude; rounded half to even in 64 bits
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        v = (v / step).round() * step
        rows[:, :512] = v.float().to(torch.float8_e4m3fn).view(torch.uint8).view(n, 512)
        rows[:, 512:528] = sc.view(n, 4).contiguous().view(torch.uint8)
    else:
        y = y.view(n, 32, 16)
        m = (y.abs().amax(2, keepdim=True) / 6.0).clamp(max=448.0)
        step = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
        sc = ((m / step).round() * step).float().to(torch.float8_e4m3fn)
        f = sc.double()
        a = (y / torch.where(f > 0, f, 1.0)).clamp(-6, 6) * (f > 0)
        mag = a.abs()
        code = ((mag > 0.25).to(torch.uint8) + (mag >= 0.75) + (mag > 1.25) + (mag >= 1.75)
                + (mag > 2.5) + (mag >= 3.5) + (mag > 5.0))
        code = (code + torch.signbit(a).to(torch.uint8) * 8).view(n, 256, 2)
        rows[:, :256] = code[:, :, 0] | (code[:, :, 1] << 4)
        rows[:, 256:288] = sc.view(torch.uint8).view(n, 32)
    rows[:, -128:] = rope.to(torch.bfloat16).view(torch.uint8).view(n, 128)
    s["pool"][s["slots"][live].long()] = rows
    return _plain_gather(s["pool"], s["slots"], fmt, torch.bfloat16)


def _plain_attend(q, pool, slots, fmt):
    """Softmax attention of q [T, H, 576] over pool rows slots [T, K] (-1: masked)."""
    k = _values(pool[slots.clamp(min=0)], fmt)
    sc = torch.matmul(q.float(), k.transpose(1, 2)) * SCALE
    sc = torch.where((slots >= 0)[:, None], sc, NEG_INF)
    m = sc.amax(2, keepdim=True)
    e = torch.exp(sc - torch.where(m > NEG_INF, m, 0.0))
    l = e.sum(2, keepdim=True)
    out = torch.matmul(e, k[..., :512]) / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l))[..., 0]
    return out.to(torch.bfloat16), lse


def _plain_slots(s, ids, req, D, I, bs):
    """Rows of the stacked pools that hold the requests' positions ids."""
    v = ids.clamp(min=0).long()
    d = (v // I) % D
    lp = (v // (I * D)) * I + v % I
    blk = s["bt"][d, req.long(), lp // bs].long()
    return torch.where(ids >= 0, s["base"][d] + blk * bs + lp % bs, -1)


def _plain_window(s):
    c = s["case"]
    B, S, D, I, W, N = c["B"], c["S"], c["D"], c["I"], c["window"], c["sinks"]
    dev = s["q"].device
    n = min(c["ctx_hi"], W + N)
    p = (s["ctx"].long()[:, None] - S + torch.arange(S, device=dev)).view(-1, 1)
    w0 = (p + 1 - W).clamp(min=0)
    s1 = w0.clamp(max=N)
    j = torch.arange(n, device=dev)[None]
    ids = torch.where(j < s1, j, j - s1 + w0)
    keep = ids <= p
    if c["rank"] >= 0:
        keep = keep & ((ids // I) % D == c["rank"])
    req = torch.arange(B * S, device=dev)[:, None] // S
    slots = _plain_slots(s, torch.where(keep, ids, -1), req, D, I, c["bs"])
    return _plain_attend(s["q"], s["pool"], slots, c["fmt"])


def run(s):
    if own:
        return _run_own(s)
    c, op = s["case"], s["op"]
    if op == "maps":
        return _plain_maps(s)
    if op == "write":
        return _plain_write(s)
    if op == "gather":
        return _plain_gather(s["pool"], s["slots"], c["fmt"],
                             torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
    if op == "sparse4":
        slots = (s["slots"].long() if c["D"] == 1 else
                 _plain_slots(s, s["topk"], s["req"][:, None], c["D"], 1, c["bs"]))
        return _plain_attend(s["q"], s["pool"], slots, "fp4")
    return _plain_window(s)


# --------------------------------------------------------------------------
# the definitions in 64 bits, row by row
# --------------------------------------------------------------------------
def _e4m3_table(dev):
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if code & 127 == 127 else -x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=dev)


def _exact_rows(rows, fmt):
    dev, n = rows.device, rows.shape[0]
    e4m3 = _e4m3_table(dev)
    if fmt == "fp8":
        sc = rows[:, 512:528].contiguous().view(torch.float32).double()
        lat = e4m3[rows[:, :512].long()] * sc.repeat_interleave(128, 1)
    else:
        mag = torch.tensor(E2M1, dtype=torch.float64, device=dev)
        nib = torch.empty((n, 512), dtype=torch.int64, device=dev)
        nib[:, 0::2] = rows[:, :256].long() % 16
        nib[:, 1::2] = rows[:, :256].long() // 16
        lat = mag[nib % 8] * torch.where(nib >= 8, -1.0, 1.0)
        lat = lat * e4m3[rows[:, 256:288].long()].repeat_interleave(16, 1)
    rope = (rows[:, -128::2].int() + rows[:, -127::2].int() * 256).to(torch.int32)
    rope = (rope << 16).view(torch.float32).double()
    return torch.cat([lat, rope], 1)


def _nearest(values, x):
    """The entry of the ascending table `values` nearest to x >= 0, ties to
    the even index."""
    at = torch.searchsorted(values, x.contiguous()).clamp(1, values.numel() - 1)
    lo, hi = values[at - 1], values[at]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (at % 2 == 0))
    return torch.where(up, hi, lo)


def _exact_write(s, case):
    dev = s["kv"].device
    x = s["kv"].double()
    lat = x[:, :512]
    y = lat / torch.sqrt((lat * lat).sum(1, keepdim=True) / 512 + EPS) * s["gamma"].double()[None]
    table = _e4m3_table(dev)[:127]
    if case["fmt"] == "fp8":
        g = y.reshape(-1, 4, 128)
        sc = (g.abs().amax(2, keepdim=True) / 448).float().double()
        v = _nearest(table, g.abs() / sc) * g.sign() * sc
    else:
        g = y.reshape(-1, 32, 16)
        sc = _nearest(table, g.abs().amax(2, keepdim=True) / 6)
        v = _nearest(torch.tensor(E2M1, dtype=torch.float64, device=dev), g.abs() / sc) * g.sign() * sc
    cs = s["cos_sin"].double()[s["pos"].long()]
    z = torch.complex(cs[:, :32], cs[:, 32:])
    r = x[:, 512:]
    r = r.reshape(-1, 32, 2) if case["pairs"] else r.reshape(-1, 2, 32).transpose(1, 2)
    z = torch.view_as_real(torch.view_as_complex(r.contiguous()) * z)
    z = (z if case["pairs"] else z.transpose(1, 2)).reshape(-1, 64)
    out = torch.cat([v.reshape(-1, 512), z], 1)
    out[s["slots"] < 0] = 0
    return out


def _exact_attend(q, keys):
    """One row: q [H, 576], keys [n, 576]."""
    if keys.shape[0] == 0:
        return q.new_zeros((q.shape[0], 512)), q.new_full((q.shape[0],), NEG_INF)
    sc = (q @ keys.T) * SCALE
    lse = torch.logsumexp(sc, 1)
    return torch.softmax(sc, 1) @ keys[:, :512], lse


def exact(case, seed):
    op = case["op"]
    if op == "maps":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "write":
        return _exact_write(s, case)
    if op == "gather":
        v = torch.zeros((case["N"], 576), dtype=torch.float64, device=s["pool"].device)
        at = torch.nonzero(s["slots"] >= 0)[:, 0]
        v[at] = _exact_rows(s["pool"][s["slots"][at].long()], case["fmt"])
        return v
    D, bs = case["D"], case["bs"]
    I = case.get("I", 1)
    bt = s["bt"].cpu()
    outs, lses = [], []
    rows = s["q"].shape[0]
    ctx = None if op == "sparse4" else s["ctx"].tolist()
    topk = s["topk"].cpu() if op == "sparse4" else None
    base = s["base"].tolist()
    for t in range(rows):
        if op == "sparse4":
            b = t
            ids = topk[t].long()
            ids = ids[ids >= 0]
        else:
            b, i = divmod(t, case["S"])
            p = ctx[b] - case["S"] + i
            ids = torch.arange(p + 1)
            ids = ids[(ids < case["sinks"]) | (ids > p - case["window"])]
            if case["rank"] >= 0:
                ids = ids[torch.div(ids, I, rounding_mode="floor") % D == case["rank"]]
        d = torch.div(ids, I, rounding_mode="floor") % D
        lp = torch.div(ids, I * D, rounding_mode="floor") * I + ids % I
        slot = bt[d, b, torch.div(lp, bs, rounding_mode="floor")].long() * bs + lp % bs
        slot = slot + torch.tensor(base)[d]
        keys = _exact_rows(s["pool"][slot.to(s["pool"].device)], case.get("fmt", "fp4"))
        o, l = _exact_attend(s["q"][t].double(), keys)
        outs.append(o)
        lses.append(l)
    return torch.stack(outs), torch.stack(lses)
