"""Measured cases of the 8-bit paged cache: writing it, reading it back, and
decode and prefill attention over it.

The cache holds e4m3 values in block pools [num_blocks, 16, n_kv, head_dim]
with one fp32 scale, a power of two, per (block, KV head) and pool; an element
stands for its e4m3 value times its block's and head's scale.
"""
import math
import random

import torch

own = False  # False: the plain forms below; True: the framework's own calls

BS = 16  # tokens per block
E_MIN, E_MAX = -60, 60  # exponents of the scales
F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases

def _case(name, op, dtype, heads, n_kv, head_dim, seqs, lo, hi, new=0, spread="even"):
    """`seqs` sequences of `lo` .. `hi` tokens; `new` of each are this step's
    (0: the whole sequence is)."""
    c = dict(op=op, dtype=dtype, heads=heads, n_kv=n_kv, head_dim=head_dim, seqs=seqs, lo=lo,
             hi=hi, new=new, spread=spread)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of each of a few toy sequences: what a call costs by itself
        _case("write toy step f32", "write", "f32", 8, 4, 16, 4, 7, 100, 1),
        # a decode step of a 64-user server: one token a sequence, most into part-filled blocks
        _case("write decode step", "write", "bf16", 32, 8, 64, 64, 512, 2048, 1),
        # whole prompts of 32 users arriving together
        _case("write prompts", "write", "bf16", 32, 8, 64, 32, 128, 2048, 0),
        # reading a toy cache back in fp32
        _case("read back toy f32", "gather", "f32", 8, 4, 16, 4, 7, 100, 0),
        # reading a batch's whole cache back (moving sequences out, checking a cache)
        _case("read back batch", "gather", "bf16", 32, 8, 64, 64, 512, 2048, 0),
        # the smallest decode call, in fp32
        _case("decode toy f32", "decode", "f32", 8, 4, 16, 4, 7, 100, 1),
        # 30 users of a small model: odd head counts, bound by latency
        _case("decode 30 users", "decode", "bf16", 9, 3, 64, 30, 33, 612, 1),
        # 64 users, head_dim 64, four query heads to a KV head
        _case("decode 64 users", "decode", "bf16", 32, 8, 64, 64, 512, 2048, 1),
        # 256 users of a large model, very uneven lengths
        _case("decode 256 users", "decode", "bf16", 64, 8, 128, 256, 16, 8192, 1, "lognormal"),
        # ragged chunks over ragged histories in fp32
        _case("prefill ragged f32", "prefill", "f32", 8, 4, 16, 6, 40, 230, 37),
        # the prompts of 30 users of a small model, each whole
        _case("prefill 30 prompts", "prefill", "bf16", 9, 3, 64, 30, 33, 612, 0),
        # 512-token chunks of four long prompts of a large model
        _case("prefill 4 chunks", "prefill", "bf16", 64, 8, 128, 4, 512, 4608, 512),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "gather", "decode", "decode", "prefill"])
    heads, n_kv = rng.choice([(8, 4), (9, 3), (32, 8), (32, 32), (64, 8), (12, 1), (10, 5)])
    head_dim = rng.choice([16, 32, 64, 64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "prefill":
        seqs = log_int(1, 16)
        hi = log_int(20, 2048)
        new = rng.choice([0, log_int(1, hi)])
    else:
        seqs = log_int(1, 128)
        hi = log_int(20, 4096)
        new = 0 if op == "gather" else 1 if op == "decode" else rng.choice([1, 1, 0, log_int(2, 64)])
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    # no more tokens than the largest listed cases have
    while seqs > 1 and seqs * hi * n_kv * head_dim > (3.0e8 if op == "decode" else 9.0e7):
        seqs = (seqs + 1) // 2
    while op == "prefill" and seqs > 1 and seqs * hi * (new or hi) * heads * head_dim > 3.0e10:
        seqs = (seqs + 1) // 2
    return _case("", op, dtype, heads, n_kv, head_dim, seqs, lo, hi, new, rng.choice(["even", "lognormal"]))


def _lengths(case):
    """Tokens of each sequence and how many of them are new; fixed by the case."""
    r = random.Random(case["seqs"] * 1000003 + case["hi"] * 1009 + case["lo"])
    lens = []
    for _ in range(case["seqs"]):
        if case["spread"] == "lognormal":
            x = int(round(r.lognormvariate(math.log(max(1.0, case["hi"] / 8)), 1.0)))
            lens.append(min(case["hi"], max(case["lo"], x)))
        else:
            lens.append(r.randint(case["lo"], case["hi"]))
    return lens, [min(n, case["new"]) if case["new"] else n for n in lens]


def work(case):
    lens, new = _lengths(case)
    row = case["n_kv"] * case["head_dim"]
    es = 4 if case["dtype"] == "f32" else 2
    blocks = sum(-(-n // BS) for n in lens)
    table = 4 * (blocks + 2 * len(lens))
    cache = 2 * sum(lens) * row + 2 * blocks * case["n_kv"] * 4 + table
    q = case["heads"] * case["head_dim"]
    if case["op"] == "write":
        touched = sum((n - 1) // BS - (n - c) // BS + 1 for n, c in zip(lens, new))
        return {"bytes": 2 * sum(new) * row * (es + 1) + 2 * touched * case["n_kv"] * 4
                + 4 * (touched + 2 * len(lens)), "flops": 4 * sum(new) * row}
    if case["op"] == "gather":
        return {"bytes": cache + 2 * sum(lens) * row * es, "flops": 2 * sum(lens) * row}
    seen = sum(c * (n - c) + c * (c + 1) // 2 for n, c in zip(lens, new))  # (query, key) pairs
    return {"bytes": cache + 2 * sum(new) * q * es, "flops": 4 * seen * q}


# ------------------------------------------------------------------ inputs

def _pow2(e):
    """2^e as fp32 for an integer tensor e (normal range)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _fit(a):
    """Smallest exponent e in [E_MIN, E_MAX] with a <= 448 * 2^e (a >= 0)."""
    m, e = torch.frexp(a.double() / 448.0)  # in 64 bits: a may sit next to a border
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(a > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _values(g, shape, n_kv, head_dim, dev, keys):
    """Keys have a few large channels and heads of different sizes, values less so."""
    x = torch.randn(shape, generator=g, device=dev)
    head = torch.exp(0.5 * torch.randn((n_kv, 1), generator=g, device=dev))
    if keys:
        big = torch.rand((n_kv, head_dim), generator=g, device=dev) < 0.04
        head = head * torch.where(big, 4.0, 1.0)
    return x * head


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _lengths(case)
    n_kv, hd, H = case["n_kv"], case["head_dim"], case["heads"]
    dt = TYPES[case["dtype"]]
    held = [-(-n // BS) for n in lens]
    nb = sum(held) + 3  # a dummy block 0 and two that nobody holds
    W = max(held)
    ids = torch.randperm(nb - 1, generator=g, device=dev)[: sum(held)] + 1
    bt = torch.zeros((len(lens), W), dtype=torch.int32, device=dev)
    slot = torch.arange(W, device=dev)[None, :] < torch.tensor(held, device=dev)[:, None]
    bt[slot] = ids.to(torch.int32)
    pools, scales = [], []
    for keys in (True, False):
        x = _values(g, (nb, BS, n_kv, hd), n_kv, hd, dev, keys)
        s = _pow2(_fit(x.abs().amax(dim=(1, 3))))
        pools.append((x / s[:, None, :, None]).to(F8))
        scales.append(s)
        del x
    T = sum(new)
    st = dict(op=case["op"], bt=bt, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
              kp=pools[0], vp=pools[1], ks=scales[0], vs=scales[1], scale=1.0 / math.sqrt(hd),
              max_len=max(lens), max_new=max(new), tokens=T, dt=dt, rep=H // n_kv)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["op"] == "write":
        st["k"] = _values(g, (T, n_kv, hd), n_kv, hd, dev, True).to(dt)
        st["v"] = _values(g, (T, n_kv, hd), n_kv, hd, dev, False).to(dt)
    elif case["op"] == "gather":
        st["k_out"] = torch.empty((T, n_kv, hd), dtype=dt, device=dev)
        st["v_out"] = torch.empty_like(st["k_out"])
    else:
        st["q"] = (1.5 * torch.randn((T, H, hd), generator=g, device=dev)).to(dt)
        st["out"] = torch.empty_like(st["q"])
    st["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if own and case["op"] == "decode":  # the scratch that a serving loop keeps
        import paged_kv_cache_write_gb300 as pkv
        n = pkv.decode_fp8_workspace_bytes(len(lens), H, hd, st["max_len"])
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return st


# --------------------------------------------------------------- the calls

def run(s):
    if own:
        return _run_own(s)
    return {"write": _plain_write, "gather": _plain_gather, "decode": _plain_attention,
            "prefill": _plain_attention}[s["op"]](s)


def _run_own(s):
    import paged_kv_cache_write_gb300 as pkv
    if s["op"] == "write":
        pkv.kv_write_fp8(s["k"], s["v"], s["bt"], s["lens"], s["cu"], s["kp"], s["vp"], s["ks"],
                         s["vs"], err=s["err"])
        return s["kp"], s["vp"], s["ks"], s["vs"]
    if s["op"] == "gather":
        return pkv.kv_gather_fp8(s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["cu"],
                                 s["tokens"], k_out=s["k_out"], v_out=s["v_out"], err=s["err"])
    if s["op"] == "decode":
        return pkv.paged_attention_decode_fp8(
            s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["scale"],
            s["max_len"], out=s["out"], workspace=s["workspace"], err=s["err"])
    return pkv.paged_attention_prefill_fp8(
        s["q"], s["cu"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["scale"],
        s["max_new"], s["max_len"], out=s["out"], err=s["err"])


# --------------------------------------------------------- the plain forms

def _take(pool, scale, blocks):
    """fp32 values [*blocks.shape, BS, n_kv, hd] of whole blocks."""
    x = pool.view(torch.uint8)[blocks].view(F8).float()
    return x * scale[blocks][..., None, :, None]


def _owners(s, tokens):
    """Sequence of each row of a ragged batch, and the row's position among the
    sequence's tokens (the rows are each sequence's last ones)."""
    t = torch.arange(tokens, device=s["cu"].device)
    b = torch.searchsorted(s["cu"], t.to(torch.int32), right=True) - 1
    cu = s["cu"].long()
    pos = s["lens"].long()[b] - cu[b + 1] + t
    return b, pos


def _plain_write(s):
    b, pos = _owners(s, s["tokens"])
    blk = s["bt"].long()[b, pos // BS]
    first = (s["lens"] - (s["cu"][1:] - s["cu"][:-1])).long()  # each sequence's first new position
    older = (pos // BS) * BS < first[b]  # the token's block holds earlier tokens
    # the block that each sequence's first new token goes into, and its earlier rows
    has = (s["cu"][1:] > s["cu"][:-1]) & (first % BS > 0)
    edge = s["bt"].long()[torch.arange(len(first), device=first.device),
                          (first // BS).clamp(max=s["bt"].shape[1] - 1)]
    keep = has[:, None] & (torch.arange(BS, device=first.device)[None, :] < (first % BS)[:, None])
    for x, pool, scale in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        x = x.float()
        need = torch.zeros_like(scale).index_reduce_(0, blk, x.abs().amax(-1), "amax")
        fit = _pow2(_fit(need[blk]))
        to = torch.where(older[:, None], torch.maximum(fit, scale[blk]), fit)
        rows = (x / to[..., None]).clamp(-448.0, 448.0).to(F8)
        was = scale[edge]
        scale[blk] = to
        old = pool.view(torch.uint8)[edge].view(F8).float() * (was / scale[edge])[:, None, :, None]
        flat = pool.view(torch.uint8).view(-1, *pool.shape[2:])
        at = (edge[:, None] * BS + torch.arange(BS, device=edge.device)[None, :])[keep]
        flat[at] = old.to(F8).view(torch.uint8)[keep]
        flat[blk * BS + pos % BS] = rows.view(torch.uint8)
    return s["kp"], s["vp"], s["ks"], s["vs"]


def _plain_gather(s):
    b, pos = _owners(s, s["tokens"])
    blk = s["bt"].long()[b, pos // BS]
    out = []
    for pool, scale in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
        flat = pool.view(torch.uint8).view(-1, *pool.shape[2:])
        x = flat[blk * BS + pos % BS].view(F8).float()
        out.append((x * scale[blk][..., None]).to(s["dt"]))
    return tuple(out)


def _plain_attention(s):
    """Queries padded to the longest chunk, keys to the longest sequence."""
    B, W = s["bt"].shape
    n_kv, hd = s["kp"].shape[2:]
    T, H, _ = s["q"].shape
    b, pos = _owners(s, T)
    i = torch.arange(T, device=b.device) - s["cu"].long()[b]
    C = s["max_new"]
    q = torch.zeros((B, C, H, hd), device=b.device)
    q[b, i] = s["q"].float()
    last = torch.full((B, C), -1, dtype=torch.long, device=b.device)
    last[b, i] = pos
    k = _take(s["kp"], s["ks"], s["bt"].long()).view(B, W * BS, n_kv, hd)
    # [B, n_kv, C * rep, hd] x [B, n_kv, hd, keys]
    q = q.view(B, C, n_kv, s["rep"], hd).permute(0, 2, 1, 3, 4).reshape(B, n_kv, C * s["rep"], hd)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    del k
    key = torch.arange(W * BS, device=b.device)
    seen = (key[None, None, :] <= last[:, :, None])[:, None, :, None, :]
    x = x.view(B, n_kv, C, s["rep"], W * BS).masked_fill_(~seen, float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3.0e38)  # a padded row sees no key
    p = torch.exp(x - m)
    p = p / p.sum(-1, keepdim=True).clamp(min=1.0e-30)
    v = _take(s["vp"], s["vs"], s["bt"].long()).view(B, W * BS, n_kv, hd)
    # rows past a sequence's end hold anything: they take no part
    v = v * (key[None, :] < s["lens"].long()[:, None])[:, :, None, None]
    o = torch.matmul(p.view(B, n_kv, C * s["rep"], W * BS), v.permute(0, 2, 1, 3))
    o = o.view(B, n_kv, C, s["rep"], hd).permute(0, 2, 1, 3, 4).reshape(B, C, H, hd)
    return o[b, i].to(s["dt"])


# ------------------------------------------------------------ in 64 bits

def _round_e4m3(x):
    """Nearest e4m3 value of each x (|x| <= 448), ties to the even one."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40)))
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)  # log2 may round up to the next power
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, e)
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_scale(a):
    """Smallest power of two in range that brings a to at most 448, by search."""
    s = torch.full_like(a, 2.0 ** E_MIN)
    for _ in range(E_MAX - E_MIN):
        s = torch.where(a > 448.0 * s, s * 2.0, s)
    return s


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lengths(case)
    bt = s["bt"].tolist()
    D = torch.float64
    if case["op"] == "write":
        res = []
        for x, pool, scale in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
            val, sc, at = pool.to(D), scale.to(D), 0
            for b, (n, c) in enumerate(zip(lens, new)):
                p0 = n - c
                for j in range(p0 // BS, (n - 1) // BS + 1):
                    lo, hi = max(p0, j * BS), min(n, (j + 1) * BS)
                    rows = x[at + lo - p0: at + hi - p0].to(D)
                    to = _exact_scale(rows.abs().amax(dim=(0, 2)))
                    if lo > j * BS:  # earlier tokens stay, under a scale that may have grown
                        to = torch.maximum(to, sc[bt[b][j]])
                        old = val[bt[b][j], : lo - j * BS]
                        val[bt[b][j], : lo - j * BS] = _round_e4m3(old * (sc[bt[b][j]] / to)[:, None])
                    val[bt[b][j], lo - j * BS: hi - j * BS] = _round_e4m3(rows / to[:, None])
                    sc[bt[b][j]] = to
                at += c
            res.append((val, sc))
        return res[0][0], res[1][0], res[0][1], res[1][1]
    out, at = [], 0
    for b, (n, c) in enumerate(zip(lens, new)):
        row = s["bt"][b, : -(-n // BS)].long()
        k, v = ((p.view(torch.uint8)[row].view(F8).to(D) * z[row].to(D)[:, None, :, None]).flatten(0, 1)[:n]
                for p, z in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))
        if case["op"] == "gather":
            out.append((k, v))
            continue
        q = s["q"][at: at + c].to(D)
        k, v = (z.repeat_interleave(s["rep"], dim=1) for z in (k, v))
        x = torch.einsum("chd,nhd->hcn", q, k) / math.sqrt(case["head_dim"])
        ahead = torch.arange(n, device=x.device)[None, :] > torch.arange(n - c, n, device=x.device)[:, None]
        w = torch.softmax(x.masked_fill(ahead, float("-inf")), dim=-1)
        out.append(torch.einsum("hcn,nhd->chd", w, v))
        at += c
    if case["op"] == "gather":
        return torch.cat([k for k, _ in out]), torch.cat([v for _, v in out])
    return torch.cat(out)
