"""Timed cases of the serving operators around the low-bit MLA cache.

  append   norm + rotation + quantize + paged write of new tokens, straight from the projections
  read     dequantized rows of a range of every request, read back from the paged cache
  digest   mean key of every page that an append completed
  scores   attention mass that every candidate page is expected to hold, per query
  select   the pages a query reads: first, newest, and best by score
  sparse   one decode step over the selected pages (scores, selection, attention)

`run` computes each in its plain form (elementary torch operations in 32 bits, 64
for the norm and the key rotation, whose results sit next to the quantizer's
borders), or through the framework's entry points where `own` is true.
`exact` states the same definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

D_C, D_R, D_QK, PAGE = 512, 64, 576, 64
SCALE = 1.0 / math.sqrt(192.0)
EPS = float(np.float32(1e-6))
FORMATS = {"i4g64": (4, 64, 4, 64), "i2g32_r4g64": (2, 32, 4, 64), "i4g32_r2g64": (4, 32, 2, 64), "i2g64_r2g32": (2, 64, 2, 32)}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a serving batch: every request appends its newest token (smallest call, latency)
        dict(name="append_step", op="append", B=32, n=1, H=128, t_lo=4095, t_hi=4095, fmt="i4g64", conv="interleaved"),
        # a prefill chunk of a padded batch, 128 heads of queries rotated with it
        dict(name="append_prefill", op="append", B=4, n=2048, H=128, t_lo=0, t_hi=4096, fmt="i2g32_r4g64", conv="half"),
        # a short prefix read back for one request
        dict(name="read_short", op="read", B=1, t_lo=1021, t_hi=1021, fmt="i4g64"),
        # the cached prefixes of a ragged batch read back for a prefill over them
        dict(name="read_ragged", op="read", B=64, t_lo=2048, t_hi=16384, fmt="i2g32_r4g64"),
        # a speculative step: few of the requests complete a page
        dict(name="digest_step", op="digest", B=128, n=2, t_lo=1024, t_hi=4096, fmt="i2g32_r4g64"),
        # after a prefill: every page of every prompt
        dict(name="digest_prefill", op="digest", B=32, n=4096, t_lo=0, t_hi=0, fmt="i4g64"),
        # 16 heads a GPU (tensor-parallel shard), many long requests
        dict(name="scores_h16", op="scores", B=64, s_q=1, H=16, t_lo=32768, t_hi=32768),
        # few very long requests, every head
        dict(name="scores_long", op="scores", B=4, s_q=1, H=128, t_lo=131072, t_hi=131072),
        # ragged batch with two queries a request
        dict(name="select_ragged", op="select", B=128, s_q=2, t_lo=1024, t_hi=32768, k=64, sink=1, recent=2),
        # few very long requests, many pages each
        dict(name="select_long", op="select", B=4, s_q=1, t_lo=131072, t_hi=131072, k=255, sink=2, recent=4),
        # a decode step over 128K tokens that reads 4K of them
        dict(name="sparse_long", op="sparse", B=4, s_q=1, H=128, t_lo=131072, t_hi=131072, k=64, sink=1, recent=2,
             fmt="i4g64"),
        # the speculative-verify step of a ragged batch: two queries of a request select on their own (largest)
        dict(name="sparse_ragged", op="sparse", B=128, s_q=2, H=128, t_lo=1024, t_hi=32768, k=32, sink=1, recent=2,
             fmt="i2g32_r4g64"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "read", "digest", "scores", "select", "sparse"])
    fmt = rng.choice(sorted(FORMATS))
    H = rng.choice([1, 8, 16, 20, 32, 40, 64, 96, 128])
    if op == "append":
        B = _log_int(rng, 1, 128)
        n = _log_int(rng, 1, max(1, 8192 // B))
        t_hi = _log_int(rng, 1, 16384)
        return dict(op=op, B=B, n=n, H=H, t_lo=rng.randint(0, t_hi), t_hi=t_hi, fmt=fmt,
                    conv=rng.choice(["interleaved", "half"]))
    if op == "read":
        B = _log_int(rng, 1, 64)
        t_hi = _log_int(rng, 1, 16384)
        return dict(op=op, B=B, t_lo=rng.randint(0, t_hi // 2), t_hi=t_hi, fmt=fmt)
    if op == "digest":
        B = _log_int(rng, 1, 128)
        n = _log_int(rng, 1, max(1, 131072 // B))
        t_hi = _log_int(rng, 1, 8192)
        return dict(op=op, B=B, n=n, t_lo=rng.randint(0, t_hi), t_hi=t_hi, fmt=fmt)
    B = _log_int(rng, 1, 128)
    s_q = rng.choice([1, 1, 2, 3])
    t_hi = _log_int(rng, 1, min(131072, (1 << 21) // B))
    t_lo = rng.randint(max(1, t_hi // 8), t_hi)
    if op == "scores":
        return dict(op=op, B=B, s_q=s_q, H=H, t_lo=t_lo, t_hi=t_hi)
    k = _log_int(rng, 4, 256)
    sink, recent = rng.randint(0, 2), rng.randint(1, 2)
    if op == "select":
        return dict(op=op, B=B, s_q=s_q, t_lo=t_lo, t_hi=t_hi, k=k, sink=sink, recent=recent)
    k = max(4, min(k, 8192 // (B * s_q)))
    return dict(op=op, B=B, s_q=s_q, H=H, t_lo=t_lo, t_hi=t_hi, k=k, sink=sink, recent=recent, fmt=fmt)


def _token_bytes(fmt):
    bc, gc, br, gr = FORMATS[fmt]
    return D_C * bc // 8 + D_R * br // 8 + 4 * (D_C // gc) + 4 * (D_R // gr)


def work(case):
    """Bytes and operations of one pass, with lengths at their mean."""
    B, op = case["B"], case["op"]
    T = 0.5 * (case["t_lo"] + case["t_hi"])
    if op == "append":
        rows = B * case["n"]
        return {"bytes": rows * (2 * D_QK + 2 * D_QK + _token_bytes(case["fmt"]) + 2 * case["H"] * D_R * 2 + 4 * D_R),
                "flops": rows * (4 * D_C + 10 * D_QK + 3 * (case["H"] + 1) * D_R)}
    if op == "read":
        rows = B * T * 0.75 if case["t_hi"] != case["t_lo"] else B * T
        return {"bytes": rows * (_token_bytes(case["fmt"]) + 2 * D_QK), "flops": rows * 2 * D_QK}
    if op == "digest":
        pages = B * case["n"] / PAGE
        return {"bytes": pages * (PAGE * _token_bytes(case["fmt"]) + 2 * D_QK) + 8 * B, "flops": pages * PAGE * 3 * D_QK}
    s_q, P = case["s_q"], T / PAGE
    if op == "select":
        return {"bytes": B * s_q * (4 * P + 8 * case["k"]), "flops": B * s_q * P}
    rows = B * s_q * case["H"]
    w = {"bytes": rows * 2 * D_QK + B * P * 2 * D_QK, "flops": rows * P * (2 * D_QK + 4)}
    if op == "scores":
        w["bytes"] += 4 * B * s_q * P
        return w
    keys = min(case["k"] * PAGE, T)
    w["bytes"] += B * keys * _token_bytes(case["fmt"]) + rows * 2 * D_C
    w["flops"] += rows * keys * 2 * (D_QK + D_C)
    return w


# ---------------------------------------------------------------- inputs

def _quantize(x, bits, group):
    """(codes, s, z) of fp32 x [..., D], per group of channels: the cache's quantizer."""
    g = x.reshape(*x.shape[:-1], -1, group)
    mn, mx = g.amin(-1) + 0.0, g.amax(-1)
    top = torch.full((), float(2 ** bits - 1), device=x.device)  # a tensor: division by it rounds once
    s, z = ((mx - mn) / top).half(), mn.half()
    s32, z32 = s.float().unsqueeze(-1), z.float().unsqueeze(-1)
    u = torch.where(s32 == 0, torch.zeros_like(g), torch.minimum(((g - z32) / s32).round().clamp_min(0), top))
    return u, s, z


def _pack(u, bits):
    """codes [..., D/group, group] -> packed bytes [..., D*bits/8]."""
    per = 8 // bits
    u = u.reshape(*u.shape[:-2], -1, per).to(torch.int32)
    sh = bits * torch.arange(per, device=u.device, dtype=torch.int32)
    return (u << sh).sum(-1).to(torch.uint8)


def _page_bytes(x, fmt):
    """Bytes [n, page_bytes] of whole pages of fp32 tokens x [n, 64, 576]."""
    bc, gc, br, gr = FORMATS[fmt]
    uc, sc, zc = _quantize(x[..., :D_C], bc, gc)
    ur, sr, zr = _quantize(x[..., D_C:], br, gr)
    meta = lambda s, z: torch.stack([s, z], -1).contiguous().view(torch.uint8)  # noqa: E731
    parts = [_pack(uc, bc), _pack(ur, br), meta(sc, zc), meta(sr, zr)]
    return torch.cat([p.reshape(x.shape[0], -1) for p in parts], 1)


def _lengths(case, rng):
    """(lengths, tokens given of the padded n, first token read) of each request: a case's
    own set, so that its outputs have one shape, dealt to the requests by the seed."""
    B, n = case["B"], case.get("n", 1)
    own_rng = np.random.default_rng([B, n, case["t_lo"], case["t_hi"]])
    lens = own_rng.integers(case["t_lo"], case["t_hi"] + 1, size=B)
    lens[0] = case["t_hi"]
    if case["op"] == "digest" and n < PAGE:
        lens[0] = case["t_hi"] // PAGE * PAGE + PAGE - 1  # one request at least completes a page
    new = own_rng.integers(max(1, n - n // 4), n + 1, size=B)
    new[0] = n
    first = np.zeros(B, np.int64) if case["t_lo"] == case["t_hi"] else own_rng.integers(0, lens // 2 + 1)
    order = rng.permutation(B)
    return lens[order].astype(np.int64), new[order], first[order]


def _table(case, rng, capacity):
    """Random pages for requests of `capacity` tokens: (table [B, max_pages] int32, owner and index of each page)."""
    pages = np.maximum((capacity + PAGE - 1) // PAGE, 1)
    n = int(pages.sum())
    perm = rng.permutation(n)
    table = np.full((len(pages), int(pages.max())), -1, dtype=np.int32)
    at = np.concatenate([[0], np.cumsum(pages)])
    owner, index = np.zeros(n, np.int64), np.zeros(n, np.int64)
    for b, m in enumerate(pages):
        mine = perm[at[b]:at[b + 1]]
        table[b, :m] = mine
        owner[mine], index[mine] = b, np.arange(m)
    return torch.from_numpy(table).cuda(), owner, index, n


def _fill_pool(st, case, gen, offset=None):
    """Random tokens in every page: N(0,1) times a magnitude for each channel, plus the page's offset [pages, 576]."""
    n = st["num_pages"]
    mag = torch.exp(0.5 * torch.randn(D_QK, generator=gen, device="cuda"))
    pool = torch.empty((n, PAGE * _token_bytes(case["fmt"])), dtype=torch.uint8, device="cuda")
    for p in range(0, n, 2048):
        x = torch.randn((min(2048, n - p), PAGE, D_QK), generator=gen, device="cuda") * mag
        if offset is not None:
            x += offset[p:p + 2048, None, :]
        pool[p:p + 2048] = _page_bytes(x.bfloat16().float(), case["fmt"])
    st["pool"] = pool


def _queries(st, case, gen):
    """Queries of a request share a direction; `hot` pages hold keys along it."""
    B, s_q, H = case["B"], case["s_q"], case["H"]
    u = torch.randn((B, 1, 1, D_QK), generator=gen, device="cuda")
    q = (u + 0.5 * torch.randn((B, s_q, H, D_QK), generator=gen, device="cuda")).bfloat16()
    st["q_c"], st["q_r"] = q[..., :D_C].contiguous(), q[..., D_C:].contiguous()
    return (u / u.norm(dim=-1, keepdim=True))[:, 0, 0]


def _hot_offsets(case, rng, owner, index, pages_of, direction, hot):
    """Offset along the request's direction for about `hot` of its pages, one strength each."""
    gain = np.where(rng.random(len(owner)) < hot / np.maximum(pages_of[owner], 1), rng.uniform(1.0, 3.5, len(owner)), 0.0)
    g = torch.from_numpy(gain.astype(np.float32)).cuda()
    return direction[torch.from_numpy(owner).cuda()] * g[:, None]


def prepare(case, seed):
    rng = np.random.default_rng([int(seed), 17])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) + 1)
    op, B = case["op"], case["B"]
    st = {"op": op, "case": dict(case)}
    lens, new, first = _lengths(case, rng)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    if op in ("append", "digest"):
        n = case["n"]
        st["before"] = i32(lens)
        st["table"], _, _, st["num_pages"] = _table(case, rng, lens + n)
        st["new_lens"] = i32(new) if n > 1 else None  # the batch is padded to n
    if op == "append":
        H = case["H"]
        # the down-projections' fused output [B, n, 1536 + 576] and the queries' [B, n, H, 128 + 64]
        kv = torch.randn((B, n, 1536 + D_QK), generator=gen, device="cuda")
        kv *= torch.exp(0.5 * torch.randn(1536 + D_QK, generator=gen, device="cuda"))
        st["kv"] = kv.bfloat16()[..., 1536:]
        st["q"] = torch.randn((B, n, H, 192), generator=gen, device="cuda", dtype=torch.bfloat16)[..., 128:]
        st["weight"] = (1.0 + 0.2 * torch.randn(D_C, generator=gen, device="cuda")).bfloat16()
        pos = torch.arange(case["t_hi"] + n, device="cuda", dtype=torch.float64)
        ang = pos[:, None] * 10000.0 ** (-torch.arange(D_R // 2, device="cuda", dtype=torch.float64) / (D_R // 2))
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["pool"] = torch.zeros((st["num_pages"], PAGE * _token_bytes(case["fmt"])), dtype=torch.uint8, device="cuda")
        st["q_out"] = torch.zeros((B, n, H, D_R), dtype=torch.bfloat16, device="cuda")
        st["rows"] = torch.zeros((B, n, D_QK), dtype=torch.bfloat16, device="cuda")
    elif op == "digest":
        _fill_pool(st, case, gen)
        st["digests"] = torch.zeros((st["num_pages"] + 1, D_QK), dtype=torch.bfloat16, device="cuda")
    elif op == "read":
        st["table"], _, _, st["num_pages"] = _table(case, rng, lens)
        _fill_pool(st, case, gen)
        st["start"] = i32(first)
        rows = np.concatenate([[0], np.cumsum(lens - first)])
        st["cu_rows"], st["n_rows"], st["max_rows"] = i32(rows), int(rows[-1]), int((lens - first).max())
        out = torch.zeros((max(st["n_rows"], 1), D_QK), dtype=torch.bfloat16, device="cuda")
        st["out"], st["out_c"], st["out_kr"] = out, out[:, :D_C], out[:, D_C:]
    else:
        st["lens"], st["max_len"] = i32(lens), case["t_hi"]
        st["table"], owner, index, st["num_pages"] = _table(case, rng, lens)
        pages_of = (lens + PAGE - 1) // PAGE
        width = max(1, (case["t_hi"] + PAGE - 1) // PAGE)
        if op == "select":
            # scores of an earlier call: sums over heads of softmax weights, many equal after a long tail's underflow
            sc = torch.rand((B, case["s_q"], width), generator=gen, device="cuda") ** 6
            sc = torch.where(sc < 1e-3, torch.zeros_like(sc), sc * 16).bfloat16().float()
            L = st["lens"].long()[:, None] - case["s_q"] + 1 + torch.arange(case["s_q"], device="cuda")
            cand = ((L - 1) // PAGE).clamp_min(0)
            st["scores"] = sc.masked_fill(torch.arange(width, device="cuda") >= cand[..., None], -math.inf)
        else:
            direction = _queries(st, case, gen)
            hot = case["k"] / 2 if op == "sparse" else 24
            off = _hot_offsets(case, rng, owner, index, pages_of, direction, hot)
            if op == "sparse":
                _fill_pool(st, case, gen, off)
                st["digests"] = torch.empty((st["num_pages"], D_QK), dtype=torch.bfloat16, device="cuda")
                for p in range(0, st["num_pages"], 2048):
                    ids = torch.arange(p, min(p + 2048, st["num_pages"]), device="cuda")
                    st["digests"][p:p + 2048] = _values(st["pool"], case["fmt"], ids).mean(1).bfloat16()
            else:
                st["digests"] = (torch.randn((st["num_pages"], D_QK), generator=gen, device="cuda") * 0.125 + off).bfloat16()
    return st


# ---------------------------------------------------------------- plain forms

def _values(pool, fmt, pages, slots=None):
    """fp32 values [..., 64, 576] of whole pages, or [..., 576] of one slot of each."""
    bc, gc, br, gr = FORMATS[fmt]
    n = pool.shape[0]
    widths = (D_C * bc // 8, D_R * br // 8, 4 * (D_C // gc), 4 * (D_R // gr))
    segs = torch.split(pool, [PAGE * w for w in widths], 1)
    take = [s.view(n, PAGE, w)[pages] if slots is None else s.view(n, PAGE, w)[pages, slots] for s, w in zip(segs, widths)]

    def part(codes, meta, bits, group):
        sh = bits * torch.arange(8 // bits, device=pool.device, dtype=torch.uint8)
        u = ((codes.unsqueeze(-1) >> sh) & (2 ** bits - 1)).flatten(-2)
        sz = meta.contiguous().view(torch.float16).float().unflatten(-1, (-1, 2))
        u = u.float().unflatten(-1, (-1, group))
        return (u * sz[..., :1] + sz[..., 1:]).flatten(-2)

    return torch.cat([part(take[0], take[2], bc, gc), part(take[1], take[3], br, gr)], -1)


def _rotate(x, cos, sin, conv, dtype):
    """Rotary pairs of x [..., 64] turned by the angles of cos, sin [..., 32]."""
    x, cos, sin = x.to(dtype), cos.to(dtype), sin.to(dtype)
    if conv == "half":
        a, b = x[..., :D_R // 2], x[..., D_R // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _plain_append(st):
    case = st["case"]
    B, n = case["B"], case["n"]
    bc, gc, br, gr = FORMATS[case["fmt"]]
    j = torch.arange(n, device="cuda")
    pos = st["before"].long()[:, None] + j
    cos, sin = st["cos_sin"][pos].split(D_R // 2, -1)
    x = st["kv"][..., :D_C].double()
    inv = 1.0 / (x.square().sum(-1, keepdim=True) / D_C + EPS).sqrt()
    c = (x * inv * st["weight"].double()).float().bfloat16().float()
    kr = _rotate(st["kv"][..., D_C:], cos, sin, case["conv"], torch.float64).float().bfloat16().float()
    hat = []
    for v, bits, group in ((c, bc, gc), (kr, br, gr)):
        u, s, z = _quantize(v, bits, group)
        hat.append((u * s.float().unsqueeze(-1) + z.float().unsqueeze(-1)).flatten(-2))
    rows = torch.cat(hat, -1).bfloat16()
    q = _rotate(st["q"], cos[:, :, None], sin[:, :, None], case["conv"], torch.float32).bfloat16()
    if st["new_lens"] is not None:
        keep = (j < st["new_lens"][:, None])[..., None]
        rows = torch.where(keep, rows, st["rows"])
        q = torch.where(keep[..., None], q, st["q_out"])
    return {"q": q, "rows": rows}


def _plain_read(st):
    r = torch.arange(st["n_rows"], device="cuda")
    b = torch.searchsorted(st["cu_rows"].long(), r, right=True) - 1
    t = st["start"].long()[b] + r - st["cu_rows"].long()[b]
    return _values(st["pool"], st["case"]["fmt"], st["table"].long()[b, t // PAGE], t % PAGE).bfloat16()


def _plain_digest(st):
    n = st["case"]["n"]
    before = st["before"].long()
    new = st["new_lens"].long() if st["new_lens"] is not None else torch.full_like(before, n)
    idx = before[:, None] // PAGE + torch.arange(n // PAGE + 1, device="cuda")
    full = idx < ((before + new) // PAGE)[:, None]
    page = torch.gather(st["table"].long(), 1, idx.clamp_max(st["table"].shape[1] - 1))
    mean = _values(st["pool"], st["case"]["fmt"], torch.where(full, page, 0)).mean(-2).bfloat16()
    out = st["digests"].clone()
    out[torch.where(full, page, st["num_pages"])] = mean  # the others go to a row behind the last page
    return out[:st["num_pages"]]


def _visible(st):
    s_q = st["case"]["s_q"]
    return st["lens"].long()[:, None] - s_q + 1 + torch.arange(s_q, device="cuda")  # [B, s_q]


def _plain_scores(st):
    width = max(1, -(-st["max_len"] // PAGE))
    cand = ((_visible(st) - 1) // PAGE).clamp_min(0)
    ok = torch.arange(width, device="cuda") < cand[..., None]  # [B, s_q, width]
    d = st["digests"][st["table"][:, :width].long().clamp_min(0)].float()
    B, s_q, H = st["q_c"].shape[:3]
    q = torch.cat([st["q_c"], st["q_r"]], -1).float().reshape(B, s_q * H, D_QK)
    s = (torch.bmm(q, d.transpose(1, 2)) * SCALE).view(B, s_q, H, width)
    s = s.masked_fill(~ok[:, :, None], -math.inf)
    e = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-1e30))
    mass = (e / e.sum(-1, keepdim=True).clamp_min(1e-30)).sum(2)
    return mass.masked_fill(~ok, -math.inf)


def _plain_select(st, scores):
    case = st["case"]
    k, width = case["k"], scores.shape[-1]
    L = _visible(st)
    last = torch.where(L > 0, (L - 1) // PAGE, -1)[..., None]  # the page a query's own position is in
    p = torch.arange(width, device="cuda")
    rank = scores.masked_fill(p > last - case["recent"], math.inf).masked_fill(p < case["sink"], math.inf)
    rank = rank.masked_fill(p > last, -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :k]  # the lower of two equal ones first
    best = torch.where(best <= last, best, width)
    best = torch.sort(best, dim=-1)[0]
    if best.shape[-1] < k:
        best = torch.nn.functional.pad(best, (0, k - best.shape[-1]), value=width)
    real = best < width
    page = torch.gather(st["table"].long()[:, None, :].expand(-1, L.shape[1], -1), 2, best.clamp_max(st["table"].shape[1] - 1))
    count = real.sum(-1)
    lens = torch.where(L > 0, (count - 1) * PAGE + (L - 1) % PAGE + 1, 0)
    return torch.where(real, page, -1).int(), torch.where(real, best, -1).int(), lens.int()


def _plain_sparse(st):
    table, _, lens = _plain_select(st, _plain_scores(st))
    k = _values(st["pool"], st["case"]["fmt"], table.long().clamp_min(0)).flatten(2, 3)  # [B, s_q, keys, 576]
    q = torch.cat([st["q_c"], st["q_r"]], -1).float()
    s = torch.matmul(q, k.transpose(-1, -2)) * SCALE
    ok = torch.arange(k.shape[2], device="cuda") < lens[..., None, None]
    s = s.masked_fill(~ok, -math.inf)
    e = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-1e30))
    o = torch.matmul(e, k[..., :D_C]) / e.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.bfloat16()


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if own:
        from bit_mla_kv_qdecode_b200 import api
        case = st["case"]
        if "fmt" in case and "desc" not in st:  # the cache's description, made once and kept with the pool
            st["desc"] = api.make_desc(*FORMATS[case["fmt"]], num_pages=st["num_pages"])
        if op == "append":
            api.mla_qcache_append_norm_rope(st["desc"], st["pool"], st["table"], st["before"], st["kv"], st["weight"], EPS,
                                            st["cos_sin"], convention=case["conv"], q=st["q"], q_out=st["q_out"],
                                            new_lens=st["new_lens"], rows_out=st["rows"])
            return {"q": st["q_out"], "rows": st["rows"]}
        if op == "read":
            api.mla_qcache_read(st["desc"], st["pool"], st["table"], st["start"], st["cu_rows"], st["max_rows"],
                                st["out_c"], st["out_kr"])
            return st["out"]
        if op == "digest":
            api.mla_page_digest(st["desc"], st["pool"], st["table"], st["before"], case["n"], st["digests"][:-1],
                                new_lens=st["new_lens"])
            return st["digests"][:-1]
        if op == "scores":
            return api.mla_page_scores(st["table"], st["lens"], st["max_len"], st["digests"], st["q_c"], st["q_r"], SCALE)
        if op == "select":
            return list(api.mla_select_pages(st["table"], st["lens"], st["max_len"], st["scores"], case["k"],
                                             n_sink=case["sink"], n_recent=case["recent"]))
        return api.mla_qdecode_sparse(st["desc"], st["pool"], st["table"], st["lens"], st["max_len"], st["digests"],
                                      st["q_c"], st["q_r"], SCALE, case["k"], n_sink=case["sink"],
                                      n_recent=case["recent"])[0]
    if op == "append":
        return _plain_append(st)
    if op == "read":
        return _plain_read(st)
    if op == "digest":
        return _plain_digest(st)
    if op == "scores":
        return _plain_scores(st)
    if op == "select":
        return list(_plain_select(st, st["scores"]))
    return _plain_sparse(st)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_tokens(pool, fmt, page):
    """float64 [64, 576] tokens of one page's bytes, by the layout's definition."""
    bc, gc, br, gr = FORMATS[fmt]
    raw, at, got = pool[page], 0, []
    for d, bits in ((D_C, bc), (D_R, br)):
        n = PAGE * d * bits // 8
        b = raw[at:at + n].view(PAGE, -1).long()
        got.append(torch.stack([b.bitwise_right_shift(bits * i) % (1 << bits) for i in range(8 // bits)], 2).view(PAGE, d).double())
        at += n
    for i, (d, group) in enumerate(((D_C, gc), (D_R, gr))):
        n = PAGE * 4 * (d // group)
        m = raw[at:at + n].clone().view(torch.float16).view(PAGE, d // group, 2).double()
        got[i] = got[i] * m[:, :, 0].repeat_interleave(group, 1) + m[:, :, 1].repeat_interleave(group, 1)
        at += n
    return torch.cat(got, 1)


def _exact_scores(st, b, i, L):
    """float64 mass of each candidate page for query i of request b."""
    cand = max(0, (L - 1) // PAGE)
    if cand == 0:
        return torch.zeros(0, dtype=torch.float64, device="cuda")
    d = st["digests"][st["table"][b, :cand].long()].double()
    s = SCALE * (st["q_c"][b, i].double() @ d[:, :D_C].T + st["q_r"][b, i].double() @ d[:, D_C:].T)
    return torch.softmax(s, 1).sum(0)


def exact(case, seed):
    op = case["op"]
    if op == "select" or (op == "sparse" and case["B"] * case["s_q"] * case["k"] > 16384):
        return None
    st = prepare(case, seed)
    if op == "append":
        B, n = case["B"], case["n"]
        before = st["before"].long().cpu()
        count = st["new_lens"].cpu() if st["new_lens"] is not None else torch.full((B,), n)
        q, rows = torch.zeros_like(st["q_out"], dtype=torch.float64), torch.zeros_like(st["rows"], dtype=torch.float64)
        bc, gc, br, gr = FORMATS[case["fmt"]]
        half = D_R // 2
        first = torch.arange(half, device="cuda") if case["conv"] == "half" else 2 * torch.arange(half, device="cuda")
        second = first + (half if case["conv"] == "half" else 1)
        for b in range(B):
            m = int(count[b])
            cs = st["cos_sin"][int(before[b]):int(before[b]) + m].double()
            rot = torch.complex(cs[:, :half], cs[:, half:])
            v = st["q"][b, :m].double()
            w = torch.complex(v[..., first], v[..., second]) * rot[:, None]
            q[b, :m, :, first], q[b, :m, :, second] = w.real, w.imag
            k = st["kv"][b, :m].double()
            w = torch.complex(k[:, D_C + first], k[:, D_C + second]) * rot
            c = k[:, :D_C] * torch.rsqrt(k[:, :D_C].pow(2).mean(1, keepdim=True) + EPS) * st["weight"].double()
            kr = torch.empty((m, D_R), dtype=torch.float64, device="cuda")
            kr[:, first], kr[:, second] = w.real, w.imag
            at = 0
            for x, bits, group in ((c, bc, gc), (kr, br, gr)):
                # the quantizer's own roundings are part of the definition: bf16 input, fp16 step and offset, fp32 quotient
                for g in x.float().bfloat16().float().split(group, 1):
                    lo, hi = g.min(1, keepdim=True)[0], g.max(1, keepdim=True)[0]
                    step = ((hi - lo).double() / (2 ** bits - 1)).float().half().float()
                    off = lo.half().float()
                    code = ((g - off).double() / step.double()).float().round().clamp(0, 2 ** bits - 1)
                    code = torch.where(step == 0, torch.zeros_like(code), code)
                    rows[b, :m, at:at + group] = code.double() * step.double() + off.double()
                    at += group
        return {"q": q, "rows": rows}
    if op == "read":
        out = torch.zeros((st["out"].shape[0], D_QK), dtype=torch.float64, device="cuda")
        cu, start = st["cu_rows"].tolist(), st["start"].tolist()
        table = st["table"].tolist()
        for b in range(case["B"]):
            t, end, at = start[b], start[b] + cu[b + 1] - cu[b], cu[b]
            while t < end:
                stop = min(end, (t // PAGE + 1) * PAGE)
                v = _exact_tokens(st["pool"], case["fmt"], table[b][t // PAGE])
                out[at:at + stop - t] = v[t % PAGE:t % PAGE + stop - t]
                at, t = at + stop - t, stop
        return out[:st["n_rows"]]
    if op == "digest":
        out = torch.zeros((st["num_pages"], D_QK), dtype=torch.float64, device="cuda")
        table, before = st["table"].tolist(), st["before"].tolist()
        new = st["new_lens"].tolist() if st["new_lens"] is not None else [case["n"]] * case["B"]
        for b in range(case["B"]):
            for p in range(before[b] // PAGE, (before[b] + new[b]) // PAGE):
                out[table[b][p]] = _exact_tokens(st["pool"], case["fmt"], table[b][p]).mean(0)
        return out
    lens = st["lens"].tolist()
    if op == "scores":
        width = max(1, -(-case["t_hi"] // PAGE))
        out = torch.full((case["B"], case["s_q"], width), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            for i in range(case["s_q"]):
                s = _exact_scores(st, b, i, lens[b] - case["s_q"] + 1 + i)
                out[b, i, :s.numel()] = s
        return out
    out = torch.zeros(st["q_c"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        for i in range(case["s_q"]):
            L = lens[b] - case["s_q"] + 1 + i
            if L <= 0:
                continue
            last = (L - 1) // PAGE
            must = [p for p in range(last + 1) if p < case["sink"] or p > last - case["recent"]]
            if last + 1 <= case["k"]:
                pages = list(range(last + 1))
            else:
                s = _exact_scores(st, b, i, L)
                rest = sorted((p for p in range(last) if p not in set(must)), key=lambda p, s=s.tolist(): (-s[p], p))
                pages = sorted(must + rest[:case["k"] - len(must)])
            v = torch.cat([_exact_tokens(st["pool"], case["fmt"], int(st["table"][b, p])) for p in pages])
            v = v[:(len(pages) - 1) * PAGE + (L - 1) % PAGE + 1]
            w = torch.softmax(SCALE * (st["q_c"][b, i].double() @ v[:, :D_C].T + st["q_r"][b, i].double() @ v[:, D_C:].T), 1)
            out[b, i] = w @ v[:, :D_C]
    return out
