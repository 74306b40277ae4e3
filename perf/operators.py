"""Measured cases of the paged-cache operators: kda_kv_append, kda_kv_read and kda_kv_attend.

They are what a full-attention layer of a hybrid model runs beside the KDA layer step: the queries and keys are normalised
per head and rotated, keys and values go to the pages of the cache (as they are, or as e4m3 with a power-of-two scale per
token and head), and the newest tokens of every sequence attend to the cache.  Head counts, batch sizes, draft lengths and
prompt lengths are those of this repository's workloads (64 heads of 128 channels, batches of 1 and 64, 8 drafts, prompts of
1K to 64K tokens); 8 cache heads, the smaller heads and the page sizes are generic.

With ``own`` false, run() computes the plain form with elementary torch operations in 32 bits; with ``own`` true it makes the
library's calls."""

import math

import torch

own = False

BF16, F32 = "bf16", "f32"
E4M3_MAX = 448.0


# ---- cases ------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # the newest token of one conversation: latency
        dict(name="append_decode_1", op="append", act=BF16, kv="act", heads=64, kv_heads=8, dim=128, page=64, n=1, new_lo=1,
             new_hi=1, ctx_lo=4096, ctx_hi=4096, rot=128, inter=False, norm=True, pad=0),
        # one decode step of a full batch into a quantised cache, and those tokens read back
        dict(name="append_read_decode_64_e4m3", op="append_read", act=BF16, kv="e4m3", heads=64, kv_heads=8, dim=128, page=64,
             n=64, new_lo=1, new_hi=1, ctx_lo=1024, ctx_hi=65536, rot=128, inter=False, norm=True, pad=0),
        # a prompt of eight ragged sequences, rotated in part, rows inside a wider projection
        dict(name="append_prefill_8_bf16", op="append", act=BF16, kv="act", heads=64, kv_heads=8, dim=128, page=64, n=8,
             new_lo=511, new_hi=2049, ctx_lo=0, ctx_hi=1000, rot=64, inter=True, norm=True, pad=64),
        # a whole long prompt written in e4m3 and read back, as when a request moves to another replica
        dict(name="append_read_32768_e4m3", op="append_read", act=BF16, kv="e4m3", heads=64, kv_heads=8, dim=128, page=64, n=1,
             new_lo=32768, new_hi=32768, ctx_lo=0, ctx_hi=0, rot=128, inter=False, norm=True, pad=0),
        # 32-bit activations, small heads, no norm
        dict(name="append_f32_d32", op="append", act=F32, kv="act", heads=12, kv_heads=4, dim=32, page=16, n=5, new_lo=100,
             new_hi=333, ctx_lo=0, ctx_hi=77, rot=32, inter=False, norm=False, pad=4),
        # one conversation's decode: a short cache (latency) and the longest prompt, quantised
        dict(name="attend_decode_1_1k", op="attend", act=BF16, kv="act", heads=64, kv_heads=8, dim=128, page=64, n=1, new_lo=1,
             new_hi=1, ctx_lo=1023, ctx_hi=1023),
        dict(name="attend_decode_1_64k_e4m3", op="attend", act=BF16, kv="e4m3", heads=64, kv_heads=8, dim=128, page=64, n=1,
             new_lo=1, new_hi=1, ctx_lo=65535, ctx_hi=65535),
        # a full batch's decode step over ragged caches
        dict(name="attend_decode_64_ragged", op="attend", act=BF16, kv="act", heads=64, kv_heads=8, dim=128, page=64, n=64,
             new_lo=1, new_hi=1, ctx_lo=4001, ctx_hi=16384),
        # speculative verify of 8 drafts each, quantised cache
        dict(name="attend_verify_64_t8_e4m3", op="attend", act=BF16, kv="e4m3", heads=64, kv_heads=8, dim=128, page=64, n=64,
             new_lo=8, new_hi=8, ctx_lo=1000, ctx_hi=8192),
        # a chunk of a prompt behind a long context, and a whole prompt at once
        dict(name="attend_chunk_512_32k", op="attend", act=BF16, kv="act", heads=64, kv_heads=8, dim=128, page=64, n=1,
             new_lo=512, new_hi=512, ctx_lo=32256, ctx_hi=32256),
        dict(name="attend_prefill_8192", op="attend", act=BF16, kv="act", heads=64, kv_heads=8, dim=128, page=64, n=1,
             new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0),
        # 32-bit activations: ragged prompts of a small model, short pages
        dict(name="attend_prefill_f32_d64", op="attend", act=F32, kv="act", heads=12, kv_heads=4, dim=64, page=16, n=3,
             new_lo=777, new_hi=1500, ctx_lo=0, ctx_hi=300),
    ]


def _log(rng, lo, hi):
    return int(math.floor(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    while True:
        op = rng.choice(["append", "append_read", "attend", "attend", "attend"])
        # quantised pages are compared as the values read back
        kv = "act" if op == "append" else rng.choice(["act", "e4m3"])
        act = rng.choice([BF16, BF16, BF16, F32])
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        c = dict(op=op, act=act, kv=kv, heads=kv_heads * group, kv_heads=kv_heads,
                 dim=rng.choice([16, 32, 64, 64, 128, 128, 128]), page=rng.choice([16, 32, 64, 128]))
        step = rng.choice(["decode", "verify", "chunk", "chunk"])
        if step == "decode":
            c["n"], c["new_lo"], c["new_hi"] = _log(rng, 1, 128), 1, 1
        elif step == "verify":
            c["n"], c["new_lo"], c["new_hi"] = _log(rng, 1, 64), rng.randint(1, 4), rng.randint(4, 16)
        else:
            c["n"], c["new_hi"] = _log(rng, 1, 8), _log(rng, 17, 8192)
            c["new_lo"] = max(1, int(c["new_hi"] * rng.uniform(0.5, 1.0)))
        c["ctx_hi"] = _log(rng, 1, 65536) - 1
        c["ctx_lo"] = int(c["ctx_hi"] * rng.uniform(0.4, 1.0))
        if op != "attend":
            c["rot"] = rng.choice([0, c["dim"] // 2, c["dim"], c["dim"]])
            c["inter"] = rng.random() < 0.5
            c["norm"] = rng.random() < 0.8
            c["pad"] = rng.choice([0, 8, 64])
        new, total = _lengths(c)
        w = work(c)
        scores = c["n"] * c["heads"] * max(new) * max(total)
        if w["bytes"] > 2e9 or sum(total) * c["kv_heads"] * c["dim"] > 1e9:
            continue
        if op == "attend" and (w["flops"] > 1e12 or (act == F32 and w["flops"] > 1e11) or scores > 4.2e9):
            continue
        return c


def _spread(lo, hi, n, turn):
    """n whole numbers spread over [lo, hi] by the golden ratio; the same for every seed."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + turn) % 1.0)) for i in range(n)]


def _lengths(c):
    new = _spread(c["new_lo"], c["new_hi"], c["n"], 0.25)
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["n"], 0.5)
    return new, [a + b for a, b in zip(new, ctx)]


def work(c):
    new, total = _lengths(c)
    rows, act, kv = sum(new), 4 if c["act"] == F32 else 2, (4 if c["act"] == F32 else 2) if c["kv"] == "act" else 1
    vec = 1 if c["kv"] == "e4m3" else 0  # a scale's byte
    hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "attend":
        pairs = sum(t * (n - t) + t * (t + 1) // 2 for t, n in zip(new, total))
        return {"bytes": 2 * sum(total) * hk * (d * kv + vec) + 2 * rows * hq * d * act, "flops": 4 * d * hq * pairs}
    b = rows * (hq + 2 * hk) * d * act + rows * hq * d * act + 2 * rows * hk * (d * kv + vec)
    if c["op"] == "append_read":  # the cache's part is written once; what is read back goes out once
        b += 2 * rows * hk * d * act
    return {"bytes": b, "flops": 10 * rows * (hq + hk) * d}


# ---- inputs -----------------------------------------------------------------------------------------------------------

def _act(c):
    return torch.float32 if c["act"] == F32 else torch.bfloat16


def _quantise(x):
    """fp32 vectors (last axis) -> e4m3 values and biased scale exponents: the smallest power of two that brings the
    largest magnitude to at most 448."""
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m > 0, (e - 9 + (m > 0.875).to(e.dtype) + 127).clamp(1, 254), torch.zeros_like(e))
    y = x * torch.exp2((127 - e).to(torch.float32)).unsqueeze(-1)
    return y.to(torch.float8_e4m3fn), e.to(torch.uint8)


def _pages(c, num_pages, gen, dev):
    """A cache in use: keys and values near N(0, 1)."""
    shape = (num_pages, c["kv_heads"], c["page"], c["dim"])
    made = []
    for _ in range(2):
        if c["kv"] == "act":
            made.append((torch.randn(shape, generator=gen, device=dev, dtype=_act(c)), None))
            continue
        x = torch.empty(shape, device=dev, dtype=torch.float8_e4m3fn)
        e = torch.empty(shape[:3], device=dev, dtype=torch.uint8)
        for i in range(0, num_pages, 4096):
            part = torch.randn((min(4096, num_pages - i),) + shape[1:], generator=gen, device=dev)
            x[i:i + 4096], e[i:i + 4096] = _quantise(part)
        made.append((x, e))
    return made


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    new, total = _lengths(c)
    n, rows = c["n"], sum(new)
    act, hq, hk, d = _act(c), c["heads"], c["kv_heads"], c["dim"]
    per_seq = [-(-t // c["page"]) for t in total]
    num_pages, width = sum(per_seq) + 3, max(per_seq)
    perm = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    start = torch.tensor([sum(per_seq[:i]) for i in range(n)], device=dev)
    table = perm[(start[:, None] + torch.arange(width, device=dev)).clamp(max=num_pages - 1)].contiguous()
    s = {"case": c, "max_new": max(new), "max_total": max(total), "table": table,
         "cu": torch.tensor([sum(new[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev),
         "lens": torch.tensor(total, dtype=torch.int32, device=dev), "rows": rows}
    if c["op"] == "attend":
        (s["k"], s["ke"]), (s["v"], s["ve"]) = _pages(c, num_pages, gen, dev)
        s["q"] = torch.randn((rows, hq, d), generator=gen, device=dev, dtype=act)
        s["out"] = torch.empty_like(s["q"])
    else:
        # q, k and v are slices of one projection's rows; pad: columns of the projection that are something else
        row = torch.randn((rows, (hq + 2 * hk) * d + c["pad"]), generator=gen, device=dev).to(act)
        s["proj"] = row
        s["xq"] = row[:, :hq * d].unflatten(1, (hq, d))
        s["xk"] = row[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["xv"] = row[:, (hq + hk) * d:(hq + 2 * hk) * d].unflatten(1, (hk, d))
        s["wq"], s["wk"] = ((1 + 0.1 * torch.randn((2, d), generator=gen, device=dev)).to(act) if c["norm"] else (None, None))
        s["inv_freq"] = [10000.0 ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)]
        s["freq"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device=dev)
        kv = act if c["kv"] == "act" else torch.float8_e4m3fn
        s["k"] = torch.zeros((num_pages, hk, c["page"], d), device=dev).to(kv)
        s["v"] = torch.zeros((num_pages, hk, c["page"], d), device=dev).to(kv)
        s["ke"], s["ve"] = (torch.zeros((2, num_pages, hk, c["page"]), dtype=torch.uint8, device=dev)
                            if c["kv"] == "e4m3" else (None, None))
        s["q_out"] = torch.empty((rows, hq, d), dtype=act, device=dev)
        if c["op"] == "append_read":
            s["k_out"], s["v_out"] = torch.empty((2, rows, hk, d), dtype=act, device=dev)
    if own:  # what a program keeps: the cache, the batch's tables and the argument records
        from hybrid_linear_attention_03_gb300 import kda

        s["cache"] = kda.PagedKV(num_pages, c["page"], hq, hk, d, act, kv_format=c["kv"], k=s["k"], v=s["v"],
                                 k_scale=s["ke"], v_scale=s["ve"])
        s["batch"] = kda.make_kv_batch(s["cu"], s["lens"], table, max_rows=rows, max_new=max(new))
        if c["op"] == "attend":
            s["io"] = kda.make_attn_io(s["q"], s["out"])
            s["ws"] = torch.empty(kda.kda_kv_attend_workspace_bytes(s["cache"], s["batch"]), dtype=torch.uint8, device=dev)
        else:
            s["qk"] = kda.make_qk_params(s["wq"], s["wk"], eps=1e-5, inv_freq=s["inv_freq"], interleaved=c["inter"])
            s["io"] = kda.make_kv_io(s["xq"], s["xk"], s["xv"], s["q_out"])
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return _attend(s) if s["case"]["op"] == "attend" else _append(s)


def _run_own(s):
    from hybrid_linear_attention_03_gb300 import kda

    op = s["case"]["op"]
    if op == "attend":
        kda.kda_kv_attend(s["cache"], s["io"], s["batch"], s["ws"])
        return {"out": s["out"]}
    kda.kda_kv_append(s["cache"], s["qk"], s["io"], s["batch"])
    if op == "append":
        return {"q": s["q_out"], "k_pages": s["k"], "v_pages": s["v"]}
    kda.kda_kv_read(s["cache"], s["batch"], s["k_out"], s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _rows(s):
    """Per row: its sequence and position."""
    r = torch.arange(s["rows"], device=s["cu"].device)
    n = torch.searchsorted(s["cu"], r, right=True, out_int32=True).long() - 1
    return n, s["lens"][n] - s["cu"][n + 1] + r


def _norm_rotate(x, w, pos, s):
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w.float()
    rot = c["rot"]
    if rot:
        ang = pos.double()[:, None] * s["freq"]  # 64 bits: a far position times a frequency
        cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        ra, rb = a * cos - b * sin, a * sin + b * cos
        turned = torch.stack((ra, rb), -1).flatten(-2) if c["inter"] else torch.cat((ra, rb), -1)
        x = torch.cat((turned, x[..., rot:]), -1)
    return x


def _append(s):
    c = s["case"]
    n, pos = _rows(s)
    q = _norm_rotate(s["xq"], s["wq"], pos, s).to(_act(c))
    k, v = _norm_rotate(s["xk"], s["wk"], pos, s), s["xv"].float()
    page, line = s["table"][n, pos // c["page"]].long(), pos % c["page"]
    if c["kv"] == "act":
        s["k"][page, :, line], s["v"][page, :, line] = k.to(_act(c)), v.to(_act(c))
    else:
        for pages, scales, x in ((s["k"], s["ke"], k), (s["v"], s["ve"], v)):
            y, e = _quantise(x)
            pages.view(torch.uint8)[page, :, line], scales[page, :, line] = y.view(torch.uint8), e
    if c["op"] == "append":
        return {"q": q, "k_pages": s["k"], "v_pages": s["v"]}
    k, v = _stored(s, "k", page, line), _stored(s, "v", page, line)
    return {"q": q, "k": k.to(_act(c)), "v": v.to(_act(c))}


def _stored(s, which, page, line):
    """The cached vectors [..., kv_heads, dim] at these pages and lines, in 32 bits."""
    x = s[which]
    if s["case"]["kv"] == "act":
        return x[page, :, line].float()
    y = x.view(torch.uint8)[page, :, line].view(torch.float8_e4m3fn).float()
    return y * torch.exp2(s[which + "e"][page, :, line].float() - 127.0).unsqueeze(-1)


def _attend(s):
    """Padded to the longest sequence and the longest chunk of new tokens."""
    c = s["case"]
    hk, d, g = c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    n, dev = c["n"], s["q"].device
    j = torch.arange(s["max_total"], device=dev)
    page, line = s["table"][:, j // c["page"]].long(), (j % c["page"]).expand(n, -1)
    k, v = _stored(s, "k", page, line).permute(0, 2, 3, 1), _stored(s, "v", page, line).permute(0, 2, 1, 3)
    new = s["cu"][1:] - s["cu"][:-1]
    t = torch.arange(s["max_new"], device=dev)
    at = (s["cu"][:-1, None] + t).clamp(max=s["rows"] - 1)
    q = s["q"][at].float() * (1.0 / math.sqrt(d))  # [n, t, heads, d]
    q = q.view(n, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    p = torch.matmul(q, k).view(n, hk, g, s["max_new"], -1)
    seen = j <= (s["lens"] - new)[:, None, None] + t[:, None]  # [n, t, j]
    keep = (j < s["lens"][:, None])[:, None, :, None]
    p.masked_fill_(~seen[:, None, None], float("-inf"))
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    o = torch.matmul(p.view(n, hk, -1, s["max_total"]), v.masked_fill(~keep, 0.0))
    o = o.view(n, hk, g, s["max_new"], d).permute(0, 3, 1, 2, 4).reshape(n, s["max_new"], c["heads"], d)
    return {"out": o[t < new[:, None]].to(_act(c))}


# ---- the definition in 64 bits ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c, dev = case, "cuda"
    new, total = _lengths(c)
    hq, hk, d, ps = c["heads"], c["kv_heads"], c["dim"], c["page"]
    if c["op"] == "attend":
        out = torch.zeros((s["rows"], hq, d), dtype=torch.float64, device=dev)
        row = 0
        for i in range(c["n"]):
            pages = s["table"][i, :-(-total[i] // ps)].long()
            for h in range(hk):
                kv = []
                for pool, exps in ((s["k"], s["ke"]), (s["v"], s["ve"])):
                    x = pool[:, h][pages] if c["kv"] == "act" else pool.view(torch.uint8)[:, h][pages].view(pool.dtype)
                    x = x.double() if c["kv"] == "act" else x.float().double()
                    if exps is not None:
                        x = x * (2.0 ** (exps[:, h][pages].double() - 127)).unsqueeze(-1)
                    kv.append(x.reshape(-1, d)[:total[i]])
                for t0 in range(0, new[i], 1024):
                    t1 = min(new[i], t0 + 1024)
                    last = total[i] - new[i] + t1  # keys that the last of these rows sees
                    q = s["q"][row + t0:row + t1, h * (hq // hk):(h + 1) * (hq // hk)].double()
                    z = torch.einsum("tgd,jd->tgj", q, kv[0][:last]) / math.sqrt(d)
                    own_pos = torch.arange(last - (t1 - t0), last, device=dev)
                    z[(torch.arange(last, device=dev)[None] > own_pos[:, None])[:, None].expand_as(z)] = -math.inf
                    out[row + t0:row + t1, h * (hq // hk):(h + 1) * (hq // hk)] = torch.einsum(
                        "tgj,jd->tgd", torch.softmax(z, -1), kv[1][:last])
            row += new[i]
        return {"out": out}
    seqs = [i for i in range(c["n"]) for _ in range(new[i])]
    pos = [total[i] - new[i] + t for i in range(c["n"]) for t in range(new[i])]
    P = torch.tensor(pos, dtype=torch.float64, device=dev)
    turned = []
    for x, w in ((s["xq"], s["wq"]), (s["xk"], s["wk"])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + 1e-5) * w.double()
        y = y.clone()
        for f in range(c["rot"] // 2):
            a, b = (2 * f, 2 * f + 1) if c["inter"] else (f, f + c["rot"] // 2)
            z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(P), P * s["inv_freq"][f])[:, None]
            y[..., a], y[..., b] = z.real, z.imag
        turned.append(y)
    q, k, v = turned[0], turned[1], s["xv"].double()
    page = torch.tensor([int(x) for x in s["table"].cpu()[seqs, [p // ps for p in pos]]], device=dev)
    line = torch.tensor([p % ps for p in pos], device=dev)
    if c["kv"] == "act":
        pools = torch.zeros((2,) + tuple(s["k"].shape), dtype=torch.float64, device=dev)
        pools[0][page, :, line], pools[1][page, :, line] = k, v
        if c["op"] == "append":
            return {"q": q, "k_pages": pools[0], "v_pages": pools[1]}
        return {"q": q, "k": k, "v": v}
    held = []
    for x in (k, v):
        e = torch.ceil(torch.log2((x.abs().amax(-1) / E4M3_MAX).clamp(min=1e-300)))
        unit = (2.0 ** e).unsqueeze(-1)
        held.append((x / unit).float().to(torch.float8_e4m3fn).double() * unit)
    return {"q": q, "k": held[0], "v": held[1]}
