"""Measured cases of the latent-attention operators: kda_latent_append, kda_latent_read, kda_latent_attend, kda_latent_prefill.

They are what a latent-attention layer of a hybrid model runs beside the KDA layer step.  A token leaves one latent vector c,
normalised, and one key part kr, rotated, that all heads share.  Its attention has two forms: absorbed, over the pages of the
cache, with queries already in the latent space (decode, drafts, short chunks), and expanded, over keys and values per head
that a product made from the latents (prompts).  Head counts, batch sizes, draft lengths and prompt lengths are those of this
repository's workloads (64 heads of 128 channels, batches of 1 and 64, 8 drafts, prompts of 1K to 64K tokens); a latent of 512
channels with a shared key part of 64, the smaller sizes and the page sizes are generic.

With ``own`` false, run() computes the plain form with elementary torch operations in 32 bits (64 where a value goes to 8 bits);
with ``own`` true it makes the library's calls."""

import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-5
E4M3_MAX = 448.0


# ---- cases ------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # the newest token of one conversation: latency
        dict(name="append_decode_1", op="append", act=BF16, kv="act", heads=64, latent=512, rope=64, page=64, n=1, new_lo=1,
             new_hi=1, ctx_lo=4096, ctx_hi=4096, rot=64, inter=False, norm=True, pad=0),
        # a prompt of eight ragged sequences behind cached prefixes, rows inside a wider projection, and those tokens read back
        dict(name="append_read_8_ragged", op="append_read", act=BF16, kv="act", heads=64, latent=512, rope=64, page=64, n=8,
             new_lo=511, new_hi=2049, ctx_lo=0, ctx_hi=1000, rot=64, inter=True, norm=True, pad=64),
        # a whole long prompt written in e4m3 and read back, as for the expanded form or a move to another replica
        dict(name="append_read_32768_e4m3", op="append_read", act=BF16, kv="e4m3", heads=64, latent=512, rope=64, page=64, n=1,
             new_lo=32768, new_hi=32768, ctx_lo=0, ctx_hi=0, rot=64, inter=False, norm=True, pad=0),
        # one conversation's decode: a short cache (latency) and the longest prompt, quantised
        dict(name="attend_decode_1_4k", op="attend", act=BF16, kv="act", heads=64, latent=512, rope=64, page=64, n=1, new_lo=1,
             new_hi=1, ctx_lo=4095, ctx_hi=4095),
        dict(name="attend_decode_1_64k_e4m3", op="attend", act=BF16, kv="e4m3", heads=64, latent=512, rope=64, page=64, n=1,
             new_lo=1, new_hi=1, ctx_lo=65535, ctx_hi=65535),
        # a full batch's decode step over ragged caches
        dict(name="attend_decode_64_ragged", op="attend", act=BF16, kv="act", heads=64, latent=512, rope=64, page=64, n=64,
             new_lo=1, new_hi=1, ctx_lo=4001, ctx_hi=16384),
        # speculative verify of 8 drafts each, quantised cache
        dict(name="attend_verify_64_t8_e4m3", op="attend", act=BF16, kv="e4m3", heads=64, latent=512, rope=64, page=64, n=64,
             new_lo=8, new_hi=8, ctx_lo=1000, ctx_hi=8192),
        # 32-bit activations of a small model, short pages, a few tokens each
        dict(name="attend_f32_small", op="attend", act=F32, kv="act", heads=12, latent=128, rope=32, page=16, n=5, new_lo=3,
             new_hi=40, ctx_lo=50, ctx_hi=777),
        # a whole prompt, eight ragged ones behind prefixes, and a chunk behind a long context
        dict(name="prefill_8192", op="prefill", act=BF16, heads=64, nope=128, rope=64, value=128, n=1, new_lo=8192, new_hi=8192,
             ctx_lo=0, ctx_hi=0),
        dict(name="prefill_8_ragged", op="prefill", act=BF16, heads=64, nope=128, rope=64, value=128, n=8, new_lo=511,
             new_hi=2049, ctx_lo=0, ctx_hi=1000),
        dict(name="prefill_chunk_512_32k", op="prefill", act=BF16, heads=64, nope=128, rope=64, value=128, n=1, new_lo=512,
             new_hi=512, ctx_lo=32256, ctx_hi=32256),
        # 32-bit activations: ragged prompts of a small model
        dict(name="prefill_f32_small", op="prefill", act=F32, heads=12, nope=64, rope=32, value=64, n=3, new_lo=300,
             new_hi=700, ctx_lo=0, ctx_hi=100),
    ]


def _log(rng, lo, hi):
    return int(math.floor(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    while True:
        op = rng.choice(["append", "append_read", "attend", "attend", "attend", "prefill", "prefill"])
        act = rng.choice([BF16, BF16, BF16, F32])
        c = dict(op=op, act=act, heads=rng.choice([1, 3, 8, 12, 16, 16, 32, 64, 64, 128]), rope=rng.choice([16, 32, 64, 64, 64]))
        step = "chunk" if op == "prefill" else rng.choice(["decode", "decode", "verify", "chunk"])
        if step == "decode":
            c["n"], c["new_lo"], c["new_hi"] = _log(rng, 1, 128), 1, 1
        elif step == "verify":
            c["n"], c["new_lo"], c["new_hi"] = _log(rng, 1, 64), rng.randint(1, 4), rng.randint(4, 16)
        else:
            c["n"], c["new_hi"] = _log(rng, 1, 8), _log(rng, 17, 1024 if op == "attend" else 8192)
            c["new_lo"] = max(1, int(c["new_hi"] * rng.uniform(0.5, 1.0)))
        c["ctx_hi"] = _log(rng, 1, 65536) - 1
        c["ctx_lo"] = int(c["ctx_hi"] * rng.uniform(0.4, 1.0))
        if op == "prefill":
            c["nope"], c["value"] = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
        else:
            # quantised pages are compared as the values read back
            c["kv"] = "act" if op == "append" else rng.choice(["act", "e4m3"])
            c["latent"], c["page"] = rng.choice([128, 256, 512, 512, 512]), rng.choice([16, 32, 64, 128])
        if op in ("append", "append_read"):
            c["rot"] = rng.choice([0, c["rope"] // 2, c["rope"], c["rope"]])
            c["inter"] = rng.random() < 0.5
            c["norm"] = rng.random() < 0.8
            c["pad"] = rng.choice([0, 8, 64])
        new, total = _lengths(c)
        w = work(c)
        scores = c["n"] * c["heads"] * max(new) * max(total)
        if w["bytes"] > 1.5e9 or sum(total) * 576 > 1e9:
            continue
        if op in ("attend", "prefill") and (w["flops"] > 1.2e12 or (act == F32 and w["flops"] > 5e10) or scores > 4.2e9):
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
    rows, act, h, r = sum(new), 4 if c["act"] == F32 else 2, c["heads"], c["rope"]
    pairs = sum(t * (n - t) + t * (t + 1) // 2 for t, n in zip(new, total))
    if c["op"] == "prefill":
        dq, dv = c["nope"] + r, c["value"]
        return {"bytes": act * (rows * h * (dq + dv) + sum(total) * (h * (c["nope"] + dv) + r)), "flops": 2 * h * pairs * (dq + dv)}
    latent = c["latent"]
    line = (latent + 1 if c["kv"] == "e4m3" else latent * act) + r * act
    if c["op"] == "attend":
        return {"bytes": sum(total) * line + rows * h * (2 * latent + r) * act, "flops": 2 * h * pairs * (2 * latent + r)}
    b = rows * ((latent + r + 2 * h * r) * act + line)
    if c["op"] == "append_read":  # the cache's part is written once; what is read back goes out once
        b += rows * (latent + r) * act
    return {"bytes": b, "flops": 10 * rows * (latent + r + h * r)}


# ---- inputs -----------------------------------------------------------------------------------------------------------

def _act(c):
    return torch.float32 if c["act"] == F32 else torch.bfloat16


def _quantise(x):
    """Vectors (last axis) in 32 or 64 bits -> e4m3 values and biased scale exponents: the smallest power of two that brings
    the largest magnitude to at most 448."""
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m > 0, (e - 9 + (m > 0.875).to(e.dtype) + 127).clamp(1, 254), torch.zeros_like(e))
    y = x * torch.exp2((127 - e).to(x.dtype)).unsqueeze(-1)
    return y.to(torch.float8_e4m3fn), e.to(torch.uint8)


def _scale(c):
    """Of the scores: heads of 128 channels beside the shared part, whatever the latent's size."""
    return (c.get("nope", 128) + c["rope"]) ** -0.5


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    new, total = _lengths(c)
    n, rows, act, h, r = c["n"], sum(new), _act(c), c["heads"], c["rope"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=act)

    s = {"case": c, "rows": rows, "max_new": max(new), "max_total": max(total), "new": new, "total": total,
         "cu": torch.tensor([sum(new[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev),
         "lens": torch.tensor(total, dtype=torch.int32, device=dev)}
    if c["op"] == "prefill":
        dn, dv = c["nope"], c["value"]
        s["cu_kv"] = torch.tensor([sum(total[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev)
        q, kv = normal(rows, h, dn + r), normal(sum(total), h, dn + dv)  # one projection each
        s["qn"], s["qr"], s["k"], s["v"] = q[..., :dn], q[..., dn:], kv[..., :dn], kv[..., dn:]
        s["kr"] = normal(sum(total), r)
        s["out"] = torch.empty((rows, h, dv), dtype=act, device=dev)
        if own:
            from hybrid_linear_attention_03_gb300 import kda

            s["cache"] = kda.PagedLatent(1, 16, h, 128, r, act)  # the layer's cache, whose pages this form does not read
            s["batch"] = kda.make_latent_prefill_batch(s["cu"], s["cu_kv"], max_rows=rows, max_kv_rows=sum(total),
                                                       max_new=max(new))
            s["io"] = kda.make_latent_prefill_io(s["qn"], s["qr"], s["k"], s["kr"], s["v"], s["out"], _scale(c))
            s["ws"] = torch.empty(kda.kda_latent_prefill_workspace_bytes(s["cache"], s["io"], s["batch"]), dtype=torch.uint8,
                                  device=dev)
        return s

    latent, ps = c["latent"], c["page"]
    per_seq = [-(-t // ps) for t in total]
    num_pages, width = sum(per_seq) + 3, max(per_seq)
    perm = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    start = torch.tensor([sum(per_seq[:i]) for i in range(n)], device=dev)
    s["table"] = perm[(start[:, None] + torch.arange(width, device=dev)).clamp(max=num_pages - 1)].contiguous()
    if c["op"] == "attend":  # a cache in use: normalised latents and key parts near N(0, 1)
        s["c"], s["ce"] = normal(num_pages, ps, latent), None
        if c["kv"] == "e4m3":
            s["c"], s["ce"] = _quantise(s["c"].float())
        s["kr"] = normal(num_pages, ps, r)
        s["qc"], s["qr"] = normal(rows, h, latent), normal(rows, h, r)
        s["out"] = torch.empty((rows, h, latent), dtype=act, device=dev)
    else:
        # c and kr are slices of one projection's rows, q_r of the queries'; pad: columns that are something else
        row = normal(rows, latent + r + c["pad"])
        s["xc"], s["xk"] = row[:, :latent], row[:, latent:latent + r]
        s["xq"] = normal(rows, h, 128 + r)[..., 128:]
        s["w"] = (1 + 0.1 * torch.randn(latent, generator=gen, device=dev)).to(act) if c["norm"] else None
        s["inv_freq"] = [10000.0 ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)]
        s["freq"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device=dev)
        s["c"] = torch.zeros((num_pages, ps, latent), device=dev).to(torch.float8_e4m3fn if c["kv"] == "e4m3" else act)
        s["ce"] = torch.zeros((num_pages, ps), dtype=torch.uint8, device=dev) if c["kv"] == "e4m3" else None
        s["kr"] = torch.zeros((num_pages, ps, r), dtype=act, device=dev)
        s["q_out"] = torch.empty((rows, h, r), dtype=act, device=dev)
        if c["op"] == "append_read":
            s["c_out"] = torch.empty((rows, latent), dtype=act, device=dev)
            s["kr_out"] = torch.empty((rows, r), dtype=act, device=dev)
    if own:  # what a program keeps: the cache, the batch's tables and the argument records
        from hybrid_linear_attention_03_gb300 import kda

        s["cache"] = kda.PagedLatent(num_pages, ps, h, latent, r, act, kv_format=c["kv"], c=s["c"], kr=s["kr"],
                                     c_scale=s["ce"])
        s["batch"] = kda.make_kv_batch(s["cu"], s["lens"], s["table"], max_rows=rows, max_new=max(new))
        if c["op"] == "attend":
            s["io"] = kda.make_latent_attn_io(s["qc"], s["qr"], s["out"], _scale(c))
            s["ws"] = torch.empty(kda.kda_latent_attend_workspace_bytes(s["cache"], s["batch"]), dtype=torch.uint8, device=dev)
        else:
            s["params"] = kda.make_latent_params(s["w"], eps=EPS, inv_freq=s["inv_freq"], interleaved=c["inter"])
            s["io"] = kda.make_latent_io(s["xc"], s["xk"], s["xq"], s["q_out"])
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"prefill": _prefill, "attend": _attend}.get(s["case"]["op"], _append)(s)


def _run_own(s):
    from hybrid_linear_attention_03_gb300 import kda

    op = s["case"]["op"]
    if op == "prefill":
        kda.kda_latent_prefill(s["cache"], s["io"], s["batch"], s["ws"])
        return {"out": s["out"]}
    if op == "attend":
        kda.kda_latent_attend(s["cache"], s["io"], s["batch"], s["ws"])
        return {"out": s["out"]}
    kda.kda_latent_append(s["cache"], s["params"], s["io"], s["batch"])
    if op == "append":
        return {"q": s["q_out"], "c_pages": s["c"], "kr_pages": s["kr"]}
    kda.kda_latent_read(s["cache"], s["batch"], s["c_out"], s["kr_out"])
    return {"q": s["q_out"], "c": s["c_out"], "kr": s["kr_out"]}


def _rows(s):
    """Per row: its sequence and position."""
    r = torch.arange(s["rows"], device=s["cu"].device)
    n = torch.searchsorted(s["cu"], r, right=True, out_int32=True).long() - 1
    return n, s["lens"][n] - s["cu"][n + 1] + r


def _rotate(x, cos, sin, c):
    x, rot = x.float(), c["rot"]
    if rot == 0:
        return x
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((ra, rb), -1).flatten(-2) if c["inter"] else torch.cat((ra, rb), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _append(s):
    c = s["case"]
    n, pos = _rows(s)
    ang = pos.double()[:, None] * s["freq"]  # 64 bits: a far position times a frequency
    cos, sin = ang.cos().float(), ang.sin().float()
    q = _rotate(s["xq"], cos[:, None], sin[:, None], c).to(_act(c))
    kr = _rotate(s["xk"], cos, sin, c).to(_act(c))
    x = s["xc"].double() if c["kv"] == "e4m3" else s["xc"].float()  # 64 bits: next to a border of e4m3
    if s["w"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["w"].to(x.dtype)
    page, line = s["table"][n, pos // c["page"]].long(), pos % c["page"]
    s["kr"][page, line] = kr
    if c["kv"] == "act":
        s["c"][page, line] = x.to(_act(c))
    else:
        y, e = _quantise(x)
        s["c"].view(torch.uint8)[page, line], s["ce"][page, line] = y.view(torch.uint8), e
    if c["op"] == "append":
        return {"q": q, "c_pages": s["c"], "kr_pages": s["kr"]}
    return {"q": q, "c": _latents(s, page, line).to(_act(c)), "kr": s["kr"][page, line]}


def _latents(s, page, line):
    """The cached latents at these pages and lines, in 32 bits."""
    if s["ce"] is None:
        return s["c"][page, line].float()
    y = s["c"].view(torch.uint8)[page, line].view(torch.float8_e4m3fn).float()
    return y * torch.exp2(s["ce"][page, line].float() - 127.0).unsqueeze(-1)


def _attend(s):
    """Padded to the longest sequence and the longest run of new tokens."""
    c = s["case"]
    n, h, latent, dev = c["n"], c["heads"], c["latent"], s["cu"].device
    j = torch.arange(s["max_total"], device=dev)
    page, line = s["table"][:, j // c["page"]].long(), (j % c["page"]).expand(n, -1)
    keys = _latents(s, page, line)  # [n, j, latent]
    new = s["cu"][1:] - s["cu"][:-1]
    t = torch.arange(s["max_new"], device=dev)
    at = (s["cu"][:-1, None] + t).clamp(max=s["rows"] - 1)
    q = torch.cat((s["qc"], s["qr"]), -1)[at].float().mul_(_scale(c)).view(n, -1, latent + c["rope"])  # [n, t heads, .]
    p = torch.matmul(q, torch.cat((keys, s["kr"][page, line].float()), -1).transpose(1, 2)).view(n, s["max_new"], h, -1)
    seen = j <= (s["lens"] - new)[:, None, None] + t[:, None]  # [n, t, j]
    p.masked_fill_(~seen[:, :, None], float("-inf"))
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    keep = (j < s["lens"][:, None])[..., None]
    o = torch.matmul(p.view(n, -1, s["max_total"]), keys.masked_fill_(~keep, 0.0)).view(n, s["max_new"], h, latent)
    return {"out": o[t < new[:, None]].to(_act(c))}


def _prefill(s):
    """Sequence by sequence."""
    c = s["case"]
    dev, out, row, key = s["cu"].device, [], 0, 0
    for t, total in zip(s["new"], s["total"]):
        q = torch.cat((s["qn"][row:row + t], s["qr"][row:row + t]), -1).float().mul_(_scale(c)).transpose(0, 1)
        kr = s["kr"][key:key + total, None].float().expand(-1, c["heads"], -1)
        k = torch.cat((s["k"][key:key + total].float(), kr), -1)
        p = torch.matmul(q, k.permute(1, 2, 0))  # [heads, t, total]
        hidden = torch.arange(total, device=dev) > torch.arange(total - t, total, device=dev)[:, None]
        p.masked_fill_(hidden, float("-inf"))
        p.sub_(p.amax(-1, keepdim=True)).exp_()
        p.div_(p.sum(-1, keepdim=True))
        out.append(torch.matmul(p, s["v"][key:key + total].float().transpose(0, 1)).transpose(0, 1).to(_act(c)))
        row, key = row + t, key + total
    return {"out": torch.cat(out)}


# ---- the definition in 64 bits ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c, dev, h = case, "cuda", case["heads"]
    new, total = _lengths(c)
    f64 = torch.float64
    if c["op"] == "prefill":
        out = torch.zeros((s["rows"], h, c["value"]), dtype=f64, device=dev)
        r0 = k0 = 0
        for t, n in zip(new, total):
            for head in range(h):
                kk, vv = s["k"][k0:k0 + n, head].double(), s["v"][k0:k0 + n, head].double()
                shared = s["kr"][k0:k0 + n].double()
                for a in range(0, t, 2048):
                    b = min(t, a + 2048)
                    last = n - t + b  # keys that the last of these rows sees
                    z = s["qn"][r0 + a:r0 + b, head].double() @ kk[:last].T + s["qr"][r0 + a:r0 + b, head].double() @ shared[:last].T
                    z = z * _scale(c)
                    z = torch.where(torch.arange(last, device=dev) <= torch.arange(last - (b - a), last, device=dev)[:, None], z,
                                    torch.full((), -math.inf, dtype=f64, device=dev))
                    out[r0 + a:r0 + b, head] = torch.softmax(z, -1) @ vv[:last]
            r0, k0 = r0 + t, k0 + n
        return {"out": out}
    ps = c["page"]
    if c["op"] == "attend":
        out = torch.zeros((s["rows"], h, c["latent"]), dtype=f64, device=dev)
        r0 = 0
        for i in range(c["n"]):
            pages = s["table"][i, :-(-total[i] // ps)].long()
            if c["kv"] == "act":
                lat = s["c"][pages].double()
            else:
                lat = s["c"].view(torch.uint8)[pages].view(s["c"].dtype).float().double()
                lat = lat * (2.0 ** (s["ce"][pages].double() - 127)).unsqueeze(-1)
            lat, shared = lat.reshape(-1, c["latent"])[:total[i]], s["kr"][pages].double().reshape(-1, c["rope"])[:total[i]]
            for a in range(0, new[i], 64):
                b = min(new[i], a + 64)
                last = total[i] - new[i] + b
                z = torch.einsum("thl,jl->thj", s["qc"][r0 + a:r0 + b].double(), lat[:last])
                z += torch.einsum("thr,jr->thj", s["qr"][r0 + a:r0 + b].double(), shared[:last])
                z *= _scale(c)
                own_pos = torch.arange(last - (b - a), last, device=dev)
                z[(torch.arange(last, device=dev)[None] > own_pos[:, None])[:, None].expand_as(z)] = -math.inf
                out[r0 + a:r0 + b] = torch.einsum("thj,jl->thl", torch.softmax(z, -1), lat[:last])
            r0 += new[i]
        return {"out": out}
    seqs = [i for i in range(c["n"]) for _ in range(new[i])]
    pos = [total[i] - new[i] + t for i in range(c["n"]) for t in range(new[i])]
    P = torch.tensor(pos, dtype=f64, device=dev)
    turned = []
    for x in (s["xq"].double().clone(), s["xk"].double().clone()):
        for f in range(c["rot"] // 2):
            a, b = (2 * f, 2 * f + 1) if c["inter"] else (f, f + c["rot"] // 2)
            turn = torch.polar(torch.ones_like(P), P * s["inv_freq"][f])
            z = torch.complex(x[..., a], x[..., b]) * turn.view((-1,) + (1,) * (x.dim() - 2))
            x[..., a], x[..., b] = z.real, z.imag
        turned.append(x)
    q, kr = turned
    lat = s["xc"].double()
    if s["w"] is not None:
        lat = lat / torch.sqrt((lat * lat).sum(-1, keepdim=True) / c["latent"] + EPS) * s["w"].double()
    if c["op"] == "append_read":
        if c["kv"] == "e4m3":
            unit = (2.0 ** torch.ceil(torch.log2((lat.abs().amax(-1) / E4M3_MAX).clamp(min=1e-300)))).unsqueeze(-1)
            lat = (lat / unit).float().to(torch.float8_e4m3fn).double() * unit
        return {"q": q, "c": lat, "kr": kr}
    page = torch.tensor([int(x) for x in s["table"].cpu()[seqs, [p // ps for p in pos]]], device=dev)
    line = torch.tensor([p % ps for p in pos], device=dev)
    pools = torch.zeros(s["c"].shape, dtype=f64, device=dev), torch.zeros(s["kr"].shape, dtype=f64, device=dev)
    pools[0][page, line], pools[1][page, line] = lat, kr
    return {"q": q, "c_pages": pools[0], "kr_pages": pools[1]}
