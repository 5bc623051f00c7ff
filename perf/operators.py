"""The cache-writing and block-scaled operators, and what they are measured on.

Three passes a serving program makes over a paged KV cache:

``append``  rotate q and k at their positions and write k and v into the pages
            of the cache, stored as they are or as E4M3 with a scale per
            tensor, per kv head, per token or per block (page x kv head);
``attend``  decode attention over an E4M3 cache with one scale per block;
``step``    one after the other, as a decode step runs them.

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through this package's plans.
"""
import math
import random

import torch

own = False

PAGE = 16
E4M3 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases

def _append(name, batch, ctx, new, heads, d=128, dtype="bf16", scales="none", offset=0,
            rotary=None, interleaved=False):
    return {"name": name, "op": "append", "batch": batch, "ctx_min": ctx[0], "ctx_max": ctx[1],
            "new_min": new[0], "new_max": new[1], "hq": heads[0], "hkv": heads[1], "d": d,
            "dtype": dtype, "scales": scales, "offset": offset,
            "rotary": d if rotary is None else rotary, "interleaved": interleaved}


def _attention(name, batch, ctx, heads, d=128, dtype="bf16", drafts=1, op="attend"):
    return {"name": name, "op": op, "batch": batch, "ctx_min": ctx[0], "ctx_max": ctx[1],
            "new_min": 1, "new_max": drafts, "hq": heads[0], "hkv": heads[1], "d": d,
            "dtype": dtype, "scales": "block", "offset": 0, "rotary": d, "interleaved": False}


def listed():
    return [
        # an interactive session: a few requests, one token each; latency counts
        _append("append few", 4, (17, 255), (1, 1), (32, 8)),
        # a large serving batch, one token each, far positions behind a shared prefix
        _append("append decode", 450, (256, 2048), (1, 1), (32, 8), offset=62000),
        # short prompts of odd lengths, f16, partial interleaved rotation
        _append("append prompts f16", 24, (0, 300), (1, 700), (16, 8), d=64, dtype="f16",
                rotary=32, interleaved=True),
        # a prefill step of long prompts
        _append("append prefill", 8, (0, 1000), (2048, 6144), (32, 8)),
        # one token each into an E4M3 cache with a scale per token
        _append("append e4m3 token", 128, (1024, 2048), (1, 1), (64, 8), scales="token"),
        # one token each into a block-scaled cache: the page's scale may grow
        _append("append e4m3 block", 128, (1024, 2048), (1, 1), (64, 8), scales="block"),
        # prompts into a block-scaled cache
        _append("append e4m3 prefill", 8, (0, 500), (1024, 4096), (64, 8), scales="block"),
        # a few short requests: latency counts
        _attention("attend few", 4, (17, 700), (32, 8)),
        # the fp8_kv workload's shapes and lengths
        _attention("attend batch", 128, (1024, 8192), (64, 8)),
        # one long sequence without grouping (the long_split workload's shape)
        _attention("attend long", 1, (65536, 65536), (32, 32)),
        # verifying 1 to 4 draft tokens a request (spec_decode_ragged's shapes)
        _attention("attend drafts", 128, (1024, 4096), (64, 8), drafts=4),
        # a decode step: append into the block-scaled cache, then attend
        _attention("step", 64, (512, 4096), (32, 8), op="step"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "append", "attend", "attend", "step"])
    d = rng.choice([64, 128, 128])
    group = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    if op == "append":
        scales = rng.choice(["none", "none", "tensor", "head", "token", "block", "block"])
        dtype = rng.choice(["f32", "bf16", "f16"] if scales == "none" else ["bf16", "f16"])
        batch = _log(rng, 1, 450)
        new_max = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(6000, 40000 // batch)))
        ctx = _log(rng, 1, 2048)
        c = _append("", batch, (rng.randint(0, ctx), ctx), (rng.randint(0, new_max), new_max),
                    (hkv * group, hkv), d, dtype, scales, offset=rng.choice([0, 0, 5, 131072]),
                    rotary=rng.choice([d, d, d // 2, 48, 16, 0]), interleaved=rng.random() < 0.3)
    else:
        drafts = 1
        dtype = rng.choice(["bf16", "bf16", "f16"])
        if dtype == "bf16" and d == 128 and rng.random() < 0.4:
            drafts = rng.randint(2, 32 // group if group > 4 else 8)
        batch = _log(rng, 1, 128)
        ctx = _log(rng, 1, min(65536, 500000 // batch))
        c = _attention("", batch, (rng.randint(0, ctx), ctx), (hkv * group, hkv), d, dtype,
                       drafts, op)
    del c["name"]
    return c


def _lengths(case):
    """Per request: tokens in the cache before the pass, and new tokens.
    Fixed by the case, so that work() knows them too."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    pairs = [(r.randint(case["ctx_min"], case["ctx_max"]),
              r.randint(case["new_min"], case["new_max"])) for _ in range(case["batch"])]
    if case["op"] == "attend":
        # the query tokens' own keys are the last of the cache already; a
        # request without a context has no query token either
        pairs = [(max(c - n, 0), min(n, c)) for c, n in pairs]
        if case["new_max"] == 1:
            return [c for c, _ in pairs], [n for _, n in pairs], [1] * case["batch"]
    return [c for c, _ in pairs], [n for _, n in pairs], [n for _, n in pairs]


# ---------------------------------------------------------------- inputs

def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s; 0 for 0."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875).to(e.dtype)))
    return torch.where(amax > 0, s, torch.zeros_like(amax))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    ctx, new, rows = _lengths(case)
    B, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    qt = TYPES[case["dtype"]]
    kvt = qt if case["scales"] == "none" else E4M3
    total = torch.tensor(ctx) + torch.tensor(new)
    pages = (total + PAGE - 1) // PAGE
    indptr = torch.zeros(B + 1, dtype=torch.int64)
    indptr[1:] = pages.cumsum(0)
    last = torch.where(pages > 0, total - (pages - 1) * PAGE, torch.full_like(total, PAGE))
    num_pages = int(indptr[-1]) + 3
    host = torch.Generator().manual_seed(seed)
    ids = torch.randperm(num_pages, generator=host)[:int(indptr[-1])].to(torch.int32).to(dev)
    row_ptr = torch.zeros(B + 1, dtype=torch.int64)
    row_ptr[1:] = torch.tensor(rows).cumsum(0)
    T = int(row_ptr[-1])

    s = {"case": case, "indptr": indptr.to(torch.int32), "last": last.to(torch.int32),
         "ids": ids, "row_ptr": row_ptr.to(torch.int32), "num_pages": num_pages}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    # what a projection gives: q, k and v side by side in one row a token,
    # magnitudes that differ from token to token
    s["qkv"] = (normal(T, hq + 2 * hkv, d) * torch.exp2(normal(T, 1, 1))).to(qt)
    s["q"], s["k"], s["v"] = s["qkv"].split([hq, hkv, hkv], dim=1)
    if case["op"] == "attend":
        s["q"] = s["q"].contiguous()
    # the cache as earlier passes left it
    if kvt == E4M3:
        s["kv"] = torch.empty((num_pages, 2, PAGE, hkv, d), dtype=E4M3, device=dev)
        sc = []
        for half in range(2):
            x = normal(num_pages, PAGE, hkv, d).mul_(torch.exp2(normal(num_pages, 1, hkv, 1)))
            if case["scales"] == "token":
                a = x.abs().amax(-1) / 448
                sc.append(a.permute(0, 2, 1).contiguous())
                a = a[..., None]
            elif case["scales"] == "block":
                a = _pow2_scale(x.abs().amax((1, 3)))
                sc.append(a)
                a = a[:, None, :, None]
            else:
                a = torch.full((hkv,), 0.03125 * (1 + half), device=dev)
                a = a * (1 + torch.arange(hkv, device=dev) % 3) if case["scales"] == "head" else a
                sc.append(a)
                a = a[:, None]
            s["kv"][:, half] = x.div_(a).clamp_(-448, 448).to(E4M3)
            del x
        s["ks"], s["vs"] = sc
        if case["scales"] == "tensor":
            s["ks1"], s["vs1"] = float(sc[0][0]), float(sc[1][0])
    else:
        s["kv"] = torch.randn((num_pages, 2, PAGE, hkv, d), generator=g, device=dev, dtype=qt)
    s["qo"] = torch.empty((T, hq, d), dtype=qt, device=dev)

    # where each new token goes (device copies of the page table's arithmetic)
    req = torch.repeat_interleave(torch.arange(B), row_ptr[1:] - row_ptr[:-1])
    j = torch.arange(T) - row_ptr[req]
    pos = total[req] - torch.tensor(rows)[req] + j
    s["req"], s["j"], s["pos"] = req.to(dev), j.to(dev), pos.to(dev)
    s["entry"] = (indptr[req] + pos.clamp(min=0) // PAGE).to(dev)
    s["slot"] = (pos % PAGE).to(dev)
    s["rows"] = torch.tensor(rows).to(dev)
    s["total"] = total.to(dev)
    s["pages_of"] = pages.to(dev)
    s["first_entry"] = indptr[:-1].to(dev)
    s["max_pages"], s["max_rows"] = int(pages.max()), max(rows)
    # the pages the new tokens touch, in order, and how full each was before
    if case["op"] != "attend":
        ent = indptr[req] + pos // PAGE
        s["touched"], s["unit"] = (x.to(dev) for x in torch.unique(ent, return_inverse=True))
        before = torch.full((len(s["touched"]),), PAGE, dtype=torch.int64)
        before.scatter_reduce_(0, s["unit"].cpu(), pos % PAGE, "amin")
        s["before"] = before.to(dev)
    s["inv_freq"] = 10000.0 ** (-2.0 * torch.arange(case["rotary"] // 2, dtype=torch.float64)
                                / max(case["rotary"], 1))
    if own:
        _plans(s, qt, kvt)
    s["inv_freq"] = s["inv_freq"].to(dev)
    return s


def _plans(s, qt, kvt):
    import paged_kv_decode_fa_gb300 as fa
    c = s["case"]
    shape = (c["hq"], c["hkv"], c["d"], PAGE)
    if c["op"] != "attend":
        rotary = None
        if c["rotary"]:
            rotary = fa.RotaryTable(c["rotary"], inv_freq=s["inv_freq"],
                                    interleaved=c["interleaved"])
        s["append"] = fa.plan_append(s["indptr"], s["ids"], s["last"], s["row_ptr"], *shape,
                                     q_data_type=qt, kv_data_type=kvt, rotary=rotary,
                                     position_offset=[c["offset"]] * c["batch"])
    if c["op"] != "append":
        if c["new_max"] == 1:
            s["decode"] = fa.plan(s["indptr"], s["ids"], s["last"], *shape, q_data_type=qt,
                                  kv_data_type=kvt)
        else:
            s["decode"] = fa.plan_ragged_q(s["indptr"], s["ids"], s["last"], s["row_ptr"],
                                           *shape, q_data_type=qt, kv_data_type=kvt)


# ---------------------------------------------------------------- the passes

def run(s):
    op = s["case"]["op"]
    if op == "append":
        return _append_own(s) if own else _append_plain(s)
    if op == "attend":
        return _attend_own(s, s["q"]) if own else _attend_plain(s, s["q"])
    out = _append_own(s) if own else _append_plain(s)
    out.update(_attend_own(s, out["q"]) if own else _attend_plain(s, out["q"]))
    return out


def _append_own(s):
    p, scales = s["append"], s["case"]["scales"]
    kw = {"q": s["q"], "q_out": s["qo"]}
    if scales == "none":
        q = p.run(s["k"], s["v"], s["kv"], **kw)
    elif scales == "tensor":
        q = p.run(s["k"], s["v"], s["kv"], k_scale=s["ks1"], v_scale=s["vs1"], **kw)
    elif scales == "head":
        q = p.run_head_scales(s["k"], s["v"], s["kv"], s["ks"], s["vs"], **kw)
    elif scales == "token":
        q = p.run_token_scales(s["k"], s["v"], s["kv"], s["ks"], s["vs"], **kw)
    else:
        q = p.run_block_scales(s["k"], s["v"], s["kv"], s["ks"], s["vs"], **kw)
    return _append_out(s, q)


def _append_out(s, q):
    out = {"q": q, "kv": s["kv"]}
    if s["case"]["scales"] in ("token", "block"):
        out["ks"], out["vs"] = s["ks"], s["vs"]
    return out


def _attend_own(s, q):
    o, lse = s["decode"].run_block_scales(q, s["kv"], s["ks"], s["vs"])
    return {"o": o, "lse": lse}


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] float, cos / sin [T, 1, rotary / 2]."""
    n = cos.shape[-1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = a * cos - b * sin, b * cos + a * sin
    return y


def _codes(x, inv):
    """E4M3 codes of x * inv: finite values saturate, others become NaN."""
    y = (x * inv).clamp(-448, 448)
    return torch.where(x.isfinite(), y, torch.full_like(y, math.nan)).to(E4M3)


def _inverse(scale):
    return torch.where(scale > 0, 1 / scale, torch.zeros_like(scale))


def _amax(x, dims):
    return torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(dims)


def _append_plain(s):
    c = s["case"]
    kv, scales = s["kv"], c["scales"]
    angle = (s["pos"] + c["offset"]).double()[:, None, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    s["qo"].copy_(_rotate(s["q"].float(), cos, sin, c["interleaved"]))
    k, v = _rotate(s["k"].float(), cos, sin, c["interleaved"]), s["v"].float()
    page = s["ids"][s["entry"]].long() if len(s["entry"]) else s["entry"]
    raw = kv.view(torch.uint8) if kv.dtype == E4M3 else kv
    if scales == "none":
        raw[page, 0, s["slot"]] = k.to(kv.dtype)
        raw[page, 1, s["slot"]] = v.to(kv.dtype)
    elif scales in ("tensor", "head"):
        raw[page, 0, s["slot"]] = _codes(k, 1 / s["ks"][:, None]).view(torch.uint8)
        raw[page, 1, s["slot"]] = _codes(v, 1 / s["vs"][:, None]).view(torch.uint8)
    elif scales == "token":
        ka, va = _amax(k, -1), _amax(v, -1)
        s["ks"][page, :, s["slot"]], s["vs"][page, :, s["slot"]] = ka / 448, va / 448
        raw[page, 0, s["slot"]] = _codes(k, _inverse(ka / 448)[..., None]).view(torch.uint8)
        raw[page, 1, s["slot"]] = _codes(v, _inverse(va / 448)[..., None]).view(torch.uint8)
    else:
        _block_half(s, raw, 0, k, s["ks"], page)
        _block_half(s, raw, 1, v, s["vs"], page)
    return _append_out(s, s["qo"])


def _block_half(s, raw, half, x, scale, page):
    ids = s["ids"][s["touched"]].long()
    need = torch.zeros((len(ids), x.shape[1]), device=x.device)
    need = need.scatter_reduce(0, s["unit"][:, None].expand(-1, x.shape[1]), _amax(x, -1), "amax")
    old = torch.where(s["before"][:, None] > 0, scale[ids], torch.zeros_like(need))
    new = torch.maximum(old, _pow2_scale(need))
    # the page's earlier codes under its new scale
    held = raw[ids, half].view(E4M3).float()
    moved = _codes(held, (old * _inverse(new))[:, None, :, None]).view(torch.uint8)
    keep = (torch.arange(PAGE, device=x.device) < s["before"][:, None])[..., None, None]
    keep = keep & (new > old)[:, None, :, None]
    raw[ids, half] = torch.where(keep, moved, raw[ids, half])
    raw[page, half, s["slot"]] = _codes(x, _inverse(new)[s["unit"]][..., None]).view(torch.uint8)
    scale[ids] = new


def _pages_table(s):
    p = torch.arange(s["max_pages"], device=s["ids"].device)
    entry = (s["first_entry"][:, None] + p).clamp(max=max(len(s["ids"]) - 1, 0))
    return s["ids"][entry].long() if len(s["ids"]) else entry * 0


def _attend(s, q, wide):
    """softmax(q k / sqrt(d)) v over each request's pages, in the type `wide`."""
    c, dev = s["case"], q.device
    hkv, d, B = c["hkv"], c["d"], c["batch"]
    table = _pages_table(s)
    L = s["max_pages"] * PAGE
    raw = s["kv"].view(torch.uint8)
    seen = torch.arange(L, device=dev) < s["total"][:, None]

    def half(i, scale):
        x = raw[table, i].view(E4M3).to(wide) * scale.to(wide)[table][:, :, None, :, None]
        return torch.where(seen[..., None, None], x.view(B, L, hkv, d), x.new_zeros(()))

    qs = torch.zeros((B, s["max_rows"]) + q.shape[1:], dtype=wide, device=dev)
    qs[s["req"], s["j"]] = q.to(wide)
    qs = qs.view(B, s["max_rows"], hkv, -1, d) / math.sqrt(d)
    logits = torch.einsum("bnhgd,blhd->bhgnl", qs, half(0, s["ks"]))
    # query row n of a request with r rows sees positions up to total - r + n
    limit = s["total"][:, None] - s["rows"][:, None] + torch.arange(s["max_rows"], device=dev)
    ok = torch.arange(L, device=dev) <= limit[..., None]
    logits = logits.masked_fill(~(ok & seen[:, None])[:, None, None], -math.inf)
    m = logits.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (logits - m).exp()
    z = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgnl,blhd->bnhgd", p, half(1, s["vs"]))
    o = o / z.permute(0, 3, 1, 2, 4).clamp(min=1e-30)
    lse = (m + z.log()).squeeze(-1).permute(0, 3, 1, 2)
    return (o.reshape(B, -1, c["hq"], d)[s["req"], s["j"]],
            lse.reshape(B, -1, c["hq"])[s["req"], s["j"]])


def _attend_plain(s, q):
    c = s["case"]
    if s["max_pages"] == 0:
        return {"o": torch.zeros_like(q),
                "lse": torch.full(q.shape[:2], -math.inf, device=q.device)}
    o, lse = _attend(s, q, torch.float32)
    return {"o": o.to(TYPES[c["dtype"]]), "lse": lse}


# ---------------------------------------------------------------- what a pass needs

def work(case):
    ctx, new, rows = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    es = 4 if case["dtype"] == "f32" else 2
    ce = es if case["scales"] == "none" else 1
    T = sum(rows)
    nbytes = flops = 0
    if case["op"] != "attend":
        # q, k, v read; q and the cache's new rows written
        nbytes += T * d * (hq * 2 * es + 2 * hkv * (es + ce))
        touched = sum((c + n + PAGE - 1) // PAGE - c // PAGE for c, n in zip(ctx, new) if n)
        per = {"token": T, "block": 2 * touched}.get(case["scales"], 0)
        nbytes += per * hkv * 2 * 4
        flops += T * (hq + hkv) * case["rotary"] * 3
    if case["op"] != "append":
        tokens = sum(ctx) + sum(new)
        pages = sum((c + n + PAGE - 1) // PAGE for c, n in zip(ctx, new))
        nbytes += tokens * hkv * d * 2 * ce + pages * (hkv * 8 + 4) + T * hq * (2 * d * es + 4)
        flops += sum(4 * (c + n) * r * hq * d for c, n, r in zip(ctx, new, rows))
    return {"bytes": max(nbytes, 1), "flops": flops}


# ---------------------------------------------------------------- the definition, in 64 bits

def _grid(x):
    """x (float64) rounded to the nearest E4M3 value, ties to even."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -30))).clamp(min=-6)
    # log2 may land on the wrong side next to a power of two
    e = e + (a >= torch.exp2(e + 1)).double() - ((a < torch.exp2(e)) & (e > -6)).double()
    step = torch.exp2(e - 3)
    y = torch.round(a / step) * step
    return torch.sign(x) * y.clamp(max=448)


def exact(case, seed):
    s = prepare(case, seed)
    c, dev, out = case, s["kv"].device, {}
    hkv, d = c["hkv"], c["d"]
    q = s["q"].double()
    if c["op"] != "attend":
        n = c["rotary"] // 2
        freq = torch.tensor([10000.0 ** (-2.0 * i / max(c["rotary"], 1)) for i in range(n)],
                            dtype=torch.float64, device=dev)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev),
                           (s["pos"].double() + c["offset"])[:, None] * freq)[:, None]

        def rotated(x):
            part = x[..., :2 * n].unflatten(-1, (n, 2) if c["interleaved"] else (2, n))
            a, b = part.unbind(-1 if c["interleaved"] else -2)
            z = torch.complex(a.contiguous(), b.contiguous()) * turn
            pair = torch.stack([z.real, z.imag], -1 if c["interleaved"] else -2)
            return torch.cat([pair.flatten(-2), x[..., 2 * n:]], -1)

        q = rotated(q)
        out["q"] = q
        news = [rotated(s["k"].double()), s["v"].double()]
        kv = s["kv"].double()
        ids = s["ids"].long()
        for i, x in enumerate(news):
            page, slot = ids[s["entry"]], s["slot"]
            if c["scales"] == "none":
                kv[page, i, slot] = x
            elif c["scales"] in ("tensor", "head"):
                sc = (s["ks"], s["vs"])[i].double()
                kv[page, i, slot] = _grid(x / sc[:, None])
            elif c["scales"] == "token":
                sc = x.abs().amax(-1) / 448
                s["ks" if i == 0 else "vs"] = full = (s["ks"], s["vs"])[i].double()
                full[page, :, slot] = sc
                kv[page, i, slot] = _grid(x / sc[..., None].clamp(min=1e-300))
            else:
                full = (s["ks"], s["vs"])[i].double()
                at = ids[s["touched"]]
                top = torch.zeros((len(at), hkv), dtype=torch.float64, device=dev)
                top.scatter_reduce_(0, s["unit"][:, None].expand(-1, hkv), x.abs().amax(-1),
                                    "amax")
                need = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-60) / 448)))
                # log2 may land on either side next to a power of two
                need = need * torch.where(top > 448 * need, 2.0, 1.0)
                need = need * torch.where(top <= 224 * need, 0.5, 1.0)
                had = s["before"] > 0
                old = full[at] * had[:, None]
                now = torch.maximum(old, need)
                ratio = (old / now)[:, None, :, None]
                rows = kv[at, i]
                older = (torch.arange(PAGE, device=dev) < s["before"][:, None])[..., None, None]
                kv[at, i] = torch.where(older & (ratio < 1), _grid(rows * ratio), rows)
                full[at] = now
                kv[page, i, slot] = _grid(x / now[s["unit"]][..., None])
                s["ks" if i == 0 else "vs"] = full
        out["kv"] = kv
        if c["scales"] in ("token", "block"):
            out["ks"], out["vs"] = s["ks"], s["vs"]
    if c["op"] != "append":
        if "kv" in out:
            s["kv"] = out["kv"].to(E4M3)  # values on the E4M3 grid: exact
        o, lse = _softmax_rows(s, q)
        out["o"], out["lse"] = o, lse
    return out


def _softmax_rows(s, q):
    """Request by request, in 64 bits."""
    c, dev = s["case"], q.device
    hkv, d, hq = c["hkv"], c["d"], c["hq"]
    o = torch.zeros((len(q), hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((len(q), hq), -math.inf, dtype=torch.float64, device=dev)
    ptr, row_ptr = s["indptr"].tolist(), s["row_ptr"].tolist()
    total = s["total"].tolist()
    if c["op"] == "step":
        # the rotated q as the attention is given it
        q = q.to(TYPES[c["dtype"]]).double()
    raw = s["kv"].view(torch.uint8)
    for b in range(c["batch"]):
        n, r0, r1 = total[b], row_ptr[b], row_ptr[b + 1]
        if n == 0 or r0 == r1:
            continue
        at = s["ids"][ptr[b]:ptr[b + 1]].long()
        kv = raw[at].view(E4M3).double()
        k = (kv[:, 0] * s["ks"].double()[at][:, None, :, None]).flatten(0, 1)[:n]
        v = (kv[:, 1] * s["vs"].double()[at][:, None, :, None]).flatten(0, 1)[:n]
        x = q[r0:r1].view(r1 - r0, hkv, -1, d).permute(1, 2, 0, 3)     # [hkv, g, r, d]
        w = x @ k.permute(1, 2, 0)[:, None] / math.sqrt(d)             # [hkv, g, r, n]
        behind = torch.arange(n, device=dev) > (n - (r1 - r0)
                                                + torch.arange(r1 - r0, device=dev))[:, None]
        w = w.masked_fill(behind, -math.inf)
        top = torch.logsumexp(w, -1)
        y = (w - top[..., None]).exp() @ v.permute(1, 0, 2)[:, None]   # [hkv, g, r, d]
        o[r0:r1] = y.permute(2, 0, 1, 3).reshape(r1 - r0, hq, d)
        lse[r0:r1] = top.permute(2, 0, 1).reshape(r1 - r0, hq)
    return o, lse
