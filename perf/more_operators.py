"""The prompt operators, and what they are measured on.

What a serving program does around decode, over a paged KV cache:

``prefill``  causal attention of packed query rows (whole prompts, chunks of
             them, single tokens) over each request's pages;
``axes``     append with a rotation of several position axes (time, height,
             width), as image and video tokens need it;
``weights``  add to each cached token the attention weight that a batch of
             query rows gave it;
``evict``    keep each kv head's most attended and most recent tokens, and
             compact the pages in place.

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

def _case(name, op, batch, ctx, new, heads, d=128, dtype="bf16", scales="none", **more):
    c = {"name": name, "op": op, "batch": batch, "ctx_min": ctx[0], "ctx_max": ctx[1],
         "new_min": new[0], "new_max": new[1], "hq": heads[0], "hkv": heads[1], "d": d,
         "dtype": dtype, "scales": scales}
    c.update(more)
    return c


def listed():
    return [
        # an interactive session: two short prompts; latency counts
        _case("prefill few", "prefill", 2, (0, 40), (5, 60), (32, 8)),
        # a prefill step of whole prompts
        _case("prefill prompts", "prefill", 8, (0, 0), (2048, 6144), (32, 8)),
        # the last chunk of one long prompt
        _case("prefill long", "prefill", 1, (24576, 24576), (8192, 8192), (32, 8)),
        # a mixed step, f16: single tokens, short prompts and chunks together
        _case("prefill mixed f16", "prefill", 48, (0, 2000), (1, 700), (16, 8), d=64, dtype="f16"),
        # chunks of prompts over an E4M3 cache with a scale per block
        _case("prefill e4m3 block", "prefill", 16, (1024, 8192), (500, 520), (64, 8),
              scales="block"),
        # prompts with images: text and height x width grids, three axes
        _case("axes images", "axes", 8, (0, 500), (1024, 4096), (32, 8), rotary=128,
              interleaved=False),
        # a decode step of a video chat: one token each, its axes apart
        _case("axes tokens", "axes", 128, (1024, 2048), (1, 1), (64, 8), rotary=128,
              interleaved=False),
        # a few short requests; latency counts
        _case("weights few", "weights", 4, (17, 700), (1, 1), (32, 8)),
        # a decode step's weights
        _case("weights decode", "weights", 128, (1024, 8192), (1, 1), (64, 8)),
        # the last 32 rows of each prompt look back, E4M3 with a scale per block
        _case("weights window e4m3", "weights", 16, (2048, 8192), (32, 32), (32, 8),
              scales="block"),
        # a serving batch trimmed to its budget
        _case("evict batch", "evict", 64, (2048, 8192), (0, 0), (64, 8), keep=2048, recent=256),
        # one long sequence, E4M3 with a scale per token, weights that tie
        _case("evict long e4m3", "evict", 1, (65536, 65536), (0, 0), (32, 8), scales="token",
              keep=8000, recent=33, ties=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "axes", "weights", "evict"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    heads = (hkv * rng.choice([1, 2, 4, 8]), hkv)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    e4m3 = rng.choice(["none", "none", "tensor", "head", "token", "block"])
    if op == "prefill":
        scales = e4m3 if dtype == "bf16" else "none"
        batch = _log(rng, 1, 128)
        new = _log(rng, 1, max(2, min(8192, 24000 // batch)))
        ctx = _log(rng, 1, max(2, min(24000, 200000 // batch)))
        c = _case("", op, batch, (rng.randint(0, ctx), ctx), (rng.randint(0, new), new), heads, d,
                  dtype, scales)
    elif op == "axes":
        dtype = rng.choice(["f32", "bf16", "f16"])
        batch = _log(rng, 1, 400)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(4000, 24000 // batch)))
        ctx = _log(rng, 1, 2048)
        scales = rng.choice(["none", e4m3]) if dtype != "f32" else "none"
        if scales not in ("none", "tensor", "head"):
            scales = "head"
        c = _case("", op, batch, (rng.randint(0, ctx), ctx), (rng.randint(0, new), new), heads, d,
                  dtype, scales, rotary=rng.choice([d, d, d // 2, 48, 16]),
                  interleaved=rng.random() < 0.3)
    elif op == "weights":
        batch = _log(rng, 1, 128)
        new = 1 if rng.random() < 0.5 else _log(rng, 2, 64)
        ctx = _log(rng, 1, max(2, min(65536, 500000 // batch)))
        c = _case("", op, batch, (rng.randint(0, ctx), ctx), (rng.randint(0, new), new), heads, d,
                  dtype, e4m3)
    else:
        batch = _log(rng, 1, 128)
        ctx = _log(rng, 2, max(2, min(65536, 300000 // batch)))
        keep = _log(rng, 1, ctx)
        scales = rng.choice(["none", "none", "tensor", "token"])
        c = _case("", op, batch, (rng.randint(0, ctx), ctx), (0, 0), heads, d,
                  rng.choice(["f32", "bf16"]) if scales == "none" else dtype, scales, keep=keep,
                  recent=rng.choice([0, 1, keep // 8, keep // 2, keep]),
                  ties=rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(case):
    """Per request: tokens in the cache before its query rows, and query rows.
    Fixed by the case, so that work() knows them too."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    pairs = [(r.randint(case["ctx_min"], case["ctx_max"]),
              r.randint(case["new_min"], case["new_max"])) for _ in range(case["batch"])]
    return [c for c, _ in pairs], [n for _, n in pairs]


# ---------------------------------------------------------------- inputs

def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s; 0 for 0."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875).to(e.dtype)))
    return torch.where(amax > 0, s, torch.zeros_like(amax))


def _axis_positions(case, ctx, new):
    """[3, rows]: text advances all three axes together, an image stands still
    in time while it walks a grid of height and width."""
    r = random.Random(repr(case["batch"]) + repr(case["new_max"]))
    out = [[], [], []]
    for c, n in zip(ctx, new):
        at, done = c // 2, 0
        while done < n:
            text = min(n - done, r.randint(1, 60))
            for axis in out:
                axis.extend(range(at, at + text))
            at, done = at + text, done + text
            h, w = r.randint(1, 32), r.randint(1, 32)
            cells = [(at, at + i // w, at + i % w) for i in range(min(h * w, n - done))]
            for a, axis in enumerate(out):
                axis.extend(cell[a] for cell in cells)
            done += len(cells)
            at += max(h, w)
    return torch.tensor(out, dtype=torch.int32).view(3, -1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    ctx, rows = _lengths(case)
    op, B, hq, hkv, d = case["op"], case["batch"], case["hq"], case["hkv"], case["d"]
    qt = TYPES[case["dtype"]]
    kvt = qt if case["scales"] == "none" else E4M3
    total = [c + n for c, n in zip(ctx, rows)]
    pages = [(t + PAGE - 1) // PAGE for t in total]
    ptr, row_ptr = [0], [0]
    for p, n in zip(pages, rows):
        ptr.append(ptr[-1] + p)
        row_ptr.append(row_ptr[-1] + n)
    num_pages, T = ptr[-1] + 3, row_ptr[-1]
    host = torch.Generator().manual_seed(seed)
    ids = torch.randperm(num_pages, generator=host)[:ptr[-1]].to(torch.int32).to(dev)
    s = {"case": case, "total": total, "rows": rows, "ptr": ptr, "row_ptr": row_ptr, "ids": ids,
         "num_pages": num_pages,
         "indptr": torch.tensor(ptr, dtype=torch.int32),
         "qo_indptr": torch.tensor(row_ptr, dtype=torch.int32),
         "last": torch.tensor([t - (p - 1) * PAGE if p else PAGE for t, p in zip(total, pages)],
                              dtype=torch.int32)}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    # the cache as appends left it; an E4M3 one by its scales
    if kvt == E4M3:
        s["kv"] = torch.empty((num_pages, 2, PAGE, hkv, d), dtype=E4M3, device=dev)
        sc = []
        for half in range(2):
            x = normal(num_pages, PAGE, hkv, d)
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

    if op == "axes":
        # what a projection gives: q, k and v side by side in one row a token
        s["qkv"] = (normal(T, hq + 2 * hkv, d) * torch.exp2(normal(T, 1, 1))).to(qt)
        s["q"], s["k"], s["v"] = s["qkv"].split([hq, hkv, hkv], dim=1)
        s["qo"] = torch.empty((T, hq, d), dtype=qt, device=dev)
        s["positions"] = _axis_positions(case, ctx, rows).to(dev)
        n = case["rotary"] // 2
        # a quarter of the pairs turn with time, the others with height and width
        s["axis"] = torch.tensor([0] * (n - 2 * (3 * n // 8)) + [1] * (3 * n // 8)
                                 + [2] * (3 * n // 8))
        s["inv_freq"] = 10000.0 ** (-2.0 * torch.arange(n, dtype=torch.float64) / (2 * n))
        entry, slot = [], []
        for b in range(B):
            for t in range(ctx[b], total[b]):
                entry.append(ptr[b] + t // PAGE)
                slot.append(t % PAGE)
        s["entry"] = torch.tensor(entry, dtype=torch.int64, device=dev)
        s["slot"] = torch.tensor(slot, dtype=torch.int64, device=dev)
    elif op in ("prefill", "weights"):
        # rows whose logits spread by about one, some rows more
        s["q"] = (normal(T, hq, d) * torch.exp2(normal(T, 1, 1) / 2)).to(qt)
    if op == "weights":
        # the lse that the attention of these rows gave, and the weights so far
        s["lse"] = _attention_plain(s, False)[1]
        s["w"] = torch.rand((num_pages, hkv, PAGE), generator=g, device=dev)
    if op == "evict":
        # weights fall off steeply from token to token; they tie where few rows were seen
        w = torch.rand((num_pages, hkv, PAGE), generator=g, device=dev).pow(8)
        s["w"] = (w * 64).floor() / 64 if case.get("ties") else w
    if own:
        _plans(s, qt, kvt)
    return s


def _plans(s, qt, kvt):
    import paged_kv_decode_fa_gb300 as fa
    c = s["case"]
    shape = (c["hq"], c["hkv"], c["d"], PAGE)
    lay = (s["indptr"], s["ids"], s["last"])
    types = {"q_data_type": qt, "kv_data_type": kvt}
    if c["op"] == "prefill":
        s["plan"] = fa.plan_prefill(*lay, s["qo_indptr"], *shape, **types)
    elif c["op"] == "axes":
        rotary = fa.RotaryTable(c["rotary"], inv_freq=s["inv_freq"], axes=s["axis"],
                                interleaved=c["interleaved"])
        s["plan"] = fa.plan_append(*lay, s["qo_indptr"], *shape, rotary=rotary,
                                   positions=s["positions"], **types)
    elif c["op"] == "weights":
        s["plan"] = fa.plan_weights(*lay, s["qo_indptr"], *shape, **types)
    else:
        s["plan"] = fa.plan_evict(*lay, c["keep"], *shape[1:], recent=c["recent"],
                                  kv_data_type=kvt)


# ---------------------------------------------------------------- the passes

def run(s):
    op = s["case"]["op"]
    if op == "prefill":
        o, lse = _prefill_own(s) if own else _attention_plain(s, True)
        return {"o": o, "lse": lse}
    if op == "axes":
        return _axes_own(s) if own else _axes_plain(s)
    if op == "weights":
        return {"w": _weights_own(s) if own else _weights_plain(s)}
    if own:
        _evict_own(s)
    else:
        _evict_plain(s)
    return _evict_out(s)


def _evict_out(s):
    out = {"kv": s["kv"], "w": s["w"]}
    if s["case"]["scales"] == "token":
        out["ks"], out["vs"] = s["ks"], s["vs"]
    return out


def _prefill_own(s):
    p, scales, q, kv = s["plan"], s["case"]["scales"], s["q"], s["kv"]
    if scales == "none":
        return p.run(q, kv)
    if scales == "tensor":
        return p.run(q, kv, k_scale=s["ks1"], v_scale=s["vs1"])
    if scales == "head":
        return p.run_head_scales(q, kv, s["ks"], s["vs"])
    if scales == "token":
        return p.run_token_scales(q, kv, s["ks"], s["vs"])
    return p.run_block_scales(q, kv, s["ks"], s["vs"])


def _weights_own(s):
    p, scales, args = s["plan"], s["case"]["scales"], (s["q"], s["kv"], s["lse"], s["w"])
    if scales == "none":
        return p.run(*args)
    if scales == "tensor":
        return p.run(*args, k_scale=s["ks1"])
    if scales == "head":
        return p.run_head_scales(*args, s["ks"])
    if scales == "token":
        return p.run_token_scales(*args, s["ks"])
    return p.run_block_scales(*args, s["ks"])


def _evict_own(s):
    if s["case"]["scales"] == "token":
        s["plan"].run(s["kv"], s["w"], k_scales=s["ks"], v_scales=s["vs"])
    else:
        s["plan"].run(s["kv"], s["w"])


def _axes_own(s):
    p, scales, kw = s["plan"], s["case"]["scales"], {"q": s["q"], "q_out": s["qo"]}
    if scales == "none":
        q = p.run(s["k"], s["v"], s["kv"], **kw)
    elif scales == "tensor":
        q = p.run(s["k"], s["v"], s["kv"], k_scale=s["ks1"], v_scale=s["vs1"], **kw)
    else:
        q = p.run_head_scales(s["k"], s["v"], s["kv"], s["ks"], s["vs"], **kw)
    return {"q": q, "kv": s["kv"]}


def _cached(s, b, half, wide):
    """Request b's keys (half 0) or values (1), [tokens, hkv, d], as `wide`."""
    at = s["ids"][s["ptr"][b]:s["ptr"][b + 1]].long()
    kv = s["kv"]
    if kv.dtype != E4M3:
        return kv[at, half].to(wide).flatten(0, 1)[:s["total"][b]]
    x = kv.view(torch.uint8)[at, half].view(E4M3).to(wide)
    scale = (s["ks"], s["vs"])[half].to(wide)
    kind = s["case"]["scales"]
    if kind == "token":
        x = x * scale[at].permute(0, 2, 1)[..., None]
    elif kind == "block":
        x = x * scale[at][:, None, :, None]
    else:
        x = x * scale[:, None]
    return x.flatten(0, 1)[:s["total"][b]]


def _logits(s, b, k, r0, r1):
    """Rows r0 .. r1 of request b against its keys, [hkv, group, rows, tokens]."""
    c, n = s["case"], s["total"][b]
    x = s["q"][s["row_ptr"][b] + r0:s["row_ptr"][b] + r1].to(k.dtype)
    x = x.view(r1 - r0, c["hkv"], -1, c["d"]).permute(1, 2, 0, 3) / math.sqrt(c["d"])
    w = torch.matmul(x.flatten(1, 2), k.permute(1, 2, 0)).view(c["hkv"], -1, r1 - r0, n)
    row = torch.arange(r0, r1, device=k.device) + (n - s["rows"][b])
    return w.masked_fill_(torch.arange(n, device=k.device) > row[:, None], -math.inf)


def _chunks(s, b):
    """Row ranges of request b whose logits stay below 2^29 values."""
    n, step = s["rows"][b], max(1, (1 << 29) // max(1, s["total"][b] * s["case"]["hq"]))
    return [(r, min(n, r + step)) for r in range(0, n, step)]


def _attention_plain(s, values):
    c, q = s["case"], s["q"]
    o = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    for b in range(c["batch"]):
        if s["rows"][b] == 0:
            continue
        k = _cached(s, b, 0, torch.float32)
        v = _cached(s, b, 1, torch.float32) if values else None
        for r0, r1 in _chunks(s, b):
            w = _logits(s, b, k, r0, r1)
            m = w.amax(-1, keepdim=True)
            w = w.sub_(m).exp_()
            z = w.sum(-1, keepdim=True)
            a0, a1 = s["row_ptr"][b] + r0, s["row_ptr"][b] + r1
            lse[a0:a1] = (m + z.log()).squeeze(-1).permute(2, 0, 1).flatten(1)
            if values:
                y = torch.matmul(w.flatten(1, 2), v.permute(1, 0, 2)).view(*w.shape[:3], -1) / z
                o[a0:a1] = y.permute(2, 0, 1, 3).flatten(1, 2)
    return o.to(q.dtype), lse


def _weights_plain(s):
    c = s["case"]
    for b in range(c["batch"]):
        if s["rows"][b] == 0:
            continue
        n = s["total"][b]
        k = _cached(s, b, 0, torch.float32)
        add = torch.zeros((c["hkv"], n), device=k.device)
        for r0, r1 in _chunks(s, b):
            w = _logits(s, b, k, r0, r1)
            lse = s["lse"][s["row_ptr"][b] + r0:s["row_ptr"][b] + r1]
            w = w.sub_(lse.view(r1 - r0, c["hkv"], -1).permute(1, 2, 0)[..., None]).exp_()
            add += w.sum((1, 2))
        at = s["ids"][s["ptr"][b]:s["ptr"][b + 1]].long()
        t = torch.arange(n, device=k.device)
        s["w"][at[t // PAGE], :, t % PAGE] += add.T
    return s["w"]


def _evict_plain(s):
    c, dev = s["case"], s["w"].device
    raw = s["kv"].view(torch.uint8) if s["kv"].dtype == E4M3 else s["kv"]
    heads = torch.arange(c["hkv"], device=dev)
    for b in range(c["batch"]):
        length = s["total"][b]
        n = min(length, c["keep"])
        if n == length:
            continue
        recent = min(c["recent"], n)
        t = torch.arange(length, device=dev)
        page, slot = s["ids"][s["ptr"][b] + t // PAGE].long(), t % PAGE
        w = s["w"][page, :, slot]                                    # [length, hkv]
        order = w[:length - recent].sort(dim=0, descending=True, stable=True)[1][:n - recent]
        kept = torch.cat([order, t[length - recent:, None].expand(-1, c["hkv"])]).sort(0)[0]
        src = (page[kept], slot[kept])                               # [n, hkv] each
        dst = (page[:n, None], slot[:n, None])
        for half in range(2):
            raw[dst[0], half, dst[1], heads] = raw[src[0], half, src[1], heads]
        s["w"][page, :, slot] = 0.0
        s["w"][dst[0], heads, dst[1]] = w.gather(0, kept)
        if c["scales"] == "token":
            for name in ("ks", "vs"):
                s[name][dst[0], heads, dst[1]] = s[name][src[0], heads, src[1]]


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


def _axes_plain(s):
    c, kv, dev = s["case"], s["kv"], s["kv"].device
    angle = s["positions"][s["axis"].to(dev)].T.double() * s["inv_freq"].to(dev)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s["qo"].copy_(_rotate(s["q"].float(), cos, sin, c["interleaved"]))
    k, v = _rotate(s["k"].float(), cos, sin, c["interleaved"]), s["v"].float()
    page = s["ids"][s["entry"]].long()
    for half, x in ((0, k), (1, v)):
        if kv.dtype == E4M3:
            scale = (s["ks"], s["vs"])[half]
            codes = (x * (1 / scale)[:, None]).clamp(-448, 448).to(E4M3)
            kv.view(torch.uint8)[page, half, s["slot"]] = codes.view(torch.uint8)
        else:
            kv[page, half, s["slot"]] = x.to(kv.dtype)
    return {"q": s["qo"], "kv": kv}


# ---------------------------------------------------------------- what a pass needs

def work(case):
    ctx, rows = _lengths(case)
    op, hq, hkv, d = case["op"], case["hq"], case["hkv"], case["d"]
    es = 4 if case["dtype"] == "f32" else 2
    ce = es if case["scales"] == "none" else 1
    T = sum(rows)
    nbytes = flops = 0
    if op == "axes":
        # q, k, v and the positions read; q and the cache's new rows written
        nbytes = T * (d * (hq * 2 * es + 2 * hkv * (es + ce)) + 12)
        flops = T * (hq + hkv) * case["rotary"] * 3
    elif op in ("prefill", "weights"):
        scale = {"token": 4, "block": 4 / PAGE}.get(case["scales"], 0)
        for c, n in zip(ctx, rows):
            if n == 0:
                continue
            seen = n * c + n * (n + 1) // 2
            halves = 2 if op == "prefill" else 1
            nbytes += (c + n) * hkv * (d * ce + scale) * halves + (c + n) / 4
            flops += seen * hq * d * 2 * halves
            # q read; o and lse written, or lse read and the weights added to
            nbytes += n * hq * (d * es * halves + 4)
            nbytes += 0 if op == "prefill" else (c + n) * hkv * 8
    else:
        per = 2 * d * ce + (8 if case["scales"] == "token" else 0)
        for c in ctx:
            n = min(c, case["keep"])
            if n < c:
                # all weights read, cleared or moved; the kept tokens that are
                # not in place (at least those behind the budget's slots) move
                far = n * (c - n) // c
                nbytes += hkv * (8 * c + far * 2 * per)
                flops += hkv * c
    return {"bytes": max(int(nbytes), 1), "flops": int(flops)}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefill":
        return _exact_prefill(s)
    if op == "axes":
        return _exact_axes(s)
    if op == "weights":
        return _exact_weights(s)
    return _exact_evict(s)


def _tokens(s, b):
    """(pages, slots) of request b's tokens."""
    t = torch.arange(s["total"][b], device=s["ids"].device)
    return s["ids"].long()[s["ptr"][b] + t // PAGE], t % PAGE


def _values64(s, b, half):
    page, slot = _tokens(s, b)
    kv, kind = s["kv"], s["case"]["scales"]
    if kv.dtype != E4M3:
        return kv[page, half, slot].double()
    x = kv.view(torch.uint8)[page, half, slot].view(E4M3).double()
    scale = (s["ks"] if half == 0 else s["vs"]).double()
    if kind == "token":
        return x * scale[page, :, slot].unsqueeze(-1)
    if kind == "block":
        return x * scale[page].unsqueeze(-1)
    return x * scale.view(1, -1, 1)


def _exact_rows(s, b, h, k, lo, hi):
    """Logits of query head h, rows lo .. hi of request b, masked, [rows, tokens]."""
    c = s["case"]
    x = s["q"][s["row_ptr"][b] + lo:s["row_ptr"][b] + hi, h].double()
    w = x @ k[:, h // (c["hq"] // c["hkv"])].T * c["d"] ** -0.5
    before = s["total"][b] - s["rows"][b]
    return w + torch.full_like(w, -math.inf).triu(before + lo + 1)


def _exact_prefill(s):
    c, q = s["case"], s["q"]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b in range(c["batch"]):
        n = s["rows"][b]
        if not n:
            continue
        k, v = _values64(s, b, 0), _values64(s, b, 1)
        for h in range(c["hq"]):
            for lo in range(0, n, 4096):
                hi, a = min(n, lo + 4096), s["row_ptr"][b]
                w = _exact_rows(s, b, h, k, lo, hi)
                top = torch.logsumexp(w, -1)
                o[a + lo:a + hi, h] = (w - top[:, None]).exp() @ v[:, h // (c["hq"] // c["hkv"])]
                lse[a + lo:a + hi, h] = top
    return {"o": o, "lse": lse}


def _exact_weights(s):
    c, out = s["case"], s["w"].double()
    for b in range(c["batch"]):
        n = s["rows"][b]
        if not n:
            continue
        k = _values64(s, b, 0)
        page, slot = _tokens(s, b)
        for h in range(c["hq"]):
            w = _exact_rows(s, b, h, k, 0, n)
            seen = s["lse"][s["row_ptr"][b]:s["row_ptr"][b] + n, h].double()
            out[page, h // (c["hq"] // c["hkv"]), slot] += (w - seen[:, None]).exp().sum(0)
    return {"w": out}


def _exact_axes(s):
    c, dev = s["case"], s["kv"].device
    n = c["rotary"] // 2
    axis = s["axis"].tolist()
    freq = torch.tensor([10000.0 ** (-i / n) for i in range(n)], dtype=torch.float64, device=dev)
    pos = torch.stack([s["positions"][a] for a in axis], -1).double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev), pos * freq)[:, None]

    def rotated(x):
        part = x[..., :2 * n].unflatten(-1, (n, 2) if c["interleaved"] else (2, n))
        a, b = part.unbind(-1 if c["interleaved"] else -2)
        z = torch.complex(a.contiguous(), b.contiguous()) * turn
        pair = torch.stack([z.real, z.imag], -1 if c["interleaved"] else -2)
        return torch.cat([pair.flatten(-2), x[..., 2 * n:]], -1)

    kv = s["kv"].double()
    page = s["ids"].long()[s["entry"]]
    for half, x in ((0, rotated(s["k"].double())), (1, s["v"].double())):
        if s["kv"].dtype == E4M3:
            x = _grid(x / (s["ks"], s["vs"])[half].double()[:, None])
        kv[page, half, s["slot"]] = x
    return {"q": rotated(s["q"].double()), "kv": kv}


def _grid(x):
    """x (float64) rounded to the nearest E4M3 value, ties to even."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -30))).clamp(min=-6)
    # log2 may land on the wrong side next to a power of two
    e = e + (a >= torch.exp2(e + 1)).double() - ((a < torch.exp2(e)) & (e > -6)).double()
    step = torch.exp2(e - 3)
    y = torch.round(a / step) * step
    return torch.sign(x) * y.clamp(max=448)


def _exact_evict(s):
    c = s["case"]
    for b in range(c["batch"]):
        length = s["total"][b]
        n = min(length, c["keep"])
        if n == length:
            continue
        old = length - min(c["recent"], n)
        want = n - (length - old)
        page, slot = _tokens(s, b)
        for h in range(c["hkv"]):
            w = s["w"][page, h, slot]
            keep = torch.zeros(length, dtype=torch.bool, device=w.device)
            keep[old:] = True
            if want:
                border = torch.kthvalue(w[:old], old - want + 1)[0]
                above, level = w[:old] > border, w[:old] == border
                keep[:old] = above | (level & (level.cumsum(0) <= want - above.sum()))
            kept = keep.nonzero()[:, 0]
            at, to = (page[kept], slot[kept]), (page[:n], slot[:n])
            raw = s["kv"].view(torch.uint8) if s["kv"].dtype == E4M3 else s["kv"]
            raw[to[0], :, to[1], h] = raw[at[0], :, at[1], h]
            moved = torch.zeros_like(w)
            moved[:n] = w[kept]
            s["w"][page, h, slot] = moved
            if c["scales"] == "token":
                for name in ("ks", "vs"):
                    s[name][to[0], h, to[1]] = s[name][at[0], h, at[1]]
    return _evict_out(s)
