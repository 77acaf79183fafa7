"""Workloads of the paged KV cache: block tables and slots, appending, reading back, attention.

A request's cached tokens live in pages of `page` tokens, anywhere in a pool.
K and V rows (128 columns) are rotated, y = (x * s) H / sqrt(128), and stored
as INT8 or INT4 codes with one float32 scale per `group` columns.  A serving
step is: find the slots of the new tokens (`slots`), quantise their K and V
into them (`append`), attend from the new tokens over everything cached
(`attention`); `gather` reads cached rows back as bf16.

With `own` false, `run` computes each of them with elementary torch operations
in 32 bits; with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DIM = 128
SCRATCH_BYTES = 48 << 20  # attention scratch that a program allocates once


# --------------------------------------------------------------------- cases

def _attention(name, batch, new, ctx, bits, group, page, q_heads=32, kv_heads=8, signs=True, causal=True, window=0, sinks=0,
               lens=1):
    return {"name": name, "op": "attention", "batch": batch, "new_min": new[0], "new_max": new[1], "ctx_min": ctx[0], "ctx_max": ctx[1],
            "bits": bits, "group": group, "page": page, "q_heads": q_heads, "kv_heads": kv_heads, "signs": signs, "causal": causal,
            "window": window, "sinks": sinks, "lens": lens}


def listed():
    return [
        # a decode step of a small server: a few requests grow by one token
        {"name": "slots_b16", "op": "slots", "batch": 16, "new_min": 1, "new_max": 1, "ctx_min": 1, "ctx_max": 4096, "page": 16, "lens": 1},
        # admission of a large ragged batch: some requests empty, some whole prompts
        {"name": "slots_b2048_prompts", "op": "slots", "batch": 2048, "new_min": 0, "new_max": 512, "ctx_min": 0, "ctx_max": 8191,
         "page": 32, "lens": 2},
        # the K and V rows of one decode step, written to the cache and read back
        {"name": "append_64_int4", "op": "append", "tokens": 64, "kv_heads": 8, "bits": 4, "group": 128, "page": 16, "signs": True},
        # a prompt chunk of a model without shared heads, INT8, one scale per 64 columns
        {"name": "append_4099_int8_g64", "op": "append", "tokens": 4099, "kv_heads": 32, "bits": 8, "group": 64, "page": 64, "signs": False},
        # a short cached prefix handed to another consumer
        {"name": "gather_333_int8", "op": "gather", "tokens": 333, "kv_heads": 8, "bits": 8, "group": 128, "page": 16, "signs": False},
        # a long cached prefix of 131072 tokens
        {"name": "gather_131072_int4", "op": "gather", "tokens": 131072, "kv_heads": 8, "bits": 4, "group": 128, "page": 64, "signs": True},
        # one request in a short conversation, one new token: latency
        _attention("decode_b1_short_int8", 1, (1, 1), (500, 500), 8, 128, 16),
        # one request over the 131072-token cache of the decode workload
        _attention("decode_b1_131072_int4", 1, (1, 1), (131071, 131071), 4, 128, 64),
        # a ragged decode batch, one scale per 32 columns
        _attention("decode_b64_int4_g32", 64, (1, 1), (17, 8191), 4, 32, 16, lens=3),
        # speculative tokens checked under sinks and a window, no shared heads
        _attention("verify_b24_int8_stream", 24, (1, 6), (0, 12000), 8, 128, 32, q_heads=32, kv_heads=32, signs=False, window=4096, sinks=4,
                   lens=4),
        # prompt chunks over a cached prefix: the compute-bound end
        _attention("chunk_b4_2048_int4", 4, (1500, 2048), (2000, 8192), 4, 128, 64, lens=5),
        # decoder tokens over an encoder's cached states of another length
        _attention("cross_b16_int8", 16, (40, 448), (1500, 1500), 8, 128, 16, q_heads=20, kv_heads=20, causal=False, lens=6),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["slots", "append", "gather", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1, 1 << 20)
    if op == "slots":
        return {"op": op, "batch": _log(rng, 1, 2048), "new_min": rng.choice([0, 1]), "new_max": _log(rng, 1, 512), "ctx_min": rng.choice([0, 1]),
                "ctx_max": _log(rng, 64, 8192), "page": page, "lens": lens}
    kv = rng.choice([1, 2, 4, 8, 8, 32])
    bits, group = rng.choice([4, 8]), rng.choice([128, 128, 64, 32])
    if op in ("append", "gather"):
        return {"op": op, "tokens": _log(rng, 1, (65536 if op == "append" else 131072) // kv), "kv_heads": kv, "bits": bits, "group": group,
                "page": page, "signs": rng.random() < 0.5}
    g = rng.choice([1, 4, 5, 7, 8]) if kv <= 8 else 1
    kind = rng.choice(["decode", "decode", "verify", "chunk", "chunk", "cross"])
    stream = kind != "cross" and rng.random() < 0.3
    c = {"op": op, "batch": 1, "new_min": 1, "new_max": 1, "ctx_min": 0, "ctx_max": 0, "bits": bits, "group": group, "page": page,
         "q_heads": kv * g, "kv_heads": kv, "signs": rng.random() < 0.5, "causal": kind != "cross",
         "window": _log(rng, 32, 4096) if stream else 0, "sinks": rng.choice([0, 4, 64]) if stream else 0, "lens": lens}
    if kind in ("decode", "verify"):
        c["batch"] = _log(rng, 1, 64)
        c["ctx_max"] = _log(rng, 16, max(16, min(131071, 4194304 // (kv * c["batch"]))))
        if kind == "verify":
            c["new_max"] = rng.randrange(2, 9)
    else:
        c["batch"] = _log(rng, 1, 16)
        c["new_max"] = _log(rng, 9, max(9, min(2048, 8192 // c["batch"])))
        c["new_min"] = rng.choice([0, 1, c["new_max"]])
        # the score matrix of the plain form has batch * q_heads * new_max * length entries
        c["ctx_max"] = _log(rng, 16, int(max(16, min(8192, 5e8 / (c["batch"] * c["q_heads"] * c["new_max"])))))
        if kind == "cross":
            c["ctx_min"] = rng.choice([1, c["ctx_max"]])
    return c


def _lengths(case):
    """Cached and new tokens of each request (the case fixes them up to their order)."""
    r = np.random.RandomState(case["lens"])
    ctx = r.randint(case["ctx_min"], case["ctx_max"] + 1, case["batch"])
    new = r.randint(case["new_min"], case["new_max"] + 1, case["batch"])
    if case["ctx_min"] != case["ctx_max"]:
        ctx[0] = case["ctx_max"]
    if not new.any():
        new[-1] = max(1, case["new_max"])
    if not case.get("causal", True):
        return ctx, new, ctx
    return ctx, new, ctx + new


# -------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)


def _rows(g, *shape):
    """bf16 activations with a few columns that run large, as keys have them."""
    x = torch.randn(*shape, generator=g, device="cuda")
    hot = torch.randint(0, DIM, (3,), generator=g, device="cuda")
    x[..., hot] *= 20.0
    return x.to(torch.bfloat16)


def _pool(g, pages, heads, page, bits, group, mean):
    """Codes and scales of rotated rows: after the rotation a row is close to
    Gaussian, around a direction that all rows of a head share."""
    y = torch.randn(pages, heads, page, DIM // group, group, generator=g, device="cuda")
    y += mean * torch.randn(heads, 1, DIM // group, group, generator=g, device="cuda")
    y *= torch.exp(0.3 * torch.randn(pages, heads, page, 1, 1, generator=g, device="cuda"))
    qmax = 127.0 if bits == 8 else 7.0
    scales = y.abs().amax(-1) / qmax
    codes = torch.round(y / scales.unsqueeze(-1)).clamp_(-qmax, qmax).to(torch.int8).view(pages, heads, page, DIM)
    if bits == 4:
        lo, hi = codes[..., 0::2].to(torch.uint8) & 15, codes[..., 1::2].to(torch.uint8) & 15
        codes = lo | (hi << 4)
    return codes.contiguous(), scales.contiguous()


def _signs(g, case):
    return (torch.randint(0, 2, (DIM,), generator=g, device="cuda") * 2 - 1).to(torch.int8) if case["signs"] else None


def prepare(case, seed):
    g = _generator(seed)
    dev = "cuda"
    s = {"case": case}
    if case["op"] == "slots":
        ctx, new, total = _lengths(case)
        order = np.random.RandomState(seed % (1 << 31)).permutation(len(ctx))
        ctx, new, total = ctx[order], new[order], total[order]
        old, all_ = -(-ctx // case["page"]), -(-total // case["page"])
        wide = int(all_.max()) + 1
        ids = torch.randperm(int(all_.sum()) + 64, generator=g, device=dev).to(torch.int32)
        table = torch.full((len(ctx), wide), -1, dtype=torch.int32, device=dev)
        have = torch.arange(wide, device=dev)[None, :] < torch.from_numpy(old).to(dev)[:, None]
        n_old = int(old.sum())
        table[have] = ids[:n_old]
        s.update(table=table, free=ids[n_old:].contiguous(), cached=torch.from_numpy(ctx.astype(np.int32)).to(dev),
                 new=torch.from_numpy(new.astype(np.int32)).to(dev), capacity=int(new.sum()) + 7)
        return s
    s["signs"] = _signs(g, case)
    page, heads, bits, group = case["page"], case["kv_heads"], case["bits"], case["group"]
    if case["op"] in ("append", "gather"):
        n = case["tokens"]
        pages = -(-n // page) + 2
        s["slots"] = torch.randperm(pages, generator=g, device=dev)[:, None].mul(page).add(torch.arange(page, device=dev)).view(-1)[:n].to(torch.int32)
        if case["op"] == "gather":
            s["codes"], s["scales"] = _pool(g, pages, heads, page, bits, group, 0.5)
        else:
            # K and V as a projection leaves them: columns of one wide row per token
            qkv = _rows(g, n, 3 * heads, DIM)
            s["k"], s["v"] = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
            for kv in "kv":
                s[kv + "_codes"] = torch.zeros((pages, heads, page, DIM * bits // 8), dtype=torch.uint8, device=dev)
                s[kv + "_scales"] = torch.zeros((pages, heads, page, DIM // group), dtype=torch.float32, device=dev)
        return s
    ctx, new, total = _lengths(case)
    order = np.random.RandomState(seed % (1 << 31)).permutation(len(ctx))
    new, total = new[order], total[order]
    need = -(-total // page)
    wide = max(1, int(need.max()))
    pages = int(need.sum()) + 3
    table = torch.full((len(new), wide), -1, dtype=torch.int32, device=dev)
    have = torch.arange(wide, device=dev)[None, :] < torch.from_numpy(need).to(dev)[:, None]
    table[have] = torch.randperm(pages, generator=g, device=dev)[:int(need.sum())].to(torch.int32)
    s["k_codes"], s["k_scales"] = _pool(g, pages, heads, page, bits, group, 0.5)
    s["v_codes"], s["v_scales"] = _pool(g, pages, heads, page, bits, group, 0.1)
    rows = int(new.sum())
    wide_q = torch.randn(rows, case["q_heads"] + 2 * heads, DIM, generator=g, device=dev)  # a projection's rows: q, k, v
    s.update(q=wide_q.to(torch.bfloat16)[:, :case["q_heads"]], table=table,
             lens=torch.from_numpy(total.astype(np.int32)).to(dev),
             cu=torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev),
             max_new=int(new.max()), max_len=int(total.max()), scratch=torch.zeros(SCRATCH_BYTES, dtype=torch.uint8, device=dev))
    return s


# ------------------------------------------------------------ the plain forms

_H = {}


def _hadamard(device):
    """The normalised Sylvester matrix of 128 points."""
    if device not in _H:
        h = torch.ones(1, 1, device=device)
        while h.shape[0] < DIM:
            h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
        _H[device] = h / math.sqrt(DIM)
    return _H[device]


def _rotate(x, signs):
    x = x.float()
    if signs is not None:
        x = x * signs.float()
    return x @ _hadamard(x.device)


def _unrotate(y, signs):
    y = y @ _hadamard(y.device)
    return y if signs is None else y * signs.float()


def _values(codes, scales, bits, group):
    """Codes [..., bytes] and scales [..., 128 / group] -> float32 [..., 128] in the rotated basis."""
    if bits == 4:
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int8)
        c = ((c + 8) & 15) - 8
    else:
        c = codes.view(torch.int8)
    return (c.unflatten(-1, (DIM // group, group)).float() * scales.unsqueeze(-1)).flatten(-2)


def _plain_slots(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    cached, new = s["cached"].long(), s["new"].long()
    old, all_ = (cached + page - 1) // page, (cached + new + page - 1) // page
    need = all_ - old
    first = need.cumsum(0) - need
    fits = (first + need <= free.numel()) & (all_ <= table.shape[1])
    cols = torch.arange(table.shape[1], device=table.device)
    fresh = fits[:, None] & (cols >= old[:, None]) & (cols < all_[:, None])
    at = (first[:, None] + cols - old[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at], table))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(s["capacity"], device=table.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    live = b < new.numel()
    b = b.clamp(max=new.numel() - 1)
    pos = cached[b] + t - cu[b]
    live = live & fits[b]
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    slots = torch.where(live, slot, -1).int()
    total = torch.where(fits, cached + new, 0).int()
    counts = torch.stack([(need * fits).sum(), (~fits).sum()]).int()
    return {"table": table, "slots": slots, "total": total, "cu": cu.int(), "counts": counts}


def _plain_gather(codes, scales, s):
    c = s["case"]
    slots = s["slots"].long()
    p, o = slots // c["page"], slots % c["page"]
    return _unrotate(_values(codes[p, :, o], scales[p, :, o], c["bits"], c["group"]), s["signs"]).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    qmax = 127.0 if c["bits"] == 8 else 7.0
    slots = s["slots"].long()
    p, o = slots // c["page"], slots % c["page"]
    for kv in "kv":
        y = _rotate(s[kv], s["signs"]).unflatten(-1, (DIM // c["group"], c["group"]))
        scale = y.abs().amax(-1) / qmax
        q = torch.round(y / torch.where(scale > 0, scale, 1.0).unsqueeze(-1)).clamp(-qmax, qmax).flatten(-2).to(torch.int8)
        q = q.view(torch.uint8)
        if c["bits"] == 4:
            q = (q[..., 0::2] & 15) | (q[..., 1::2] << 4)
        s[kv + "_codes"][p, :, o] = q
        s[kv + "_scales"][p, :, o] = scale


def _plain_attention(s):
    c = s["case"]
    q, lens, cu, page = s["q"], s["lens"].long(), s["cu"].long(), c["page"]
    batch, hq, hkv, tq, tk = c["batch"], c["q_heads"], c["kv_heads"], s["max_new"], s["max_len"]
    new = cu[1:] - cu[:-1]
    i = torch.arange(tq, device=q.device)
    live = i < new[:, None]
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    # [batch, kv head, (head of its group, token), 128]
    qr = _rotate(q[row], s["signs"]) * (1.0 / math.sqrt(DIM))
    qr = qr.view(batch, tq, hkv, hq // hkv, DIM).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, DIM)
    pages = s["table"][:, :-(-tk // page)].long().clamp(min=0)

    def cached(codes, scales):
        x = _values(codes[pages], scales[pages], c["bits"], c["group"])
        return x.permute(0, 2, 1, 3, 4).reshape(batch, hkv, -1, DIM)[:, :, :tk]

    j = torch.arange(tk, device=q.device)
    see = (j < lens[:, None])[:, None, :].expand(batch, tq, tk)
    if c["causal"]:
        pos = (lens - new)[:, None] + i
        ok = j <= pos[..., None]
        if c["window"]:
            ok = ok & ((j > pos[..., None] - c["window"]) | (j < c["sinks"]))
        see = see & ok
    score = torch.matmul(qr, cached(s["k_codes"], s["k_scales"]).transpose(-1, -2)).view(batch, hkv, hq // hkv, tq, tk)
    score = score.masked_fill(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = torch.matmul(p.view(batch, hkv, -1, tk), cached(s["v_codes"], s["v_scales"]))
    o = _unrotate(o, s["signs"]).view(batch, hkv, hq // hkv, tq, DIM).permute(0, 3, 1, 2, 4).reshape(batch, tq, hq, DIM)
    out = torch.empty((q.shape[0], hq, DIM), dtype=torch.bfloat16, device=q.device)
    out[row[live]] = o[live].to(torch.bfloat16)
    return out


def run(s):
    c = s["case"]
    if own:
        import hadamard_rotation_outlier_b200 as hq
        if c["op"] == "slots":
            slots, total, cu, counts = hq.hadq_paged_slots(s["cached"], s["new"], s["free"], s["table"], c["page"], capacity=s["capacity"])
            return {"table": s["table"], "slots": slots, "total": total, "cu": cu, "counts": counts}
        how = {"signs": s["signs"], "bits": c["bits"], "group": c["group"]}
        if c["op"] == "gather":
            return hq.hadq_paged_gather(s["codes"], s["scales"], s["slots"], **how)
        if c["op"] == "append":
            hq.hadq_paged_append(s["k"], s["v"], s["slots"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], **how)
            return {"k_scales": s["k_scales"], "v_scales": s["v_scales"],
                    "k": hq.hadq_paged_gather(s["k_codes"], s["k_scales"], s["slots"], **how),
                    "v": hq.hadq_paged_gather(s["v_codes"], s["v_scales"], s["slots"], **how)}
        return hq.hadq_paged_attention(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["table"], s["lens"], s["cu"],
                                       s["max_new"], causal=c["causal"], window=c["window"], sinks=c["sinks"], workspace=s["scratch"], **how)
    if c["op"] == "slots":
        return _plain_slots(s)
    if c["op"] == "gather":
        return _plain_gather(s["codes"], s["scales"], s)
    if c["op"] == "append":
        # codes come back as the values they stand for: read back in the basis of the input
        _plain_append(s)
        return {"k_scales": s["k_scales"], "v_scales": s["v_scales"], "k": _plain_gather(s["k_codes"], s["k_scales"], s),
                "v": _plain_gather(s["v_codes"], s["v_scales"], s)}
    return _plain_attention(s)


# ---------------------------------------------------------------------- work

def _seen(case):
    """(query, key) pairs per head, and cached tokens that some query of their request sees."""
    pairs = tokens = 0
    _, new, total = _lengths(case)
    for n, t in zip(new.tolist(), total.tolist()):
        if n == 0 or t == 0:
            continue
        if not case["causal"]:
            pairs, tokens = pairs + n * t, tokens + t
            continue
        w, k = case["window"], case["sinks"]
        pos = np.arange(t - n, t, dtype=np.int64)
        if not w:
            pairs, tokens = pairs + int((pos + 1).sum()), tokens + t
        else:
            start = np.maximum(0, pos - w + 1)
            pairs += int((pos + 1 - start + np.minimum(start, k)).sum())
            tokens += int(t - start[0] + min(start[0], k))
    return pairs, tokens


def work(case):
    if case["op"] == "slots":
        _, new, total = _lengths(case)
        ctx = _lengths(case)[0]
        taken = int((-(-total // case["page"]) - -(-ctx // case["page"])).sum())
        return {"bytes": 4.0 * (4 * case["batch"] + 1 + 2 * taken + int(new.sum()) + 9), "flops": 0.0}
    row = DIM * case["bits"] / 8 + 4 * DIM / case["group"]  # one cached row: codes and scales
    if case["op"] == "gather":
        n = case["tokens"] * case["kv_heads"]
        return {"bytes": n * (row + 2 * DIM) + 4.0 * case["tokens"], "flops": n * DIM * 8.0}
    if case["op"] == "append":  # both of K and V: written, and read back
        n = 2 * case["tokens"] * case["kv_heads"]
        return {"bytes": n * (2 * row + 4 * DIM) + 12.0 * case["tokens"], "flops": n * DIM * 18.0}
    pairs, tokens = _seen(case)
    rows = int(_lengths(case)[1].sum()) * case["q_heads"]
    return {"bytes": 2 * tokens * case["kv_heads"] * row + 4.0 * DIM * rows, "flops": 4.0 * DIM * pairs * case["q_heads"]}


# ----------------------------------------------------------- 64-bit reference

def _exact_h():
    i = torch.arange(DIM, device="cuda")
    x = i[:, None] & i[None, :]
    for shift in (4, 2, 1):
        x = x ^ (x >> shift)
    return (1.0 - 2.0 * (x & 1).double()) / math.sqrt(float(DIM))


def _exact_codes(codes, bits):
    if bits == 8:
        return codes.to(torch.int16).sub((codes > 127).to(torch.int16) * 256).double()
    both = torch.empty(*codes.shape[:-1], DIM, dtype=torch.float64, device=codes.device)
    both[..., 0::2] = (codes % 16).double()
    both[..., 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    return torch.where(both > 7, both - 16, both)


def _exact_rows(codes, scales, slots, case):
    """float64 rows [tokens, heads, 128] in the rotated basis."""
    page = case["page"]
    flat_c = codes.transpose(1, 2).reshape(-1, codes.shape[1], codes.shape[3])
    flat_s = scales.transpose(1, 2).reshape(-1, scales.shape[1], scales.shape[3])
    assert flat_c.shape[0] % page == 0
    return _exact_codes(flat_c[slots], case["bits"]) * flat_s[slots].double().repeat_interleave(case["group"], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "slots":
        return None
    h = _exact_h()
    sg = torch.ones(DIM, dtype=torch.float64, device="cuda") if s["signs"] is None else s["signs"].double()
    if case["op"] == "gather":
        return _exact_rows(s["codes"], s["scales"], s["slots"].long(), case) @ h * sg
    if case["op"] == "append":
        top = 2.0 ** (case["bits"] - 1) - 1
        got = {}
        for kv in "kv":
            y = (s[kv].double() * sg) @ h
            y = y.reshape(*y.shape[:-1], -1, case["group"])
            scale = y.abs().max(-1).values / top
            q = torch.round(y / scale[..., None])
            got[kv] = (q * scale[..., None]).reshape(*y.shape[:-2], DIM) @ h * sg
            whole = torch.zeros(s[kv + "_scales"].shape, dtype=torch.float64, device="cuda").transpose(1, 2).contiguous()
            whole.view(-1, *whole.shape[2:])[s["slots"].long()] = scale
            got[kv + "_scales"] = whole.transpose(1, 2).contiguous()
        return got
    page, per = case["page"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        first, last = cu[b], cu[b + 1]
        if first == last or n == 0:
            continue
        at = torch.arange(n, device="cuda")
        slots = s["table"][b].long()[at // page] * page + at % page
        k, v = _exact_rows(s["k_codes"], s["k_scales"], slots, case), _exact_rows(s["v_codes"], s["v_scales"], slots, case)
        where = torch.arange(n - (last - first), n, device="cuda")[:, None]
        hidden = torch.zeros(last - first, n, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden = at[None] > where
            if case["window"]:
                hidden |= (at[None] <= where - case["window"]) & (at[None] >= case["sinks"])
        for head in range(case["q_heads"]):
            x = ((s["q"][first:last, head].double() * sg) @ h) @ k[:, head // per].T / math.sqrt(float(DIM))
            x[hidden] = -math.inf
            out[first:last, head] = torch.softmax(x, -1) @ v[:, head // per] @ h * sg
    return out
