"""The paged-cache operators, as cases that can be timed and compared.

Four paths that a decoder layer with a full (uncompressed) cache runs beside the
fixed-budget one:

  heads   norm of every query and key head, then the position rotation
  write   keys and values written into the pages of a cache, as they are or
          quantised to e4m3 with one scale per token and head
  step    heads and write in one call, from the projection's rows to the cache
  read    a sequence's keys and values read back from its pages
  attend  attention of one new token per sequence over its pages

`run` computes them with elementary torch operations, or (own = True) with the
package's calls on the same inputs.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
F8 = torch.float8_e4m3fn


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def listed():
    shape = {"hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"}
    tiny = {"hq": 4, "hkv": 2, "d": 64, "dtype": "f32"}
    turn = {"rot": 128, "interleaved": False}
    return [
        # one decode step of 16 sequences: a launch's latency
        dict(shape, name="heads, 16 new tokens", op="heads", b=16, n=1, first=8191, **turn),
        # a whole prompt, from the projection's rows to the head-major layout that the prefill calls take
        dict(shape, name="heads, a prompt of 8192", op="heads", b=1, n=8192, first=0, **turn),
        # a prompt's keys and values into pages of 64 tokens as they are; rows of odd length, padded to one
        dict(shape, name="write, 3 x 2731 bf16", op="write", b=3, n=2731, cache="native", page=64, pad=100),
        # the same work with the cache held in 8 bits, pages of 16
        dict(shape, name="write, 8192 e4m3", op="write", b=1, n=8192, cache="e4m3", page=16, pad=0),
        # one decode step of 64 sequences in one call, cache in 8 bits
        dict(shape, name="step, 64 new tokens e4m3", op="step", b=64, n=1, first=8191, cache="e4m3", page=64, pad=0, **turn),
        # a chunk of a small model in 32 bits: odd length, half of each head turned, neighbouring pairs
        dict(tiny, name="step, 2 x 1021 f32", op="step", b=2, n=1021, first=100000, cache="native", page=16, pad=5, rot=32, interleaved=True),
        # four sequences read back from 8 bits, of unequal lengths
        dict(shape, name="read, 4 x 8192 e4m3", op="read", b=4, len=8192, cache="e4m3", page=64, ragged=True),
        # one short sequence read back
        dict(shape, name="read, 1 x 500 bf16", op="read", b=1, len=500, cache="native", page=16, ragged=False),
        # a conversation's first tokens: the smallest call
        dict(shape, name="attend, 1 x 117 bf16", op="attend", b=1, len=117, cache="native", page=16, ragged=False, softcap=0.0, window=0),
        # the ordinary decode step: 64 sequences of 8192 tokens
        dict(shape, name="attend, 64 x 8192 bf16", op="attend", b=64, len=8192, cache="native", page=64, ragged=False, softcap=0.0, window=0),
        # long contexts of unequal lengths, cache in 8 bits
        dict(shape, name="attend, 32 x 32768 e4m3", op="attend", b=32, len=32768, cache="e4m3", page=64, ragged=True, softcap=0.0, window=0),
        # few heads in 32 bits, scores capped, the last 1000 tokens alone
        dict(tiny, name="attend, 24 x 5000 f32 capped", op="attend", b=24, len=5000, cache="native", page=32, ragged=True, softcap=30.0, window=1000),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["heads", "write", "step", "read", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8])
    case = {"op": op, "hq": hkv * rng.choice([1, 2, 3, 4, 5, 8]), "hkv": hkv, "d": rng.choice([64, 128, 128]), "dtype": dtype}
    if op in ("heads", "write", "step"):
        case["b"] = _spread(rng, 1, 64)
        case["n"] = 1 if rng.random() < 0.3 else _spread(rng, 1, max(1, 8192 // case["b"]))
    if op in ("heads", "step"):
        case["first"] = rng.choice([0, rng.randrange(40000), rng.randrange(1 << 20)])
        case["rot"] = rng.choice([case["d"], case["d"], case["d"] // 2, 24])
        case["interleaved"] = rng.random() < 0.3
    if op != "heads":
        case["cache"] = "native" if dtype == "f32" else rng.choice(["native", "e4m3"])
        case["page"] = rng.choice([16, 32, 64, 128])
    if op in ("write", "step"):
        case["pad"] = rng.choice([0, case["n"] // 7])
    if op in ("read", "attend"):
        case["b"] = _spread(rng, 1, 64)
        case["len"] = _spread(rng, 1, min(32768, (32768 if op == "read" else 1 << 18) // case["b"]))
        case["ragged"] = rng.random() < 0.6
    if op == "attend":
        case["softcap"] = rng.choice([0.0, 0.0, 30.0])
        case["window"] = rng.choice([0, 0, _spread(rng, 1, case["len"])])
    return case


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _lens(case, seed):
    """Tokens of each sequence, on the host: all of them alike, or spread with an empty and a one-token sequence among them."""
    b, n = case["b"], case["len"]
    if not case["ragged"]:
        return [n] * b
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(1 + n // 2, n + 1, (b,), generator=g).tolist()
    lens[0] = n
    if b > 4:
        lens[1], lens[2] = 0, 1
    return lens


def _tables(case, seed, lens):
    """Pages in a random order: table [b][width] (-1 behind a sequence's last page), and the pool's size."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed + 1))
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m].int()
        at += m
    return table.cuda(), n_pages


def _pool(case, n_pages):
    """An empty pool of pages, key rows before value rows, with a last page where rows that belong nowhere go."""
    shape = (n_pages + 1, case["hkv"], 2, case["page"], case["d"])
    if case["cache"] == "e4m3":
        return torch.zeros(shape, device="cuda", dtype=torch.uint8).view(F8), torch.zeros(shape[:-1], device="cuda")
    return torch.zeros(shape, device="cuda", dtype=_dtype(case)), None


def _handle(case, n_pages):
    import fixed_budget_kv_kvpop_b200 as kp
    return kp.KVPopPagedCache(kp.make_paged_config(
        n_layers=1, n_q_heads=case["hq"], n_kv_heads=case["hkv"], head_dim=case["d"], page_size=case["page"],
        n_pages=n_pages, max_batch=case["b"], dtype=case["dtype"], cache=case["cache"]))


def _rows(case, seed):
    """A projection's output, [b][n][hq + 2 hkv heads][d], and views of its queries, keys and values; 2% of the keys are three times as long."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv = case["hq"], case["hkv"]
    x = _normal(g, (case["b"], case["n"], hq + 2 * hkv, case["d"]), _dtype(case))
    long = torch.rand(case["b"], case["n"], hkv, 1, generator=g, device="cuda") < 0.02
    x[:, :, hq:hq + hkv] *= torch.where(long, 3.0, 1.0).to(x.dtype)
    return x, x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]


def _turn(case, seed):
    """Norm weights, frequencies and positions."""
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    qw, kw = (1 + 0.1 * torch.randn(case["d"], generator=g, device="cuda") for _ in range(2))
    rot = case["rot"]
    freq = 1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    pos = (case["first"] + torch.arange(case["n"], device="cuda")).repeat(case["b"], 1)
    return qw, kw, freq, (pos + torch.arange(case["b"], device="cuda").unsqueeze(1) * 7).int()


def _slots(case, seed):
    """Where each token goes: rows of n tokens in pages of a random order; the last `pad` of every second row go nowhere (-1)."""
    b, n, page = case["b"], case["n"], case["page"]
    table, n_pages = _tables(case, seed, [n] * b)
    i = torch.arange(n, device="cuda")
    slots = table[:, i // page] * page + i % page
    if case["pad"]:
        slots[::2, n - case["pad"]:] = -1
    return slots.int().contiguous(), n_pages


def _prompt(case, seed):
    """Keys and values of `b` sequences, [b][len][hkv][d], bf16 or f32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (case["b"], case["len"], case["hkv"], case["d"])
    k = _normal(g, shape, _dtype(case))
    k *= torch.where(torch.rand(shape[:-1] + (1,), generator=g, device="cuda") < 0.02, 3.0, 1.0).to(k.dtype)
    return k, _normal(g, shape, _dtype(case))


def _filled(case, seed):
    """Lengths, page table and slots of a cache that holds `_prompt`."""
    lens = _lens(case, seed)
    table, n_pages = _tables(case, seed, lens)
    i = torch.arange(case["len"], device="cuda")
    n = torch.tensor(lens, device="cuda", dtype=torch.int32)
    slots = table[:, (i // case["page"]).clamp(max=table.shape[1] - 1)] * case["page"] + i % case["page"]
    return n, table, torch.where(i < n.unsqueeze(1), slots, -1).int().contiguous(), n_pages


def prepare(case, seed):
    s = {"case": case}
    op = case["op"]
    if op in ("heads", "write", "step"):
        s["x"], s["q"], s["k"], s["v"] = _rows(case, seed)
    if op in ("heads", "step"):
        s["qw"], s["kw"], s["freq"], s["pos"] = _turn(case, seed)
        if own:
            import fixed_budget_kv_kvpop_b200 as kp
            s["rope"] = kp.make_rope(s["freq"], q_weight=s["qw"], k_weight=s["kw"], interleaved=case["interleaved"])
            s["q_out"] = torch.empty(case["b"], case["hq"], case["n"], case["d"], device="cuda", dtype=_dtype(case))
            if op == "heads":
                s["k_out"] = torch.empty(case["b"], case["hkv"], case["n"], case["d"], device="cuda", dtype=_dtype(case))
    if op in ("write", "step"):
        s["slots"], n_pages = _slots(case, seed)
    if op in ("read", "attend"):
        s["lens"], s["table"], slots, n_pages = _filled(case, seed)
        k, v = _prompt(case, seed)
    if op != "heads":
        if own:
            s["cache"] = _handle(case, n_pages)
        else:
            s["pages"], s["scales"] = _pool(case, n_pages)
        if op in ("read", "attend"):
            if own:
                s["cache"].append(0, k, v, slots)
            else:
                _store(s["pages"], s["scales"], k, v, slots)
    if op == "read":
        s["k_out"], s["v_out"] = (torch.zeros(case["b"], case["hkv"], case["len"], case["d"], device="cuda", dtype=_dtype(case)) for _ in range(2))
    if op == "attend":
        g = torch.Generator(device="cuda").manual_seed(seed + 3)
        s["q"] = _normal(g, (case["b"], case["hq"], case["d"]), _dtype(case))
        if own:
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(case["b"], case["hq"], device="cuda")
    return s


def _heads(x, weight, freq, pos, interleaved):
    """[b][n][h][d] in 32 bits: x / rms(x) * weight, then its first 2 * len(freq) values turned by pos * freq."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight
    angle = torch.remainder(pos.double().unsqueeze(-1) * freq, 2 * math.pi).unsqueeze(2)
    cos, sin = angle.cos().float(), angle.sin().float()
    rot = 2 * freq.numel()
    turned, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turned[..., :rot // 2], turned[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _quantised(x):
    """Values over scale in e4m3, and the scale: the row's largest magnitude stands for 448."""
    scale = x.abs().amax(-1) / E4M3_MAX
    return (x / torch.where(scale > 0, scale, 1.0).unsqueeze(-1)).to(F8), scale


def _store(pages, scales, k, v, slots):
    """Writes rows [b][n][hkv][d] to their slots, rows without one to the last page."""
    page = pages.shape[3]
    at = torch.where(slots < 0, (pages.shape[0] - 1) * page, slots).reshape(-1).long()
    where, row = at // page, at % page
    kv = torch.stack((k, v), 3).flatten(0, 1)
    if scales is None:
        pages[where, :, :, row] = kv.to(pages.dtype)
    else:
        x, scale = _quantised(kv.float())
        pages.view(torch.uint8)[where, :, :, row] = x.view(torch.uint8)
        scales[where, :, :, row] = scale


def _fetch(pages, scales, table):
    """[b][hkv][2][tokens][d] in 32 bits: what the pages of a table hold."""
    at = table.clamp(min=0).long()
    if scales is None:
        x = pages[at].float()
    else:
        x = pages.view(torch.uint8)[at].view(F8).float()
        x *= scales[at].unsqueeze(-1)
    b, p, h, _, page, d = x.shape
    return x.permute(0, 2, 3, 1, 4, 5).reshape(b, h, 2, p * page, d)


def _attend(q, kv, lens, softcap, window):
    """Softmax attention of q [b][hq][d] over the first `lens` keys (the last `window` of them): output and the log of the softmax's sum."""
    b, h, _, n, d = kv.shape
    scores = q.float().view(b, h, -1, d) @ kv[:, :, 0].transpose(-1, -2) / math.sqrt(d)
    if softcap:
        scores = softcap * torch.tanh(scores / softcap)
    i, m = torch.arange(n, device=q.device), lens.view(b, 1, 1, 1)
    seen = i < m
    if window:
        seen = seen & (i >= m - window)
    scores = scores.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(scores, -1)
    p = torch.exp(scores - torch.where(lse.isinf(), 0.0, lse).unsqueeze(-1))
    return (p @ kv[:, :, 1]).flatten(1, 2), lse.flatten(1, 2)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if op == "heads":
            import fixed_budget_kv_kvpop_b200 as kp
            kp.qk_norm_rope(s["rope"], s["q"], s["k"], s["pos"], s["q_out"].transpose(1, 2), s["k_out"].transpose(1, 2))
            return {"q": s["q_out"], "k": s["k_out"]}
        cache = s["cache"]
        if op == "write":
            cache.append(0, s["k"], s["v"], s["slots"])
            return {"pages": cache.pages(0), "scales": cache.scales(0)}
        if op == "step":
            cache.append_qkv(0, s["rope"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["q_out"].transpose(1, 2))
            return {"q": s["q_out"], "pages": cache.pages(0), "scales": cache.scales(0)}
        if op == "read":
            cache.gather(0, s["table"], s["lens"], s["k_out"].transpose(1, 2), s["v_out"].transpose(1, 2))
            return {"k": s["k_out"], "v": s["v_out"]}
        cache.attend(0, s["q"], s["table"], s["lens"], s["out"], lse=s["lse"], softcap=case["softcap"], window=case["window"])
        return {"out": s["out"], "lse": s["lse"]}
    if op in ("heads", "step"):
        q, k = (_heads(x, w, s["freq"], s["pos"], case["interleaved"]) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
        q = q.transpose(1, 2).to(_dtype(case)).contiguous()
        if op == "heads":
            return {"q": q, "k": k.transpose(1, 2).to(_dtype(case)).contiguous()}
        _store(s["pages"], s["scales"], k, s["v"].float(), s["slots"])
        return {"q": q, "pages": s["pages"][:-1], "scales": None if s["scales"] is None else s["scales"][:-1]}
    if op == "write":
        _store(s["pages"], s["scales"], s["k"], s["v"], s["slots"])
        return {"pages": s["pages"][:-1], "scales": None if s["scales"] is None else s["scales"][:-1]}
    kv = _fetch(s["pages"], s["scales"], s["table"])
    if op == "read":
        kv = kv[:, :, :, :case["len"]]
        held = (torch.arange(kv.shape[3], device="cuda") < s["lens"].view(-1, 1, 1, 1)).unsqueeze(-1)
        kv = torch.where(held, kv, 0.0).to(_dtype(case))
        s["k_out"][:, :, :kv.shape[3]], s["v_out"][:, :, :kv.shape[3]] = kv[:, :, 0], kv[:, :, 1]
        return {"k": s["k_out"], "v": s["v_out"]}
    out, lse = _attend(s["q"], kv, s["lens"], case["softcap"], case["window"])
    return {"out": out.to(_dtype(case)), "lse": lse}


def work(case):
    """Bytes that a pass has to read and write, and the operations of its products, norms and turns."""
    size = 4 if case["dtype"] == "f32" else 2
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["b"]
    held = d + 4 if case.get("cache") == "e4m3" else d * size
    op = case["op"]
    if op in ("heads", "write", "step"):
        rows, kept = b * case["n"], b * case["n"] - (b + 1) // 2 * case.get("pad", 0)
        if op == "heads":
            return {"bytes": rows * ((hq + hkv) * d * size * 2 + 4), "flops": rows * (hq + hkv) * d * 7}
        if op == "write":
            return {"bytes": kept * hkv * 2 * (d * size + held) + rows * 4, "flops": kept * hkv * 2 * d * 2}
        return {"bytes": rows * (hq * d * size * 2 + 8) + kept * hkv * 2 * (d * size + held), "flops": rows * (hq + hkv) * d * 7}
    spread = case["len"] * (0.75 if case["ragged"] else 1.0)
    tokens = b * (min(spread, case["window"]) if case.get("window") else spread)
    if op == "read":
        return {"bytes": tokens * hkv * 2 * (held + d * size), "flops": tokens * hkv * 2 * d}
    return {"bytes": tokens * hkv * 2 * held + b * hq * (2 * d * size + 4), "flops": tokens * hq * d * 4}


# ---- the definitions again, in 64 bits, sequence by sequence ----

def _exact_heads(x, weight, freq, pos, interleaved):
    x = x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * weight.double()
    turn = torch.exp(1j * (pos.double().unsqueeze(-1) * freq))
    half = freq.numel()
    out = y.clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    z = torch.complex(y[..., first], y[..., second]) * turn.unsqueeze(2)
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_store(case, k, v, slots, n_pages):
    page, hkv, d = case["page"], case["hkv"], case["d"]
    pages = torch.zeros(n_pages * page, hkv, 2, d, device="cuda", dtype=torch.float64)
    at = slots.reshape(-1).long()
    kept = at >= 0
    pages[at[kept]] = torch.stack((k.double(), v.double()), 3).reshape(-1, hkv, 2, d)[kept]
    pages = pages.view(n_pages, page, hkv, 2, d).permute(0, 2, 3, 1, 4).contiguous()
    if case["cache"] != "e4m3":
        return pages, None
    scales = pages.abs().amax(-1) / E4M3_MAX
    ratio = torch.where(scales.unsqueeze(-1) > 0, pages / scales.unsqueeze(-1), 0.0)
    # e4m3 has three bits after the leading one, and steps of 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(ratio.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(ratio / step) * step, scales


def exact(case, seed):
    op = case["op"]
    if op in ("heads", "write", "step"):
        _, q, k, v = _rows(case, seed)
        if op in ("heads", "step"):
            qw, kw, freq, pos = _turn(case, seed)
            q, k = _exact_heads(q, qw, freq, pos, case["interleaved"]), _exact_heads(k, kw, freq, pos, case["interleaved"])
            if op == "heads":
                return {"q": q.transpose(1, 2), "k": k.transpose(1, 2)}
        pages, scales = _exact_store(case, k, v, *_slots(case, seed))
        return dict({"pages": pages, "scales": scales}, **({"q": q.transpose(1, 2)} if op == "step" else {}))
    lens, table, slots, n_pages = _filled(case, seed)
    k, v = _prompt(case, seed)
    b, n, hkv, d = k.shape
    hq = case["hq"]
    if op == "read":
        k_out, v_out = (torch.zeros(b, hkv, n, d, device="cuda", dtype=torch.float64) for _ in range(2))
    else:
        g = torch.Generator(device="cuda").manual_seed(seed + 3)
        q = _normal(g, (b, hq, d), _dtype(case)).double()
        out, lse = torch.zeros(b, hq, d, device="cuda", dtype=torch.float64), torch.full((b, hq), -math.inf, device="cuda", dtype=torch.float64)
    for i, m in enumerate(lens.tolist()):
        if not m:
            continue
        rows = torch.stack((k[i, :m], v[i, :m]))
        if case["cache"] == "e4m3":  # what the cache holds is what is read: 8 bits and a scale in 32
            scale = (rows.float().abs().amax(-1, keepdim=True) / E4M3_MAX)
            rows = (rows.float() / torch.where(scale > 0, scale, 1.0)).to(F8).double() * scale.double()
        rows = rows.double().transpose(1, 2)
        if op == "read":
            k_out[i, :, :m], v_out[i, :, :m] = rows[0], rows[1]
            continue
        lo = max(0, m - case["window"]) if case["window"] else 0
        x = torch.einsum("hgd,hnd->hgn", q[i].view(hkv, hq // hkv, d), rows[0, :, lo:]) * d ** -0.5
        if case["softcap"]:
            x = torch.tanh(x / case["softcap"]) * case["softcap"]
        top = x.amax(-1, keepdim=True)
        e = (x - top).exp()
        out[i] = (torch.einsum("hgn,hnd->hgd", e, rows[1, :, lo:]) / e.sum(-1, keepdim=True)).reshape(hq, d)
        lse[i] = (top + e.sum(-1, keepdim=True).log()).reshape(hq)
    return {"k": k_out, "v": v_out} if op == "read" else {"out": out, "lse": lse}
