"""Cases that measure the decoding operators of this package: appending to and
attending over a paged 8-bit key/value cache, and beam search's selection and
reordering of rows.

``own`` False: each operator in its plain form, elementary torch operations.
``own`` True: the calls a user makes of stateful_decoding_b200.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
FP8 = torch.float8_e4m3fn
LEAST = -110                      # a block's scale is 2^e with e >= LEAST


def listed():
    return [
        # one generated token per row of the large tied model (64 rows at 4k+ positions, 16 heads x 128)
        {"name": "append one token", "op": "append", "rows": 64, "n": 1, "kv_heads": 16, "dh": 128, "page": 64,
         "type": "bf16", "lo": 4096, "hi": 4608, "cmin": 1, "rot": 128, "interleaved": False},
        # prompts of unequal length, straight from an fp32 projection (8 heads x 64)
        {"name": "append ragged prompts", "op": "append", "rows": 16, "n": 1999, "kv_heads": 8, "dh": 64, "page": 32,
         "type": "fp32", "lo": 0, "hi": 301, "cmin": 400, "rot": 64, "interleaved": False},
        # the prompts of the large model's batch, the largest append; interleaved pairs on part of the head
        {"name": "append large prompts", "op": "append", "rows": 32, "n": 4096, "kv_heads": 16, "dh": 128, "page": 64,
         "type": "bf16", "lo": 0, "hi": 0, "cmin": 4096, "rot": 64, "interleaved": True},
        # one sequence, one token: latency
        {"name": "attend one row", "op": "attend", "rows": 1, "n": 1, "heads": 8, "kv_heads": 8, "dh": 64, "page": 16,
         "type": "bf16", "lo": 300, "hi": 300, "rot": 64, "interleaved": False},
        # the parity workload's decoder step: 256 rows within 256 positions
        {"name": "attend parity rows", "op": "attend", "rows": 256, "n": 1, "heads": 8, "kv_heads": 8, "dh": 64,
         "page": 16, "type": "fp32", "lo": 1, "hi": 256, "rot": 64, "interleaved": False},
        # the large model's generation step: 64 rows at 4k+ positions, 16 heads x 128
        {"name": "attend large rows", "op": "attend", "rows": 64, "n": 1, "heads": 16, "kv_heads": 16, "dh": 128,
         "page": 64, "type": "bf16", "lo": 4096, "hi": 4608, "rot": 128, "interleaved": False},
        # blocks of four positions, eight query heads to a key head, very unequal lengths
        {"name": "attend shared heads", "op": "attend", "rows": 16, "n": 4, "heads": 32, "kv_heads": 4, "dh": 128,
         "page": 32, "type": "bf16", "lo": 103, "hi": 20011, "rot": 0, "interleaved": False},
        # one sequence with a very long prefix: work has to be split along it
        {"name": "attend long row", "op": "attend", "rows": 1, "n": 1, "heads": 16, "kv_heads": 8, "dh": 128,
         "page": 128, "type": "bf16", "lo": 131072, "hi": 131072, "rot": 128, "interleaved": False},
        # one search of four beams over the large model's vocabulary: latency
        {"name": "select one search", "op": "select", "groups": 1, "beams": 4, "vocab": 32000, "type": "fp32",
         "temperature": 1.0},
        # a batch of searches over a large odd vocabulary, 16-bit logits
        {"name": "select many searches", "op": "select", "groups": 128, "beams": 5, "vocab": 100003, "type": "bf16",
         "temperature": 0.8},
        # a few beams of a small model, generated part only
        {"name": "reorder few rows", "op": "reorder", "groups": 4, "beams": 4, "planes": 16, "cap": 288, "width": 64,
         "start": 256, "stop": 273, "type": "bf16"},
        # many beams: the generated half of a long cache
        {"name": "reorder many rows", "op": "reorder", "groups": 16, "beams": 8, "planes": 32, "cap": 1024,
         "width": 128, "start": 512, "stop": 1023, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "select", "reorder"])
    if op in ("append", "attend"):
        dh = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8, 16])
        c = {"op": op, "rows": _log(rng, 1, 256), "n": 1, "kv_heads": kv, "dh": dh,
             "page": rng.choice([16, 32, 64, 128]), "type": rng.choice(["bf16", "fp32"]),
             "rot": rng.choice([0, dh // 2, dh]), "interleaved": rng.random() < 0.4}
        most = 250_000_000                    # values of K (and of V) that a drawn case holds
        if op == "append":
            c["n"] = rng.choice([1, _log(rng, 2, 4096)])
            while c["rows"] * c["n"] * kv * dh > most:
                c["n"] = (c["n"] + 1) // 2
            c["hi"] = _log(rng, 1, 2048)
            c["lo"] = rng.randint(0, c["hi"])
            c["cmin"] = rng.randint(1, c["n"])
        else:
            c["heads"] = kv * rng.choice([1, 1, 2, 4, 8])
            c["n"] = rng.choice([1, 1, 1, rng.randint(2, 16)])
            c["hi"] = max(c["n"], _log(rng, 16, 100_000))
            while c["rows"] * c["hi"] * kv * dh * c["heads"] // kv * c["n"] > 16 * most or c["rows"] * c["hi"] * kv * dh > most:
                if c["rows"] > 1:
                    c["rows"] = (c["rows"] + 1) // 2
                else:
                    c["hi"] = (c["hi"] + 1) // 2
            c["hi"] = max(c["n"], c["hi"])
            c["lo"] = rng.randint(c["n"], c["hi"])
        return c
    if op == "select":
        c = {"op": op, "groups": _log(rng, 1, 128), "beams": rng.randint(1, 16), "vocab": _log(rng, 1000, 130_000),
             "type": rng.choice(["fp32", "bf16"]), "temperature": rng.choice([1.0, 0.7])}
        while c["groups"] * c["beams"] * c["vocab"] > 64_000_000:
            c["groups"] = (c["groups"] + 1) // 2
        return c
    c = {"op": op, "groups": _log(rng, 1, 32), "beams": rng.randint(2, 16), "planes": _log(rng, 1, 64),
         "cap": _log(rng, 8, 1024), "width": rng.choice([64, 128]), "type": rng.choice(["bf16", "fp32"])}
    while c["groups"] * c["beams"] * c["planes"] * c["cap"] * c["width"] > 250_000_000:
        c["cap"] = (c["cap"] + 1) // 2
    c["start"] = rng.randint(0, c["cap"] - 1)
    c["stop"] = rng.randint(c["start"] + 1, c["cap"])
    return c


def _spread(lo, hi, rows):
    """`rows` whole numbers from lo to hi, evenly spread."""
    return [hi if rows == 1 else lo + (hi - lo) * b // (rows - 1) for b in range(rows)]


def work(case):
    if case["op"] == "append":
        tokens = sum(_spread(case["cmin"], case["n"], case["rows"]))
        values = 2 * tokens * case["kv_heads"] * case["dh"]
        return {"bytes": values * ((2 if case["type"] == "bf16" else 4) + 1), "flops": 5 * values}
    if case["op"] == "attend":
        keys = sum(_spread(case["lo"], case["hi"], case["rows"]))
        io = 2 * case["rows"] * case["n"] * case["heads"] * case["dh"] * (2 if case["type"] == "bf16" else 4)
        kv = 2 * keys * case["kv_heads"] * case["dh"]
        blocks = 2 * case["kv_heads"] * keys / case["page"]
        return {"bytes": kv + 4 * blocks + io, "flops": 4 * keys * case["n"] * case["heads"] * case["dh"]}
    if case["op"] == "select":
        values = case["groups"] * case["beams"] * case["vocab"]
        return {"bytes": values * (2 if case["type"] == "bf16" else 4), "flops": 4 * values}
    # of all rows the moved ones alone have to be written, and the rows that they take read
    g, k = case["groups"], case["beams"]
    kept = (k + 1) // 2
    part = case["planes"] * (case["stop"] - case["start"]) * case["width"] * (2 if case["type"] == "bf16" else 4)
    return {"bytes": g * (k - kept + min(kept, k - kept)) * part, "flops": 0}


# ------------------------------------------------------------------ inputs
def _cache(case, g, longest):
    """Pages in a shuffled order, a few more of them than the rows need, holding e4m3 values and their scales."""
    page, rows, kv, dh = case["page"], case["rows"], case["kv_heads"], case["dh"]
    row_pages = -(-longest // page)
    n_pages = rows * row_pages + 3
    pages = torch.empty(n_pages, 2, kv, page, dh, dtype=torch.uint8, device="cuda")
    step = max(1, 64_000_000 // (2 * kv * page * dh))
    for i in range(0, n_pages, step):          # keys and values about N(0, 1) with scales of 2^-7 and 2^-6
        x = torch.randn(pages[i:i + step].shape, generator=g, device="cuda", dtype=torch.float32)
        pages[i:i + step] = (x * 96).clamp(-448, 448).to(FP8).view(torch.uint8)
    scales = torch.exp2(torch.randint(-7, -5, (n_pages, 2, kv), generator=g, device="cuda").float())
    table = torch.randperm(n_pages, generator=g, device="cuda")[: rows * row_pages].to(torch.int32)
    return {"pages": pages, "scales": scales, "table": table.view(rows, row_pages)}


def _rope(case, longest):
    if not case["rot"]:
        return None, None
    half = case["rot"] // 2
    at = torch.arange(longest + 1, dtype=torch.float64, device="cuda")[:, None]
    angle = at * 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    return angle.cos().float(), angle.sin().float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["type"]]
    s = {"case": case}
    if case["op"] in ("append", "attend"):
        rows = case["rows"]
        mix = torch.randperm(rows, generator=g, device="cuda")
        longest = case["hi"] + (case["n"] if case["op"] == "append" else 0)
        s.update(_cache(case, g, longest))
        s["cos"], s["sin"] = _rope(case, longest)
        lens = torch.tensor(_spread(case["lo"], case["hi"], rows), dtype=torch.int32, device="cuda")[mix]
        if case["op"] == "append":
            mix = torch.randperm(rows, generator=g, device="cuda")
            s["start"] = lens
            s["counts"] = torch.tensor(_spread(case["cmin"], case["n"], rows), dtype=torch.int32, device="cuda")[mix]
            # keys and values as one fused projection leaves them, side by side; now and then a much larger value
            kv = torch.randn(rows, case["n"], 2, case["kv_heads"], case["dh"], generator=g, device="cuda", dtype=t)
            kv[:, ::97] *= 3.0
            s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        else:
            s["lens"] = lens
            s["q"] = 1.5 * torch.randn(rows, case["n"], case["heads"], case["dh"], generator=g, device="cuda", dtype=t)
            s["out"] = torch.empty_like(s["q"])
    elif case["op"] == "select":
        G, K, V = case["groups"], case["beams"], case["vocab"]
        x = torch.randn(G, K, V, generator=g, device="cuda", dtype=torch.float32)
        s["logits"] = (3.0 * x).to(t)
        s["scores"] = -20.0 * torch.rand(G, K, generator=g, device="cuda")
        s["scores"][::5, 1:] = float("-inf")              # searches at their first token: one beam alive
        s["finished"] = (torch.rand(G, K, generator=g, device="cuda") < 0.1).to(torch.uint8)
        s["finished"][:, 0] = 0
        s["parents"] = torch.empty(G, K, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.empty(G, K, dtype=torch.int32, device="cuda")
        s["picked"] = torch.empty(G, K, dtype=torch.float32, device="cuda")
    else:
        G, K = case["groups"], case["beams"]
        s["rows"] = torch.randn(G * K, case["planes"], case["cap"], case["width"], generator=g, device="cuda", dtype=t)
        # half of the beams survive in their place, each of the others takes up one of those
        order = torch.rand(G, K, generator=g, device="cuda").argsort(1)
        kept = (K + 1) // 2
        parents = torch.empty(G, K, dtype=torch.int64, device="cuda")
        parents.scatter_(1, order[:, :kept], order[:, :kept])
        if K > kept:
            parents.scatter_(1, order[:, kept:], order[:, : K - kept])
        s["parents"] = parents.to(torch.int32)
    return s


# ------------------------------------------------------------------ plain forms
def _rotated(x, cos, sin, at, case):
    """x fp32 [..., heads, dh] turned by the angles of the positions `at` (the shape of x without its last two)."""
    if cos is None:
        return x
    c, s, rot = cos[at][..., None, :], sin[at][..., None, :], case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _power(amax):
    """The smallest power of two that brings amax within e4m3's 448 = 1.75 * 2^8."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.exp2(torch.where(amax > 0, e, LEAST).clamp(LEAST, 120).to(amax.dtype))


def _append(s):
    case, page = s["case"], s["case"]["page"]
    pages, scales, table = s["pages"], s["scales"], s["table"].long()
    start, counts = s["start"].long(), s["counts"].long()
    rows, n = case["rows"], case["n"]
    # rows with fewer tokens repeat their last one: written again, it changes nothing
    i = torch.minimum(torch.arange(n, device="cuda")[None], counts[:, None] - 1)
    b = torch.arange(rows, device="cuda")[:, None]
    at = start[:, None] + i
    k = _rotated(s["k"][b, i].float(), s["cos"], s["sin"], at, case)
    x = torch.stack((k, s["v"][b, i].float()), 2).flatten(0, 1)          # [tokens][2][heads][dh]
    home, slot = table[b, at // page].flatten(), (at % page).flatten()
    top = torch.zeros_like(scales).index_reduce_(0, home, x.abs().amax(-1), "amax")
    new = _power(top)
    # the block that a row begins in keeps its tokens, at the larger of the two scales
    first = table[torch.arange(rows, device="cuda"), start // page]
    old_there = (start % page > 0)[:, None, None]
    new[first] = torch.where(old_there, torch.maximum(new[first], scales[first]), new[first])
    old = pages[first].view(FP8).float() * (scales[first] / new[first])[..., None, None]
    is_old = (torch.arange(page, device="cuda") < (start % page)[:, None])[:, None, None, :, None]
    pages[first] = torch.where(is_old, old.to(FP8).view(torch.uint8), pages[first])
    pages[home, :, :, slot] = (x / new[home][..., None]).to(FP8).view(torch.uint8)
    touched = torch.zeros(len(scales), dtype=torch.bool, device="cuda").index_fill_(0, home, True)
    scales.copy_(torch.where(touched[:, None, None], new, scales))
    return {"pages": pages.view(FP8), "scales": scales}


def _attend(s):
    case = s["case"]
    rows, n, kv, dh = case["rows"], case["n"], case["kv_heads"], case["dh"]
    lens = s["lens"].long()
    at = lens[:, None] - n + torch.arange(n, device="cuda")
    q = _rotated(s["q"].float(), s["cos"], s["sin"], at, case) / math.sqrt(dh)
    q = q.view(rows, n, kv, -1, dh).permute(0, 2, 3, 1, 4)               # [rows][kv][group][n][dh]
    t = s["table"].long()
    x = s["pages"][t].view(FP8).float() * s["scales"][t][..., None, None]
    x = x.permute(2, 0, 3, 1, 4, 5).flatten(3, 4)                        # [2][rows][kv][keys][dh]
    score = q.flatten(2, 3) @ x[0].transpose(-1, -2)
    seen = torch.arange(x.shape[3], device="cuda") <= at[..., None]      # [rows][n][keys]
    score = score.unflatten(2, (-1, n)).masked_fill(~seen[:, None, None], float("-inf"))
    p = (score - score.amax(-1, keepdim=True)).exp()
    o = (p.flatten(2, 3) @ x[1]).unflatten(2, (-1, n)) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(rows, n, -1, dh))
    return s["out"]


def _select(s):
    K, V = s["case"]["beams"], s["case"]["vocab"]
    x = s["logits"].double() / s["case"]["temperature"]
    x = x - x.amax(-1, keepdim=True)
    x = s["scores"].double()[..., None] + (x - x.exp().sum(-1, keepdim=True).log())
    done = torch.full((V,), float("-inf"), dtype=torch.float64, device="cuda")
    alone = torch.where(torch.arange(V, device="cuda") == 2, s["scores"].double()[..., None], done)
    x = torch.where(s["finished"].bool()[..., None], alone, x).flatten(1)
    top, at = x.sort(dim=1, descending=True, stable=True)
    s["parents"].copy_(at[:, :K] // V)
    s["tokens"].copy_(at[:, :K] % V)
    s["picked"].copy_(top[:, :K])
    return s["parents"], s["tokens"], s["picked"]


def _reorder(s):
    G, K = s["parents"].shape
    source = (s["parents"].long() + K * torch.arange(G, device="cuda")[:, None]).flatten()
    part = s["rows"][:, :, s["case"]["start"]:s["case"]["stop"]]
    part.copy_(part[source])
    return s["rows"]


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import stateful_decoding_b200 as sd
    case, stream = s["case"], torch.cuda.current_stream()
    if case["op"] in ("append", "attend"):
        if "cache" not in s:                   # the handles that a program keeps beside its buffers
            s["cache"] = sd.Cache8(s["pages"], s["scales"], s["table"])
            s["rope"] = sd.Rope(s["cos"], s["sin"], interleaved=case["interleaved"]) if case["rot"] else None
        if case["op"] == "append":
            s["cache"].append(s["k"], s["v"], s["start"], counts=s["counts"], rope=s["rope"], stream=stream)
            return {"pages": s["pages"].view(FP8), "scales": s["scales"]}
        s["cache"].attend(s["q"], s["lens"], s["out"], rope=s["rope"], stream=stream)
        return s["out"]
    if case["op"] == "select":
        sd.beam_select(s["logits"], s["scores"], s["parents"], s["tokens"], s["picked"], finished=s["finished"],
                       eos=2, temperature=case["temperature"], stream=stream)
        return s["parents"], s["tokens"], s["picked"]
    sd.rows_reorder(s["rows"], s["parents"], start=case["start"], stop=case["stop"], stream=stream)
    return s["rows"]


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "select": _select, "reorder": _reorder}[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _turn64(x, cos, sin, at, case):
    """Each pair as a complex number times exp(i angle), the angle's cosine and sine as the table holds them."""
    rot = case["rot"]
    if not rot:
        return x
    w = torch.complex(cos.double(), sin.double())[at].unsqueeze(-2)
    pair = (lambda y: y.unflatten(-1, (rot // 2, 2))) if case["interleaved"] else (lambda y: y.unflatten(-1, (2, rot // 2)).transpose(-1, -2))
    z = torch.view_as_complex(pair(x[..., :rot]).contiguous()) * w
    z = torch.view_as_real(z)
    z = z if case["interleaved"] else z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), x[..., rot:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        page, table = case["page"], s["table"].tolist()
        if sum(len(t) for t in table) > 4000:
            return None
        pages, scales = s["pages"].view(FP8).double() * s["scales"].double()[..., None, None], s["scales"].double()
        eight, rows = s["pages"].view(FP8).clone(), list(zip(table, s["start"].tolist(), s["counts"].tolist()))
        for b, (mine, start, count) in enumerate(rows):
            at = torch.arange(start, start + count, device="cuda")
            k = _turn64(s["k"][b, :count].double(), s["cos"], s["sin"], at, case)
            x = torch.stack((k, s["v"][b, :count].double()), 1).permute(1, 2, 0, 3)
            for block in range(start // page, (start + count - 1) // page + 1):
                lo, hi = max(start, block * page), min(start + count, (block + 1) * page)
                p, a, z = mine[block], lo - block * page, hi - block * page
                new = x[:, :, lo - start:hi - start]
                # (an exact power of two may come out of log2 a rounding above its whole number)
                scale = torch.exp2(((new.abs().amax((-1, -2)) / 448).log2() - 1e-9).ceil().clamp(LEAST, 120))
                scale = torch.maximum(scale, scales[p]) if a else scale
                if a:
                    eight[p, :, :, :a] = (pages[p, :, :, :a] / scale[..., None, None]).float().to(FP8)
                eight[p, :, :, a:z] = (new / scale[..., None, None]).float().to(FP8)
                scales[p] = scale
        return {"pages": eight, "scales": scales}
    if case["op"] == "attend":
        n, dh, share = case["n"], case["dh"], case["heads"] // case["kv_heads"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, keys in enumerate(s["lens"].tolist()):
            mine = s["table"][b, : -(-keys // case["page"])].long()
            x = s["pages"][mine].view(FP8).double() * s["scales"][mine].double()[..., None, None]
            x = x.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :keys].repeat_interleave(share, 1)
            q = _turn64(s["q"][b].double(), s["cos"], s["sin"], torch.arange(keys - n, keys, device="cuda"), case)
            w = torch.einsum("nhd,hkd->hnk", q, x[0]) / dh ** 0.5
            w = w + torch.full((n, keys), float("-inf"), dtype=torch.float64, device="cuda").triu(keys - n + 1)
            out[b] = torch.einsum("hnk,hkd->nhd", torch.softmax(w, -1), x[1])
        return out
    if case["op"] == "select":
        G, K, V = case["groups"], case["beams"], case["vocab"]
        parents, tokens, picked = (torch.zeros(G, K, dtype=d, device="cuda") for d in (torch.int32, torch.int32, torch.float64))
        done = s["finished"].tolist()
        for g in range(G):
            each = s["scores"][g].double()[:, None] + torch.log_softmax(s["logits"][g].double() / case["temperature"], -1)
            for k in range(K):
                if done[g][k]:
                    each[k] = float("-inf")
                    each[k, 2] = s["scores"][g, k].double()
            each = each.flatten()
            for k in range(K):                 # the largest left, the first of equals
                best = each.max()
                at = (each == best).nonzero()[0, 0]
                parents[g, k], tokens[g, k], picked[g, k] = at // V, at % V, best
                each[at] = float("-inf")
        return parents, tokens, picked
    rows = s["rows"].clone()
    for r, p in enumerate(s["parents"].flatten().tolist()):
        source = s["rows"][r - r % case["beams"] + p]
        rows[r, :, case["start"]:case["stop"]] = source[:, case["start"]:case["stop"]]
    return rows.double()
