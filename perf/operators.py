"""The page operators of a shared cache and the attention that reads it, as
cases to measure: copying pages, forking a prompt into many requests (and
releasing them), compacting a fragmented pool, and decode attention of a
batch that shares long prefixes.

`run` computes each in elementary torch operations (`own` false) or through
the package's entry points (`own` true) on the same inputs.  Pools are bytes:
e4m3 codes, or bf16.
"""
import math
import random

import torch

own = False

DEV = "cuda"
KEYS = {
    "prefix": ("q_heads", "kv_heads", "dim", "page", "groups", "members", "loose", "prefix_tokens", "suffix_lo",
               "suffix_hi", "cache", "out", "tags", "append"),
    "copy": ("kv_heads", "dim", "page", "pool", "pages", "cache", "ragged"),
    "fork": ("kv_heads", "dim", "page", "parents", "forks", "tokens", "cache", "tags"),
    "compact": ("kv_heads", "dim", "page", "pool", "rows", "fill", "shared", "cache"),
}


# ------------------------------------------------------------------ cases


def _prefix(name, q_heads, kv_heads, dim, page, groups, members, loose, prefix_tokens, suffix_lo, suffix_hi, cache,
            out, tags=False, append=False):
    return {"name": name, "op": "prefix", "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "groups": groups, "members": members, "loose": loose, "prefix_tokens": prefix_tokens,
            "suffix_lo": suffix_lo, "suffix_hi": suffix_hi, "cache": cache, "out": out, "tags": tags,
            "append": append}


def listed():
    return [
        # four samples of one short prompt, a few tokens in: what a call costs when there is next to nothing to do
        _prefix("prefix_4_samples", 8, 2, 64, 16, 1, 4, 0, 128, 1, 37, "fp8", "float32"),
        # a served batch behind one system prompt, FP8 cache, output in the type the next product takes
        _prefix("prefix_system_prompt", 32, 8, 128, 16, 1, 32, 0, 4096, 64, 1024, "fp8", "bfloat16", tags=True),
        # several prompts of different lengths and some requests of their own, per-token scales, odd sizes
        _prefix("prefix_mixed_groups", 24, 8, 128, 16, 5, 13, 7, 7000, 1, 1500, "fp8_token", "float32", tags=True),
        # the prefill pool's own precision
        _prefix("prefix_bf16_cache", 32, 8, 128, 16, 2, 24, 0, 8192, 16, 512, "bf16", "bfloat16"),
        # a long document and many questions about it, the step's new token written on the way
        _prefix("prefix_document_step", 64, 8, 128, 64, 1, 64, 0, 32768, 32, 640, "fp8", "bfloat16", tags=True,
                append=True),
        # the same reading with an output of 32 bits, as the plain decode gives it
        _prefix("prefix_document_fp32", 32, 8, 128, 16, 1, 64, 0, 16384, 32, 640, "fp8", "float32"),
        # copy-on-write of a few partly filled pages
        {"name": "copy_tails", "op": "copy", "kv_heads": 8, "dim": 128, "page": 16, "pool": 4096, "pages": 24,
         "cache": "fp8_token", "ragged": True},
        # whole requests copied inside the pool
        {"name": "copy_requests", "op": "copy", "kv_heads": 8, "dim": 128, "page": 64, "pool": 8192, "pages": 3800,
         "cache": "fp8", "ragged": False},
        # four samples branch off one request
        {"name": "fork_4_samples", "op": "fork", "kv_heads": 8, "dim": 128, "page": 16, "parents": 1, "forks": 4,
         "tokens": 1000, "cache": "fp8", "tags": True},
        # a search over several long requests: every row forks, then the branches are given back
        {"name": "fork_beams", "op": "fork", "kv_heads": 8, "dim": 128, "page": 16, "parents": 8, "forks": 64,
         "tokens": 30000, "cache": "bf16", "tags": True},
        # a small pool with holes
        {"name": "compact_small", "op": "compact", "kv_heads": 8, "dim": 128, "page": 16, "pool": 1500, "rows": 16,
         "fill": 0.5, "shared": True, "cache": "fp8_token"},
        # a served pool, half of it given back in no order
        {"name": "compact_pool", "op": "compact", "kv_heads": 8, "dim": 128, "page": 64, "pool": 14000, "rows": 96,
         "fill": 0.55, "shared": False, "cache": "fp8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefix", "prefix", "prefix", "copy", "fork", "compact"))
    cache = rng.choice(("fp8", "fp8_token", "bf16"))
    dim, page = rng.choice((64, 128)), rng.choice((16, 32, 64))
    kv = rng.choice((1, 2, 4, 8))
    if op == "prefix":
        group = rng.choice((1, 2, 3, 4, 7, 8))
        return {"op": op, "q_heads": kv * group, "kv_heads": kv, "dim": dim, "page": page,
                "groups": rng.randint(1, 4), "members": _log(rng, 2, 48), "loose": rng.choice((0, 0, 3)),
                "prefix_tokens": _log(rng, 100, 12000), "suffix_lo": 1, "suffix_hi": _log(rng, 8, 1500),
                "cache": cache, "out": rng.choice(("float32", "bfloat16")), "tags": rng.random() < 0.5,
                "append": rng.random() < 0.3}
    if op == "copy":
        pages = _log(rng, 3, 3000)
        return {"op": op, "kv_heads": kv, "dim": dim, "page": page, "pool": 2 * pages + rng.randint(1, 99),
                "pages": pages, "cache": cache, "ragged": rng.random() < 0.5}
    if op == "fork":
        return {"op": op, "kv_heads": kv, "dim": dim, "page": page, "parents": rng.randint(1, 8),
                "forks": _log(rng, 1, 60), "tokens": _log(rng, 20, 28000), "cache": cache,
                "tags": rng.random() < 0.7}
    return {"op": op, "kv_heads": kv, "dim": dim, "page": page, "pool": _log(rng, 200, 12000),
            "rows": _log(rng, 3, 90), "fill": round(rng.uniform(0.2, 0.8), 2), "shared": rng.random() < 0.5,
            "cache": cache}


# ------------------------------------------------------------------ sizes (of the case alone, not of the seed)


def _sizes(case):
    rng = random.Random("|".join("%s=%s" % (k, case[k]) for k in KEYS[case["op"]]))
    S = case["page"]
    if case["op"] == "prefix":
        group, pages = [], []
        for g in range(case["groups"]):
            full = max(1, case["prefix_tokens"] // S)
            pages.append(full if g == 0 else _log(rng, 1, full))
            group += [g] * (case["members"] if g == 0 else rng.randint(1, case["members"]))
        group += [-1] * case["loose"]
        rng.shuffle(group)
        suffix = [rng.randint(case["suffix_lo"], case["suffix_hi"]) for _ in group]
        # a request of its own has a context of its own, of the prompts' kind of length
        lens = [(pages[g] * S if g >= 0 else rng.randint(1, case["prefix_tokens"])) + s for g, s in zip(group, suffix)]
        return {"group": group, "pages": pages, "lens": lens}
    if case["op"] == "copy":
        return {"slots": [rng.randint(1, S) if case["ragged"] else S for _ in range(case["pages"])]}
    if case["op"] == "fork":
        lens = [case["tokens"]] + [rng.randint(max(1, case["tokens"] // 4), case["tokens"])
                                   for _ in range(case["parents"] - 1)]
        parents = [i % case["parents"] for i in range(case["forks"])]
        return {"parent_lens": lens, "parents": parents, "lens": [lens[p] for p in parents]}
    held = min(max(case["rows"], int(case["pool"] * case["fill"])), case["pool"])
    cuts = [0] + sorted(rng.sample(range(1, held), case["rows"] - 1)) + [held]
    return {"held": held, "rows": [b - a for a, b in zip(cuts, cuts[1:])]}


def _row_bytes(case):
    """Bytes of one (token, KV head) of K and V together, with its scales."""
    e = 2 if case["cache"] == "bf16" else 1
    return 2 * case["dim"] * e + (8 if case["cache"] == "fp8_token" else 0)


def work(case):
    z, S, H = _sizes(case), case["page"], case["kv_heads"]
    row = _row_bytes(case) * H
    if case["op"] == "prefix":
        own_tokens = sum(n - (z["pages"][g] * S if g >= 0 else 0) for n, g in zip(z["lens"], z["group"]))
        tokens = own_tokens + sum(z["pages"]) * S
        entries = sum(-(-n // S) for n in z["lens"])
        B, out = len(z["lens"]), 4 if case["out"] == "float32" else 2
        nbytes = tokens * row + entries * (12 if case["tags"] else 4) + B * case["q_heads"] * case["dim"] * (2 + out)
        if case["append"]:
            nbytes += B * H * case["dim"] * 4
        return {"bytes": nbytes, "flops": 4 * case["dim"] * case["q_heads"] * sum(z["lens"])}
    if case["op"] == "copy":
        return {"bytes": 2 * sum(z["slots"]) * row + 12 * case["pages"], "flops": 0}
    if case["op"] == "fork":
        shared = sum(n // S for n in z["lens"])
        # fork: entry and tag read, written, count read and written, page tag read; release: entry read, count
        # read and written
        return {"bytes": 2 * sum(n % S for n in z["lens"]) * row + shared * (8 + 8 + 8 + 4 + 12), "flops": 0}
    H_, P = z["held"], case["pool"]
    moved = H_ * (P - H_) / P  # held pages above the held count, expected of a random placement
    return {"bytes": 2 * moved * S * row + 9 * P + 16 * H_, "flops": 0}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * (seed + 1))


def _rows(shape, g):
    """Normal rows of the keys' and values' kind: one in a hundred is twenty times as large."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    return torch.where(torch.rand(shape, generator=g, device=DEV, dtype=torch.bfloat16) < 0.01, x * 20, x)


def _pool(case, P, g):
    """One pool [P][H][S][D] as bytes (or bf16) with its scales."""
    x = _rows((P, case["kv_heads"], case["page"], case["dim"]), g)
    if case["cache"] == "bf16":
        return x, None
    amax = x.abs().amax(-1).float() if case["cache"] == "fp8_token" else x.abs().amax((0, 2, 3)).float()
    scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    if case["cache"] == "fp8":
        scale = scale.clamp(min=60 / 448)
    wide = scale[..., None] if case["cache"] == "fp8_token" else scale[None, :, None, None]
    codes = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    for i in range(0, P, 512):  # in slices: the quotients are wide
        w = wide[i:i + 512] if case["cache"] == "fp8_token" else wide
        codes[i:i + 512] = (x[i:i + 512].float() / w).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def prepare(case, seed):
    z, S, g = _sizes(case), case["page"], _gen(seed)
    s = {"case": case, "sizes": z, "kept": {}}
    r = random.Random(seed)
    if case["op"] == "prefix":
        lens = z["lens"]
        B, MP = len(lens), max(-(-n // S) for n in lens) + 2
        need = [-(-n // S) for n in lens]
        P = sum(z["pages"]) + sum(n - (z["pages"][q] if q >= 0 else 0) for n, q in zip(need, z["group"]))
        P += P // 8 + 1
        perm = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).tolist()
        shared = [[perm.pop() for _ in range(n)] for n in z["pages"]]
        table = torch.full((B, MP), -1, dtype=torch.int32)
        for b in range(B):
            row = list(shared[z["group"][b]]) if z["group"][b] >= 0 else []
            row += [perm.pop() for _ in range(need[b] - len(row))]
            table[b, :need[b]] = torch.tensor(row, dtype=torch.int32)
        s["P"], s["table"] = P, table.to(DEV)
        s["page_tags"] = torch.randint(-2**31, 2**31 - 1, (P,), generator=g, device=DEV).int()
        s["tags"] = torch.where(s["table"] >= 0, s["page_tags"][s["table"].clamp(min=0).long()], 0).int()
        s["lens"], s["group"], s["prefix_pages"] = _ints(lens), _ints(z["group"]), _ints(z["pages"])
        s["k"], s["ks"] = _pool(case, P, g)
        s["v"], s["vs"] = _pool(case, P, g)
        s["q"] = torch.randn((B, case["q_heads"], case["dim"]), generator=g, device=DEV).bfloat16()
        s["scale"] = 1 / math.sqrt(case["dim"])
        s["k_new"] = _rows((B, case["kv_heads"], case["dim"]), g)
        s["v_new"] = _rows((B, case["kv_heads"], case["dim"]), g)
        return s
    if case["op"] == "copy":
        P, n = case["pool"], case["pages"]
        ids = torch.randperm(P, generator=torch.Generator().manual_seed(seed))[:2 * n].int()
        s["P"], s["src"], s["dst"] = P, ids[:n].to(DEV), ids[n:].to(DEV)
        s["slots"] = _ints(z["slots"])
        s["page_tags"] = torch.zeros(P, dtype=torch.int32, device=DEV)
        s["k"], s["ks"] = _pool(case, P, g)
        s["v"], s["vs"] = _pool(case, P, g)
        return s
    if case["op"] == "fork":
        need = [-(-n // S) for n in z["parent_lens"]]
        n_par, n = len(need), case["forks"]
        P = sum(need) + n + 16
        held = torch.randperm(P, generator=torch.Generator().manual_seed(seed))[:sum(need)].int()
        MP = max(need) + 2
        table = torch.full((n_par + n, MP), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = held[at:at + k]
            at += k
        s["held_pages"] = held.to(DEV)
        children = list(range(n_par, n_par + n))
        r.shuffle(children)
        s["parents"], s["children"], s["fork_lens"] = _ints(z["parents"]), _ints(children), _ints(z["lens"])
        # where in the table the children's pages stand, child by child: what is given back
        s["given_back"] = _ints([c * MP + i for c, m in zip(children, z["lens"]) for i in range(-(-m // S))],
                                torch.int64)
    else:
        P, H = case["pool"], z["held"]
        perm = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).int()
        held = perm[:H]
        parts = list(torch.split(held, z["rows"]))
        if case["shared"]:  # the rows after the first begin with the first one's pages, as forks do
            k = max(1, len(parts[0]) // 2)
            parts = [parts[0]] + [torch.cat([parts[0][:k], q]) for q in parts[1:]]
        MP = max(len(q) for q in parts) + 1
        table = torch.full((len(parts), MP), -1, dtype=torch.int32)
        for b, q in enumerate(parts):
            table[b, :len(q)] = q
        s["used"] = _ints([len(q) for q in parts])
        s["held_pages"] = held.to(DEV)
    s["P"], s["table"] = P, table.to(DEV)
    s["page_tags"] = torch.randint(-2**31, 2**31 - 1, (P,), generator=g, device=DEV).int()
    s["tags"] = torch.where(s["table"] >= 0, s["page_tags"][s["table"].clamp(min=0).long()], 0).int()
    entries = s["table"][s["table"] >= 0].long()
    s["refs"] = torch.zeros(P, dtype=torch.int32, device=DEV)  # holders beyond the first
    s["refs"].index_add_(0, entries, torch.ones_like(entries, dtype=torch.int32))
    s["refs"] = (s["refs"] - 1).clamp(min=0)
    held = torch.zeros(P, dtype=torch.bool, device=DEV)
    held[s["held_pages"].long()] = True
    s["held"] = held
    free = torch.nonzero(~held)[:, 0].flip(0).int()  # the smallest id on top
    s["stack"] = torch.cat([free, torch.zeros(P - len(free), dtype=torch.int32, device=DEV)])
    s["n_free"] = len(free)
    s["k"], s["ks"] = _pool(case, P, g)
    s["v"], s["vs"] = _pool(case, P, g)
    if case["op"] == "compact":  # every pass starts from the same holes
        s["saved"] = {k: s[k].clone() for k in ("table", "tags", "page_tags", "refs", "held", "stack")}
    return s


# ------------------------------------------------------------------ plain forms


def _values(t):
    """A pool as the values it holds."""
    return t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t


def _pools(s):
    """Every per-page array of the cache: codes or values, and per-token scales."""
    return [s["k"], s["v"]] + ([s["ks"], s["vs"]] if s["case"]["cache"] == "fp8_token" else [])


def _read(s, which, ids, dtype):
    """Pages ids [...] of one pool as real values [..., S, H, D]."""
    case, pool, scale = s["case"], s[which], s[which + "s"]
    x = _values(pool[ids]).to(dtype)
    if case["cache"] == "fp8_token":
        x = x * scale[ids].to(dtype)[..., None]
    elif case["cache"] == "fp8":
        x = x * scale.to(dtype)[:, None, None]
    return x.transpose(-2, -3)


def _append_plain(s):
    case, S = s["case"], s["case"]["page"]
    pos = (s["lens"] - 1).long()
    page = s["table"].gather(1, (pos // S)[:, None])[:, 0].long()
    slot = pos % S
    for which, new in (("k", s["k_new"]), ("v", s["v_new"])):
        if case["cache"] == "bf16":
            s[which][page, :, slot] = new
            continue
        if case["cache"] == "fp8_token":
            amax = new.abs().amax(-1).float()
            scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
            s[which + "s"][page, :, slot] = scale
        else:
            scale = s[which + "s"][None].expand(len(page), -1)
        codes = (new.float() / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s[which][page, :, slot] = codes.view(torch.uint8)


def _attend(s, dtype):
    """Softmax over the shared pages and a request's own pages together; shared pages are read once for a group."""
    case, S = s["case"], s["case"]["page"]
    B, Hq, D = s["q"].shape
    H = case["kv_heads"]
    G, n_groups = Hq // H, case["groups"]
    q = (s["q"].to(dtype) * s["scale"]).view(B, H, G, D)
    cols = torch.arange(n_groups, device=DEV)
    member = s["group"][:, None] == cols  # [B, groups]
    rank = (member.int().cumsum(0) * member).sum(1) - 1  # a request's place in its group
    grp = s["group"].clamp(min=0).long()
    loose = s["group"] < 0
    skip = torch.where(loose, 0, s["prefix_pages"][grp]).long()  # pages before a request's own
    # the groups' rows, padded to the largest group
    lead = member.int().argmax(0)
    n_max, p_max = case["members"], max(s["sizes"]["pages"])
    qg = torch.zeros((n_groups, n_max, H, G, D), dtype=dtype, device=DEV)
    gi, ri = torch.where(loose, n_groups - 1, grp), torch.where(loose, n_max - 1, rank)
    qg.index_put_((gi, ri), torch.where(loose[:, None, None, None], 0, q), accumulate=True)
    ids = s["table"][lead][:, :p_max].clamp(min=0).long()
    kp = _read(s, "k", ids, dtype).reshape(n_groups, p_max * S, H, D)
    zp = torch.einsum("gmhjd,gthd->gmhjt", qg, kp)
    t = torch.arange(p_max * S, device=DEV)
    zp = zp.masked_fill((t >= s["prefix_pages"][:, None] * S)[:, None, None, None], -math.inf)
    # own pages
    own_pages = max(-(-n // S) - (s["sizes"]["pages"][g] if g >= 0 else 0)
                    for n, g in zip(s["sizes"]["lens"], s["sizes"]["group"]))
    idx = (skip[:, None] + torch.arange(own_pages, device=DEV)).clamp(max=s["table"].shape[1] - 1)
    ids2 = s["table"].gather(1, idx).clamp(min=0).long()
    ko = _read(s, "k", ids2, dtype).reshape(B, own_pages * S, H, D)
    zo = torch.einsum("bhjd,bthd->bhjt", q, ko)
    u = torch.arange(own_pages * S, device=DEV)
    zo = zo.masked_fill((u >= (s["lens"] - skip * S)[:, None])[:, None, None], -math.inf)
    zb = zp[gi, ri].masked_fill(loose[:, None, None, None], -math.inf)  # a request's scores of its prefix
    m = torch.maximum(zb.amax(-1), zo.amax(-1))[..., None]
    pb, po = torch.exp(zb - m), torch.exp(zo - m)
    norm = pb.sum(-1) + po.sum(-1)
    del zb, zo, zp
    pg = torch.zeros((n_groups, n_max, H, G, p_max * S), dtype=dtype, device=DEV)
    pg.index_put_((gi, ri), pb, accumulate=True)  # a loose request adds zeros
    vp = _read(s, "v", ids, dtype).reshape(n_groups, p_max * S, H, D)
    shared = torch.einsum("gmhjt,gthd->gmhjd", pg, vp)[gi, ri].masked_fill(loose[:, None, None, None], 0)
    vo = _read(s, "v", ids2, dtype).reshape(B, own_pages * S, H, D)
    return ((shared + torch.einsum("bhjt,bthd->bhjd", po, vo)) / norm[..., None]).reshape(B, Hq, D)


def _prefix_plain(s):
    if s["case"]["append"]:
        _append_plain(s)
    out = _attend(s, torch.float32).to(getattr(torch, s["case"]["out"]))
    status = torch.zeros(len(s["lens"]), dtype=torch.int32, device=DEV)
    if s["case"]["tags"]:  # a page that has moved on marks its request
        at = s["table"].clamp(min=0).long()
        used = torch.arange(at.shape[1], device=DEV) < ((s["lens"] + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
        stale = ((s["page_tags"][at] != s["tags"]) & used).any(1)
        status = stale.int()
        out = torch.where(stale[:, None, None], torch.zeros_like(out), out)
    return out, status


def _copy_plain(s):
    S, src, dst = s["case"]["page"], s["src"].long(), s["dst"].long()
    if not s["case"]["ragged"]:
        for x in _pools(s):
            x[dst] = x[src]
        return
    m = torch.arange(S, device=DEV) < s["slots"][:, None]
    for x in _pools(s):
        w = m[:, None, :, None] if x.dim() == 4 else m[:, None]
        x[dst] = torch.where(w, x[src], x[dst])


def _fork_plain(s):
    S, table, tags = s["case"]["page"], s["table"], s["tags"]
    par, chi, lens = s["parents"].long(), s["children"].long(), s["fork_lens"].long()
    full, tail = lens // S, lens % S
    cols = torch.arange(table.shape[1], device=DEV)
    m = cols < full[:, None]
    rows = table[par]
    table[chi] = torch.where(m, rows, table[chi])
    tags[chi] = torch.where(m, tags[par], tags[chi])
    s["refs"].index_add_(0, rows.clamp(min=0).long().flatten(), m.int().flatten())
    who = torch.nonzero(tail > 0)[:, 0]  # those whose last page is partly filled
    k = len(who)
    new = s["stack"][s["n_free"] - 1 - torch.arange(k, device=DEV)].long()
    old = table[par[who], full[who]].long()
    s["page_tags"][new] += 1
    table[chi[who], full[who]] = new.int()
    tags[chi[who], full[who]] = s["page_tags"][new]
    keep = torch.arange(S, device=DEV) < tail[who][:, None]
    for x in _pools(s):
        w = keep[:, None, :, None] if x.dim() == 4 else keep[:, None]
        x[new] = torch.where(w, x[old], x[new])
    s["held"][new] = True
    return k


def _release_plain(s, pages, n_free):
    p = pages.long()
    s["refs"].index_add_(0, p, torch.full_like(pages, -1))
    gone = s["refs"][p] < 0
    at = torch.arange(len(p), device=DEV)
    last = torch.full((s["P"],), -1, dtype=torch.int64, device=DEV).scatter_reduce_(0, p, at, "amax")
    freed = p[gone & (last[p] == at)]
    s["stack"][n_free:n_free + len(freed)] = freed.int()
    s["refs"][freed] = 0
    s["held"][freed] = False


def _compact_plain(s):
    P, held, refs = s["P"], s["held"], s["refs"]
    n = s["sizes"]["held"]
    src = n + torch.nonzero(held[n:])[:, 0].flip(0)
    dst = torch.nonzero(~held[:n])[:, 0]
    for x in _pools(s):
        x[dst] = x[src]
    s["page_tags"][dst] += 1
    refs[dst] = refs[src]
    refs[src] = 0
    held[dst] = True
    held[src] = False
    to = torch.full((P,), -1, dtype=torch.int32, device=DEV)
    to[src] = dst.int()
    at = s["table"].clamp(min=0).long()
    used = torch.arange(at.shape[1], device=DEV) < s["used"][:, None]
    moved = used & (to[at] >= 0) & (s["page_tags"][at] == s["tags"])
    s["table"].copy_(torch.where(moved, to[at], s["table"]))
    s["tags"].copy_(torch.where(moved, s["page_tags"][s["table"].clamp(min=0).long()], s["tags"]))
    s["stack"][:P - n] = torch.nonzero(~held)[:, 0].flip(0).int()
    return src.int(), dst.int()


# ------------------------------------------------------------------ one pass


def _handles(s):
    """The cache descriptor, allocator and workspace that a program keeps."""
    kept = s["kept"]
    if kept:
        return kept
    from paged_fp8_kv_quantize_gb300 import abi

    case = s["case"]
    bf16 = case["cache"] == "bf16"
    cache = abi.PagedCache(s["P"], case["page"], case["kv_heads"], case["dim"],
                           dtype=abi.DTYPE_BF16 if bf16 else abi.DTYPE_FP8_E4M3,
                           scale_mode=abi.SCALE_PER_TOKEN if case["cache"] == "fp8_token" else abi.SCALE_PER_HEAD,
                           device=DEV, alloc_pools=False)
    cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale = s["k"], s["v"], s["ks"], s["vs"]
    cache.page_tags = s["page_tags"]
    kept["abi"], kept["cache"] = abi, cache
    if case["op"] in ("fork", "compact"):
        kept["alloc"] = abi.PageAllocator(s["P"], held_pages=s["held_pages"], device=DEV)
        kept["alloc"].refs = s["refs"]
        kept["saved"] = kept["alloc"].state.clone()
    if case["op"] == "prefix":
        n = abi.prefix_workspace_bytes(cache, len(s["lens"]), case["q_heads"], case["groups"])
        kept["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return kept


def run(s):
    case = s["case"]
    kept = _handles(s) if own else None
    if case["op"] == "prefix":
        if own:
            abi = kept["abi"]
            out, status = abi.paged_decode_attention_prefix(
                kept["cache"], s["q"], s["lens"], s["table"], s["tags"], s["group"], s["prefix_pages"], s["scale"],
                flags=abi.FLAG_TAG_CHECK if case["tags"] else 0, k_new=s["k_new"] if case["append"] else None,
                v_new=s["v_new"] if case["append"] else None, workspace=kept["workspace"],
                out_dtype=getattr(torch, case["out"]))
        else:
            out, status = _prefix_plain(s)
        got = {"out": out, "status": status}
        if case["append"]:
            got["k"], got["v"] = _values(s["k"]), _values(s["v"])
            if case["cache"] == "fp8_token":
                got["ks"], got["vs"] = s["ks"], s["vs"]
        return got
    if case["op"] == "copy":
        if own:
            kept["abi"].page_copy(kept["cache"], s["src"], s["dst"], s["slots"] if case["ragged"] else None)
        else:
            _copy_plain(s)
        return [_values(x) for x in _pools(s)]
    if case["op"] == "fork":
        if own:
            abi, alloc = kept["abi"], kept["alloc"]
            alloc.fork(kept["cache"], s["parents"], s["children"], s["fork_lens"], s["table"], s["tags"],
                       flags=abi.FLAG_TAG_CHECK if case["tags"] else 0)
            alloc.release(s["table"].view(-1)[s["given_back"]])
            stack = alloc.state[256:256 + 4 * s["P"]].view(torch.int32)
        else:
            k = _fork_plain(s)
            _release_plain(s, s["table"].view(-1)[s["given_back"]], s["n_free"] - k)
            stack = s["stack"]
        return {"table": s["table"], "tags": s["tags"], "page_tags": s["page_tags"], "refs": s["refs"],
                "free": stack[:s["n_free"]], "pools": [_values(x) for x in _pools(s)]}
    back = s["saved"]
    s["table"].copy_(back["table"])
    s["tags"].copy_(back["tags"])
    s["page_tags"].copy_(back["page_tags"])
    s["refs"].copy_(back["refs"])
    if own:
        alloc = kept["alloc"]
        alloc.state.copy_(kept["saved"])
        src, dst, _ = alloc.compact(kept["cache"], s["table"], s["tags"], used=s["used"])
        n = s["sizes"]["held"]
        stack = alloc.state[256:256 + 4 * s["P"]].view(torch.int32)
    else:
        s["held"].copy_(back["held"])
        s["stack"].copy_(back["stack"])
        src, dst = _compact_plain(s)
        n = s["sizes"]["held"]
        stack = s["stack"]
    return {"table": s["table"], "tags": s["tags"], "page_tags": s["page_tags"], "refs": s["refs"],
            "free": stack[:s["P"] - n], "pools": [_values(x) for x in _pools(s)]}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    """Attention from its definition, request by request and KV head by KV head; the page operators compute no
    numbers of their own."""
    if case["op"] != "prefix":
        return None
    s = prepare(case, seed)
    S, H, D = case["page"], case["kv_heads"], case["dim"]
    G = case["q_heads"] // H
    if case["append"]:
        _append_plain(s)
    out = torch.empty((len(s["lens"]), case["q_heads"], D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["sizes"]["lens"]):
        ids = s["table"][b, :-(-n // S)].long()
        kv = []
        for which in ("k", "v"):
            x = _values(s[which][ids]).double()  # [pages, H, S, D]
            if case["cache"] == "fp8_token":
                x = x * s[which + "s"][ids].double().unsqueeze(-1)
            elif case["cache"] == "fp8":
                x = x * s[which + "s"].double().view(1, H, 1, 1)
            kv.append(x.permute(1, 0, 2, 3).reshape(H, -1, D)[:, :n])
        z = torch.bmm(s["q"][b].double().view(H, G, D), kv[0].transpose(1, 2)) / math.sqrt(D)
        out[b] = torch.bmm(torch.softmax(z, -1), kv[1]).view(-1, D)
    got = {"out": out, "status": None}
    if case["append"]:
        got["k"] = got["v"] = None
        if case["cache"] == "fp8_token":
            got["ks"] = got["vs"] = None
    return got
