"""Timing cases of the cache's serving operators around block-sparse decoding.

Five operators, each with its plain form (elementary torch operations) and the library's
call, chosen by the module's ``own``:

  rope    rotate q and k by position, quantize k and v at their widths and append them; the
          appended rows are read back as values, so the pass returns all that it changed
  read    the dequantized K and V of the last tokens of each sequence
  bounds  per block of consecutive keys, each channel's minimum and maximum
  select  score every block from its bounds (an upper bound of its logits) and pick k
  attn    one new token per sequence attends over the picked blocks (full queries), over the
          local window (local queries) or not at all (skip queries)

Cases are dicts of plain values. ``lens`` lists the sequences' lengths ("8192*64" is 64 times
8192). Widths are drawn per (token, head) with the probabilities of WIDTHS_P.
"""
import math

import torch

own = False

WIDTHS = (2, 4, 8, 16)
WIDTHS_P = (0.25, 0.45, 0.2, 0.1)
MEAN_WIDTH = sum(b * p for b, p in zip(WIDTHS, WIDTHS_P))
TILE = 64                       # blocks per tile of the bounds layout [B, H, tiles, 2, D, TILE]
SKIP, LOCAL, FULL = 0, 1, 2


def _lens(case):
    out = []
    for part in case["lens"].split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * int(times or 1)
    return out


def listed():
    return [
        # one decode step of 64 sequences from one fused projection's output
        {"name": "rope_step", "op": "rope", "lens": "1*64", "before": 1023, "H": 16, "G": 1, "D": 128, "rot": 128,
         "interleaved": False, "fused": True, "page": 0},
        # a ragged prompt batch
        {"name": "rope_ragged_prefill", "op": "rope", "lens": "1024,3000,8192,5555", "before": 0, "H": 16, "G": 1,
         "D": 128, "rot": 128, "interleaved": False, "fused": False, "page": 0},
        # prompts of a small model that rotates neighbouring channels of half the head, on a paged cache
        {"name": "rope_prefill_160m", "op": "rope", "lens": "2048*8", "before": 0, "H": 12, "G": 1, "D": 64, "rot": 32,
         "interleaved": True, "fused": True, "page": 65536},
        # the whole cached prompt batch as fp16 rows, for a layer that wants plain K and V
        {"name": "read_ragged_prefill", "op": "read", "lens": "1024,3000,8192,5555", "tail": 8192, "H": 16, "G": 1,
         "D": 128, "dtype": "float16", "page": 0},
        # the newest tokens of many sequences in full precision, as a check or a migration reads them
        {"name": "read_tails", "op": "read", "lens": "1000*31,37", "tail": 65, "H": 4, "G": 4, "D": 128,
         "dtype": "float32", "page": 4096},
        # block bounds after a long prompt batch
        {"name": "bounds_build", "op": "bounds", "lens": "8192*7,5555", "new": 0, "block": 64, "H": 16, "G": 1,
         "D": 128, "page": 0},
        # the same kept up in a decode step: one new token a sequence
        {"name": "bounds_step", "op": "bounds", "lens": "1023*32,1024*31,65", "new": 1, "block": 64, "H": 16, "G": 1,
         "D": 128, "page": 0},
        # block choice in a decode step at context 8192
        {"name": "select_1p3b", "op": "select", "lens": "8192*64", "block": 64, "k": 16, "first": 1, "last": 1,
         "H": 16, "G": 1, "D": 128},
        # block choice over long contexts with KV heads shared by four query heads
        {"name": "select_long_gqa", "op": "select", "lens": "65536*4,50001", "block": 64, "k": 64, "first": 1,
         "last": 2, "H": 4, "G": 4, "D": 128},
        # a decode step at batch 64 and context 8192, 16 blocks of 64 keys per full query
        {"name": "attn_1p3b", "op": "attn", "lens": "8192*64", "block": 64, "k": 16, "w": 512, "H": 16, "G": 1,
         "D": 128, "p_skip": 0.15, "p_local": 0.45, "page": 0},
        # a decode step over long contexts, shared KV heads, paged, every query full
        {"name": "attn_long_gqa", "op": "attn", "lens": "65536*4,50001", "block": 64, "k": 64, "w": 0, "H": 4, "G": 4,
         "D": 128, "p_skip": 0.0, "p_local": 0.0, "page": 65536},
        # one short sequence: latency
        {"name": "attn_single", "op": "attn", "lens": "777", "block": 32, "k": 5, "w": 100, "H": 4, "G": 2, "D": 64,
         "p_skip": 0.1, "p_local": 0.2, "page": 0},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("rope", "read", "bounds", "select", "attn"))
    d = rng.choice((64, 128))
    g = rng.choice((1, 1, 2, 3, 4, 8))
    h = log(1, 16) if g == 1 else log(1, 8)
    page = rng.choice((0, 0, 4096, 65536))
    batch = log(1, 64)
    most = {"rope": 16000, "read": 16000, "bounds": 60000, "select": 200000, "attn": 200000}[op]
    top = max(2, min(8192 if op in ("rope", "read") else 65536, most // batch))
    lens = ",".join(str(log(1, top)) for _ in range(batch))
    case = {"op": op, "lens": lens, "H": h, "G": g, "D": d}
    if op == "rope":
        step = rng.random() < 0.4
        case |= {"lens": ",".join(str(rng.choice((1, 1, 1, 2))) for _ in range(batch)) if step else lens,
                 "before": log(1, 700) if step else rng.choice((0, 0, 33)), "rot": 16 * rng.randint(1, d // 16),
                 "interleaved": rng.random() < 0.5, "fused": rng.random() < 0.5, "page": page}
    elif op == "read":
        case |= {"tail": log(1, 8192), "dtype": rng.choice(("float16", "bfloat16", "float32")), "page": page}
    else:
        case["block"] = rng.choice((16, 32, 64, 128))
        k = max(2, min(64, 4096 // case["block"], log(2, 64)))
        if op == "bounds":
            case |= {"new": rng.choice((0, 1, 1, log(1, 300))), "page": page}
        elif op == "select":
            case |= {"k": k, "first": rng.randint(0, 1), "last": rng.randint(0, 1)}
        else:
            case |= {"k": k, "w": log(1, 1024), "p_skip": rng.choice((0.0, 0.15)),
                     "p_local": rng.choice((0.0, 0.45)), "page": page}
    return case


def work(case):
    lens, H, G, D = _lens(case), case["H"], case["G"], case["D"]
    B, HQ = len(lens), H * G
    record, entry = MEAN_WIDTH * D / 4, 20              # bytes of a token and head: codes; scale, zero, offset
    op = case["op"]
    if op == "rope":
        n = sum(lens)
        return {"bytes": n * (2 * HQ * D * 2 + 4 * H * D * 2 + H * (1 + record + entry) + case["rot"] * 4),
                "flops": n * ((HQ + H) * case["rot"] * 3 + H * 2 * D * 8)}
    if op == "read":
        n = sum(min(L, case["tail"]) for L in lens)
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": n * H * (record + entry + 2 * D * size), "flops": n * H * 4 * D}
    bs = case["block"]
    if op == "bounds":
        starts = [(L - min(L, case["new"] or L)) // bs * bs for L in lens]
        keys = sum(L - a for L, a in zip(lens, starts))
        blocks = sum(-(-L // bs) - a // bs for L, a in zip(lens, starts))
        return {"bytes": H * (keys * (record / 2 + 12) + blocks * 4 * D), "flops": keys * H * D * 4}
    if op == "select":
        blocks = sum(-(-L // bs) for L in lens)
        both = 2 - 2.0 ** (1 - G)                       # of a channel's two bounds, those some query's sign needs
        return {"bytes": blocks * H * (D * 2 * both + 4) + B * HQ * D * 2 + B * H * case["k"] * 4,
                "flops": blocks * HQ * D * 2}
    p_full = 1 - case["p_skip"] - case["p_local"]
    full = sum(min(L, case["k"] * bs) for L in lens)
    local = sum(min(L, case["w"] + 1) for L in lens)
    any_full, any_local = 1 - (1 - p_full) ** G, 1 - (1 - case["p_local"]) ** G
    return {"bytes": H * (full * any_full + local * any_local) * (record + entry) + B * HQ * D * 6,
            "flops": HQ * 4 * D * (full * p_full + local * case["p_local"])}


# ---------------------------------------------------------------------------- inputs

def _rows(n, H, D, g):
    """fp16 normal rows with a few stronger channels."""
    x = torch.randn((n, H, D), generator=g, device="cuda", dtype=torch.float16)
    strong = torch.where(torch.rand((H, D), generator=g, device="cuda") < 0.02, 4.0, 1.0)
    return x.mul_(strong.half())


def _widths(n, H, g):
    cum = torch.tensor(WIDTHS_P, device="cuda").cumsum(0)[:-1]
    pick = torch.bucketize(torch.rand((n, H), generator=g, device="cuda"), cum)
    return torch.tensor(WIDTHS, dtype=torch.uint8, device="cuda")[pick]


def _cu(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)


def _quantize(x, bits):
    """Asymmetric min/max codes of each row: codes (fp16 bits where the width is 16), scale, zero."""
    x32, b = x.float(), bits.float()[..., None]
    lo, hi = x32.amin(-1, keepdim=True), x32.amax(-1, keepdim=True)
    native = b == 16
    s = torch.where(native, 1.0, (hi - lo) / (torch.exp2(b) - 1))
    z = torch.where(native, 0.0, lo + 0.0)
    code = torch.where(s == 0, 0.0, ((x32 - z) / s).round()).clamp(0, 255)
    return torch.where(native, x.view(torch.int16), code.to(torch.int16)), s[..., 0], z[..., 0]


def _values(codes, s, z, bits):
    """What stored codes stand for, fp32."""
    return torch.where(bits[..., None] == 16, codes.view(torch.float16).float(),
                       codes.float() * s[..., None] + z[..., None])


def _table(n, rot, device="cuda"):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(n, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat((a.cos(), a.sin()), -1).float()


def _cache(case, lens, k, v, bits, cu):
    """The library's cache of `lens` tokens a sequence, with k and v written at their widths."""
    from mixed_precision_kv_write_b200 import kvq
    H, D, page = k.shape[1], k.shape[2], case.get("page", 0)
    pages = len(lens) * H * (max(lens) * 4 * D // page + 2) if page else 0
    cache = kvq.KVQCache(len(lens), H, D, [max(1, L) for L in lens], query_group=case["G"], page_bytes=page,
                         pool_pages=pages)
    if k.shape[0]:
        kvq.kvq_write(k, v, bits, cu, cache)
    return cache


def _held(case, lens, k, v, bits, cu):
    """A filled cache as a program has it in hand: the library's, or dense codes with scales and zeros."""
    if own:
        return {"cache": _cache(case, lens, k, v, bits, cu)}
    parts = [[*_quantize(k[a:a + 8192], bits[a:a + 8192]), *_quantize(v[a:a + 8192], bits[a:a + 8192])]
             for a in range(0, k.shape[0], 8192)]
    kc, ks, kz, vc, vs, vz = (torch.cat(p) for p in zip(*parts))
    return {"kc": kc, "ks": ks, "kz": kz, "vc": vc, "vs": vs, "vz": vz, "bits": bits}


def _raw(case, seed):
    """The case's inputs from the seed alone, before anything is stored."""
    lens, H, G, D = _lens(case), case["H"], case["G"], case["D"]
    B, HQ, op = len(lens), H * G, case["op"]
    g = torch.Generator("cuda").manual_seed(seed)
    raw = {"lens": lens, "len": torch.tensor(lens, device="cuda"), "cu": _cu(lens)}
    if op == "rope":
        n = sum(lens)
        if case["fused"]:                               # q, k, v are column ranges of one projection's rows
            qkv = _rows(n, HQ + 2 * H, D, g)
            raw |= {"q": qkv[:, :HQ], "k": qkv[:, HQ:HQ + H], "v": qkv[:, HQ + H:]}
        else:
            raw |= {"q": _rows(n, HQ, D, g), "k": _rows(n, H, D, g), "v": _rows(n, H, D, g)}
        raw |= {"bits": _widths(n, H, g), "table": _table(case["before"] + max(lens), case["rot"])}
        return raw
    if op == "select":
        nt = -(-(-(-max(lens) // case["block"])) // TILE)
        mid = 0.5 * torch.randn((B, H, nt, 1, D, TILE), generator=g, device="cuda")
        rad = (2.3 + 0.4 * torch.randn((B, H, nt, 1, D, TILE), generator=g, device="cuda")).abs()
        raw |= {"bounds": torch.cat((mid - rad, mid + rad), 3).half()}
    else:
        n = sum(lens)
        raw |= {"k": _rows(n, H, D, g), "v": _rows(n, H, D, g), "bits": _widths(n, H, g)}
    if op in ("select", "attn"):
        raw["q"] = _rows(B, HQ, D, g)
        u = torch.rand((B, HQ), generator=g, device="cuda")
        p0, p1 = case.get("p_skip", 0.1), case.get("p_local", 0.2)
        raw["modes"] = (FULL - (u < p0 + p1).to(torch.uint8) - (u < p0).to(torch.uint8)).to(torch.uint8)
    if op == "attn":                                    # distinct blocks in ascending order, the last one among them
        k, nb = case["k"], -(-raw["len"] // case["block"])
        most = max(k, int(nb.max()))
        at = torch.arange(most, device="cuda")
        rank = torch.rand((B, H, most), generator=g, device="cuda")
        rank = torch.where(at == nb[:, None, None] - 1, 2.0, torch.where(at < nb[:, None, None], rank, -1.0))
        top, ids = rank.topk(k, -1)
        ids = torch.where(top >= 0, ids, most).sort(-1).values
        raw["ids"] = torch.where(ids < most, ids, -1).to(torch.int32)
    return raw


def prepare(case, seed):
    raw = _raw(case, seed)
    lens, H, D, op = raw["lens"], case["H"], case["D"], case["op"]
    st = {"case": case, **{n: raw[n] for n in ("lens", "len", "cu")}}
    if op == "rope":
        st |= {n: raw[n] for n in ("q", "k", "v", "bits", "table")}
        st["pos"] = torch.full((len(lens),), case["before"], dtype=torch.int32, device="cuda")
        if own:
            g = torch.Generator("cuda").manual_seed(seed + 1000003)
            pre = [case["before"]] * len(lens)
            n = sum(pre)
            four = torch.full((n, H), 4, dtype=torch.uint8, device="cuda")
            st["cache"] = _cache(case, [case["before"] + L for L in lens], _rows(n, H, D, g), _rows(n, H, D, g), four,
                                 _cu(pre))
        return st
    if op == "select":
        st |= {n: raw[n] for n in ("q", "modes", "bounds")}
        if own:                                         # only the lengths matter: one row written everywhere
            two = torch.full((sum(lens), H), 2, dtype=torch.uint8, device="cuda")
            zero = torch.zeros((sum(lens), H, D), dtype=torch.float16, device="cuda")
            st["cache"] = _cache(case, lens, zero, zero, two, raw["cu"])
        return st
    st |= _held(case, lens, raw["k"], raw["v"], raw["bits"], raw["cu"])
    if op == "read":
        tails = [min(L, case["tail"]) for L in lens]
        st |= {"n": sum(tails), "cu_tail": _cu(tails)}
        if not own:
            st["rows"] = torch.cat([torch.arange(L - t, L, device="cuda") + int(c)
                                    for L, t, c in zip(lens, tails, raw["cu"][:-1].tolist())])
    elif op == "bounds":
        nt = -(-(-(-max(lens) // case["block"])) // TILE)
        st["bounds"] = torch.zeros((len(lens), H, nt, 2, D, TILE), dtype=torch.float16, device="cuda")
        new = [min(L, case["new"] or L) for L in lens]
        st["cu_new"] = _cu(new)
        st["touched"] = max(-(-L // case["block"]) - (L - n) // case["block"] for L, n in zip(lens, new))
    else:
        st |= {n: raw[n] for n in ("q", "modes", "ids")}
    return st


# ---------------------------------------------------------------------------- one pass

def _rotate(x, rows, rot, interleaved):
    """x with its first `rot` channels rotated; rows holds each token's cosines, then its sines."""
    x32 = x[..., :rot].float()
    c, s = rows[:, None, :rot // 2], rows[:, None, rot // 2:]
    a, b = (x32[..., 0::2], x32[..., 1::2]) if interleaved else (x32[..., :rot // 2], x32[..., rot // 2:])
    ra, rb = a * c - b * s, b * c + a * s
    y = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((y.half(), x[..., rot:]), -1)


def _block_tokens(st, blocks):
    """Token rows of blocks [B, ...]: row indices (clamped) and which of them exist."""
    bs, dims = st["case"]["block"], (slice(None),) + (None,) * blocks.dim()
    j = blocks[..., None].long() * bs + torch.arange(bs, device="cuda")
    there = (blocks[..., None] >= 0) & (j < st["len"][dims])
    return torch.where(there, j + st["cu"][:-1].long()[dims], 0), there


def _plain_rope(st):
    case = st["case"]
    n = st["k"].shape[0]
    at = torch.arange(n, device="cuda")
    seq = torch.searchsorted(st["cu"][1:].contiguous(), at, right=True)
    rows = st["table"][st["pos"][seq].long() + at - st["cu"][seq]]
    k = _rotate(st["k"], rows, case["rot"], case["interleaved"])
    return {"q": _rotate(st["q"], rows, case["rot"], case["interleaved"]),
            "k": _values(*_quantize(k, st["bits"]), st["bits"]).half(),
            "v": _values(*_quantize(st["v"].contiguous(), st["bits"]), st["bits"]).half()}


def _plain_read(st):
    r = st["rows"]
    dt = getattr(torch, st["case"]["dtype"])
    return {"k": _values(st["kc"][r], st["ks"][r], st["kz"][r], st["bits"][r]).to(dt),
            "v": _values(st["vc"][r], st["vs"][r], st["vz"][r], st["bits"][r]).to(dt)}


def _plain_bounds(st):
    bs = st["case"]["block"]
    new = st["cu_new"].diff()
    blocks = ((st["len"] - new) // bs)[:, None] + torch.arange(st["touched"], device="cuda")
    tok, there = _block_tokens(st, blocks)
    x = _values(st["kc"][tok], st["ks"][tok], st["kz"][tok], st["bits"][tok])          # [B, m, bs, H, D]
    there = there[..., None, None]
    lo, hi = x.masked_fill(~there, math.inf).amin(2).half(), x.masked_fill(~there, -math.inf).amax(2).half()
    s, m = (blocks * bs < st["len"][:, None]).nonzero(as_tuple=True)
    b = blocks[s, m]
    st["bounds"][s, :, b // TILE, 0, :, b % TILE] = lo[s, m]
    st["bounds"][s, :, b // TILE, 1, :, b % TILE] = hi[s, m]
    return {"bounds": st["bounds"]}


def _plain_select(st):
    case = st["case"]
    B, H, nt, _, D, _ = st["bounds"].shape
    G, k = case["G"], case["k"]
    # sums in 64 bits: two blocks' scores can lie next to one another, and the choice is exact
    q = st["q"].view(B, H, G, 1, D, 1).double()
    lo, hi = st["bounds"][:, :, None, :, 0].double(), st["bounds"][:, :, None, :, 1].double()
    score = torch.maximum(q * lo, q * hi).sum(-2).flatten(-2)                          # [B, H, G, nt * TILE]
    full = (st["modes"] == FULL).view(B, H, G)
    at = torch.arange(nt * TILE, device="cuda")
    nb = (-(-st["len"] // case["block"]))[:, None, None]
    score = score.masked_fill(~full[..., None], -math.inf).amax(2).float().masked_fill(at >= nb, -math.inf)
    forced = (at < nb) & ((at < case["first"]) | (at >= nb - case["last"]))
    ids = score.masked_fill(forced, math.inf).sort(dim=-1, descending=True, stable=True).indices[..., :k]
    taken = (ids < nb) & full.any(-1)[..., None]
    ids = torch.where(taken, ids, nt * TILE).sort(-1).values
    ids = torch.where(ids < nt * TILE, ids, -1).to(torch.int32)
    if ids.shape[-1] < k:
        ids = torch.cat((ids, ids.new_full((B, H, k - ids.shape[-1]), -1)), -1)
    return {"ids": ids, "scores": score}


def _plain_attn(st):
    case = st["case"]
    B, H, _ = st["ids"].shape
    G, D = case["G"], case["D"]
    tok, there = _block_tokens(st, st["ids"])                                          # [B, H, k, bs]
    w = min(case["w"] + 1, max(st["lens"]))
    j = st["len"][:, None] - w + torch.arange(w, device="cuda")                        # the local window
    near = torch.where(j >= 0, j + st["cu"][:-1, None], 0)[:, None].expand(B, H, w)
    tok = torch.cat((tok.flatten(2), near), -1)
    head = torch.arange(H, device="cuda")[:, None]
    kv = [_values(st[c][tok, head], st[s][tok, head], st[z][tok, head], st["bits"][tok, head])
          for c, s, z in (("kc", "ks", "kz"), ("vc", "vs", "vz"))]
    mode = st["modes"].view(B, H, G, 1)
    seen = torch.cat((there.flatten(2)[:, :, None] & (mode == FULL),
                      (j >= 0)[:, None, None] & (mode == LOCAL)), -1)
    q = st["q"].view(B, H, G, D).float()
    a = (torch.matmul(q, kv[0].transpose(-1, -2)) / math.sqrt(D)).masked_fill(~seen, -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(top == -math.inf, 0.0, top))
    out = torch.matmul(p, kv[1]) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return {"out": out.view(B, H * G, D)}


def _own_run(st):
    from mixed_precision_kv_write_b200 import kvq
    case = st["case"]
    op = case["op"]
    if op == "rope":
        q = kvq.kvq_write_rope(st["q"], st["k"], st["v"], st["bits"], st["cu"], st["cache"], st["table"],
                               interleaved=case["interleaved"], positions=st["pos"])
        k, v = kvq.kvq_read(st["cache"], st["cu"], st["k"].shape[0])
        return {"q": q, "k": k, "v": v}
    if op == "read":
        k, v = kvq.kvq_read(st["cache"], st["cu_tail"], st["n"], dtype=getattr(torch, case["dtype"]))
        return {"k": k, "v": v}
    if op == "bounds":
        return {"bounds": kvq.block_bounds(st["cache"], case["block"], st["cu_new"] if case["new"] else None,
                                           out=st["bounds"])}
    if op == "select":
        ids, scores = kvq.select_blocks(st["q"], st["cache"], st["bounds"], case["block"], case["k"], st["modes"],
                                        first=case["first"], last=case["last"])
        return {"ids": ids, "scores": scores}
    return {"out": kvq.routed_attn_decode_blocks(st["q"], st["cache"], st["ids"], case["block"], st["modes"],
                                                 case["w"])}


def run(state):
    if own:
        return _own_run(state)
    return {"rope": _plain_rope, "read": _plain_read, "bounds": _plain_bounds, "select": _plain_select,
            "attn": _plain_attn}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- 64 bits

def _exact_store(x, bits):
    """Eq.-4 values of fp16 rows in 64 bits."""
    x, top = x.double(), (2.0 ** bits.double() - 1)[..., None]
    z = x.min(-1, keepdim=True).values
    s = (x.max(-1, keepdim=True).values - z) / top
    y = torch.round((x - z) / torch.where(s > 0, s, 1.0)) * s + z
    return torch.where(bits[..., None] == 16, x, y)


def _exact_held(raw, name, rows):
    """What the stored codes of k or v stand for in 64 bits: codes, fp32 scale and fp32 zero are given."""
    c, s, z = _quantize(raw[name][rows], raw["bits"][rows])
    native = (raw["bits"][rows] == 16)[..., None]
    return torch.where(native, c.view(torch.float16).double(), c.double() * s.double()[..., None] + z.double()[..., None])


def exact(case, seed):
    raw = _raw(case, seed)
    lens, H, G, D, op = raw["lens"], case["H"], case["G"], case["D"], case["op"]
    starts = raw["cu"].tolist()
    if op == "rope":
        at = torch.cat([torch.arange(case["before"], case["before"] + L, device="cuda") for L in lens])
        t = raw["table"].double()[at]
        r, half = case["rot"], case["rot"] // 2
        first = torch.arange(half, device="cuda")
        first, second = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + half)
        turned = []
        for x in (raw["q"], raw["k"]):
            y, cs, sn = x.double(), t[:, None, :half], t[:, None, half:r]
            a, b = y[..., first], y[..., second]
            y[..., first], y[..., second] = cs * a - sn * b, sn * a + cs * b
            turned.append(y)
        return {"q": turned[0], "k": _exact_store(turned[1].half(), raw["bits"]), "v": _exact_store(raw["v"], raw["bits"])}
    if op == "read":
        rows = torch.cat([torch.arange(c + L - min(L, case["tail"]), c + L, device="cuda") for L, c in zip(lens, starts)])
        return {"k": _exact_held(raw, "k", rows), "v": _exact_held(raw, "v", rows)}
    bs = case["block"]
    if op == "bounds":
        nt = -(-(-(-max(lens) // bs)) // TILE)
        out = torch.zeros((len(lens), H, nt, 2, D, TILE), dtype=torch.float64, device="cuda")
        for s, L in enumerate(lens):
            b0 = (L - min(L, case["new"] or L)) // bs
            x = _exact_held(raw, "k", slice(starts[s] + b0 * bs, starts[s] + L))
            pad = -x.shape[0] % bs                      # the last block's missing keys repeat its last one
            x = torch.cat((x, x[-1:].expand(pad, H, D))).view(-1, bs, H, D)
            b = torch.arange(b0, b0 + x.shape[0], device="cuda")
            out[s, :, b // TILE, 0, :, b % TILE] = x.min(1).values
            out[s, :, b // TILE, 1, :, b % TILE] = x.max(1).values
        return {"bounds": out}
    if op == "select":
        q = raw["q"].double().view(len(lens), H, G, D)
        up, down = q.clamp(min=0), q.clamp(max=0)
        score = torch.einsum("bhgd,bhtdn->bhgtn", up, raw["bounds"][:, :, :, 1].double()) + \
            torch.einsum("bhgd,bhtdn->bhgtn", down, raw["bounds"][:, :, :, 0].double())
        score[(raw["modes"] != FULL).view(len(lens), H, G)] = -math.inf
        score = score.max(2).values.flatten(2)
        for s, L in enumerate(lens):
            score[s, :, -(-L // bs):] = -math.inf
        return {"ids": None, "scores": score}
    out = torch.zeros((len(lens), H * G, D), dtype=torch.float64, device="cuda")
    offs = torch.arange(bs, device="cuda")
    modes = raw["modes"].tolist()
    for s, L in enumerate(lens):
        near = torch.arange(max(0, L - 1 - case["w"]), L, device="cuda")
        used = (raw["ids"][s].clamp(min=0)[..., None] * bs + offs).flatten(1)           # [H, k * bs]
        there = ((raw["ids"][s] >= 0)[..., None].expand(-1, -1, bs).flatten(1)) & (used < L)
        rows, back = torch.cat((used[there], near)).unique(return_inverse=True)
        kd, vd = (_exact_held(raw, n, starts[s] + rows) for n in ("k", "v"))
        n_there = there.sum(-1).cumsum(0).tolist()
        for h in range(H):
            picked = back[(n_there[h - 1] if h else 0):n_there[h]]
            for i in range(h * G, (h + 1) * G):
                keys = {SKIP: back[:0], LOCAL: back[n_there[-1]:], FULL: picked}[modes[s][i]]
                if keys.numel():
                    a = kd[keys, h] @ raw["q"][s, i].double() / math.sqrt(D)
                    out[s, i] = torch.softmax(a, 0) @ vd[keys, h]
    return {"out": out}
