"""Rotary positions, the life of a cache's pages, and decode over a shared prefix, as cases to be
measured.

Three operators around Native Sparse Attention's training step and its paged decode:

  rope    queries and keys turned by their positions (half or interleaved pairs, the whole head or
          its first dimensions, frequencies scaled for long contexts), and the gradient of that
  pages   pages of a cache forked (n continuations of one request share its full pages and copy
          the last), freed, compacted, and their bytes copied
  shared  one new token per sequence attending to everything cached in 4-bit pages, where the
          sequences of a group share a prefix of pages

`run` computes them in elementary torch operations in 32 bits (angles in 64), or, where `own` is
true, through block_sparse_attention_nsa_gb300.  `exact` computes them in 64 bits from the definition.

Pages.  block_table int32 [B, W]: request b's tokens lie in the pages of its first
ceil(seq_lens[b] / P) entries.  shares int32 [num_pages]: how many rows name a page beyond the
first.  free_pages int32 [F], from entry free_head[0] on, are the pages that nobody has.
  free     a row's pages lose one owner each; those that had no other go to the free list, just
           before its head, in ascending order; the row's entries become -1, its length 0
  fork     row children[i] gets row parents[i]'s full pages (shared) and, where the last page is
           partly full, a page of the free list in its place; (copy_src, copy_dst)[i] is what has
           to be copied, -1 where nothing has
  compact  with n pages in use, those of them at n or above move, in ascending order, to the
           unused ones below n, ascending; the free list then is n ... num_pages - 1, at its end
The 4-bit pool is uint8 [num_pages, h_k, P * (d + d / 8)]; the record of a (page, KV head) is P / 32
tiles of 32 tokens:
  K codes [32, d / 2], V codes [32, d / 2], then fp16 [4, 32, d / 64]: K scale, K zero,
  V scale, V zero.
A row's codes are 32-bit words; the word at index j * (d / 64) + i holds dimensions
64 i + 8 j ... + 7, four bits each, lowest first.  A code c stands for c * scale + zero.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # q and k of one decode step, far into long sequences; column ranges of a fused projection
        {"name": "rope_step_64", "op": "rope", "tokens": 64, "hq": 16, "hk": 4, "d": 128, "rot": 128,
         "inter": 0, "dtype": "bf16", "fused": 1, "far": 1, "seqs": 64, "scaling": "ramp",
         "grad": 0, "salt": 1},
        # a packed ragged batch with small heads, half of each turned, in pairs of neighbours
        {"name": "rope_ragged_9k", "op": "rope", "tokens": 9001, "hq": 6, "hk": 3, "d": 64,
         "rot": 32, "inter": 1, "dtype": "fp16", "fused": 0, "far": 0, "seqs": 11,
         "scaling": "linear", "grad": 1, "salt": 2},
        # a training step of one 64K sequence: q and k, and their gradients
        {"name": "rope_train_64k", "op": "rope", "tokens": 65536, "hq": 16, "hk": 4, "d": 128,
         "rot": 128, "inter": 0, "dtype": "bf16", "fused": 0, "far": 0, "seqs": 1,
         "scaling": "none", "grad": 1, "salt": 3},
        # a step of a small beam search: four requests' beams are dropped and forked again
        {"name": "beams_4x4", "op": "beams", "parents": 4, "each": 4, "ctx": 517, "heads": 4,
         "d": 128, "page": 64, "salt": 4},
        # 64 prompts of up to 8K tokens with eight continuations each
        {"name": "beams_64x8", "op": "beams", "parents": 64, "each": 8, "ctx": 8192, "heads": 4,
         "d": 128, "page": 64, "salt": 5},
        # continuous batching: a third of 1000 requests ends, as many prompts are admitted
        {"name": "admit_1000", "op": "admit", "seqs": 1000, "gone": 333, "ctx": 4096, "page": 32,
         "salt": 6},
        # a pool of about 30K pages, three quarters full, is compacted: tables, list and bytes
        {"name": "compact_30k", "op": "compact", "seqs": 500, "ctx": 32768, "heads": 4, "d": 128,
         "page": 64, "fill": 0.75, "salt": 7},
        # four samples of one short prompt
        {"name": "shared_4x517", "op": "shared", "groups": 1, "seqs": 4, "prefix": 517, "suffix": 60,
         "heads": 4, "g": 4, "d": 128, "page": 64, "dtype": "bf16", "salt": 8},
        # a served batch behind one system prompt of 8K tokens
        {"name": "shared_64x8k", "op": "shared", "groups": 1, "seqs": 64, "prefix": 8192,
         "suffix": 1000, "heads": 4, "g": 4, "d": 128, "page": 64, "dtype": "bf16", "salt": 9},
        # several prompts of different length, uneven groups, small heads, fp16
        {"name": "shared_5_groups_d64", "op": "shared", "groups": 5, "seqs": 100, "prefix": 5000,
         "suffix": 300, "heads": 8, "g": 3, "d": 64, "page": 32, "dtype": "fp16", "salt": 10},
        # a large batch over one 32K document
        {"name": "shared_256x32k", "op": "shared", "groups": 1, "seqs": 256, "prefix": 32768,
         "suffix": 500, "heads": 8, "g": 4, "d": 128, "page": 64, "dtype": "bf16", "salt": 11},
        # two documents, eight query heads to a KV head, fp16, lengths that end inside pages
        {"name": "shared_2x16k_g8", "op": "shared", "groups": 2, "seqs": 96, "prefix": 16001,
         "suffix": 700, "heads": 4, "g": 8, "d": 128, "page": 128, "dtype": "fp16", "salt": 12},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "rope", "beams", "admit", "compact", "shared", "shared", "shared"])
    page = rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    salt = rng.randrange(1 << 30)
    d = rng.choice([64, 128])
    if op == "rope":
        hk = rng.choice([1, 2, 3, 4, 8])
        hq = hk * rng.choice([1, 2, 3, 4, 7])
        tokens = _log_int(rng, 1, min(65536, 1000000 // (hq + hk)))
        return {"op": op, "tokens": tokens, "hq": hq, "hk": hk, "d": d,
                "rot": rng.choice([16, 32, d // 2, d, d]), "inter": rng.choice([0, 1]),
                "dtype": dtype, "fused": rng.choice([0, 1]), "far": rng.choice([0, 1]),
                "seqs": _log_int(rng, 1, min(tokens, 300)),
                "scaling": rng.choice(["none", "linear", "base", "ramp"]),
                "grad": rng.choice([0, 1]), "salt": salt}
    if op == "beams":
        parents = _log_int(rng, 1, 64)
        return {"op": op, "parents": parents, "each": _log_int(rng, 1, 8), "ctx": _log_int(rng, 1, 8192),
                "heads": rng.choice([1, 2, 3, 4]), "d": d, "page": page, "salt": salt}
    if op == "admit":
        seqs = _log_int(rng, 2, 1000)
        return {"op": op, "seqs": seqs, "gone": _log_int(rng, 1, seqs), "ctx": _log_int(rng, 1, 4096),
                "page": page, "salt": salt}
    if op == "compact":
        seqs = _log_int(rng, 1, 200)
        return {"op": op, "seqs": seqs, "ctx": _log_int(rng, 1, 8192), "heads": rng.choice([1, 2, 3, 4]),
                "d": d, "page": max(page, 64), "fill": rng.choice([0.3, 0.6, 0.9]), "salt": salt}
    seqs = _log_int(rng, 2, 256)
    heads, g = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16])
    most = max(64, min(32768, 250000000 // (seqs * heads * g)))
    return {"op": op, "groups": rng.randint(1, min(5, seqs)), "seqs": seqs,
            "prefix": _log_int(rng, 1, most), "suffix": _log_int(rng, 1, 1000), "heads": heads, "g": g,
            "d": d, "page": page, "dtype": dtype, "salt": salt}


def _ceil(a, b):
    return -(-a // b)


def _spread(name, salt, n, hi):
    """n whole numbers of [1, hi], spread over their logarithm, one of them hi."""
    rng = random.Random("%s %d" % (name, salt))
    out = [_log_int(rng, 1, hi) for _ in range(n)]
    out[rng.randrange(n)] = hi
    return out


def _cuts(name, salt, n, total):
    """total split into n uneven parts of at least one."""
    rng = random.Random("%s %d" % (name, salt))
    at = sorted(rng.sample(range(1, total), n - 1))
    return [b - a for a, b in zip([0] + at, at + [total])]


def _shape_shared(case):
    """Sequences of each group, its prefix, and every sequence's length (its new token included)."""
    sizes = _cuts("groups", case["salt"], case["groups"], case["seqs"])
    prefixes = _spread("prefix", case["salt"], case["groups"], case["prefix"])
    own_lens = _spread("suffix", case["salt"], case["seqs"], case["suffix"])
    lens, at = [], 0
    for n, p in zip(sizes, prefixes):
        lens += [p + x for x in own_lens[at:at + n]]
        at += n
    return sizes, prefixes, lens


def work(case):
    op = case["op"]
    if op == "rope":
        values = case["tokens"] * (case["hq"] + case["hk"]) * case["d"]
        turned = case["tokens"] * (case["hq"] + case["hk"]) * case["rot"]
        times = 1 + case["grad"]
        return {"bytes": times * (4 * values + 4 * case["tokens"]), "flops": times * 3 * turned}
    if op == "admit":
        lens, gone = _spread("ctx", case["salt"], case["seqs"], case["ctx"]), _gone(case)
        pages = sum(_ceil(lens[b], case["page"]) for b in gone)
        slots = sum(lens[b] for b in gone)
        # freed: entry, shares, list; admitted: list, entry; the slots; lengths in and out
        return {"bytes": 4 * (7 * pages + slots + 4 * case["seqs"]), "flops": 0}
    page = case["page"]
    if op == "beams":
        lens = _spread("ctx", case["salt"], case["parents"], case["ctx"])
        full = case["each"] * sum(n // page for n in lens)
        part = case["each"] * sum(1 for n in lens if n % page)
        record = case["heads"] * page * (case["d"] + case["d"] // 8)
        # freed: entry, shares (read and written); forked: entry read and written, shares
        return {"bytes": 4 * (8 * full + 12 * part) + 2 * part * record, "flops": 0}
    if op == "compact":
        lens = _spread("ctx", case["salt"], case["seqs"], case["ctx"])
        pages = sum(_ceil(n, page) for n in lens)
        total = int(pages / case["fill"]) + 3
        moved = round(pages * (total - pages) / total)
        record = case["heads"] * page * (case["d"] + case["d"] // 8)
        return {"bytes": 4 * (2 * pages + 3 * total) + 2 * moved * record, "flops": 0}
    sizes, prefixes, lens = _shape_shared(case)
    d, heads, g = case["d"], case["heads"], case["g"]
    stored = sum(prefixes) + sum(lens) - sum(n * p for n, p in zip(sizes, prefixes))
    rows = case["seqs"] * heads * g
    return {"bytes": stored * heads * (d + d // 8) + rows * (4 * d + 4),
            "flops": 4 * d * sum(lens) * heads * g}


def _gone(case):
    rng = random.Random("gone %d" % case["salt"])
    return sorted(rng.sample(range(case["seqs"]), case["gone"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


SCALING = {"none": {}, "linear": {"factor": 8.0}, "base": {"factor": 4.0},
           "ramp": {"factor": 16.0, "trained": 8192, "low": 1.0, "high": 32.0}}


def _frequencies(rot, scaling):
    """Radians per position of each pair, fp64 [rot / 2], and the factor on both outputs."""
    how = SCALING[scaling]
    base = 10000.0
    if scaling == "base":
        base = base * how["factor"] ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        f = f / how["factor"]
    if scaling == "ramp":
        turns = how["trained"] * f / (2 * math.pi)
        keep = ((turns - how["low"]) / (how["high"] - how["low"])).clamp(0, 1)
        f = f * keep + f / how["factor"] * (1 - keep)
    return f.cuda(), 0.1 * math.log(how["factor"]) + 1 if scaling == "ramp" else 1.0


def _prepare_rope(case, seed):
    gen = _gen(seed)
    s = dict(case)
    n, hq, hk, d, dt = case["tokens"], case["hq"], case["hk"], case["d"], DTYPES[case["dtype"]]
    if case["fused"]:                      # q, k and v side by side in one row
        row = torch.randn((n, hq + 2 * hk, d), generator=gen, device="cuda").to(dt)
        s["q"], s["k"] = row[:, :hq], row[:, hq:hq + hk]
    else:
        s["q"] = torch.randn((n, hq, d), generator=gen, device="cuda").to(dt)
        s["k"] = torch.randn((n, hk, d), generator=gen, device="cuda").to(dt)
    if case["grad"]:
        s["dq"] = torch.randn((n, hq, d), generator=gen, device="cuda").to(dt)
        s["dk"] = torch.randn((n, hk, d), generator=gen, device="cuda").to(dt)
        s["dq_in"], s["dk_in"] = torch.empty_like(s["dq"]), torch.empty_like(s["dk"])
    s["q_out"] = torch.empty((n, hq, d), dtype=dt, device="cuda")
    s["k_out"] = torch.empty((n, hk, d), dtype=dt, device="cuda")
    sizes = _cuts("tokens", case["salt"], case["seqs"], n)
    s["cu"] = _ints([0] + sizes).cumsum(0).int()
    # sequences that go on far behind their beginning, or begin here
    s["start"] = None
    if case["far"]:
        s["start"] = torch.randint(0, 1 << 20, (case["seqs"],), generator=gen, device="cuda").int()
    s["freq"], s["mscale"] = _frequencies(case["rot"], case["scaling"])
    if own:
        import block_sparse_attention_nsa_gb300 as nsa
        s["freqs"] = nsa.rope_freqs(case["rot"], 10000.0, scaling=case["scaling"],
                                    **SCALING[case["scaling"]])
    return s


def _fill_rows(lens, page, width, order):
    """Table rows of those lengths, with the pages of `order` in turn; -1 elsewhere."""
    per = [_ceil(n, page) for n in lens]
    per_t = torch.tensor(per, device="cuda")
    first = per_t.cumsum(0) - per_t
    col = torch.arange(width, device="cuda")
    at = (first.unsqueeze(1) + col).clamp(max=order.numel() - 1)
    return torch.where(col < per_t.unsqueeze(1), order[at], -1).int(), sum(per)


def _bytes(shape, gen):
    """Pages' records as bytes: what moves them does not look at them."""
    words = shape[:-1] + (shape[-1] // 8,)
    return torch.randint(-2 ** 62, 2 ** 62, words, generator=gen, device="cuda").view(torch.uint8)


def _prepare_beams(case, seed):
    gen = _gen(seed)
    s = dict(case)
    page, n, each = case["page"], case["parents"], case["each"]
    lens = _spread("ctx", case["salt"], n, case["ctx"])
    rows = n * (each + 1)
    width = _ceil(case["ctx"], page) + 2
    used = sum(_ceil(x, page) for x in lens)
    pages = used + n * each + 9
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    at = torch.randperm(rows, generator=gen, device="cuda")
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    table[at[:n]], _ = _fill_rows(lens, page, width, order)
    seq_lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    seq_lens[at[:n]] = _ints(lens)
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[used:] = order[used:].sort().values
    s.update(table=table, lens=seq_lens, free=free, head=_ints([used]),
             shares=torch.zeros(pages, dtype=torch.int32, device="cuda"),
             from_rows=at[:n].repeat_interleave(each).int(), to_rows=at[n:].int().contiguous(),
             copy_src=torch.empty(n * each, dtype=torch.int32, device="cuda"),
             copy_dst=torch.empty(n * each, dtype=torch.int32, device="cuda"),
             pool=_bytes((pages, case["heads"], page * (case["d"] + case["d"] // 8)), gen))
    _plain_fork(s)                        # the beams of the step before
    return s


def _prepare_admit(case, seed):
    gen = _gen(seed)
    s = dict(case)
    page = case["page"]
    lens, gone = _spread("ctx", case["salt"], case["seqs"], case["ctx"]), _gone(case)
    width = _ceil(case["ctx"], page) + 1
    used = sum(_ceil(x, page) for x in lens)
    pages = used + 50
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table, _ = _fill_rows(lens, page, width, order)
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[used:] = order[used:]
    new = [0] * case["seqs"]
    for b in gone:
        new[b] = lens[b]
    s.update(table=table, lens=_ints(lens), free=free, head=_ints([used]), new=_ints(new),
             shares=torch.zeros(pages, dtype=torch.int32, device="cuda"), gone_rows=_ints(gone),
             slots=torch.empty(sum(new), dtype=torch.int32, device="cuda"),
             cu_new=torch.empty(case["seqs"] + 1, dtype=torch.int32, device="cuda"))
    _plain_admit(s)                       # the pages of the rows that change lie in order
    return s


def _prepare_compact(case, seed):
    gen = _gen(seed)
    s = dict(case)
    page = case["page"]
    lens = _spread("ctx", case["salt"], case["seqs"], case["ctx"])
    used = sum(_ceil(x, page) for x in lens)
    pages = int(used / case["fill"]) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table, _ = _fill_rows(lens, page, _ceil(case["ctx"], page) + 1, order)
    shares = torch.zeros(pages, dtype=torch.int32, device="cuda")
    if case["seqs"] > 2:                  # the second request is a fork of the first at a page's end
        both = min(lens[0], lens[1]) // page
        table[1, :both] = table[0, :both]
        shares[table[0, :both].long()] = 1
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[used:] = order[used:]
    s.update(table=table, lens=_ints(lens), free=free, shares=shares,
             table_out=torch.empty_like(table), shares_out=torch.empty_like(shares),
             free_out=torch.full_like(free, -1), head=torch.empty(1, dtype=torch.int32, device="cuda"),
             copy_src=torch.empty(pages // 2 + 1, dtype=torch.int32, device="cuda"),
             copy_dst=torch.empty(pages // 2 + 1, dtype=torch.int32, device="cuda"),
             pool=_bytes((pages, case["heads"], page * (case["d"] + case["d"] // 8)), gen))
    return s


def _values(shape, gen):
    """Key- or value-like numbers in fp32: a few dimensions much larger than the rest, and
    dimensions of different size."""
    x = torch.randn(shape, generator=gen, device="cuda")
    d = shape[-1]
    x *= torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
    x[..., ::37] *= 4.0
    return x


def _quantise(x):
    """fp32 [..., d] -> codes uint8 [..., d], scale and zero fp16 [..., d / 64]."""
    g = x.unflatten(-1, (-1, 64))
    zero = g.amin(-1).half()
    scale = ((g.amax(-1) - zero.float()) / 15).half()
    c = ((g - zero.float().unsqueeze(-1)) / scale.float().unsqueeze(-1)).round().clamp(0, 15)
    return c.flatten(-2).to(torch.uint8), scale, zero


def _pack(codes):
    """Codes uint8 [..., d] -> the bytes of a stored row [..., d / 2]."""
    c = codes.unflatten(-1, (-1, 8, 4, 2))            # group, word, byte, nibble
    b = c[..., 0] | (c[..., 1] << 4)
    return b.transpose(-3, -2).flatten(-3)            # word, group, byte


def _records(k, v):
    """fp32 [pages, h, P, d] K and V -> the pool uint8 [pages, h, P * (d + d / 8)]."""
    def tiles(t):
        return t.unflatten(2, (-1, 32))
    kc, ks, kz = (tiles(t) for t in _quantise(k))
    vc, vs, vz = (tiles(t) for t in _quantise(v))
    par = torch.stack([ks, kz, vs, vz], 3).flatten(3).view(torch.uint8)
    return torch.cat([_pack(kc).flatten(3), _pack(vc).flatten(3), par], 3).flatten(2).contiguous()


def _prepare_shared(case, seed):
    gen = _gen(seed)
    s = dict(case)
    page, heads, d, b = case["page"], case["heads"], case["d"], case["seqs"]
    sizes, prefixes, lens = _shape_shared(case)
    pages = sum(p // page for p in prefixes) + 3
    at = 0
    for n, p in zip(sizes, prefixes):
        pages += sum(_ceil(x, page) - p // page for x in lens[at:at + n])
        at += n
    shape = (pages, heads, page, d)
    pool = _records(_values(shape, gen), _values(shape, gen))
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.full((b, _ceil(max(lens), page) + 1), -1, dtype=torch.int32, device="cuda")
    at, row = 0, 0
    for n, p in zip(sizes, prefixes):
        full, mine = p // page, lens[row:row + n]
        table[row:row + n, :full] = order[at:at + full]
        at += full
        width = max(_ceil(x, page) for x in mine) - full
        own_pages, used = _fill_rows([x - full * page for x in mine], page, width, order[at:])
        table[row:row + n, full:full + width] = own_pages
        if p % page:                      # the prefix' last page is each sequence's own copy
            pool[own_pages[1:, 0].long()] = pool[own_pages[:1, 0].long()]
        at += used
        row += n
    hq, dt = heads * case["g"], DTYPES[case["dtype"]]
    s.update(pool=pool, table=table.contiguous(), lens=_ints(lens), sizes=sizes, prefixes=prefixes,
             host_lens=lens, cu=_ints([0] + sizes).cumsum(0).int(), prefix_lens=_ints(prefixes),
             q=torch.randn((b, hq, d), generator=gen, device="cuda").to(dt), scale=d ** -0.5,
             out=torch.empty((b, hq, d), dtype=dt, device="cuda"),
             lse=torch.empty((hq, b), dtype=torch.float32, device="cuda"), workspace=None)
    if own:
        import block_sparse_attention_nsa_gb300 as nsa
        need = nsa.kv4_decode_shared_workspace_size(pages, page, heads, d, b, hq, len(sizes))
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    return {"rope": _prepare_rope, "beams": _prepare_beams, "admit": _prepare_admit,
            "compact": _prepare_compact, "shared": _prepare_shared}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _pairs(x, rot, inter):
    """The two halves of each pair of the first rot dimensions."""
    if inter:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _joined(a, b, rest, inter):
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def _plain_rope(s):
    n, rot, inter = s["tokens"], s["rot"], s["inter"]
    t = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    pos = t - s["cu"][seq]
    if s["start"] is not None:
        pos = pos + s["start"][seq]
    angle = pos.double().unsqueeze(1) * s["freq"]
    cos = (angle.cos() * s["mscale"]).float().unsqueeze(1)
    sin = (angle.sin() * s["mscale"]).float().unsqueeze(1)

    def turn(x, sin):
        a, b = _pairs(x.float(), rot, inter)
        return _joined(a * cos - b * sin, b * cos + a * sin, x[..., rot:].float(), inter).to(x.dtype)
    out = (turn(s["q"], sin), turn(s["k"], sin))
    if s["grad"]:
        out += (turn(s["dq"], -sin), turn(s["dk"], -sin))
    return out


def _count(pages, n):
    """How often each page occurs."""
    return torch.zeros(n, dtype=torch.int32, device="cuda").index_add_(
        0, pages, torch.ones_like(pages, dtype=torch.int32))


def _plain_free(s, rows):
    table, lens, page = s["table"], s["lens"], s["page"]
    rows = rows.long()
    mine = table[rows]
    have = (lens[rows] + page - 1) // page
    owned = torch.arange(table.shape[1], device="cuda") < have.unsqueeze(1)
    lost = _count(mine[owned].long(), s["shares"].numel())
    gone = lost > s["shares"]
    s["shares"].copy_(torch.where(gone, 0, s["shares"] - lost))
    freed = gone.nonzero().flatten()
    s["head"] -= freed.numel()
    s["free"][s["head"] + torch.arange(freed.numel(), device="cuda")] = freed.int()
    table[rows] = torch.where(owned, -1, mine)
    lens[rows] = 0


def _plain_fork(s):
    table, lens, page = s["table"], s["lens"], s["page"]
    src, dst = s["from_rows"].long(), s["to_rows"].long()
    n = lens[src]
    full, part = n // page, n % page > 0
    old = table[src]
    shared = torch.arange(table.shape[1], device="cuda") < full.unsqueeze(1)
    s["shares"] += _count(old[shared].long(), s["shares"].numel())
    rank = part.cumsum(0) - part.long()
    fresh = s["free"][(s["head"] + rank).clamp(max=s["free"].numel() - 1)]
    last = torch.arange(table.shape[1], device="cuda") == full.unsqueeze(1)
    rows = torch.where(shared, old, table[dst])
    table[dst] = torch.where(last & part.unsqueeze(1), fresh.unsqueeze(1), rows)
    s["copy_src"].copy_(torch.where(part, old.gather(1, full.long().unsqueeze(1)).squeeze(1), -1))
    s["copy_dst"].copy_(torch.where(part, fresh, -1))
    s["head"] += part.sum().int()
    lens[dst] = n


def _plain_copy(pool, src, dst):
    real = src >= 0
    pool[dst[real].long()] = pool[src[real].long()]


def _plain_admit(s):
    _plain_free(s, s["gone_rows"])
    page, lens, new = s["page"], s["lens"], s["new"]
    have, want = (lens + page - 1) // page, (lens + new + page - 1) // page
    need = want - have
    first = s["head"] + need.cumsum(0).int() - need
    col = torch.arange(s["table"].shape[1], device="cuda")
    opened = (col >= have.unsqueeze(1)) & (col < want.unsqueeze(1))
    at = (first.unsqueeze(1) + col - have.unsqueeze(1)).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(opened, s["free"][at], s["table"]))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)]).int()
    t = torch.arange(s["slots"].numel(), device="cuda")
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    pos = (lens[b] + t - cu[b]).long()
    s["slots"].copy_(s["table"][b, pos // page] * page + pos % page)
    s["cu_new"].copy_(cu)
    s["head"] += need.sum().int()
    s["lens"] += new


def _plain_compact(s):
    table, lens, page, total = s["table"], s["lens"], s["page"], s["shares"].numel()
    owned = torch.arange(table.shape[1], device="cuda") < ((lens + page - 1) // page).unsqueeze(1)
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    live[table[owned].long()] = True
    n = int(live.sum())
    src = live[n:].nonzero().flatten() + n
    dst = (~live[:n]).nonzero().flatten()
    to = torch.arange(total, device="cuda")
    to[src] = dst
    s["table_out"].copy_(torch.where(owned, to[table.clamp(min=0).long()].int(), table))
    shares = s["shares"].clone()
    shares[dst], shares[src] = s["shares"][src], 0
    s["shares_out"].copy_(shares)
    s["head"].fill_(s["free"].numel() - (total - n))
    s["free_out"][s["free"].numel() - (total - n):] = torch.arange(n, total, device="cuda").int()
    for name, x in (("copy_src", src), ("copy_dst", dst)):
        s[name].fill_(-1)
        s[name][:x.numel()] = x.int()


def _values_of(rec, d):
    """The K and V that records uint8 [..., tiles * tile bytes] stand for: fp32
    [..., tokens, d] each."""
    ng = d // 64
    t = rec.unflatten(-1, (-1, 32 * (d + d // 8)))
    codes = t[..., :32 * d].unflatten(-1, (2, 32, 8, ng, 4)).transpose(-3, -2)
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-3)         # [.., 2, 32, ng, 64]
    par = t[..., 32 * d:].contiguous().view(torch.float16).unflatten(-1, (2, 2, 32, ng)).float()
    x = codes * par[..., 0, :, :].unsqueeze(-1) + par[..., 1, :, :].unsqueeze(-1)
    x = x.flatten(-2).transpose(-4, -3).flatten(-3, -2)     # [..., 2, tiles * 32, d]
    return x[..., 0, :, :], x[..., 1, :, :]


def _plain_shared(s):
    heads, g, d, page, scale = s["heads"], s["g"], s["d"], s["page"], s["scale"]
    row, outs, lses = 0, [], []
    for n, p in zip(s["sizes"], s["prefixes"]):
        q = s["q"][row:row + n].float().unflatten(1, (heads, g)).transpose(0, 1)    # [h, n, g, d]
        table = s["table"][row:row + n].long()
        lens = s["lens"][row:row + n]
        # the prefix, once for the group
        k, v = _values_of(s["pool"][table[0, :_ceil(p, page)]].transpose(0, 1), d)
        k, v = k.flatten(1, 2)[:, :p], v.flatten(1, 2)[:, :p]                       # [h, p, d]
        sc = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)) * scale               # [h, n g, p]
        # each sequence's own tokens
        first = p // page
        cols = max(1, _ceil(max(s["host_lens"][row:row + n]), page) - first)
        rec = s["pool"][table[:, first:first + cols].clamp(min=0)]                  # [n, cols, h, .]
        ks, vs = _values_of(rec.transpose(1, 2), d)
        ks, vs = ks.flatten(2, 3).transpose(0, 1), vs.flatten(2, 3).transpose(0, 1)  # [h, n, m, d]
        pos = torch.arange(first * page, (first + cols) * page, device="cuda")
        seen = ((pos >= p) & (pos < lens.unsqueeze(1))).view(1, n, 1, -1)
        so = torch.where(seen, torch.matmul(q, ks.transpose(2, 3)) * scale, float("-inf"))
        sc = sc.unflatten(1, (n, g))
        m = torch.maximum(sc.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
        sc, so = torch.exp(sc - m), torch.exp(so - m)
        l = sc.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
        o = torch.matmul(sc.flatten(1, 2), v).unflatten(1, (n, g)) + torch.matmul(so, vs)
        outs.append((o / l).transpose(0, 1).flatten(1, 2))
        lses.append((m + torch.log(l)).squeeze(-1).transpose(1, 2).flatten(0, 1))
        row += n
    return torch.cat(outs).to(s["q"].dtype), torch.cat(lses, 1)


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "rope":
        return _plain_rope(s)
    if op == "beams":
        _plain_free(s, s["to_rows"])
        _plain_fork(s)
        _plain_copy(s["pool"], s["copy_src"], s["copy_dst"])
        return _state_of_beams(s)
    if op == "admit":
        _plain_admit(s)
        return s["table"], s["lens"], s["shares"], s["free"], s["head"], s["slots"], s["cu_new"]
    if op == "compact":
        _plain_compact(s)
        _plain_copy(s["pool"], s["copy_src"], s["copy_dst"])
        return _state_of_compact(s)
    return _plain_shared(s)


def _state_of_beams(s):
    return (s["table"], s["lens"], s["shares"], s["free"], s["head"], s["copy_src"], s["copy_dst"],
            s["pool"].view(torch.int32))


def _state_of_compact(s):
    return (s["table_out"], s["shares_out"], s["free_out"], s["head"], s["copy_src"], s["copy_dst"],
            s["pool"].view(torch.int32))


def _own(s):
    """The calls that a user of the framework makes."""
    import block_sparse_attention_nsa_gb300 as nsa
    op = s["op"]
    if op == "rope":
        how = {"cu_seqlens": s["cu"], "start": s["start"], "interleaved": bool(s["inter"]),
               "mscale": s["mscale"]}
        out = nsa.rope(s["q"], s["k"], s["freqs"], q_out=s["q_out"], k_out=s["k_out"], **how)
        if s["grad"]:
            out += nsa.rope_bwd(s["dq"], s["dk"], s["freqs"], dq_in=s["dq_in"], dk_in=s["dk_in"],
                                **how)
        return out
    if op == "beams":
        nsa.page_free(s["table"], s["lens"], s["to_rows"], s["page"], s["shares"], s["free"],
                      s["head"], head_out=s["head"])
        nsa.page_fork(s["table"], s["lens"], s["from_rows"], s["to_rows"], s["page"], s["shares"],
                      s["free"], s["head"], copy_src=s["copy_src"], copy_dst=s["copy_dst"],
                      head_out=s["head"])
        nsa.page_copy(s["pool"], s["copy_src"], s["copy_dst"])
        return _state_of_beams(s)
    if op == "admit":
        nsa.page_free(s["table"], s["lens"], s["gone_rows"], s["page"], s["shares"], s["free"],
                      s["head"], head_out=s["head"])
        nsa.page_plan(s["lens"], s["new"], s["free"], s["head"], s["table"], s["page"],
                      s["shares"].numel(), s["slots"], s["lens"], s["cu_new"], s["head"])
        return s["table"], s["lens"], s["shares"], s["free"], s["head"], s["slots"], s["cu_new"]
    if op == "compact":
        nsa.page_compact(s["table"], s["lens"], s["page"], s["shares"], s["free"],
                         table_out=s["table_out"], shares_out=s["shares_out"],
                         free_out=s["free_out"], copy_src=s["copy_src"], copy_dst=s["copy_dst"],
                         head_out=s["head"])
        nsa.page_copy(s["pool"], s["copy_src"], s["copy_dst"])
        return _state_of_compact(s)
    return nsa.kv4_decode_shared(s["q"], s["pool"], s["table"], s["lens"], s["scale"], s["cu"],
                                 s["prefix_lens"], out=s["out"], lse=s["lse"],
                                 workspace=s["workspace"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _turned64(x, pos, rot, inter, scaling, sign):
    """x [n, h, d] turned by sign times its positions, pair by pair."""
    how, out = SCALING[scaling], x.double()
    size = 1.0
    for i in range(rot // 2):
        base = 10000.0 * (how["factor"] ** (rot / (rot - 2)) if scaling == "base" else 1.0)
        w = base ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= how["factor"]
        if scaling == "ramp":
            r = how["trained"] * w / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (r - how["low"]) / (how["high"] - how["low"])))
            w = keep * w + (1.0 - keep) * w / how["factor"]
            size = 1.0 + 0.1 * math.log(how["factor"])
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        z = torch.polar(torch.full_like(pos, size), sign * w * pos)[:, None]
        y = torch.complex(x[..., a].double(), x[..., b].double()) * z
        out[..., a], out[..., b] = y.real, y.imag
    return out


def _row64(tile, part, r, d):
    """Rows r of K (part 0) or V (part 1) of tiles uint8 [n, h, tile bytes], in fp64 [n, h, d],
    dimension by dimension from the format's description."""
    dim = torch.arange(d, device="cuda")
    i, j, n = dim // 64, dim % 64 // 8, dim % 8
    byte = (part * 32 + r.unsqueeze(1)) * (d // 2) + 4 * (j * (d // 64) + i) + n // 2
    byte = byte.unsqueeze(1).expand(-1, tile.shape[1], -1)
    code = (tile.gather(2, byte).long() >> (4 * (n % 2))) % 16
    half = tile[..., 32 * d:].contiguous().view(torch.float16)

    def number(which):
        at = ((2 * part + which) * 32 + r.unsqueeze(1)) * (d // 64) + i
        return half.gather(2, at.unsqueeze(1).expand(-1, tile.shape[1], -1)).double()
    return code.double() * number(0) + number(1)


def _cached64(s, b, lo, hi):
    """K and V of sequence b's positions lo ... hi - 1, fp64 [n, h, d]."""
    page, d, heads = s["page"], s["d"], s["heads"]
    k = torch.empty((hi - lo, heads, d), dtype=torch.float64, device="cuda")
    v = torch.empty_like(k)
    for c in range(lo, hi, 8192):
        pos = torch.arange(c, min(c + 8192, hi), device="cuda")
        tile = s["pool"].view(-1, heads, page // 32, 32 * (d + d // 8))[
            s["table"][b, pos // page].long(), :, pos % page // 32]
        at = slice(c - lo, c - lo + pos.numel())
        k[at], v[at] = _row64(tile, 0, pos % 32, d), _row64(tile, 1, pos % 32, d)
    return k, v


def exact(case, seed):
    if case["op"] not in ("rope", "shared"):
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        cu = s["cu"].tolist()
        start = [0] * case["seqs"] if s["start"] is None else s["start"].tolist()
        pos = torch.cat([torch.arange(f, f + b - a, dtype=torch.float64, device="cuda")
                         for a, b, f in zip(cu, cu[1:], start)])
        how = (pos, case["rot"], case["inter"], case["scaling"])
        out = [_turned64(s["q"], *how, 1.0), _turned64(s["k"], *how, 1.0)]
        if case["grad"]:
            out += [_turned64(s["dq"], *how, -1.0), _turned64(s["dk"], *how, -1.0)]
        return tuple(out)
    heads, g, d = case["heads"], case["g"], case["d"]
    out = torch.empty((case["seqs"], heads * g, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((heads * g, case["seqs"]), dtype=torch.float64, device="cuda")
    q = s["q"].double()
    first = 0
    for n, p in zip(s["sizes"], s["prefixes"]):
        pk, pv = _cached64(s, first, 0, p)
        for b in range(first, first + n):
            k, v = _cached64(s, b, p, s["host_lens"][b])
            k, v = torch.cat([pk, k]).transpose(0, 1), torch.cat([pv, v]).transpose(0, 1)
            w = torch.matmul(q[b].unflatten(0, (heads, g)), k.transpose(1, 2)) * s["scale"]
            lse[:, b] = torch.logsumexp(w, -1).flatten()
            out[b] = torch.matmul(torch.softmax(w, -1), v).flatten(0, 1)
        first += n
    return out, lse
