"""The 4-bit paged KV cache's operators, as cases to be measured.

Three operators of a serving step around Native Sparse Attention's decode:

  plan    block tables and slot maps built on the GPU from request lengths
  cache   K and V quantised to 4 bits into the pages of a pool (append), and the
          pages read back as 16-bit rows (read), which a prefill attends to
  decode  one new token per sequence attending to the 4-bit pages: to the blocks that
          a selection names, to a sliding window, or to everything cached

`run` computes them in elementary torch operations in 32 bits, or, where `own` is
true, through block_sparse_attention_nsa_gb300.  `exact` computes them in 64 bits from
the definition.

The pool is uint8 [num_pages, h_k, P * (d + d / 8)] with P = 32, 64 or 128 tokens a
page and d = 64 or 128.  The record of a (page, KV head) is P / 32 tiles of 32 tokens:
  K codes [32, d / 2], V codes [32, d / 2], then fp16 [4, 32, d / 64]: K scale, K zero,
  V scale, V zero.
A row's codes are 32-bit words; the word at index j * (d / 64) + i holds dimensions
64 i + 8 j ... + 7, four bits each, lowest first.  A code c stands for c * scale + zero,
with one scale and zero for each 64 dimensions of a token's head.
"""
import random

import torch

own = False

HALF_MAX = 65504.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a batch: a new token each, some of them opening a page
        {"name": "plan_step_64", "op": "plan", "seqs": 64, "ctx": 8192, "new": 1, "page": 64,
         "pad": 0, "salt": 1},
        # a large batch of mixed prompts and decode steps, padded to a bucket
        {"name": "plan_mixed_1000", "op": "plan", "seqs": 1000, "ctx": 16384, "new": 700,
         "page": 32, "pad": 777, "salt": 2},
        # the new tokens of that decode step
        {"name": "append_step_64", "op": "append", "tokens": 64, "heads": 4, "d": 128, "page": 64,
         "dtype": "bf16", "fused": 0, "pad": 0},
        # a 64K-token prompt: K and V are column ranges of a fused projection's output
        {"name": "append_prompt_64k", "op": "append", "tokens": 65536, "heads": 4, "d": 128,
         "page": 64, "dtype": "bf16", "fused": 1, "pad": 0},
        # a few short requests whose cached tokens are read back before a prefill chunk
        {"name": "read_ragged_5", "op": "read", "seqs": 5, "ctx": 517, "heads": 3, "d": 64,
         "page": 32, "dtype": "fp16", "salt": 3},
        # long requests read back
        {"name": "read_8x8k", "op": "read", "seqs": 8, "ctx": 8192, "heads": 4, "d": 128,
         "page": 128, "dtype": "bf16", "salt": 4},
        # one user's decode step over its selected blocks: latency alone
        {"name": "sel_1x4097", "op": "decode", "seqs": 1, "ctx": 4097, "equal": 1, "heads": 4,
         "g": 4, "d": 128, "page": 64, "topk": 16, "window": 0, "dtype": "bf16", "salt": 5},
        # a served batch, 64 sequences of 8K cached tokens, 16 selected blocks each
        {"name": "sel_64x8k", "op": "decode", "seqs": 64, "ctx": 8192, "equal": 1, "heads": 4,
         "g": 4, "d": 128, "page": 64, "topk": 16, "window": 0, "dtype": "bf16", "salt": 6},
        # the same with 16 query heads to a KV head, ragged lengths, fp16
        {"name": "sel_200_ragged_g16", "op": "decode", "seqs": 200, "ctx": 8192, "equal": 0,
         "heads": 2, "g": 16, "d": 128, "page": 64, "topk": 16, "window": 0, "dtype": "fp16",
         "salt": 7},
        # one sequence of 64K cached tokens attended to in full: few rows, one long axis
        {"name": "full_1x64k", "op": "decode", "seqs": 1, "ctx": 65536, "equal": 1, "heads": 4,
         "g": 4, "d": 128, "page": 64, "topk": 0, "window": 0, "dtype": "bf16", "salt": 8},
        # a ragged batch attended to in full, one token to 32K
        {"name": "full_48_ragged", "op": "decode", "seqs": 48, "ctx": 32768, "equal": 0,
         "heads": 4, "g": 8, "d": 128, "page": 64, "topk": 0, "window": 0, "dtype": "bf16",
         "salt": 9},
        # the sliding-window branch (window 512) of a large batch with small heads
        {"name": "window_256_d64", "op": "decode", "seqs": 256, "ctx": 4096, "equal": 0,
         "heads": 8, "g": 1, "d": 64, "page": 32, "topk": 0, "window": 512, "dtype": "fp16",
         "salt": 10},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "append", "read", "decode", "decode", "decode"])
    page = rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    salt = rng.randrange(1 << 30)
    if op == "plan":
        return {"op": op, "seqs": _log_int(rng, 1, 1000), "ctx": _log_int(rng, 1, 16384),
                "new": _log_int(rng, 1, 700), "page": page, "pad": rng.choice([0, 1, 300]),
                "salt": salt}
    heads, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    if op == "append":
        return {"op": op, "tokens": _log_int(rng, 1, 32768), "heads": heads, "d": d, "page": page,
                "dtype": dtype, "fused": rng.choice([0, 1]), "pad": rng.choice([0, 7])}
    if op == "read":
        return {"op": op, "seqs": _log_int(rng, 1, 16), "ctx": _log_int(rng, 1, 4096),
                "heads": heads, "d": d, "page": page, "dtype": dtype, "salt": salt}
    kind = rng.choice(["sel", "full", "window"])
    seqs = _log_int(rng, 1, 128)
    most = max(64, min(65536, 500000 // (seqs * heads)))
    return {"op": op, "seqs": seqs, "ctx": _log_int(rng, 1, most), "equal": rng.choice([0, 1]),
            "heads": heads, "g": rng.choice([1, 2, 3, 4, 7, 8, 12, 16]), "d": d, "page": page,
            "topk": rng.choice([1, 5, 16, 32]) if kind == "sel" else 0,
            "window": rng.choice([1, 100, 512]) if kind == "window" else 0, "dtype": dtype,
            "salt": salt}


def _lengths(case):
    """The sequences' cached lengths, by the case alone: spread over their logarithm."""
    if case.get("equal"):
        return [case["ctx"]] * case["seqs"]
    rng = random.Random("lengths %d" % case["salt"])
    lens = [_log_int(rng, 1, case["ctx"]) for _ in range(case["seqs"])]
    lens[rng.randrange(len(lens))] = case["ctx"]
    return lens


def _new_lengths(case):
    """New tokens of each request of a plan: decode steps (one) and prompts, some idle."""
    if case["new"] == 1:
        return [1] * case["seqs"]
    rng = random.Random("new %d" % case["salt"])
    return [rng.choice([0, 1, 1, 1, _log_int(rng, 1, case["new"])]) for _ in range(case["seqs"])]


def _ceil(a, b):
    return -(-a // b)


def _kept_blocks(case, n):
    """Selected blocks of a sequence of n cached tokens."""
    return min(case["topk"], _ceil(n, case["page"]))


def work(case):
    if case["op"] == "plan":
        new, ctx, page = _new_lengths(case), _lengths(case), case["page"]
        opened = sum(_ceil(c + n, page) - _ceil(c, page) for c, n in zip(ctx, new))
        slots = sum(new) + case["pad"]
        # lengths in and out, offsets, free pages and table entries, the page of each
        # request that continues one, slots
        return {"bytes": 4 * (5 * case["seqs"] + 2 * opened + slots), "flops": 0}
    d = case["d"]
    stored = d + d // 8                    # bytes of a token's K and V of one head
    if case["op"] == "append":
        rows = case["tokens"] * case["heads"]
        return {"bytes": rows * (4 * d + stored + 4 * d) + 4 * (case["tokens"] + case["pad"]),
                "flops": 6 * rows * 2 * d}
    lens = _lengths(case)
    if case["op"] == "read":
        n = sum(lens)
        return {"bytes": n * case["heads"] * (stored + 4 * d), "flops": 2 * n * case["heads"] * 2 * d}
    page = case["page"]
    if case["topk"]:
        # the newest block and the first are always taken; the last may be short
        keys = sum((_kept_blocks(case, n) - 1) * page + (n - 1) % page + 1 for n in lens)
    else:
        keys = sum(min(n, case["window"]) if case["window"] else n for n in lens)
    rows = case["seqs"] * case["heads"] * case["g"]
    return {"bytes": keys * case["heads"] * stored + rows * (4 * d + 4),
            "flops": 4 * d * keys * case["heads"] * case["g"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _values(shape, gen):
    """Key- or value-like numbers in fp32: a few dimensions much larger than the rest, and
    tokens of different size."""
    x = torch.randn(shape, generator=gen, device="cuda")
    d = shape[-1]
    x *= torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
    x[..., ::37] *= 4.0
    return x


def _quantise(x):
    """fp32 [..., d] -> codes int [..., d], scale and zero fp16 [..., d / 64].  The zero is the
    group's smallest value rounded to fp16, the scale (largest - zero) / 15 rounded to
    fp16, a code round((x - zero) / scale), half to even, within 0 ... 15 (0 where the scale
    is 0)."""
    g = x.clamp(-HALF_MAX, HALF_MAX).unflatten(-1, (-1, 64))
    zero = g.amin(-1).half()
    scale = ((g.amax(-1) - zero.float()) / 15).half()
    step = torch.where(scale > 0, scale.float(), float("inf")).unsqueeze(-1)
    c = ((g - zero.float().unsqueeze(-1)) / step).round().clamp(0, 15)
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


def _pool(pages, heads, page, d, gen):
    shape = (pages, heads, page, d)
    return _records(_values(shape, gen), _values(shape, gen))


def _table(lens, page, gen, spare=3):
    """A block table int32 [B, W] of pages in shuffled order (-1 where there is none), and
    the pages that are left."""
    per = [_ceil(n, page) for n in lens]
    width, total = max(1, max(per)), sum(per)
    order = torch.randperm(total + spare, generator=gen, device="cuda").int()
    per_t = torch.tensor(per, device="cuda")
    first = per_t.cumsum(0) - per_t
    col = torch.arange(width, device="cuda")
    at = (first.unsqueeze(1) + col).clamp(max=total + spare - 1)
    table = torch.where(col < per_t.unsqueeze(1), order[at], -1)
    return table.int().contiguous(), order[total:].contiguous(), total + spare


def _selection(case, lens, gen):
    """int32 [h, B, T]: the newest block, block 0 and others at random, -1 where a sequence
    has fewer; slots in any order."""
    blocks = torch.tensor([_ceil(n, case["page"]) for n in lens], device="cuda")
    width = max(int(blocks.max()), case["topk"])
    score = torch.rand((case["heads"], case["seqs"], width), generator=gen, device="cuda")
    col = torch.arange(width, device="cuda")
    last = (blocks - 1).unsqueeze(1)
    score = score + 2.0 * (col == 0) + 4.0 * (col == last) - 8.0 * (col > last)
    top, at = score.topk(case["topk"], -1)
    sel = torch.where(top < -4.0, -1, at)
    perm = torch.randperm(case["topk"], generator=gen, device="cuda")
    return sel[..., perm].int().contiguous()


def prepare(case, seed):
    gen = _gen(seed)
    s = dict(case)
    page = case["page"]
    if case["op"] == "plan":
        ctx, new = _lengths(case), _new_lengths(case)
        after = [c + n for c, n in zip(ctx, new)]
        opened = sum(_ceil(a, page) - _ceil(c, page) for a, c in zip(after, ctx))
        table, free, pages = _table(ctx, page, gen, spare=opened + 5)
        width = max(_ceil(a, page) for a in after)
        wide = torch.full((case["seqs"], max(width, table.shape[1]) + 1), -1, dtype=torch.int32,
                          device="cuda")
        wide[:, :table.shape[1]] = table
        b = case["seqs"]
        s.update(table=wide, free=free, pages=pages, max_new=sum(new) + case["pad"],
                 ctx_lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                 new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"),
                 head=torch.full((1,), 2, dtype=torch.int32, device="cuda"),
                 head_out=torch.empty(1, dtype=torch.int32, device="cuda"),
                 seq_lens=torch.empty(b, dtype=torch.int32, device="cuda"),
                 cu_new=torch.empty(b + 1, dtype=torch.int32, device="cuda"),
                 slots=torch.empty(sum(new) + case["pad"], dtype=torch.int32, device="cuda"))
        return s
    heads, d, dt = case["heads"], case["d"], DTYPES[case["dtype"]]
    if case["op"] == "append":
        n = case["tokens"]
        pages = _ceil(n, page) + 2
        k, v = (_values((n + case["pad"], heads, d), gen).to(dt) for _ in range(2))
        if case["fused"]:                 # q of 2 * heads heads, then K, then V, in one row
            row = torch.zeros((n + case["pad"], 4 * heads, d), dtype=dt, device="cuda")
            row[:, 2 * heads:3 * heads], row[:, 3 * heads:] = k, v
            k, v = row[:, 2 * heads:3 * heads], row[:, 3 * heads:]
        order = torch.randperm(pages, generator=gen, device="cuda")
        pos = torch.arange(n, device="cuda") + page // 3     # the first page is partly full
        slots = order[pos // page] * page + pos % page
        slots = torch.cat([slots, torch.full((case["pad"],), -1, device="cuda")]).int()
        s.update(k=k, v=v, slots=slots,
                 pool=torch.zeros((pages, heads, page * (d + d // 8)), dtype=torch.uint8,
                                  device="cuda"),
                 k_out=torch.empty((n + case["pad"], heads, d), dtype=dt, device="cuda"),
                 v_out=torch.empty((n + case["pad"], heads, d), dtype=dt, device="cuda"))
        return s
    lens = _lengths(case)
    table, _, pages = _table(lens, page, gen)
    s.update(table=table, pool=_pool(pages, heads, page, d, gen), lens=lens,
             seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["op"] == "read":
        n = sum(lens)
        s.update(total=n, start=torch.zeros(case["seqs"], dtype=torch.int32, device="cuda"),
                 cu=torch.empty(case["seqs"] + 1, dtype=torch.int32, device="cuda"),
                 slots=torch.empty(n, dtype=torch.int32, device="cuda"),
                 k_out=torch.empty((n, heads, d), dtype=dt, device="cuda"),
                 v_out=torch.empty((n, heads, d), dtype=dt, device="cuda"))
        return s
    hq = heads * case["g"]
    s.update(q=torch.randn((case["seqs"], hq, d), generator=gen, device="cuda").to(dt),
             scale=d ** -0.5, sel=_selection(case, lens, gen) if case["topk"] else None,
             out=torch.empty((case["seqs"], hq, d), dtype=dt, device="cuda"),
             lse=torch.empty((hq, case["seqs"]), dtype=torch.float32, device="cuda"),
             workspace=torch.empty(8 << 20, dtype=torch.uint8, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
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


def _slots_of(table, cu, start, count, page):
    """Slot of each of `count` packed tokens, -1 past the last request's."""
    t = torch.arange(count, device="cuda")
    b = torch.searchsorted(cu[1:].long(), t, right=True).clamp(max=cu.numel() - 2)
    pos = start[b].long() + t - cu[b]
    got = table[b, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    return torch.where(t < cu[-1], got, -1).int()


def _offsets(n):
    return torch.cat([n.new_zeros(1), n.cumsum(0)]).int()


def _plain_plan(s):
    page, ctx, new = s["page"], s["ctx_lens"], s["new_lens"]
    seq = ctx + new
    have, want = (ctx + page - 1) // page, (seq + page - 1) // page
    first = s["head"] + _offsets(want - have)[:-1]
    col = torch.arange(s["table"].shape[1], device="cuda")
    opened = (col >= have.unsqueeze(1)) & (col < want.unsqueeze(1))
    at = (first.unsqueeze(1) + col - have.unsqueeze(1)).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(opened, s["free"][at], s["table"]))
    cu = _offsets(new)
    slots = _slots_of(s["table"], cu, ctx, s["max_new"], page)
    return s["table"], seq, cu, slots, s["head"] + (want - have).sum().int()


def _store(pool, k, v, slots, page):
    """Writes the rows of K and V (fp32) whose slot is not negative into the pool."""
    pages, heads, _ = pool.shape
    d = k.shape[-1]
    ng = d // 64
    at = slots.long()
    rows = at >= 0
    k, v, at = k[rows], v[rows], at[rows]
    tiles = pool.view(pages, heads, page // 32, 32 * (d + d // 8))
    p, t, r = at // page, at % page // 32, at % 32
    par = tiles[..., 32 * d:].contiguous().view(torch.float16).unflatten(-1, (4, 32, ng))
    codes = tiles[..., :32 * d].unflatten(-1, (2, 32, d // 2))
    kc, ks, kz = _quantise(k)
    vc, vs, vz = _quantise(v)
    codes[p, :, t, 0, r], codes[p, :, t, 1, r] = _pack(kc), _pack(vc)
    par[p, :, t, 0, r], par[p, :, t, 1, r] = ks, kz
    par[p, :, t, 2, r], par[p, :, t, 3, r] = vs, vz
    tiles[..., 32 * d:] = par.flatten(-3).view(torch.uint8)


def _load(pool, slots, page, d, dtype):
    """K and V [n, h, d] at the slots, zeros where a slot is negative."""
    pages, heads, _ = pool.shape
    at = slots.long().clamp(min=0)
    tiles = pool.view(pages, heads, page // 32, 32 * (d + d // 8))
    p, t, r = at // page, at % page // 32, at % 32
    ng = d // 64
    codes = tiles[..., :32 * d].unflatten(-1, (2, 32, d // 2))[p, :, t, :, r]      # [n, h, 2, d / 2]
    par = tiles[..., 32 * d:].unflatten(-1, (4, 32, 2 * ng))[p, :, t, :, r]        # [n, h, 4, 2 ng]
    par = par.contiguous().view(torch.float16).unflatten(-2, (2, 2)).float()       # [n, h, 2, 2, ng]
    c = codes.unflatten(-1, (8, ng, 4)).transpose(-3, -2)
    c = torch.stack([c & 15, c >> 4], -1).flatten(-3)                              # [n, h, 2, ng, 64]
    x = (c * par[..., 0, :].unsqueeze(-1) + par[..., 1, :].unsqueeze(-1)).flatten(-2)
    x = torch.where((slots >= 0).view(-1, 1, 1, 1), x, 0.0).to(dtype)
    return x[:, :, 0].contiguous(), x[:, :, 1].contiguous()


def _attend(q, k, v, seen, scale):
    """q [B, h, g, d], k and v [B, h, n, d], seen [B, h or 1, n], all fp32: out [B, h * g, d]
    and lse [h * g, B]."""
    sc = torch.matmul(q, k.transpose(-1, -2)) * scale
    sc = torch.where(seen.unsqueeze(2), sc, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / l
    return out.flatten(1, 2), (m + torch.log(l)).flatten(1).t()


def _seen_sel(s):
    """The kept slots of the selection (valid, causal, first of its value) and the keys that
    they show: blocks [B, h, T], seen [B, h, T, P]."""
    page, sel, lens = s["page"], s["sel"].transpose(0, 1).long(), s["seq_lens"].long()
    own_block = ((lens - 1) // page).view(-1, 1, 1)
    ok = (sel >= 0) & (sel <= own_block)
    same = sel.unsqueeze(-1) == sel.unsqueeze(-2)
    ok &= ~(same & torch.ones_like(same).tril(-1)).any(-1)
    pos = sel.unsqueeze(-1) * page + torch.arange(page, device="cuda")
    return sel, ok.unsqueeze(-1) & (pos < lens.view(-1, 1, 1, 1))


def _plain_decode(s):
    d, page, heads = s["d"], s["page"], s["heads"]
    q = s["q"].float().unflatten(1, (heads, s["g"]))
    lens, table = s["seq_lens"].long(), s["table"].long()
    if s["sel"] is not None:
        sel, seen = _seen_sel(s)
        pages = table.unsqueeze(1).expand(-1, heads, -1).gather(
            2, sel.clamp(0, table.shape[1] - 1)).clamp(min=0)
        rec = s["pool"][pages, torch.arange(heads, device="cuda").view(1, -1, 1)]
    elif s["window"]:
        # the pages that hold the last `window` tokens
        first = (lens - s["window"]).clamp(min=0) // page
        col = torch.arange(_ceil(s["window"] - 1, page) + 1, device="cuda")
        at = first.unsqueeze(1) + col
        pages = table.gather(1, at.clamp(max=table.shape[1] - 1)).clamp(min=0)
        rec = s["pool"][pages].transpose(1, 2)
        pos = (at.unsqueeze(-1) * page + torch.arange(page, device="cuda")).unsqueeze(1)
        n = lens.view(-1, 1, 1, 1)
        seen = (pos < n) & (pos >= n - s["window"])
    else:
        rec = s["pool"][table.clamp(min=0)].transpose(1, 2)
        pos = torch.arange(table.shape[1] * page, device="cuda").view(1, 1, -1, page)
        seen = pos < lens.view(-1, 1, 1, 1)
    k, v = _values_of(rec, d)
    out, lse = _attend(q, k.flatten(2, 3), v.flatten(2, 3), seen.flatten(2), s["scale"])
    return out.to(s["q"].dtype), lse.contiguous()


def run(s):
    if own:
        return _own(s)
    if s["op"] == "plan":
        return _plain_plan(s)
    if s["op"] == "append":
        _store(s["pool"], s["k"].float(), s["v"].float(), s["slots"], s["page"])
        return _load(s["pool"], s["slots"], s["page"], s["d"], s["k"].dtype)
    if s["op"] == "read":
        cu = _offsets(s["seq_lens"])
        slots = _slots_of(s["table"], cu, s["start"], s["total"], s["page"])
        return (slots, *_load(s["pool"], slots, s["page"], s["d"], s["k_out"].dtype))
    return _plain_decode(s)


def _own(s):
    """The calls that a user of the framework makes."""
    import block_sparse_attention_nsa_gb300 as nsa
    if s["op"] == "plan":
        nsa.page_plan(s["ctx_lens"], s["new_lens"], s["free"], s["head"], s["table"], s["page"],
                      s["pages"], s["slots"], s["seq_lens"], s["cu_new"], s["head_out"])
        return s["table"], s["seq_lens"], s["cu_new"], s["slots"], s["head_out"]
    if s["op"] == "append":
        nsa.kv4_append(s["pool"], s["k"], s["v"], s["slots"])
        return nsa.kv4_read(s["pool"], s["slots"], s["d"], s["k_out"], s["v_out"])
    if s["op"] == "read":
        nsa.page_slots(s["table"], s["start"], s["seq_lens"], s["page"], s["pool"].shape[0],
                       s["slots"], s["cu"])
        return (s["slots"], *nsa.kv4_read(s["pool"], s["slots"], s["d"], s["k_out"], s["v_out"]))
    return nsa.kv4_decode(s["q"], s["pool"], s["table"], s["seq_lens"], s["scale"],
                          sel_idx=s["sel"], window=s["window"], out=s["out"], lse=s["lse"],
                          workspace=s["workspace"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
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


def _cached64(s, b, heads, lo=0):
    """K and V of sequence b's positions lo ... , fp64 [n, h, d]."""
    page, d = s["page"], s["d"]
    pos = torch.arange(lo, s["lens"][b], device="cuda")
    pg = s["table"][b, pos // page].long()
    size = 32 * (d + d // 8)
    k = torch.empty((pos.numel(), heads, d), dtype=torch.float64, device="cuda")
    v = torch.empty_like(k)
    for c in range(0, pos.numel(), 8192):
        q, g = pos[c:c + 8192] % page, pg[c:c + 8192]
        tile = s["pool"].view(-1, heads, page // 32, size)[g, :, q // 32]
        k[c:c + 8192], v[c:c + 8192] = _row64(tile, 0, q % 32, d), _row64(tile, 1, q % 32, d)
    return k, v


def _fold64(x):
    """What 4 bits keep of x [n, h, d], in fp64."""
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for c in range(0, x.shape[-1], 64):
        y = x[..., c:c + 64].double()
        low, high = y.min(-1).values, y.max(-1).values
        zero = low.to(torch.float16).double()
        step = ((high - zero) / 15.0).to(torch.float16).double()
        n = torch.round((y - zero[..., None]) / step[..., None]).clamp(0.0, 15.0)
        out[..., c:c + 64] = zero[..., None] + torch.nan_to_num(n) * step[..., None]
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    heads, d = case["heads"], case["d"]
    if case["op"] == "append":
        k, v = _fold64(s["k"]), _fold64(s["v"])
        k[s["slots"] < 0], v[s["slots"] < 0] = 0.0, 0.0
        return k, v
    seqs = range(case["seqs"])
    if case["op"] == "read":
        rows = [_cached64(s, b, heads) for b in seqs]
        return None, torch.cat([k for k, _ in rows]), torch.cat([v for _, v in rows])
    g, page = case["g"], case["page"]
    out = torch.zeros((case["seqs"], heads * g, d), dtype=torch.float64, device="cuda")
    lse = torch.full((heads * g, case["seqs"]), float("-inf"), dtype=torch.float64, device="cuda")
    q = s["q"].double()
    for b in seqs:
        n = s["lens"][b]
        lo = max(0, n - case["window"]) if case["window"] else 0
        k, v = _cached64(s, b, heads, lo)
        see = torch.ones((heads, n - lo), dtype=torch.bool, device="cuda")
        if s["sel"] is not None:
            block = torch.arange(lo, n, device="cuda") // page
            see = (block[None, None] == s["sel"][:, b, :, None]).any(1)
        for h in range(heads):
            row = (q[b, h * g:(h + 1) * g] @ k[see[h], h].t()) * s["scale"]
            lse[h * g:(h + 1) * g, b] = torch.logsumexp(row, 1)
            out[b, h * g:(h + 1) * g] = torch.softmax(row, 1) @ v[see[h], h]
    return out, lse
