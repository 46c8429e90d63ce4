"""Measured cases of a serving step with drafted tokens: rotary positions, decode of a tree of drafts, cache pages.

Every case is one pass through one entry point of ``mla_latent_kv_gb300``:

  rope    rotary positions of the heads' rope parts, written into the absorbed queries
  write   rotary positions of queries and keys, and the cache write of the new rows, in one call
  tree    decode of each request's drafted tokens, each seeing the cache and its own branch
  accept  the accepted branch's rows moved to the front of the drafted ones, in every layer
  fork    one state of the page pool to the next: rows kept, forked, grown and dropped

``own`` false computes them with elementary torch operations in 32 bits (64 for angles); ``own``
true makes the framework's calls.
"""
import math
import random

import torch

own = False

L, R, D, PAGE = 512, 64, 576, 64    # latent dims (V), rope dims, cached row, tokens per page
ROW = {"bf16": 1152, "fp8": 584}    # bytes of a cached row
SCALE = 1.0 / math.sqrt(192.0)
MAX_TREE = 1.17e12                  # flops of the largest tree case: drawn cases stay below it
YARN = (10000.0, 40.0, 4096, 32.0, 1.0)   # base, factor, trained positions, fast and slow turns


def listed():
    return [
        # two requests of one of eight head shards with four drafts each: latency is all there is
        {"name": "tree_small", "op": "tree", "kv": "bf16", "B": 2, "Sq": 4, "H": 16, "len": 700, "pad": 0},
        # the benchmark's lengths and heads, eight drafts a request, three slots of the batch empty
        {"name": "tree_batch", "op": "tree", "kv": "bf16", "B": 32, "Sq": 8, "H": 128, "len": 4096, "pad": 3},
        # one of eight head shards over long contexts: the cache stream weighs most
        {"name": "tree_shard", "op": "tree", "kv": "bf16", "B": 64, "Sq": 7, "H": 16, "len": 8192, "pad": 0},
        # wide trees over the FP8 cache: the tensor cores weigh most
        {"name": "tree_wide_fp8", "op": "tree", "kv": "fp8", "B": 16, "Sq": 32, "H": 128, "len": 8192, "pad": 0},
        # a few drafted tokens of one head shard
        {"name": "rope_small", "op": "rope", "T": 7, "H": 16, "far": 4000, "pairs": "half", "yarn": False},
        # the queries of a long prompt
        {"name": "rope_prompt", "op": "rope", "T": 8192, "H": 128, "far": 131072, "pairs": "adjacent", "yarn": True},
        # the drafted tokens of a decode batch
        {"name": "write_step", "op": "write", "kv": "bf16", "T": 256, "H": 128, "far": 8192, "pairs": "adjacent", "yarn": False},
        # the new tokens of a batch of prompts on one of eight head shards, FP8 rows
        {"name": "write_prompt_fp8", "op": "write", "kv": "fp8", "T": 32768, "H": 16, "far": 163840, "pairs": "half", "yarn": True},
        # a batch's accepted branches in the sixteen layers of a pipeline stage
        {"name": "accept_stage", "op": "accept", "kv": "bf16", "layers": 16, "B": 64, "Sq": 16, "len": 1000},
        # two requests with four drafts in one layer
        {"name": "accept_small", "op": "accept", "kv": "fp8", "layers": 1, "B": 2, "Sq": 4, "len": 300},
        # one request answered four times
        {"name": "fork_small", "op": "fork", "kv": "bf16", "layers": 1, "B": 1, "B2": 4, "len": 700, "spare": 64},
        # a step of a beam search: 128 rows choose their parents, in the sixteen layers of a stage
        {"name": "fork_beams", "op": "fork", "kv": "fp8", "layers": 16, "B": 128, "B2": 128, "len": 2000, "spare": 2048},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "rope", "write", "accept", "fork"])
    kv = rng.choice(["bf16", "fp8"])
    H = rng.choice([128, 128, 64, 32, 16, _log_int(rng, 1, 128)])
    if op == "tree":
        Sq = rng.choice([1, 4, 8, _log_int(rng, 1, 64)])
        length = _log_int(rng, 1, 131072)
        B = _log_int(rng, 1, max(1, min(64, 524288 // length)))
        while 2 * (D + L) * B * Sq * H * max(length, Sq) > MAX_TREE:
            B, Sq = max(1, B // 2), max(1, Sq // 2)
        return {"op": op, "kv": kv, "B": B, "Sq": Sq, "H": H, "len": length, "pad": rng.choice([0, 0, B // 8])}
    if op in ("rope", "write"):
        T = _log_int(rng, 1, max(1, 1048576 // max(H, 32)))
        case = {"op": op, "T": T, "H": H, "far": _log_int(rng, 64, 1048576), "pairs": rng.choice(["adjacent", "half"]),
                "yarn": rng.choice([True, False])}
        return {**case, "kv": kv} if op == "write" else case
    layers = rng.choice([1, 2, 4, 16])
    if op == "accept":
        return {"op": op, "kv": kv, "layers": layers, "B": _log_int(rng, 1, 64), "Sq": _log_int(rng, 1, 64),
                "len": _log_int(rng, 64, 2000)}
    return {"op": op, "kv": kv, "layers": layers, "B": _log_int(rng, 1, 128), "B2": _log_int(rng, 1, 128),
            "len": _log_int(rng, 1, 2000), "spare": _log_int(rng, 64, 2048)}


# ------------------------------------------------------------------------------------ inputs
def _rng(case, seed):
    """Host draws of one case (made alike for `work`)."""
    return random.Random("%d/%s" % (seed, sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case, seed):
    """Cached tokens of every request, the drafted ones among them."""
    r, B, Sq, top = _rng(case, seed), case["B"], case.get("Sq", 1), max(case["len"], case.get("Sq", 1))
    lens = [r.randint(max(Sq, top // 2), top) for _ in range(B)]
    lens[0] = top
    for b in range(B - case.get("pad", 0), B):
        lens[b] = 0
    return lens


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(kv, num_blocks, g):
    """Cache pages of N(0, 1) rows: bf16, or e4m3 rows with a scale per token."""
    out = torch.empty((num_blocks * PAGE, ROW[kv]), dtype=torch.uint8, device="cuda")
    step = 262144
    for i in range(0, out.shape[0], step):
        n = min(step, out.shape[0] - i)
        x = torch.empty((n, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        if kv == "bf16":
            out[i:i + n] = x.view(torch.uint8)
            continue
        f = x.float()
        s = (f.abs().amax(1, keepdim=True) / 448.0).clamp_min(1e-20)
        out[i:i + n, :D] = (f / s).to(torch.float8_e4m3fn).view(torch.uint8)
        out[i:i + n, D:] = torch.cat([s, s], 1).view(torch.uint8)
    return out.view(num_blocks, PAGE * ROW[kv])


def _table(pages, num_blocks, g, width=None):
    """Block table of rows with `pages[b]` scattered blocks each, -1 behind."""
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(pages), width or max(1, max(pages))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.cuda()


def _tree_masks(r, B, Sq):
    """Random trees in order of creation: bit i of word t is set where draft t sees draft i (its ancestors and itself)."""
    rows = []
    for _ in range(B):
        words = []
        for t in range(Sq):
            parent = r.randint(-1 if t else -1, t - 1) if r.random() < 0.5 else t - 1
            words.append((words[parent] if parent >= 0 else 0) | (1 << t))
        rows.append([w - (1 << 64) if w >= 1 << 63 else w for w in words])
    return torch.tensor(rows, dtype=torch.int64)


def _branch(r, Sq):
    """An accepted branch of drafts numbered level by level: the first of some levels, then later ones."""
    n = r.randint(0, min(Sq, 8))
    lead = r.randint(0, n)
    rest = sorted(r.sample(range(n, Sq), min(n - lead, Sq - n)))
    return (list(range(lead)) + rest)[:n]


def _frequencies(yarn):
    """Radians per position of the 32 pairs, doubles on the host."""
    base, factor, trained, fast, slow = YARN
    freq = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if not yarn:
        return freq

    def pair_of(turns):  # the pair that makes so many turns over the trained positions
        return R * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
    low, high = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), R - 1)
    ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(R // 2)]
    return [f / factor * a + f * (1 - a) for f, a in zip(freq, ramp)]


def _bf16(g, *shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def prepare(case, seed):
    g, op, r = _generator(seed), case["op"], _rng(case, seed + 1)
    s = {"op": op, "case": dict(case)}
    if op in ("rope", "write"):
        T, H = case["T"], case["H"]
        freq = _frequencies(case["yarn"])
        s["freq"] = torch.tensor(freq, dtype=torch.float64)           # a model's constant, on the host
        s["freq_gpu"] = s["freq"].cuda()
        # runs of consecutive positions, as of the requests of a batch
        start = torch.randint(0, case["far"], (-(-T // 32),), generator=g, device="cuda")
        s["positions"] = (start.repeat_interleave(32)[:T] + torch.arange(T, device="cuda") % 32).to(torch.int32)
        s["q_in"] = _bf16(g, T, H, 192)          # the query projection's output, nope part first
        s["q"] = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")   # the absorbed queries
        if op == "write":
            s["kv_a"] = _bf16(g, T, D)           # the latent projection's output: kv_c and k_pe side by side
            blocks = -(-T // PAGE) + 8
            s["cache"] = torch.zeros((blocks + 1, PAGE * ROW[case["kv"]]), dtype=torch.uint8, device="cuda")
            s["num_blocks"] = blocks             # the block behind them takes what the plain form leaves out
            slots = torch.randperm(blocks * PAGE, generator=g, device="cuda")[:T].contiguous()
            slots[T // 2 + 1::50] = -1              # padding tokens
            s["slots"] = slots
        return s
    lens = _lengths(case, seed)
    B = case["B"]
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pages = [-(-n // PAGE) for n in lens]
    if op == "tree":
        Sq, H = case["Sq"], case["H"]
        s["max_len"] = max(lens)
        blocks = sum(pages) + 16
        s["table"] = _table(pages, blocks, g)
        s["cache"] = _cache(case["kv"], blocks, g)
        s["q"] = _bf16(g, B, Sq, H, D)
        s["masks"] = _tree_masks(r, B, Sq).cuda()
        s["o"] = torch.empty((B, Sq, H, L), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, Sq, H), device="cuda")
        return s
    layers = case["layers"]
    if op == "accept":
        paths = [_branch(r, case["Sq"]) for _ in range(B)]
        path = torch.zeros((B, case["Sq"]), dtype=torch.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        s["path"], s["counts"] = path.cuda(), torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        blocks = B * max(pages) + 1
        s["table"] = _table(pages, blocks - 1, g)
        s["cache"] = _cache(case["kv"], layers * blocks, g).view(layers, blocks, -1)
        s["new_lens"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        return s
    # fork: rows of four share all but their last pages, as beams of one prompt do
    B2 = case["B2"]
    table, at, width = [], 0, max(pages) + 2
    for b, n in enumerate(pages):
        whole = lens[b] // PAGE
        shared = min(whole, lens[b - b % 4] // PAGE) if b % 4 else 0
        row = table[b - b % 4][:shared] if b % 4 else []
        row = row + list(range(at, at + n - len(row)))
        at += n - (shared if b % 4 else 0)
        table.append(row)
    blocks = B * max(pages) + 2 * B2 + case["spare"] + 1
    perm = torch.randperm(blocks - 1, generator=g, device="cuda").cpu()
    s["table"] = torch.full((B, width), -1, dtype=torch.int32)
    refs = torch.zeros((blocks,), dtype=torch.int32)
    refs[blocks - 1] = 1                          # a block that is nobody's: the plain form's scratch
    for b, row in enumerate(table):
        held = perm[torch.tensor(row, dtype=torch.int64)].to(torch.int32)
        s["table"][b, :len(row)] = held
        refs[held.long()] += 1
    s["table"], s["refs"] = s["table"].cuda(), refs.cuda()
    s["counts"] = torch.tensor(pages, dtype=torch.int32, device="cuda")
    parents = [r.randrange(-1 if r.random() < 0.1 else 0, B) for _ in range(B2)]
    s["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
    # every row gets room for one more token, a new one for its first
    s["room"] = torch.tensor([(lens[p] if p >= 0 else 0) + 1 for p in parents], dtype=torch.int32, device="cuda")
    s["cache"] = _cache(case["kv"], layers * blocks, g).view(layers, blocks, -1)
    s["new"] = (torch.empty((B2, width), dtype=torch.int32, device="cuda"), torch.empty((B2,), dtype=torch.int32, device="cuda"),
                torch.empty((B2,), dtype=torch.int32, device="cuda"), torch.empty_like(s["refs"]))
    return s


# --------------------------------------------------------------------------------- plain forms
def _rotate(x, positions, freq, pairs):
    """Rows [T, N, 64] turned by their positions, fp32."""
    turn = positions.double()[:, None] * freq
    c, n = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs == "adjacent" else (x[..., :R // 2], x[..., R // 2:])
    u, v = a * c - b * n, b * c + a * n
    return torch.stack([u, v], -1).flatten(-2) if pairs == "adjacent" else torch.cat([u, v], -1)


def _fp8_rows(rows):
    """The e4m3 values and the scales of an FP8 cache's rows [n, 584]."""
    return rows[:, :D].view(torch.float8_e4m3fn), rows[:, D:].view(torch.float32)


def _plain_rope(s):
    s["q"][..., L:] = _rotate(s["q_in"][..., 128:], s["positions"], s["freq_gpu"], s["case"]["pairs"]).to(torch.bfloat16)
    return s["q"][..., L:]


def _written(s):
    """The cache's rows as outputs."""
    rows = s["cache"][:s["num_blocks"]].view(s["num_blocks"] * PAGE, -1)
    return rows.view(torch.bfloat16) if s["case"]["kv"] == "bf16" else _fp8_rows(rows)


def _plain_write(s):
    c = s["case"]
    _plain_rope(s)
    k = _rotate(s["kv_a"][:, None, L:], s["positions"], s["freq_gpu"], c["pairs"])[:, 0]
    row = torch.cat([s["kv_a"][:, :L].float(), k], 1)
    at = torch.where(s["slots"] >= 0, s["slots"], torch.full_like(s["slots"], s["num_blocks"] * PAGE))
    rows = s["cache"].view(-1, ROW[c["kv"]])
    if c["kv"] == "bf16":
        rows[at] = row.to(torch.bfloat16).view(torch.uint8)
    else:
        amax = row.abs().amax(1, keepdim=True)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        codes = (row * (1.0 / scale)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        rows[at] = torch.cat([codes, torch.cat([scale, scale], 1).view(torch.uint8)], 1)
    return s["q"][..., L:], _written(s)


def _plain_tree(s):
    c = s["case"]
    B, Sq, H = c["B"], c["Sq"], c["H"]
    pages = s["cache"][s["table"].long().clamp_min(0)].view(B, -1, ROW[c["kv"]])
    if c["kv"] == "bf16":
        k = pages.view(torch.bfloat16).float()
        v = k[..., :L]
    else:
        x = pages[..., :D].contiguous().view(torch.float8_e4m3fn).float()
        scales = pages[..., D:].contiguous().view(torch.float32)
        k, v = x * scales[..., :1], x[..., :L] * scales[..., 1:]
    logits = torch.matmul(s["q"].float().view(B, Sq * H, D), k.transpose(1, 2)).view(B, Sq, H, -1) * SCALE
    draft = torch.arange(k.shape[1], device="cuda") - (s["seq_lens"].long()[:, None] - Sq)   # [B, tokens]
    bits = (s["masks"][:, :, None] >> draft.clamp(0, 63)[:, None]) & 1
    seen = ((draft < 0)[:, None] | ((draft < Sq)[:, None] & (bits != 0)))[:, :, None]
    logits = logits.masked_fill(~seen, -math.inf)
    m = logits.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(logits - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Sq * H, -1), v).view(B, Sq, H, L)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return o.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


def _plain_accept(s):
    c = s["case"]
    layers, blocks = s["cache"].shape[:2]
    rows = s["cache"].view(layers, blocks * PAGE, ROW[c["kv"]])
    first = s["seq_lens"].long()[:, None] - c["Sq"]
    j = torch.arange(c["Sq"], device="cuda")
    live = j < s["counts"][:, None]

    def row_of(pos):
        pos = torch.where(live, pos, torch.zeros_like(pos))
        at = s["table"].long().gather(1, pos // PAGE) * PAGE + pos % PAGE
        return torch.where(live, at, torch.full_like(at, blocks * PAGE - 1)).view(-1)
    rows[:, row_of(first + j)] = rows[:, row_of(first + s["path"])]
    return (first[:, 0] + s["counts"]).to(torch.int32), s["cache"].view(torch.int32)


def _plain_fork(s):
    c = s["case"]
    B, B2, width = c["B"], c["B2"], s["table"].shape[1]
    table, refs = s["table"].long(), s["refs"]
    has, p = s["parents"] >= 0, s["parents"].long().clamp_min(0)
    zero = torch.zeros_like(s["room"])
    n, held = torch.where(has, s["seq_lens"][p], zero), torch.where(has, s["counts"][p], zero)
    me = torch.arange(B2, device="cuda")
    first = torch.full((B,), B2, device="cuda").scatter_reduce(0, p, torch.where(has, me, torch.full_like(me, B2)), "amin")
    heir = has & (first[p] == me)
    whole = (n // PAGE)[:, None]
    need = torch.maximum((n + PAGE - 1) // PAGE, (s["room"] + PAGE - 1) // PAGE)
    j = torch.arange(width, device="cuda")
    old = table[p]
    keep = (j < whole) | (heir[:, None] & (j < torch.minimum(held, need)[:, None]) & (refs[old.clamp_min(0)] == 1))
    fresh = (j < need[:, None]) & ~keep
    rank = (torch.cumsum(fresh.view(-1), 0) - 1).view(B2, width)
    order = torch.argsort((refs != 0).to(torch.int32), stable=True)
    new = torch.where(keep, old, torch.where(fresh, order[rank.clamp_min(0)], torch.full_like(old, -1)))
    spare = refs.shape[0] - 1
    count = refs.clone()
    count.index_add_(0, torch.where(new >= 0, new, spare).view(-1), (new >= 0).to(torch.int32).view(-1))
    mine = j < s["counts"][:, None]
    count.index_add_(0, torch.where(mine, table, spare).view(-1), -mine.to(torch.int32).view(-1))
    # a page that a row holds in part is copied where another keeps it
    at = (n // PAGE).long().clamp_max(width - 1)[:, None]
    part = fresh.gather(1, at) & (n % PAGE > 0)[:, None]
    src = torch.where(part, old.gather(1, at), spare).view(-1)
    dst = torch.where(part, new.gather(1, at), spare).view(-1)
    rows = s["cache"].view(s["cache"].shape[0], -1, PAGE, ROW[c["kv"]])
    copied = (torch.arange(PAGE, device="cuda") < (n % PAGE)[:, None])[None, :, :, None]
    rows[:, dst] = torch.where(copied, rows[:, src], rows[:, dst])
    return new.to(torch.int32), need, n, count, s["cache"].view(torch.int32)


def _own(s):
    import mla_latent_kv_gb300 as mla
    c, op = s["case"], s["op"]
    if op == "rope":
        return mla.rope(s["q_in"][..., 128:], s["positions"], s["freq"], adjacent=c["pairs"] == "adjacent", out=s["q"][..., L:])
    kv = mla.KV_BF16 if c["kv"] == "bf16" else mla.KV_FP8
    if op == "write":
        mla.rope_cache_write(s["kv_a"][:, :L], s["kv_a"][:, L:], s["positions"], s["freq"], s["slots"], s["cache"], kv_dtype=kv,
                             adjacent=c["pairs"] == "adjacent", q_pe=s["q_in"][..., 128:], q_out=s["q"][..., L:],
                             num_blocks=s["num_blocks"])
        return s["q"][..., L:], _written(s)
    if op == "tree":
        return mla.decode_tree(s["q"], s["cache"], s["table"], s["seq_lens"], s["masks"], s["max_len"], SCALE, kv_dtype=kv,
                               o_latent=s["o"], lse=s["lse"])
    if op == "accept":
        new = mla.accept_tokens(s["cache"], s["table"], s["seq_lens"], s["path"], s["counts"], kv_dtype=kv, new_lens=s["new_lens"])
        return new, s["cache"].view(torch.int32)
    new = mla.fork_pages(s["cache"], s["table"], s["counts"], s["seq_lens"], s["refs"], s["parents"], s["room"], kv_dtype=kv,
                         out=s["new"])
    return (*new, s["cache"].view(torch.int32))


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "write": _plain_write, "tree": _plain_tree, "accept": _plain_accept,
            "fork": _plain_fork}[state["op"]](state)


# ------------------------------------------------------------------------------------- figures
def work(case):
    """Bytes read and written once each, and the formula's flops, for seed 0's lengths."""
    op = case["op"]
    if op in ("rope", "write"):
        T, H = case["T"], case["H"]
        q = T * H * R
        if op == "rope":
            return {"bytes": 4 * q + 4 * T, "flops": 3 * q}
        return {"bytes": 4 * q + T * (2 * D + 12 + ROW[case["kv"]]), "flops": 3 * (q + T * R)}
    lens, r = _lengths(case, 0), _rng(case, 1)
    row, B = ROW[case["kv"]], case["B"]
    if op == "tree":
        Sq, H = case["Sq"], case["H"]
        seen = sum((n - Sq) * Sq for n in lens if n) + sum(bin(w & (1 << 64) - 1).count("1")
                                                            for n, m in zip(lens, _tree_masks(r, B, Sq).tolist()) if n for w in m)
        return {"bytes": sum(lens) * row + 4 * sum(-(-n // PAGE) for n in lens) + B * Sq * H * (2 * D + 2 * L + 4) + 8 * B * Sq,
                "flops": 2 * (D + L) * H * seen}
    if op == "accept":
        moved = sum(sum(i != p for i, p in enumerate(_branch(r, case["Sq"]))) for _ in range(B))
        return {"bytes": case["layers"] * moved * 2 * row + 4 * B * case["Sq"] + 16 * B, "flops": 0}
    B2, pages = case["B2"], [-(-n // PAGE) for n in lens]
    parents = [r.randrange(-1 if r.random() < 0.1 else 0, B) for _ in range(B2)]
    kept, copied, read, seen = 0, 0, 0, set()
    for p in parents:
        n = lens[p] if p >= 0 else 0
        copied += n % PAGE if p in seen else 0
        read += pages[p] if p >= 0 else 0
        kept += n // PAGE + 1
        seen.add(p)
    return {"bytes": case["layers"] * copied * 2 * row + 4 * (sum(pages) + kept) + 8 * case["spare"] + 20 * B2, "flops": 0}


# --------------------------------------------------------------------- the definition, in 64 bits
def _turn64(x, positions, freq, pairs):
    """Each pair as a complex number times e^(i position frequency)."""
    x = x.double()
    z = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) if pairs == "adjacent" else \
        torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:].contiguous())
    angle = positions.double()[:, None, None] * freq
    z = z * torch.polar(torch.ones_like(angle), angle)
    if pairs == "adjacent":
        return torch.view_as_real(z).reshape(x.shape)
    return torch.cat([z.real, z.imag], -1)


def _exact_positions(s):
    c = s["case"]
    q = torch.cat([_turn64(x, p, s["freq_gpu"], c["pairs"]) for x, p in
                   zip(s["q_in"][..., 128:].split(4096), s["positions"].split(4096))])
    if c["op"] == "rope":
        return q
    rows = torch.zeros((s["num_blocks"] * PAGE, D), dtype=torch.float64, device="cuda")
    k = _turn64(s["kv_a"][:, None, L:], s["positions"], s["freq_gpu"], c["pairs"])[:, 0]
    live = s["slots"] >= 0
    rows[s["slots"][live]] = torch.cat([s["kv_a"][:, :L].double(), k], 1)[live]
    if c["kv"] == "bf16":
        return q, rows
    top = rows.abs().amax(1, keepdim=True)
    written = torch.zeros((rows.shape[0], 1), dtype=torch.bool, device="cuda")
    written[s["slots"][live]] = True
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    scales = torch.where(written, scale, torch.zeros_like(scale))
    return q, (rows / scale, scales.expand(-1, 2).contiguous())


def _exact_tree(s, lens):
    c = s["case"]
    B, Sq, H = c["B"], c["Sq"], c["H"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    masks = s["masks"].tolist()
    for b, n in enumerate(lens):
        if not n:
            continue
        raw = s["cache"][s["table"][b, :-(-n // PAGE)].long()].view(-1, ROW[c["kv"]])[:n]
        if c["kv"] == "bf16":
            k = raw.contiguous().view(torch.bfloat16).double()
            v = k[:, :L]
        else:
            code = raw[:, :D].contiguous().view(torch.float8_e4m3fn).double()
            k = code * raw[:, D:D + 4].contiguous().view(torch.float32).double()
            v = code[:, :L] * raw[:, D + 4:].contiguous().view(torch.float32).double()
        for t in range(Sq):
            x = s["q"][b, t].double() @ k.t() * SCALE
            hidden = [n - Sq + i for i in range(Sq) if not masks[b][t] >> i & 1]
            x[:, hidden] = -math.inf
            lse[b, t] = torch.logsumexp(x, 1)
            o[b, t] = torch.exp(x - lse[b, t][:, None]) @ v
    return o, lse


def exact(case, seed):
    if case["op"] in ("accept", "fork"):
        return None  # whole numbers: the plain form is exact
    s = prepare(case, seed)
    if case["op"] in ("rope", "write"):
        return _exact_positions(s)
    return _exact_tree(s, _lengths(case, seed))
