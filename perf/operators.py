"""The long-context operators' measured cases: decode over a shared prefix, and decode over selected pages.

Every case is one pass through one entry point of ``mla_latent_kv_gb300``:

  prefix   decode of a batch whose requests share their first ``prefix`` cached tokens
  keys     mean key of every 64-token page that holds new tokens
  scores   score of every page for every query row: max over heads of scale * <q, mean key>
  select   the K pages of each query row: first and last pages, then the best scores
  sparse   decode over each query row's selected pages

``own`` false computes them with elementary torch operations in 32 bits; ``own`` true makes the
framework's calls.
"""
import math
import random

import torch

own = False

L, D, PAGE = 512, 576, 64           # latent dims (V), cached row, tokens per page
ROW = {"bf16": 1152, "fp8": 584}    # bytes of a cached row
SCALE = 1.0 / math.sqrt(192.0)
MAX_WORK = 300e9                    # flops of the largest prefix case: drawn cases stay below it


def listed():
    return [
        # a two-request batch behind a two-page instruction: launch latency is all there is
        {"name": "prefix_tiny", "op": "prefix", "kv": "bf16", "B": 2, "Sq": 1, "H": 16, "prefix": 128, "suffix": 172, "pad": 0},
        # the benchmark's decode batch behind a common 4096-token prompt, three slots of the
        # batch empty (a step captured for 64 requests that serves 61)
        {"name": "prefix_batch", "op": "prefix", "kv": "bf16", "B": 64, "Sq": 1, "H": 128, "prefix": 4096, "suffix": 512, "pad": 3},
        # one of eight head shards: 16 heads a request, a long document asked about 128 times
        {"name": "prefix_heads16", "op": "prefix", "kv": "bf16", "B": 128, "Sq": 1, "H": 16, "prefix": 32768, "suffix": 1000, "pad": 0},
        # FP8 rows, two tokens a request (one drafted)
        {"name": "prefix_fp8_mtp", "op": "prefix", "kv": "fp8", "B": 64, "Sq": 2, "H": 128, "prefix": 8192, "suffix": 300, "pad": 0},
        # after a prefill: every page of 64 requests
        {"name": "keys_prefill", "op": "keys", "kv": "bf16", "B": 64, "len": 4096, "new": 0},
        # after a decode step over the FP8 cache: one new token a request, ragged lengths
        {"name": "keys_step_fp8", "op": "keys", "kv": "fp8", "B": 128, "len": 8192, "new": 1},
        # a decode batch at ordinary lengths
        {"name": "scores_batch", "op": "scores", "B": 64, "Sq": 1, "H": 128, "len": 4096},
        # few long requests with two query rows each
        {"name": "scores_long_mtp", "op": "scores", "B": 4, "Sq": 2, "H": 128, "len": 131072},
        # 16 of about 64 pages for a decode batch
        {"name": "select_batch", "op": "select", "B": 64, "Sq": 1, "len": 4096, "K": 16, "sink": 1, "local": 1},
        # 64 of up to 2048 pages
        {"name": "select_long", "op": "select", "B": 128, "Sq": 2, "len": 131072, "K": 64, "sink": 1, "local": 2},
        # 64 pages of long requests, two query rows each: the latency of a step at small batch
        {"name": "sparse_long_mtp", "op": "sparse", "kv": "bf16", "B": 4, "Sq": 2, "H": 128, "len": 131072, "K": 64},
        # a large batch of ragged requests over the FP8 cache
        {"name": "sparse_ragged_fp8", "op": "sparse", "kv": "fp8", "B": 128, "Sq": 1, "H": 128, "len": 8192, "K": 32},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "keys", "scores", "select", "sparse"])
    kv = rng.choice(["bf16", "fp8"])
    Sq = rng.choice([1, 1, 1, 2, 3])
    H = rng.choice([128, 128, 64, 32, 16, _log_int(rng, 1, 128)])
    if op == "prefix":
        B, prefix, suffix = _log_int(rng, 1, 128), PAGE * _log_int(rng, 1, 512), Sq + _log_int(rng, 1, 1000)
        while 2 * (D + L) * B * Sq * H * (prefix + suffix) > MAX_WORK:
            B, prefix = max(1, B // 2), max(PAGE, prefix // 128 * 64)
        return {"op": op, "kv": kv, "B": B, "Sq": Sq, "H": H, "prefix": prefix, "suffix": suffix,
                "pad": rng.choice([0, 0, B // 8])}
    if op == "keys":
        length = _log_int(rng, 1, 32768)
        return {"op": op, "kv": kv, "B": _log_int(rng, 1, max(1, min(128, 262144 // length))), "len": length,
                "new": rng.choice([0, 1, Sq, _log_int(rng, 1, length)])}
    length = _log_int(rng, Sq, 131072)
    if op == "scores":
        return {"op": op, "B": _log_int(rng, 1, max(1, min(128, 524288 // (length * Sq)))), "Sq": Sq, "H": H, "len": length}
    if op == "select":
        K = _log_int(rng, 2, 64)
        sink = rng.randint(0, K // 2)
        return {"op": op, "B": _log_int(rng, 1, 128), "Sq": Sq, "len": length, "K": K, "sink": sink,
                "local": rng.randint(0, K - sink)}
    B = _log_int(rng, 1, max(1, min(128, 1048576 // length)))
    return {"op": op, "kv": kv, "B": B, "Sq": Sq, "H": H, "len": length, "K": _log_int(rng, 1, 64)}


# ------------------------------------------------------------------------------------ inputs
def _rng(case, seed):
    """Host draws of one case: the ragged lengths and the like (made alike for `work`)."""
    return random.Random("%d/%s" % (seed, sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case, seed):
    """Cached tokens of every request, the Sq new ones among them."""
    r, B, Sq = _rng(case, seed), case["B"], case.get("Sq", 1)
    if case["op"] == "prefix":
        lens = [case["prefix"] + r.randint(Sq, max(Sq, case["suffix"])) for _ in range(B)]
        lens[0] = case["prefix"] + max(Sq, case["suffix"])
        for b in range(B - case["pad"], B):
            lens[b] = 0
        return lens
    lens = [r.randint(max(Sq, case["len"] // 2), max(Sq, case["len"])) for _ in range(B)]
    lens[0] = max(Sq, case["len"])
    return lens


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(kv, num_blocks, g):
    """Cache pages of N(0, 1) rows: bf16, or e4m3 rows with a scale per token."""
    x = torch.empty((num_blocks * PAGE, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    if kv == "bf16":
        return x.view(torch.uint8).view(num_blocks, PAGE * ROW[kv])
    out = torch.empty((num_blocks * PAGE, ROW[kv]), dtype=torch.uint8, device="cuda")
    step = 32768
    for i in range(0, x.shape[0], step):
        f = x[i:i + step].float()
        s = (f.abs().amax(1, keepdim=True) / 448.0).clamp_min(1e-20)
        out[i:i + step, :D] = (f / s).to(torch.float8_e4m3fn).view(torch.uint8)
        out[i:i + step, D:D + 4] = s.view(torch.uint8)
        out[i:i + step, D + 4:] = s.view(torch.uint8)
    return out.view(num_blocks, PAGE * ROW[kv])


def _table(lens, prefix, g):
    """Block table over scattered blocks; the first prefix / 64 entries are common to all rows."""
    common = prefix // PAGE
    pages = [max(0, -(-n // PAGE) - common) for n in lens]
    num_blocks = common + len(lens) * max(pages) + 16  # the cache's capacity; some of it is free
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32).cpu()
    width = common + max(max(pages), 1)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    table[:, :common] = perm[:common]
    at = common
    for b, n in enumerate(pages):
        table[b, common:common + n] = perm[at:at + n]
        at += n
    return table.cuda(), num_blocks


def prepare(case, seed):
    g, op, lens = _generator(seed), case["op"], _lengths(case, seed)
    B, Sq, H = case["B"], case.get("Sq", 1), case.get("H", 1)
    s = {"op": op, "case": dict(case), "max_len": max(lens),
         "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if op == "select":
        width = -(-max(lens) // PAGE)
        scores = torch.empty((B, Sq, width), device="cuda").normal_(generator=g)
        # a quarter of the rows in coarse steps: many equal scores
        scores[::4] = (scores[::4] * 8).round() / 8
        s["scores"] = scores
        s["pages"] = torch.empty((B, Sq, case["K"]), dtype=torch.int32, device="cuda")
        return s
    s["table"], s["num_blocks"] = _table(lens, case.get("prefix", 0), g)
    if op == "scores":
        keys = torch.empty((s["num_blocks"], D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        s["keys"] = keys / 8  # the mean of 64 unit normals
        s["out"] = torch.empty((B, Sq, -(-max(lens) // PAGE)), device="cuda")
    else:
        s["cache"] = _cache(case["kv"], s["num_blocks"], g)
    if op == "keys":
        s["keys"] = torch.zeros((s["num_blocks"] + 1, D), dtype=torch.bfloat16, device="cuda")
        new = case["new"]
        s["start"] = torch.tensor([max(0, n - new) if new else 0 for n in lens], dtype=torch.int32, device="cuda")
        s["max_new"] = min(new, max(lens)) if new else max(lens)
        return s
    s["q"] = torch.empty((B, Sq, H, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    if op == "sparse":
        K, r = case["K"], _rng(case, seed + 1)
        pages = torch.full((B, Sq, K), -1, dtype=torch.int32)
        for b in range(B):
            for t in range(Sq):
                total = -(-max(0, lens[b] - (Sq - 1 - t)) // PAGE)
                n = min(total, K)
                pick = set(r.sample(range(total), n))
                if n and total - 1 not in pick:  # the row's own page is always read
                    pick.remove(max(pick))
                    pick.add(total - 1)
                pages[b, t, :n] = torch.tensor(sorted(pick), dtype=torch.int32)
        s["pages"] = pages.cuda()
    if op != "scores":
        s["o"] = torch.empty((B, Sq, H, L), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, Sq, H), device="cuda")
    return s


# --------------------------------------------------------------------------------- plain forms
def _rows(s, blocks):
    """K and V (fp32) of whole pages, [..., 64, 576] and [..., 64, 512]."""
    pages = s["cache"][blocks]
    shape = blocks.shape + (PAGE,)
    if s["case"]["kv"] == "bf16":
        k = pages.view(torch.bfloat16).view(shape + (D,)).float()
        return k, k[..., :L]
    pages = pages.view(shape + (ROW["fp8"],))
    x = pages[..., :D].contiguous().view(torch.float8_e4m3fn).float()
    scales = pages[..., D:].contiguous().view(torch.float32)
    return x * scales[..., :1], x[..., :L] * scales[..., 1:]


def _visible(s, Sq):
    """Tokens that each query row sees, [B, Sq]."""
    t = torch.arange(Sq, device="cuda")
    return (s["seq_lens"].long()[:, None] - (Sq - 1 - t)).clamp_min(0)


def _finish(logits, values):
    """bf16 o and fp32 lse from masked logits and a function that multiplies by the values."""
    m = logits.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(logits - m)
    total = p.sum(-1, keepdim=True)
    o = values(p) / torch.where(total > 0, total, torch.ones_like(total))
    return o.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


def _plain_prefix(s):
    c = s["case"]
    B, Sq, H, prefix = c["B"], c["Sq"], c["H"], c["prefix"]
    common = prefix // PAGE
    n = _visible(s, Sq)[:, :, None, None]
    kp, vp = _rows(s, s["table"][0, :common].long())
    kp, vp = kp.view(prefix, D), vp.reshape(prefix, L)
    ks, vs = _rows(s, s["table"][:, common:].long().clamp_min(0))
    ks, vs = ks.view(B, -1, D), vs.reshape(B, -1, L)
    q = s["q"].float()
    a = (q.view(-1, D) @ kp.t()).view(B, Sq, H, prefix)
    b = torch.matmul(q.view(B, Sq * H, D), ks.transpose(1, 2)).view(B, Sq, H, -1)
    logits = torch.cat([a, b], -1) * SCALE
    seen = torch.arange(logits.shape[-1], device="cuda") < n
    logits = logits.masked_fill(~seen, -math.inf)

    def values(p):
        po = p[..., :prefix].reshape(-1, prefix) @ vp
        return po.view(B, Sq, H, L) + torch.matmul(p[..., prefix:].reshape(B, Sq * H, -1), vs).view(B, Sq, H, L)
    return _finish(logits, values)


def _plain_keys(s):
    seq, start = s["seq_lens"].long(), s["start"].long()
    page = torch.arange(s["table"].shape[1], device="cuda")
    written = (page * PAGE < seq[:, None]) & ((page + 1) * PAGE > start[:, None]) & (seq > start)[:, None]
    first = start // PAGE
    touched = min(s["table"].shape[1], (s["max_new"] + PAGE - 1) // PAGE + 1)
    at = (first[:, None] + torch.arange(touched, device="cuda")).clamp_max(s["table"].shape[1] - 1)
    last = torch.cat([torch.ones_like(at[:, :1], dtype=torch.bool), at[:, 1:] != at[:, :-1]], 1)
    live = written.gather(1, at) & last
    blocks = s["table"].long().gather(1, at)
    k, _ = _rows(s, blocks.clamp_min(0))
    valid = (seq[:, None] - at * PAGE).clamp(0, PAGE)
    rows = (torch.arange(PAGE, device="cuda") < valid[..., None])[..., None]
    mean = k.masked_fill(~rows, 0.0).sum(2) / valid.clamp_min(1)[..., None]
    spare = s["num_blocks"]  # the row after the last block takes what is not written
    s["keys"][torch.where(live, blocks, torch.full_like(blocks, spare))] = mean.to(torch.bfloat16)
    return s["keys"][:spare]


def _plain_scores(s):
    c = s["case"]
    B, Sq, H, width = c["B"], c["Sq"], c["H"], s["out"].shape[2]
    keys = s["keys"][s["table"][:, :width].long().clamp_min(0)].float()
    x = torch.matmul(s["q"].float().view(B, Sq * H, D), keys.transpose(1, 2)) * SCALE
    best = x.view(B, Sq, H, width).amax(2)
    seen = torch.arange(width, device="cuda") * PAGE < _visible(s, Sq)[..., None]
    return best.masked_fill(~seen, -math.inf)


def _plain_select(s):
    c = s["case"]
    K, width = c["K"], s["scores"].shape[2]
    total = (_visible(s, c["Sq"]) + PAGE - 1)[..., None] // PAGE
    page = torch.arange(width, device="cuda")
    x = s["scores"].masked_fill(page >= total, -math.inf)
    forced = ((page < c["sink"]) | (page >= total - c["local"])) & (page < total)
    x = x.masked_fill(forced, math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :K]
    order = torch.where(torch.arange(order.shape[-1], device="cuda") < total, order, torch.full_like(order, width))
    order = order.sort(-1).values
    out = torch.full(s["pages"].shape, -1, dtype=torch.int32, device="cuda")
    out[..., :order.shape[-1]] = torch.where(order < width, order, torch.full_like(order, -1)).to(torch.int32)
    return out


def _plain_sparse(s):
    c = s["case"]
    B, Sq, H, K = c["B"], c["Sq"], c["H"], c["K"]
    R = B * Sq
    pages = s["pages"].view(R, K).long()
    table = s["table"].long().repeat_interleave(Sq, 0)
    k, v = _rows(s, table.gather(1, pages.clamp_min(0)))
    k, v = k.view(R, K * PAGE, D), v.reshape(R, K * PAGE, L)
    token = pages[..., None] * PAGE + torch.arange(PAGE, device="cuda")
    seen = ((pages >= 0)[..., None] & (token < _visible(s, Sq).view(R, 1, 1))).view(R, 1, K * PAGE)
    logits = torch.matmul(s["q"].float().view(R, H, D), k.transpose(1, 2)) * SCALE
    o, lse = _finish(logits.masked_fill(~seen, -math.inf), lambda p: torch.matmul(p, v))
    return o.view(B, Sq, H, L), lse.view(B, Sq, H)


def _own(s):
    import mla_latent_kv_gb300 as mla
    c, op = s["case"], s["op"]
    if op == "select":
        return mla.select_pages(s["scores"], s["seq_lens"], c["K"], sink_pages=c["sink"], local_pages=c["local"],
                                pages=s["pages"])
    if op == "scores":
        return mla.page_scores(s["q"], s["keys"], s["table"], s["seq_lens"], s["max_len"], SCALE, scores=s["out"])
    kv = mla.KV_BF16 if c["kv"] == "bf16" else mla.KV_FP8
    if op == "keys":
        return mla.page_keys(s["cache"], s["table"], s["seq_lens"], s["max_new"], kv_dtype=kv, start_lens=s["start"],
                             page_keys=s["keys"][:s["num_blocks"]])
    if op == "prefix":
        return mla.decode_shared_prefix(s["q"], s["cache"], s["table"], s["seq_lens"], s["max_len"], c["prefix"], SCALE,
                                        kv_dtype=kv, o_latent=s["o"], lse=s["lse"])
    return mla.decode_sparse(s["q"], s["cache"], s["table"], s["seq_lens"], s["pages"], SCALE, kv_dtype=kv,
                             o_latent=s["o"], lse=s["lse"])


def run(state):
    if own:
        return _own(state)
    return {"prefix": _plain_prefix, "keys": _plain_keys, "scores": _plain_scores, "select": _plain_select,
            "sparse": _plain_sparse}[state["op"]](state)


# ------------------------------------------------------------------------------------- figures
def work(case):
    """Bytes read and written once each, and the formula's flops, for seed 0's lengths."""
    op, lens = case["op"], _lengths(case, 0)
    B, Sq, H = case["B"], case.get("Sq", 1), case.get("H", 1)
    rows = [max(0, n - (Sq - 1 - t)) for n in lens for t in range(Sq)]
    pages = [-(-n // PAGE) for n in rows]
    if op == "select":
        return {"bytes": 4 * sum(pages) + 4 * B * Sq * case["K"] + 4 * B, "flops": 0}
    if op == "scores":
        own_pages = sum(-(-n // PAGE) for n in lens)
        return {"bytes": own_pages * (2 * D + 4) + B * Sq * H * 2 * D + 4 * B * Sq * -(-max(lens) // PAGE) + 4 * B,
                "flops": 2 * D * H * sum(pages)}
    row = ROW[case["kv"]]
    if op == "keys":
        got = [(n, -(-n // PAGE) - (max(0, n - case["new"]) if case["new"] else 0) // PAGE) for n in lens]
        tokens = sum(n - (-(-n // PAGE) - p) * PAGE for n, p in got)
        touched = sum(p for _, p in got)
        return {"bytes": tokens * row + touched * (2 * D + 4) + 8 * B, "flops": tokens * D}
    out = B * Sq * H * (2 * D + 2 * L + 4) + 4 * B
    if op == "prefix":
        common = case["prefix"]
        own_tokens = sum(max(0, n - common) for n in lens)
        return {"bytes": (common + own_tokens) * row + 4 * (common + own_tokens) // PAGE + out,
                "flops": 2 * (D + L) * H * sum(rows)}
    tokens = sum(min(n, case["K"] * PAGE) for n in rows)
    return {"bytes": tokens * row + 8 * B * Sq * case["K"] + out, "flops": 2 * (D + L) * H * tokens}


# --------------------------------------------------------------------- the definition, in 64 bits
def _row64(s, block, count):
    """K and V of the first `count` tokens of one block, from its bytes, in 64 bits."""
    raw = s["cache"][block].view(PAGE, -1)[:count]
    if s["case"]["kv"] == "bf16":
        k = raw.contiguous().view(torch.bfloat16).double()
        return k, k[:, :L]
    code = raw[:, :D].contiguous().view(torch.float8_e4m3fn).double()
    ks = raw[:, D:D + 4].contiguous().view(torch.float32).double()
    vs = raw[:, D + 4:D + 8].contiguous().view(torch.float32).double()
    return code * ks, code[:, :L] * vs


def _attend64(q, k, v):
    """One request's rows against its tokens: softmax(scale q k^T) v and its log-sum."""
    if not k.shape[0]:
        return torch.zeros(q.shape[0], L, dtype=torch.float64, device="cuda"), \
            torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device="cuda")
    x = q.double() @ k.t() * SCALE
    lse = torch.logsumexp(x, 1)
    return torch.exp(x - lse[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    op, lens, Sq = case["op"], _lengths(case, seed), case.get("Sq", 1)
    if op == "select":
        return None
    table = s["table"].tolist()
    if op == "keys":
        out = torch.zeros(s["num_blocks"], D, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            start = max(0, n - case["new"]) if case["new"] else 0
            for page in range(start // PAGE, -(-n // PAGE)):
                k, _ = _row64(s, table[b][page], min(PAGE, n - page * PAGE))
                out[table[b][page]] = k.mean(0)
        return out
    if op == "scores":
        out = torch.full(s["out"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            for t in range(Sq):
                total = -(-max(0, n - (Sq - 1 - t)) // PAGE)
                if total:
                    keys = s["keys"][s["table"][b, :total].long()].double()
                    out[b, t, :total] = (s["q"][b, t].double() @ keys.t() * SCALE).max(0).values
        return out
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    chosen = s["pages"].tolist() if op == "sparse" else None
    shared = [_row64(s, blk, PAGE) for blk in table[0][:case["prefix"] // PAGE]] if op == "prefix" else []
    for b, n in enumerate(lens):
        for t in range(Sq):
            seen = max(0, n - (Sq - 1 - t))
            ids = [p for p in chosen[b][t] if p >= 0] if chosen else range(-(-seen // PAGE))
            kv = []
            for p in ids:
                count = min(PAGE, seen - p * PAGE)
                k, v = shared[p] if p < len(shared) else _row64(s, table[b][p], count)
                kv.append((k[:count], v[:count]))
            if kv:
                k, v = torch.cat([x for x, _ in kv]), torch.cat([x for _, x in kv])
                o[b, t], lse[b, t] = _attend64(s["q"][b, t], k, v)
    return o, lse
