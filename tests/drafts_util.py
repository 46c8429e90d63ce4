"""Helpers of the tests of a step with drafted tokens: the operators' definitions, plainly and in 64 bits.

Bounds of the attention are those of longctx_util. Rotary positions: the angle is off by at most 2^-25 of
a turn (its fp32 form), cosine, sine, two products and a sum by a few 2^-24 of |u| + |v|: together
under 2^-20 (|u| + |v|) mscale, and the one rounding to bf16 by 2^-8 of the result.
"""
from __future__ import annotations

import math

import numpy as np

import mla_inputs as mi
from longctx_util import D, L, PAGE, keys_values, paged_case

R = 64


def tree_masks(B, Sq, seed):
    """Random trees: a draft's parent is an earlier one or none; bit i of word t: t sees i -> int64 [B, Sq]."""
    rng = np.random.default_rng(seed)
    out = np.zeros((B, Sq), np.uint64)
    for b in range(B):
        for t in range(Sq):
            parent = int(rng.integers(-1, t)) if rng.random() < 0.6 else t - 1
            out[b, t] = (out[b, parent] if parent >= 0 else np.uint64(0)) | np.uint64(1 << t)
    return out.view(np.int64)


def tree_case(lens, Sq, H, kv, seed, masks=None, **kw):
    import torch
    c = paged_case(lens, Sq, H, kv, seed, **kw)
    c["masks_host"] = tree_masks(c["B"], Sq, seed + 1) if masks is None else np.asarray(masks).astype(np.int64)
    c["masks"] = torch.from_numpy(np.ascontiguousarray(c["masks_host"])).cuda()
    return c


def attend_tree(c):
    """o, lse and their error bounds (those of longctx_util.attend) of every draft, only over what it sees."""
    import torch
    k_all, v_all = keys_values(c)
    B, Sq, H = c["B"], c["Sq"], c["H"]
    o = torch.zeros((B, Sq, H, L), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Sq, H), -math.inf, dtype=torch.float64, device="cuda")
    tol_o, tol_lse = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        n = int(c["lens"][b])
        blocks = torch.as_tensor(c["full_table"][b, :-(-n // PAGE)].astype(np.int64), device="cuda")
        k_row, v_row = k_all[blocks].view(-1, D)[:n], v_all[blocks].view(-1, L)[:n]
        for t in range(Sq):
            word = int(c["masks_host"][b, t])
            see = [j for j in range(n) if j < n - Sq or word >> (j - (n - Sq)) & 1]
            if not see:
                continue
            at = torch.tensor(see, device="cuda")
            k, v, q = k_row[at], v_row[at], c["q"][b, t].double()
            x = q @ k.t() * c["scale"]
            lse[b, t] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b, t][:, None])
            o[b, t] = p @ v
            mag = p @ v.abs()
            tol_o[b, t] = 2.0 ** -8 * (mag + o[b, t].abs()) + 2.0 ** -12 * mag
            tol_lse[b, t] = 576 * 2.0 ** -24 * c["scale"] * (q.abs() @ k.abs().t()).amax(1) + \
                2.0 ** -18 * (1 + lse[b, t].abs())
    return o, lse, tol_o, tol_lse


def turn64(x, positions, freq, adjacent, mscale=1.0):
    """Rows [T, N, 64] turned by their positions, in 64 bits, and the error bound of the bf16 result."""
    import torch
    x = x.double()
    a = positions.double()[:, None, None] * freq.to(x.device)
    c, s = torch.cos(a) * mscale, torch.sin(a) * mscale
    u, v = (x[..., 0::2], x[..., 1::2]) if adjacent else (x[..., :R // 2], x[..., R // 2:])
    p, q = u * c - v * s, v * c + u * s
    m = (u.abs() + v.abs()) * abs(mscale)
    join = (lambda g, h: torch.stack([g, h], -1).flatten(-2)) if adjacent else (lambda g, h: torch.cat([g, h], -1))
    return join(p, q), 2.0 ** -8 * join(p, q).abs() + 2.0 ** -20 * join(m, m)


def accept_rule(cache, table, lens, path, counts):
    """accept_tokens on numpy arrays: cache [layers, blocks, 64, row] -> (new cache, new lens, whether a branch was bad)."""
    out, new, bad = cache.copy(), [], False
    Sq = path.shape[1]
    for b, n in enumerate(int(x) for x in lens):
        first, gone = max(0, n - Sq), max(0, Sq - n)
        keep = []
        for i in range(min(max(int(counts[b]), 0), Sq)):
            p = int(path[b, i])
            if p <= (keep[-1] if keep else gone - 1) or p >= Sq:
                break
            keep.append(p)
        bad |= len(keep) != int(counts[b])
        for i, p in enumerate(keep):
            s, d = n - Sq + p, first + i
            out[:, table[b, d // PAGE], d % PAGE] = cache[:, table[b, s // PAGE], s % PAGE]
        new.append(first + len(keep))
    return out, np.array(new, np.int32), bad


def fork_rule(cache, table, counts, lens, refs, parents, room):
    """fork_pages on numpy arrays, page by page -> (cache, table, counts, lens, refs), or None if pages run out."""
    free = [int(p) for p in np.flatnonzero(refs == 0)]
    cache, new_refs, rows, seen = cache.copy(), refs.astype(np.int64).copy(), [], set()
    width = table.shape[1]
    copies = []
    for r, p in enumerate(int(x) for x in parents):
        n = int(lens[p]) if p >= 0 else 0
        held = int(counts[p]) if p >= 0 else 0
        need = -(-max(n, int(room[r])) // PAGE)
        first_child = p >= 0 and p not in seen
        seen.add(p)
        row = []
        for j in range(need):
            old = int(table[p, j]) if p >= 0 and j < held else -1
            if j < n // PAGE or (first_child and old >= 0 and refs[old] == 1):
                row.append(old)
                continue
            if not free:
                return None
            row.append(free.pop(0))
            if j == n // PAGE and n % PAGE:
                copies.append((old, row[-1], n % PAGE))
        rows.append(row)
    for s, d, m in copies:
        cache[:, d, :m] = cache[:, s, :m]
    for b in range(len(lens)):
        for j in range(int(counts[b])):
            new_refs[table[b, j]] -= 1
    for row in rows:
        for page in row:
            new_refs[page] += 1
    out = np.full((len(rows), width), -1, np.int32)
    for r, row in enumerate(rows):
        out[r, :len(row)] = row
    new_lens = np.array([int(lens[p]) if p >= 0 else 0 for p in parents], np.int32)
    return cache, out, np.array([len(r) for r in rows], np.int32), new_lens, new_refs.astype(np.int32)


def random_pool(B, width, num_blocks, layers, kv, seed, top):
    """A pool state of B rows of up to `top` tokens, rows of three sharing their first pages, a page too many
    held here and there, and some pages held by nobody in the table (another holder's)."""
    rng = np.random.default_rng(seed)
    row = {mi.KV_BF16: 1152, mi.KV_FP8: 584}[kv]
    cache = rng.integers(0, 256, (layers, num_blocks, PAGE, row), dtype=np.uint8)
    perm = [int(p) for p in rng.permutation(num_blocks)]
    lens = rng.integers(0, top + 1, B).astype(np.int32)
    lens[rng.random(B) < 0.2] //= PAGE
    lens[rng.random(B) < 0.2] = 0
    table, counts, refs = np.full((B, width), -1, np.int32), np.zeros(B, np.int32), np.zeros(num_blocks, np.int32)
    for b in range(B):
        n = -(-int(lens[b]) // PAGE)
        held = min(width, n + int(rng.integers(0, 3)) * int(rng.random() < 0.4))
        lead = b - b % 3
        shared = min(int(lens[b]) // PAGE, int(lens[lead]) // PAGE) if b % 3 else 0
        pages = [int(x) for x in table[lead, :shared]] + [perm.pop() for _ in range(held - shared)]
        table[b, :held] = pages
        counts[b] = held
        for p in pages:
            refs[p] += 1
        if held and rng.random() < 0.2:  # a prefix cache holds one of them too
            refs[pages[int(rng.integers(0, held))]] += 1
    return dict(cache=cache, table=table, counts=counts, lens=lens, refs=refs)
