"""Helpers of the long-context tests: paged inputs on the device and the operators' definitions in 64
bits (plain torch float64), with the error bounds that the comparisons use.

Bounds. One rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by 2^-24.
  o    The kernels round each softmax weight to bf16 once: with weights p, values v and result o,
       |err| <= 2^-8 (sum p |v| + |o|), the second term from the weights' sum. Sums and exponentials in fp32
       add less than 2^-12 of sum p |v|. A bf16 result adds 2^-8 |o|.
  lse  A logit is an fp32 sum of 576 exact products: off by at most 576 * 2^-24 of the sum of their
       magnitudes (times scale); exp2, log2 and the sums add less than 2^-18 (1 + |lse|).
"""
from __future__ import annotations

import math

import numpy as np

import mla_inputs as mi

L, D, PAGE = mi.L, mi.D, mi.PAGE


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def paged_case(lens, Sq, H, kv, seed, prefix=0, extra_cols=0, scale_v=None):
    """Seeded inputs on the device. The first prefix / 64 table entries of every request are one
    list of pages (row 0's; the other rows hold -1 there); rows that no request may read are NaN."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int64)
    common = prefix // PAGE
    own = np.maximum(0, -(-lens // PAGE) - common)
    num_blocks = common + int(own.sum()) + 5
    perm = rng.permutation(num_blocks).astype(np.int32)
    table = np.full((len(lens), common + max(1, int(own.max(initial=0))) + extra_cols), -1, np.int32)
    table[0, :common] = perm[:common]
    at = common
    valid = np.zeros((num_blocks, PAGE), bool)
    valid[perm[:common]] = True
    for b, n in enumerate(own):
        table[b, common:common + n] = perm[at:at + n]
        at += n
        for p in range(int(n)):
            valid[table[b, common + p], :min(PAGE, int(lens[b]) - (common + p) * PAGE)] = True
    cache = mi.make_cache(num_blocks, kv, rng, valid)
    if scale_v is not None:  # a v_scale of its own, so that a swap with k_scale shows
        c = cache.reshape(num_blocks, PAGE, -1)
        vs = c[:, :, D + 4:D + 8].copy().view("<f4") * np.float32(scale_v)
        c[:, :, D + 4:D + 8] = vs.view(np.uint8)
    full = table.copy()
    full[:, :common] = table[0, :common]
    return dict(B=len(lens), Sq=Sq, H=H, kv=kv, lens=lens, prefix=prefix, num_blocks=num_blocks, scale=mi.SCALE,
                max_len=int(lens.max(initial=0)), cache=dev(cache), table=dev(table), full_table=full,
                seq_lens=dev(lens.astype(np.int32)), q=bf16(mi.normal_bf16(rng, (len(lens), Sq, H, D))))


def keys_values(c):
    """K [num_blocks, 64, 576] and V [num_blocks, 64, 512] in 64 bits."""
    import torch
    if c["kv"] == mi.KV_BF16:
        k = c["cache"].view(torch.bfloat16).view(c["num_blocks"], PAGE, D).double()
        return k, k[..., :L]
    raw = c["cache"].view(c["num_blocks"], PAGE, D + 8)
    code = raw[..., :D].contiguous().view(torch.float8_e4m3fn).double()
    sc = raw[..., D:].contiguous().view(torch.float32).double()
    return code * sc[..., :1], code[..., :L] * sc[..., 1:]


def attend(c, pages=None):
    """o, lse and their error bounds, over every visible token or over pages[b][t] (lists)."""
    import torch
    k_all, v_all = keys_values(c)
    B, Sq, H = c["B"], c["Sq"], c["H"]
    o = torch.zeros((B, Sq, H, L), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Sq, H), -math.inf, dtype=torch.float64, device="cuda")
    tol_o, tol_lse = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        for t in range(Sq):
            n = max(0, int(c["lens"][b]) - (Sq - 1 - t))
            ids = range(-(-n // PAGE)) if pages is None else pages[b][t]
            take = [(int(c["full_table"][b, p]), min(PAGE, n - p * PAGE)) for p in ids]
            if not take:
                continue
            k = torch.cat([k_all[blk, :m] for blk, m in take])
            v = torch.cat([v_all[blk, :m] for blk, m in take])
            q = c["q"][b, t].double()
            x = q @ k.t() * c["scale"]
            lse[b, t] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b, t][:, None])
            o[b, t] = p @ v
            mag = p @ v.abs()
            tol_o[b, t] = 2.0 ** -8 * (mag + o[b, t].abs()) + 2.0 ** -12 * mag
            tol_lse[b, t] = 576 * 2.0 ** -24 * c["scale"] * (q.abs() @ k.abs().t()).amax(1) + \
                2.0 ** -18 * (1 + lse[b, t].abs())
    return o, lse, tol_o, tol_lse


def check_attention(o, lse, want, bf16_out=False):
    import torch
    o_ref, lse_ref, tol_o, tol_lse = want
    empty = torch.isinf(lse_ref)
    assert torch.isfinite(o.double()).all()
    assert bool((lse[empty] == -math.inf).all()) and bool((o[empty] == 0).all())
    if bf16_out:
        tol_o = tol_o + 2.0 ** -8 * o_ref.abs()
    over = ((o.double() - o_ref).abs() - tol_o).max().item() if o.numel() else -1.0
    assert over <= 0, f"o is {over} over its bound"
    if (~empty).any():
        over = ((lse.double() - lse_ref).abs() - tol_lse)[~empty].max().item()
        assert over <= 0, f"lse is {over} over its bound"


def check_with_nan(o, lse, want):
    """check_attention where the definition is finite, and NaN exactly where it is NaN. (Of a score of +inf
    the definition's lse is +inf, the kernels' NaN.)"""
    import torch
    o_ref, lse_ref, tol_o, tol_lse = want
    bad = lse_ref.isnan() | (lse_ref == math.inf)
    assert torch.equal(o.isnan(), o_ref.isnan()) and torch.equal(lse.isnan(), bad)
    z = lambda x, m: torch.where(m, torch.zeros_like(x), x)  # noqa: E731
    check_attention(z(o, o.isnan()), z(lse, bad),
                    (z(o_ref, o_ref.isnan()), z(lse_ref, bad), z(tol_o, o_ref.isnan()), z(tol_lse, bad)))


def select_rule(scores, n, K, sink, local):
    """The selection's definition for one row: scores [width] (numpy), n visible tokens."""
    np_ = -(-n // PAGE)
    if np_ <= K:
        return list(range(np_))
    forced = list(range(sink)) + list(range(np_ - local, np_))
    others = [j for j in range(sink, np_ - local)]
    rank = sorted(others, key=lambda j: (np.isnan(scores[j]), -scores[j] if not np.isnan(scores[j]) else 0.0, j))
    return sorted(forced + rank[:K - sink - local])
