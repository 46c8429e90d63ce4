"""Decode over a shared prefix and over selected pages, on the GPU, against their definitions in 64 bits."""
import math

import numpy as np
import pytest

import mla_inputs as mi
from longctx_util import (D, L, PAGE, attend, bf16, check_attention, check_with_nan, dev, keys_values, paged_case,
                          select_rule)

pytestmark = pytest.mark.gpu
BF, F8 = mi.KV_BF16, mi.KV_FP8


def _status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------------------- shared prefix
# Small calls run on the decode kernels alone, larger ones on the prefix kernel too (`_kernel` says
# which from the workspace: its partial states come on top of the decode's).
def _prefix(c, num_splits=-1, status=None, max_len=None, **kw):
    import mla_latent_kv_gb300 as mla
    return mla.decode_shared_prefix(c["q"], c["cache"], c["table"], c["seq_lens"], max_len or c["max_len"], c["prefix"],
                                    c["scale"], kv_dtype=c["kv"], num_splits=num_splits, dev_status=status,
                                    num_blocks=c["num_blocks"], **kw)


def _kernel(c, num_splits=-1):
    import mla_latent_kv_gb300 as mla
    need = [mla.decode_shared_prefix_workspace_bytes(c["B"], c["Sq"], c["H"], prefix, c["max_len"], c["kv"], num_splits)
            for prefix in (c["prefix"], 0)]
    return need[0] != need[1]


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("B,Sq,H,prefix,suffix,kernel", [
    (1, 1, 1, 64, [1], False),                      # one row of one head, one page
    (2, 1, 16, 128, [172, 3], False),
    (3, 1, 20, 192, [1, 64, 65], False),
    (9, 3, 37, 320, [3, 5, 64, 66, 200, 4, 9, 128, 129], False),
    (2, 1, 128, 4096, [1, 100], False),
    (150, 1, 5, 448, [1 + b % 70 for b in range(150)], None),      # 750 rows: the last tile a partial one
    (160, 1, 5, 448, [1 + b % 70 for b in range(160)], True),      # 800 rows, 7 pages
    (101, 2, 7, 704, [2 + b % 130 for b in range(101)], True),     # 11 pages, ranges of an even number
    (200, 1, 1, 960, [1 + b % 64 for b in range(200)], True),      # one tile, 200 of its 256 rows
    (130, 1, 8, 1024, [1 + b % 90 for b in range(130)], True),
    (33, 3, 37, 1984, [3 + 9 * b for b in range(33)], True),       # 31 pages, 37 heads
    (36, 1, 128, 4160, [1 + 16 * b for b in range(36)], True),     # whole tiles, 65 pages
])
def test_shared_prefix(kv, B, Sq, H, prefix, suffix, kernel):
    c = paged_case([prefix + s for s in suffix], Sq, H, kv, seed=B * 100 + H, prefix=prefix,
                   scale_v=0.5 if kv == F8 else None)
    assert kernel is None or _kernel(c) == kernel  # None: on one side of the border by the cache's type
    st = _status()
    o, lse = _prefix(c, status=st)
    assert int(st.item()) == 0
    check_attention(o, lse, attend(c))


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("num_splits", [1, 3, 0, -1, -2])
@pytest.mark.parametrize("B", [4, 112, 160])
def test_shared_prefix_suffix_splits_and_bf16_output(kv, num_splits, B):
    import mla_latent_kv_gb300 as mla
    c = paged_case([640 + (1, 700, 64, 129)[b % 4] for b in range(B)], 1, 12, kv, seed=7, prefix=640)
    if B != 112:
        assert _kernel(c, num_splits) == (B == 160)
    o, lse = _prefix(c, num_splits, o_dtype=mla.DT_BF16)
    check_attention(o, lse, attend(c), bf16_out=True)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("B", [10, 140])
def test_shared_prefix_rows_inside_the_prefix(kv, B):
    """Requests shorter than the prefix see their own tokens only; empty slots give o = 0, lse = -inf."""
    lens = [[640 + 70, 0, 1, 2, 64, 100, 255, 640, 641, 0][b % 10] for b in range(B)]
    c = paged_case(lens, 2, 6, kv, seed=11, prefix=640)
    assert _kernel(c) == (B == 140)
    o, lse = _prefix(c)
    check_attention(o, lse, attend(c))


@pytest.mark.parametrize("kv", [BF, F8])
def test_shared_prefix_every_slot_empty_and_no_prefix(kv):
    c = paged_case([0] * 160, 1, 16, kv, seed=12, prefix=704)
    for max_len in (0, 704, 704 + 64):  # a captured step's bound, whatever the slots hold
        c["max_len"] = max_len
        assert _kernel(c) == (max_len > 0)
        o, lse = _prefix(dict(c, table=torch_pad(c["table"], 13)), max_len=max_len)
        check_attention(o, lse, attend(c))
    c = paged_case([300, 5], 1, 16, kv, seed=13, prefix=0)
    o, lse = _prefix(c)
    check_attention(o, lse, attend(c))


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H", [16, 40])
@pytest.mark.parametrize("num_splits", [-1, 1, 3, -2])
def test_shared_prefix_longer_than_the_bound(kv, H, num_splits):
    """A bound on the lengths that ends inside a page of the prefix: that page is read by each request itself."""
    lens = [(1800, 1792, 1799, 0, 1728, 65, 1, 1793)[b % 8] for b in range(160)]
    c = paged_case(lens, 2, H, kv, seed=24, prefix=2560)
    assert c["max_len"] == 1800 and _kernel(c, num_splits)
    st = _status()
    o, lse = _prefix(c, num_splits, st)
    assert int(st.item()) == 0
    check_attention(o, lse, attend(c))


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("num_splits", [1, 2, -2])
def test_shared_prefix_no_tokens_of_their_own(kv, num_splits):
    """Nothing behind the prefix in any request: the prefix's states alone make the result."""
    lens = [[704, 703, 64, 1, 0][b % 5] for b in range(160)]
    c = paged_case(lens, 1, 16, kv, seed=19, prefix=704, extra_cols=3)
    assert _kernel(c)
    st = _status()
    o, lse = _prefix(c, num_splits, status=st, max_len=704 + 128)
    assert int(st.item()) == 0
    check_attention(o, lse, attend(c))


@pytest.mark.parametrize("B", [3, 180])
def test_shared_prefix_length_past_the_bound_is_reported(B):
    """As for decode, such a request's result is undefined; the others' are right."""
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case([640 + 60 + b % 40 for b in range(B)], 2, 8, BF, seed=21, prefix=640)
    st = _status()
    bound = c["max_len"] - 1
    o, lse = _prefix(c, status=st, max_len=bound)
    assert int(st.item()) == mla.DEV_SEQ_TOO_LONG
    fits = torch.from_numpy(c["lens"] <= bound).cuda()
    assert 0 < int(fits.sum()) < B
    check_attention(o[fits], lse[fits], [x[fits] for x in attend(c)])


@pytest.mark.parametrize("kv,H", [(BF, 16), (BF, 128), (F8, 16), (F8, 48)])
@pytest.mark.parametrize("bound,blocks", [(0, None), (200, 0)])
def test_a_bound_of_zero_or_no_blocks_reads_no_cache(kv, H, bound, blocks):
    """Lengths above a bound of 0, or in a cache of no blocks, are reported, and every row is empty."""
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case([200, 0, 64], 1, H, kv, seed=22)
    nb = c["num_blocks"] if blocks is None else blocks
    for num_splits in (1, 3, -2):
        for call in ("decode", "prefix") + (("sparse",) if blocks == 0 else ()):  # that one has no bound
            st = _status()
            kw = dict(kv_dtype=kv, num_splits=num_splits, dev_status=st, num_blocks=nb)
            if call == "decode":
                o, lse = mla.decode(c["q"], c["cache"], c["table"], c["seq_lens"], bound, c["scale"], **kw)
            elif call == "prefix":
                o, lse = mla.decode_shared_prefix(c["q"], c["cache"], c["table"], c["seq_lens"], bound, 64, c["scale"], **kw)
            else:
                pages = torch.tensor([[[0, 1]], [[-1, -1]], [[0, -1]]], dtype=torch.int32, device="cuda")
                o, lse = mla.decode_sparse(c["q"], c["cache"], c["table"], c["seq_lens"], pages, c["scale"], **kw)
            assert int(st.item()) & mla.DEV_SEQ_TOO_LONG, (call, num_splits)
            assert bool((o == 0).all()) and bool((lse == -math.inf).all()), (call, num_splits)


def torch_pad(table, cols):
    """The table with -1 columns behind, `cols` in all."""
    import torch
    out = torch.full((table.shape[0], cols), -1, dtype=torch.int32, device="cuda")
    out[:, :table.shape[1]] = table
    return out


@pytest.mark.parametrize("B", [2, 130])
def test_shared_prefix_moving_maximum(B):
    """Keys that grow along the prefix: the running maximum moves past the rescale threshold often."""
    import torch
    c = paged_case([1024 + (40, 3)[b % 2] for b in range(B)], 1, 9, BF, seed=14, prefix=1024)
    assert _kernel(c) == (B == 130)
    rows = c["cache"].view(torch.bfloat16).view(c["num_blocks"], PAGE, D)
    for i, blk in enumerate(c["full_table"][0, :16]):
        rows[int(blk)] *= 1.0 + i
    o, lse = _prefix(c)
    check_attention(o, lse, attend(c))


def test_shared_prefix_equals_decode_at_scale():
    """2048 rows of 16 heads over 16384 shared tokens: against the same call without sharing."""
    import torch
    import mla_latent_kv_gb300 as mla
    B, H, prefix = 128, 16, 16384
    c = paged_case([prefix + 1 + 7 * b for b in range(B)], 1, H, BF, seed=15, prefix=prefix)
    st = _status()
    o, lse = _prefix(c, status=st)
    o2, lse2 = mla.decode(c["q"], c["cache"], dev(c["full_table"]), c["seq_lens"], c["max_len"], c["scale"],
                          num_splits=-1, num_blocks=c["num_blocks"])
    assert int(st.item()) == 0
    # each side rounds its weights to bf16 (2^-8); over thousands of tokens of N(0, 1) values the
    # sums |p| |v| + |o| stay below 2
    assert (o - o2).abs().max().item() <= 2 * 2 * 2.0 ** -8
    assert (lse - lse2).abs().max().item() <= 2 * (576 * 2.0 ** -24 * 40 + 2.0 ** -18 * 20)
    assert torch.isfinite(o).all()


def _mark_pages(c):
    """Prefix page i holds a large value in dim i: its part of the result's dim i is the page's own, so that
    another page's values, or another page's weights, show there."""
    import torch
    n = c["prefix"] // PAGE
    assert n <= L
    for i, blk in enumerate(c["full_table"][0, :n]):
        if c["kv"] == BF:
            c["cache"].view(torch.bfloat16).view(c["num_blocks"], PAGE, D)[int(blk), :, i] = 16.0
        else:
            c["cache"].view(c["num_blocks"], PAGE, D + 8)[int(blk), :, i] = 0x7E  # 448, the largest code


@pytest.mark.parametrize("kv,B,H", [(BF, 128, 16), (F8, 128, 16), (BF, 24, 128), (F8, 30, 128)])
def test_shared_prefix_values_at_scale(kv, B, H):
    """16384 shared tokens, in several ranges of many pages each, against the definition: the bound is of
    each element, where one page's own part of a result is several times the bound."""
    c = paged_case([16384 + 1 + 7 * b for b in range(B)], 1, H, kv, seed=23, prefix=16384,
                   scale_v=0.5 if kv == F8 else None)
    _mark_pages(c)
    assert _kernel(c)
    st = _status()
    o, lse = _prefix(c, status=st)
    assert int(st.item()) == 0
    want = attend(c)
    check_attention(o, lse, want)
    own = want[0][..., :256] / want[2][..., :256]  # dim i of page i, in units of the bound
    assert own.abs().median().item() > 2


@pytest.mark.parametrize("kv", [BF, F8])
def test_shared_prefix_repeats_bit_for_bit(kv):
    """Forty calls over a workspace of NaN: a partial state that is stored too early, or read before it
    is stored, shows as another result (the output CTAs' waits by barrier parity depend on it)."""
    import torch
    import mla_latent_kv_gb300 as mla
    B, H, prefix = 96, 16, 8192
    c = paged_case([prefix + 1 + 5 * b for b in range(B)], 1, H, kv, seed=18, prefix=prefix)
    ws = torch.empty(mla.decode_shared_prefix_workspace_bytes(B, 1, H, prefix, c["max_len"], kv), dtype=torch.uint8,
                     device="cuda")
    first = None
    for _ in range(40):
        ws.fill_(0xFF)
        o, lse = _prefix(c, workspace=ws)
        if first is None:
            first = (o, lse)
            assert torch.isfinite(o).all()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("B", [2, 160])
def test_shared_prefix_bad_prefix_block_is_reported(kv, B):
    c = paged_case([700] * B, 1, 16, kv, seed=16, prefix=640)
    assert _kernel(c) == (B == 160)
    c["table"][0, 1] = c["num_blocks"] + 3
    st = _status()
    _prefix(c, status=st)
    assert int(st.item()) & 0x1


def test_shared_prefix_workspace_is_checked():
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case([700 + b for b in range(160)], 1, 16, BF, seed=17, prefix=640)
    need = mla.decode_shared_prefix_workspace_bytes(160, 1, 16, 640, c["max_len"])
    if need:
        with pytest.raises(mla.MlaError) as e:
            _prefix(c, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.status == mla.ERR_WORKSPACE_TOO_SMALL
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN bytes
    o, lse = _prefix(c, workspace=ws[:need])
    check_attention(o, lse, attend(c))
    assert bool((ws[need:] == 0xFF).all())


# --------------------------------------------------------------------------- NaN in cached rows
def _plant(c, b, token, what):
    """Token `token` of request b holds NaN: one value of its row, or (FP8) its k_scale or v_scale. "inf" is
    an infinite value in its row (bf16), "page" a NaN in every row of its page."""
    import torch
    blk = int(c["full_table"][b, token // PAGE])
    rows = slice(None) if what == "page" else token % PAGE
    if c["kv"] == BF:
        c["cache"].view(torch.bfloat16).view(c["num_blocks"], PAGE, D)[blk, rows, 70] = \
            math.inf if what == "inf" else math.nan
    else:
        sc = c["cache"].view(c["num_blocks"], PAGE, D + 8)[blk, rows, D:].view(torch.float32)
        sc[..., 1 if what == "v" else 0] = math.nan


_NAN = [(BF, 128, "row"), (BF, 128, "page"), (BF, 128, "inf"), (BF, 16, "row"), (BF, 16, "page"), (BF, 32, "inf"),
        (F8, 128, "row"), (F8, 128, "page"), (F8, 128, "v"), (F8, 16, "row"), (F8, 16, "page"), (F8, 32, "v")]


@pytest.mark.parametrize("kv,H,what", _NAN)
@pytest.mark.parametrize("num_splits", [1, 3, 7, -2])
def test_a_nan_key_is_a_nan_result(kv, H, what, num_splits):
    """A row that sees a NaN key has a NaN result, whatever its split and its place; the others none."""
    import mla_latent_kv_gb300 as mla
    lens = [700, 700, 700, 64, 3, 700, 129]
    c = paged_case(lens, 2, H, kv, seed=200)
    for b, token in ((0, 0), (1, 300), (2, 699), (3, 1), (5, 639)):  # the third: seen by its last row only
        _plant(c, b, token, what)
    want = attend(c)
    assert want[0].isnan().any()
    o, lse = mla.decode(c["q"], c["cache"], c["table"], c["seq_lens"], c["max_len"], c["scale"], kv_dtype=kv,
                        num_splits=num_splits, num_blocks=c["num_blocks"])
    check_with_nan(o, lse, want)
    lists, K = [], 6
    table = np.full((len(lens), 2, K), -1, np.int32)
    for b, n in enumerate(lens):
        lists.append([])
        for t in range(2):
            total = -(-(n - (1 - t)) // PAGE)
            ids = [p for p in (0, 2, 4, 9, 10) if p < total and not (b == 5 and p == 9)]
            table[b, t, :len(ids)] = ids
            lists[-1].append(ids)
    o, lse = _sparse(c, table, num_splits)
    check_with_nan(o, lse, attend(c, lists))


@pytest.mark.parametrize("kv,H,what", _NAN)
@pytest.mark.parametrize("B", [4, 160])
def test_a_nan_key_in_the_shared_prefix(kv, H, what, B):
    """Every request that sees it has a NaN result, also over many ranges; a NaN among one request's own
    tokens stays with that request."""
    c = paged_case([1024 + 1 + 11 * (b % 20) for b in range(B)], 1, H, kv, seed=201, prefix=1024)
    assert H != 16 or _kernel(c) == (B == 160)
    _plant(c, 1, 1024 + 5, what)
    want = attend(c)
    o, lse = _prefix(c)
    check_with_nan(o, lse, want)
    assert want[0][1].isnan().any() and not want[0][0].isnan().any()
    for token in (0, 500, 1023):
        c = paged_case([1024 + 1 + 11 * (b % 20) for b in range(B)], 1, H, kv, seed=202, prefix=1024)
        _plant(c, 0, token, what)
        want = attend(c)
        o, lse = _prefix(c)
        check_with_nan(o, lse, want)
        assert want[0].isnan().any(-1).all()


@pytest.mark.parametrize("kv,H,what", _NAN)
@pytest.mark.parametrize("B,prefix,num_splits", [(10, 640, -1), (160, 960, -1), (160, 960, 1), (160, 960, 3), (160, 960, -2),
                                                 (40, 8192, -1), (40, 8192, -2)])
def test_nan_in_the_prefix_past_a_request_that_ends_inside_it(kv, H, what, B, prefix, num_splits):
    """Requests that see only a part of the prefix are not touched by what its other tokens hold."""
    lens = [(prefix + 70, 0, 1, 2, 64, 301, 302, 303, 512, prefix - 1, prefix, prefix + 1, 600)[b % 13] for b in range(B)]
    c = paged_case(lens, 2, H, kv, seed=203, prefix=prefix)
    assert H != 16 or _kernel(c, num_splits) == (B > 10)
    _plant(c, 0, 301, what)
    _plant(c, 0, prefix - 1, what)
    want = attend(c)
    st = _status()
    o, lse = _prefix(c, num_splits, st)
    assert int(st.item()) == 0
    check_with_nan(o, lse, want)
    touched = want[0].isnan().view(B, -1).any(1).tolist()
    assert touched[:5] == [True, False, False, False, False] and touched[6]  # length 302: it sees the first one


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("B", [4, 160])
def test_nan_codes_read_alike_everywhere(H, B, monkeypatch):
    """The e4m3 codes 0x7F and 0xFF, which the cache writer stores for no number, read +-480 in the decode
    kernels: so they do in a shared prefix, whichever kernel reads it, and in the page keys."""
    import torch
    import longctx_util
    import mla_latent_kv_gb300 as mla
    c = paged_case([1024 + 30 + b % 100 for b in range(B)], 1, H, F8, seed=204, prefix=1024)
    assert H != 16 or _kernel(c) == (B > 4)
    raw = c["cache"].view(c["num_blocks"], PAGE, D + 8)
    for page, row, dim, code in ((0, 3, 7, 0x7F), (5, 63, 511, 0xFF), (15, 0, 570, 0x7F), (16, 1, 100, 0xFF)):
        raw[int(c["full_table"][0, page]), row, dim] = code

    def read_480(case):
        r = case["cache"].view(case["num_blocks"], PAGE, D + 8)
        code = r[..., :D].contiguous()
        x = code.view(torch.float8_e4m3fn).double()
        x = torch.where(x.isnan(), torch.where(code > 127, -480.0, 480.0), x)
        sc = r[..., D:].contiguous().view(torch.float32).double()
        return x * sc[..., :1], x[..., :L] * sc[..., 1:]

    monkeypatch.setattr(longctx_util, "keys_values", read_480)
    o, lse = _prefix(c)
    check_attention(o, lse, attend(c))
    keys = mla.page_keys(c["cache"], dev(c["full_table"]), c["seq_lens"], c["max_len"], kv_dtype=F8,
                         num_blocks=c["num_blocks"])
    for page in (0, 5, 15, 16):
        blk = int(c["full_table"][0, page])
        rows = read_480(c)[0][blk, :min(PAGE, int(c["lens"][0]) - page * PAGE)]
        tol = 2.0 ** -8 * rows.mean(0).abs() + 66 * 2.0 ** -24 * rows.abs().mean(0)
        assert bool(((keys[blk].double() - rows.mean(0)).abs() <= tol).all()), page


# ------------------------------------------------------------------------------------ page keys
@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("lens,starts", [
    ([1, 63, 64, 65, 0, 1000], None),
    ([1, 64, 130, 700, 5, 0, 640], [0, 63, 129, 128, 5, 0, 639]),  # nothing new in the fifth
    ([129, 200], [64, 250]),                                       # start past the length
])
def test_page_keys(kv, lens, starts):
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case(lens, 1, 1, kv, seed=30, extra_cols=2)
    k, _ = keys_values(c)
    start = [0] * len(lens) if starts is None else starts
    max_new = max(0, max(n - s for n, s in zip(lens, start)))
    keys = torch.full((c["num_blocks"], D), 7.0, dtype=torch.bfloat16, device="cuda")
    st = _status()
    out = mla.page_keys(c["cache"], c["table"], c["seq_lens"], max_new, kv_dtype=kv, page_keys=keys, dev_status=st,
                        start_lens=None if starts is None else dev(np.asarray(starts, np.int32)),
                        num_blocks=c["num_blocks"])
    assert out is keys and int(st.item()) == 0
    left = torch.ones(c["num_blocks"], dtype=torch.bool)
    for b, n in enumerate(lens):
        for p in range(start[b] // PAGE, -(-n // PAGE)) if n > start[b] else []:
            blk = int(c["full_table"][b, p])
            rows = k[blk, :min(PAGE, n - p * PAGE)]
            want = rows.mean(0)
            # 64 fp32 additions (and the FP8 format's product), one rounding to bf16
            tol = 2.0 ** -8 * want.abs() + 66 * 2.0 ** -24 * rows.abs().mean(0)
            assert bool(((keys[blk].double() - want).abs() <= tol).all()), (b, p)
            left[blk] = False
    assert bool((keys[left.cuda()] == 7.0).all())  # pages without new tokens keep their keys


def test_page_keys_reports_bad_blocks_and_lengths():
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case([200, 100], 1, 1, BF, seed=31)
    c["table"][1, 0] = -1
    st = _status()
    keys = mla.page_keys(c["cache"], c["table"], c["seq_lens"], 200, dev_status=st, num_blocks=c["num_blocks"])
    assert int(st.item()) == mla.DEV_BAD_BLOCK_ID and torch.isfinite(keys).all()
    st.zero_()
    c = paged_case([200, 100], 1, 1, BF, seed=31)
    mla.page_keys(c["cache"], c["table"], c["seq_lens"], 150, dev_status=st, num_blocks=c["num_blocks"])
    assert int(st.item()) == mla.DEV_SEQ_TOO_LONG


# ---------------------------------------------------------------------------------- page scores
def _scores_ref(c, keys, b, t):
    n = max(0, int(c["lens"][b]) - (c["Sq"] - 1 - t))
    ids = [int(x) for x in c["full_table"][b, :-(-n // PAGE)]]
    if not ids:
        return None, None
    k, q = keys[ids].double(), c["q"][b, t].double()
    s = (q @ k.t() * c["scale"]).amax(0)
    tol = 577 * 2.0 ** -24 * c["scale"] * (q.abs() @ k.abs().t()).amax(0) + 2.0 ** -24 * s.abs()
    return s, tol


@pytest.mark.parametrize("H", [1, 7, 16, 33, 100, 128])
@pytest.mark.parametrize("Sq,lens", [(1, [0, 1, 64, 65, 5000]), (2, [1, 2, 8192, 8193, 128, 129])])
def test_page_scores(H, Sq, lens):
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case(lens, Sq, H, BF, seed=50 + H)
    rng = np.random.default_rng(51)
    keys = bf16(mi.normal_bf16(rng, (c["num_blocks"], D), std=0.125))
    st = _status()
    s = mla.page_scores(c["q"], keys, c["table"], c["seq_lens"], c["max_len"], c["scale"], dev_status=st)
    assert int(st.item()) == 0 and s.shape[2] == -(-c["max_len"] // PAGE)
    for b in range(c["B"]):
        for t in range(Sq):
            want, tol = _scores_ref(c, keys, b, t)
            m = 0 if want is None else want.numel()
            if m:
                assert bool(((s[b, t, :m].double() - want).abs() <= tol).all()), (b, t)
            assert bool((s[b, t, m:] == -math.inf).all())


def test_page_scores_nan_and_bad_blocks():
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case([640], 1, 20, BF, seed=60)
    keys = bf16(mi.normal_bf16(np.random.default_rng(61), (c["num_blocks"], D)))
    ids = c["full_table"][0]
    keys[int(ids[3]), 100] = math.nan
    keys[int(ids[4]), 5] = math.inf
    c["table"][0, 7] = -5
    st = _status()
    s = mla.page_scores(c["q"], keys, c["table"], c["seq_lens"], c["max_len"], c["scale"], dev_status=st)[0, 0].cpu()
    assert int(st.item()) == mla.DEV_BAD_BLOCK_ID
    assert math.isnan(s[3]) and s[4] == math.inf and s[7] == -math.inf
    assert torch.isfinite(s[[0, 1, 2, 5, 6, 8, 9]]).all()


# --------------------------------------------------------------------------------------- select
@pytest.mark.parametrize("K,sink,local", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (4, 0, 0), (16, 1, 1), (16, 8, 8), (64, 2, 3)])
@pytest.mark.parametrize("width", [1, 31, 64, 129, 300, 2049, 5001, 16385])
def test_select_pages(K, sink, local, width):
    import torch
    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(width * 100 + K)
    Sq, B = 2, 7
    lens = rng.integers(0, width * PAGE + 1, size=B)
    lens[:3] = [width * PAGE, 0, 1]
    s = rng.standard_normal((B, Sq, width)).astype(np.float32)
    s[3] = np.round(s[3] * 2) / 2                       # many ties
    s[4] = -1.5                                         # nothing but ties
    s[5, :, ::3] = np.nan
    s[5, :, 1::5] = -np.inf
    s[6, :, ::4] = np.inf
    s[6, :, 1::4] = 0.0
    s[6, :, 2::4] = -0.0
    st = _status()
    pages = mla.select_pages(dev(s), dev(lens.astype(np.int32)), K, sink, local, dev_status=st).cpu().numpy()
    assert int(st.item()) == 0
    for b in range(B):
        for t in range(Sq):
            want = select_rule(s[b, t], max(0, int(lens[b]) - (Sq - 1 - t)), K, sink, local)
            assert list(pages[b, t]) == want + [-1] * (K - len(want)), (b, t)


def test_page_scores_length_past_the_bound_is_reported_and_cut():
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case([64 * 4, 64 * 7, 9], 1, 16, BF, seed=46)
    keys = bf16(mi.normal_bf16(np.random.default_rng(47), (c["num_blocks"], D), std=0.125))
    st = _status()
    args = (c["q"], keys, c["table"], c["seq_lens"])
    got = mla.page_scores(*args, 64 * 5, c["scale"], dev_status=st)
    assert int(st.item()) == mla.DEV_SEQ_TOO_LONG
    want = mla.page_scores(*args, 64 * 7, c["scale"])
    assert torch.equal(got, want[:, :, :5]) and torch.isfinite(got[1]).all()


def test_select_pages_widest_strided_and_too_long():
    import torch
    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(5)
    wide = rng.standard_normal((1, 1, 32768)).astype(np.float32)
    lens = dev(np.array([32768 * PAGE], np.int32))
    got = mla.select_pages(dev(wide), lens, 100, 1, 1).cpu().numpy()[0, 0]
    assert list(got) == select_rule(wide[0, 0], 32768 * PAGE, 100, 1, 1)
    s = dev(rng.standard_normal((3, 1, 40)).astype(np.float32))[:, :, :20]  # rows 40 apart
    st = _status()
    lens = np.array([1000, 20 * PAGE, 20 * PAGE + 1], np.int32)
    got = mla.select_pages(s, dev(lens), 5, 1, 1, dev_status=st).cpu().numpy()
    assert int(st.item()) == mla.DEV_SEQ_TOO_LONG  # the third: cut at the scores' width
    for b, n in enumerate([1000, 20 * PAGE, 20 * PAGE]):
        assert list(got[b, 0]) == select_rule(s[b, 0].cpu().numpy(), n, 5, 1, 1)


# --------------------------------------------------------------------------------- sparse decode
def _pick(c, K, seed, gaps=False):
    """Random ascending pages [B, Sq, K] and the lists they stand for; gaps: -1 between entries too."""
    rng = np.random.default_rng(seed)
    pages = np.full((c["B"], c["Sq"], K), -1, np.int32)
    lists = []
    for b in range(c["B"]):
        lists.append([])
        for t in range(c["Sq"]):
            total = -(-max(0, int(c["lens"][b]) - (c["Sq"] - 1 - t)) // PAGE)
            m = int(rng.integers(0, min(total, K) + 1)) if gaps else min(total, K)
            ids = np.sort(rng.choice(total, m, replace=False)) if m else np.zeros(0, np.int64)
            at = np.sort(rng.choice(K, m, replace=False)) if gaps else np.arange(m)
            pages[b, t, at] = ids
            lists[-1].append([int(x) for x in ids])
    return pages, lists


def _sparse(c, pages, num_splits=-1, status=None, **kw):
    import mla_latent_kv_gb300 as mla
    return mla.decode_sparse(c["q"], c["cache"], c["table"], c["seq_lens"], dev(pages), c["scale"], kv_dtype=c["kv"],
                             num_splits=num_splits, dev_status=status, num_blocks=c["num_blocks"], **kw)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("num_splits", [1, 4, -1, -2])
@pytest.mark.parametrize("Sq,H,K,lens", [
    (1, 128, 6, [0, 1, 63, 64, 65, 700, 1000, 384]),
    (2, 20, 1, [1, 2, 64, 65, 66, 300]),
    (3, 16, 70, [5000, 200, 4]),       # more entries than a warp, more than one per row's pages
])
def test_sparse_decode(kv, num_splits, Sq, H, K, lens):
    c = paged_case(lens, Sq, H, kv, seed=80 + K)
    for gaps in (False, True):
        pages, lists = _pick(c, K, 81, gaps)
        st = _status()
        o, lse = _sparse(c, pages, num_splits, st)
        assert int(st.item()) == 0
        check_attention(o, lse, attend(c, lists))


@pytest.mark.parametrize("kv,H", [(BF, 16), (BF, 128), (F8, 16), (F8, 48)])
def test_sparse_decode_length_past_the_table_is_reported_and_cut(kv, H):
    import mla_latent_kv_gb300 as mla
    c = paged_case([64 * 6, 64 * 6, 70], 2, H, kv, seed=88)
    pages, lists = _pick(c, 4, 89)
    pages[0, :, :], lists[0] = np.array([0, 2, 4, 5], np.int32), [[0, 2, 4, 5]] * 2
    c["seq_lens"][0] = c["table"].shape[1] * PAGE + 1  # read as the table's 384 tokens
    st = _status()
    o, lse = _sparse(c, pages, status=st)
    assert int(st.item()) == mla.DEV_SEQ_TOO_LONG
    check_attention(o, lse, attend(c, lists))


@pytest.mark.parametrize("H", [1, 8, 16, 17, 32, 33, 48, 49, 64, 65])
@pytest.mark.parametrize("num_splits", [1, 3])
@pytest.mark.parametrize("kv", [BF, F8])
def test_sparse_decode_head_counts_over_long_rows(kv, H, num_splits):
    """Few heads take a kernel of their own; rings wrap several times."""
    import torch
    lens = [64 * 40 + 7, 64 * 23, 1, 130]
    c = paged_case(lens, 1, H, kv, seed=84, scale_v=0.5 if kv == F8 else None)
    if kv == BF:
        rows = c["cache"].view(torch.bfloat16).view(c["num_blocks"], PAGE, D)
    else:  # the two scales of each row, views into the cache
        rows = c["cache"].view(c["num_blocks"], PAGE, D + 8).view(torch.float32)[..., D // 4:]
    for i, blk in enumerate(c["full_table"][0, :41]):  # a running maximum that moves late, too
        if i in (9, 30):
            rows[int(blk)] *= 6.0
    pages, lists = _pick(c, 45, 85, gaps=True)
    pages[0], lists[0] = _all(lens[0], 45)
    st = _status()
    o, lse = _sparse(c, pages, num_splits, st)
    assert int(st.item()) == 0
    check_attention(o, lse, attend(c, lists))


def _all(n, K):
    ids = list(range(-(-n // PAGE)))
    return np.array([ids + [-1] * (K - len(ids))], np.int32), [ids]


def test_sparse_decode_many_rows_bf16_output():
    import mla_latent_kv_gb300 as mla
    lens = [1 + (37 * b) % 900 for b in range(100)]
    c = paged_case(lens, 1, 16, BF, seed=90)
    pages, lists = _pick(c, 5, 91, gaps=True)
    o, lse = _sparse(c, pages, o_dtype=mla.DT_BF16)
    check_attention(o, lse, attend(c, lists), bf16_out=True)


def test_sparse_decode_of_all_pages_is_decode():
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case([700, 64, 1, 1000], 1, 65, BF, seed=92)
    pages = np.full((4, 1, 16), -1, np.int32)
    for b, n in enumerate(c["lens"]):
        pages[b, 0, :-(-int(n) // PAGE)] = np.arange(-(-int(n) // PAGE))
    o, lse = _sparse(c, pages, 1)
    o2, lse2 = mla.decode(c["q"], c["cache"], c["table"], c["seq_lens"], c["max_len"], c["scale"], num_splits=1,
                          num_blocks=c["num_blocks"])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_sparse_decode_skips_and_reports_bad_entries():
    """Out of order, twice, out of range, below -1: skipped and reported, the rest is attended to."""
    import mla_latent_kv_gb300 as mla
    c = paged_case([640] * 6, 1, 16, BF, seed=93)
    rows = [([3, 3, 5, -1], [3, 5]), ([5, 2, 6, -1], [5, 6]), ([1, 10, 4, 9], [1, 4, 9]), ([-2, 0, 1, 2], [0, 1, 2]),
            ([2147483647, 0, 9, 9], [0, 9]), ([4, 5, 6, 7], [4, 5, 6, 7])]
    pages = np.array([[r[0]] for r in rows], np.int32)
    st = _status()
    o, lse = _sparse(c, pages, 2, st)
    assert int(st.item()) == mla.DEV_BAD_PAGE
    check_attention(o, lse, attend(c, [[r[1]] for r in rows]))


# ------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("stream", [False, True])
def test_write_score_select_attend(kv, stream):
    """A decode step over selected pages: write the new rows, refresh their pages' keys, score,
    select, attend; eager, then captured in a graph and replayed after new inputs."""
    import torch
    import mla_latent_kv_gb300 as mla
    lens = [3000, 64, 65, 1, 900, 2049]
    B, H, K = len(lens), 32, 6
    c = paged_case(lens, 1, H, kv, seed=95)
    rng = np.random.default_rng(96)
    slots = dev(np.array([int(c["full_table"][b, (n - 1) // PAGE]) * PAGE + (n - 1) % PAGE for b, n in enumerate(lens)],
                         np.int64))
    new_c, new_pe = bf16(mi.normal_bf16(rng, (B, 512))), bf16(mi.normal_bf16(rng, (B, 64)))
    start = c["seq_lens"] - 1
    keys = mla.page_keys(c["cache"], c["table"], c["seq_lens"], c["max_len"], kv_dtype=kv, num_blocks=c["num_blocks"])
    scores = torch.empty((B, 1, -(-c["max_len"] // PAGE)), device="cuda")
    pages = torch.empty((B, 1, K), dtype=torch.int32, device="cuda")
    ws = torch.empty(mla.decode_sparse_workspace_bytes(B, 1, H, K, kv), dtype=torch.uint8, device="cuda")
    o = torch.empty((B, 1, H, L), device="cuda")
    lse = torch.empty((B, 1, H), device="cuda")
    st = _status()

    def step():
        mla.cache_write(new_c, new_pe, slots, c["cache"], kv_dtype=kv, num_blocks=c["num_blocks"], dev_status=st)
        mla.page_keys(c["cache"], c["table"], c["seq_lens"], 1, kv_dtype=kv, start_lens=start, page_keys=keys,
                      num_blocks=c["num_blocks"], dev_status=st)
        mla.page_scores(c["q"], keys, c["table"], c["seq_lens"], c["max_len"], c["scale"], scores=scores, dev_status=st)
        mla.select_pages(scores, c["seq_lens"], K, pages=pages, dev_status=st)
        mla.decode_sparse(c["q"], c["cache"], c["table"], c["seq_lens"], pages, c["scale"], kv_dtype=kv, workspace=ws,
                          o_latent=o, lse=lse, num_blocks=c["num_blocks"], dev_status=st)

    def check():
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        sc = scores.cpu().numpy()
        lists = [[select_rule(sc[b, 0], n, K, 1, 1)] for b, n in enumerate(lens)]
        got = pages.cpu().numpy()
        for b in range(B):
            assert list(got[b, 0][got[b, 0] >= 0]) == lists[b][0]
        k64, _ = keys_values(c)
        for b, n in enumerate(lens):  # the refreshed page's key and its score
            blk = int(c["full_table"][b, (n - 1) // PAGE])
            rows = k64[blk, :(n - 1) % PAGE + 1]
            tol = 2.0 ** -8 * rows.mean(0).abs() + 66 * 2.0 ** -24 * rows.abs().mean(0)
            assert bool(((keys[blk].double() - rows.mean(0)).abs() <= tol).all())
        check_attention(o, lse, attend(c, lists))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side if stream else torch.cuda.current_stream()):
        step()
        check()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        c["q"].copy_(bf16(mi.normal_bf16(rng, (B, 1, H, D))))
        new_c.copy_(bf16(mi.normal_bf16(rng, (B, 512))))
        o.zero_()
        g.replay()
        check()


@pytest.mark.parametrize("kv", [BF, F8])
def test_shared_prefix_step_in_a_graph(kv):
    """absorb -> decode over the shared prefix -> out_proj captured, replayed after new queries, and
    two captured calls that take turns on one workspace."""
    import torch
    import mla_latent_kv_gb300 as mla
    B, H, prefix = 180, 16, 640
    c = paged_case([prefix + (1, 70, 300, 64, 5, 129)[b % 6] for b in range(B)], 1, H, kv, seed=97, prefix=prefix)
    assert _kernel(c)
    rng = np.random.default_rng(98)
    e = mi.e2e_case(B, 1, H, [64] * B, seed=99)
    qn, qp = bf16(e["q_nope"]).view(B, H, 128), bf16(e["q_pe"]).view(B, H, 64)
    wk, wv = bf16(e["w_uk_t"]), bf16(e["w_uv"])
    q2 = c["q"].view(B, H, D)
    need = max(1, mla.decode_shared_prefix_workspace_bytes(B, 1, H, prefix, c["max_len"], kv))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ol, lse = torch.empty((B, 1, H, L), device="cuda"), torch.empty((B, 1, H), device="cuda")
    out = torch.empty((B, H, 128), device="cuda")

    def step():
        mla.absorb_q(qn, qp, wk, out=q2)
        _prefix(c, workspace=ws, o_latent=ol, lse=lse)
        mla.out_proj(ol.view(B, H, L), wv, out=out)

    step()
    torch.cuda.synchronize()
    check_attention(ol, lse, attend(c))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        step()
    with torch.cuda.graph(g2):
        step()
    first = out.clone()
    for g in (g1, g2, g1):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    qn.copy_(bf16(mi.normal_bf16(rng, (B, H, 128))))
    g2.replay()
    torch.cuda.synchronize()
    check_attention(ol, lse, attend(c))
    assert not torch.equal(out, first)


@pytest.mark.parametrize("H", [16, 128])
def test_two_streams_at_once(H):
    """Calls of two streams, each with its own workspace, do not disturb one another."""
    import torch
    import mla_latent_kv_gb300 as mla
    B, prefix = 64, 4096
    cases = [paged_case([prefix + 1 + (37 * b + s) % 400 for b in range(B)], 1, H, kv, seed=140 + s, prefix=prefix)
             for s, kv in enumerate((BF, F8))]
    streams = [torch.cuda.Stream() for _ in cases]
    full = [dev(c["full_table"]) for c in cases]
    pages = [torch.sort(torch.stack([torch.randperm(64)[:24] for _ in range(B)]), 1)[0].int().view(B, 1, 24).cuda()
             for _ in cases]

    def both(i):
        c = cases[i]
        o, lse = _prefix(c)
        o2, lse2 = mla.decode_sparse(c["q"], c["cache"], full[i], c["seq_lens"], pages[i], c["scale"],
                                     kv_dtype=c["kv"], num_blocks=c["num_blocks"])
        return o, lse, o2, lse2

    alone = [both(i) for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(both(i))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(out, alone[i]))


@pytest.mark.parametrize("H", [16, 128])
def test_stream_argument_with_buffers_of_the_calls_own(H):
    """Calls given stream= and no buffers, issued from one thread for two streams while the current stream
    takes and fills memory: each gives what it gives alone."""
    import torch
    import mla_latent_kv_gb300 as mla
    B, prefix = 64, 4096
    cases = [paged_case([prefix + 1 + (37 * b + s) % 400 for b in range(B)], 1, H, kv, seed=170 + s, prefix=prefix)
             for s, kv in enumerate((BF, F8))]
    full = [dev(c["full_table"]) for c in cases]
    pages = [torch.sort(torch.stack([torch.randperm(64)[:24] for _ in range(B)]), 1)[0].int().view(B, 1, 24).cuda()
             for _ in cases]
    junk = []

    def busy():  # whatever the current stream's pool holds free is taken and overwritten
        junk[:] = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in (1 << 14, 1 << 20, 1 << 23, 1 << 26)]
        junk.clear()

    def calls(i, stream):
        c = cases[i]
        kw = dict(kv_dtype=c["kv"], num_blocks=c["num_blocks"], stream=stream)
        out = []
        out += mla.decode_shared_prefix(c["q"], c["cache"], c["table"], c["seq_lens"], c["max_len"], prefix, c["scale"], **kw)
        busy()
        out += mla.decode_sparse(c["q"], c["cache"], full[i], c["seq_lens"], pages[i], c["scale"], **kw)
        busy()
        out += mla.decode(c["q"], c["cache"], full[i], c["seq_lens"], c["max_len"], c["scale"], num_splits=3, **kw)
        busy()
        keys = mla.page_keys(c["cache"], full[i], c["seq_lens"], c["max_len"], **kw)
        busy()
        s = mla.page_scores(c["q"], keys, full[i], c["seq_lens"], c["max_len"], c["scale"], stream=stream)
        busy()
        return out + [keys, s, mla.select_pages(s, c["seq_lens"], 8, stream=stream)]

    alone = [calls(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            busy()
            got[i].append(calls(i, streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(out, alone[i]))


@pytest.mark.parametrize("kv,H", [(BF, 16), (BF, 128), (F8, 16), (F8, 48)])
def test_calls_take_turns_on_one_workspace(kv, H):
    """Calls with other caches, scales, tables and pages, back to back over one workspace: each reads what
    its own kernels wrote there, not what the call before left."""
    import torch
    import mla_latent_kv_gb300 as mla
    B, prefix, K = 160, 704, 7
    cases = [paged_case([prefix + 1 + (37 * b + s) % 200 for b in range(B)], 1, H, kv, seed=150 + s, prefix=prefix,
                        scale_v=(0.5, 3.0)[s] if kv == F8 else None) for s in range(2)]
    assert H > 16 or all(_kernel(c) for c in cases)  # many heads: as the rule has it
    full = [dev(c["full_table"]) for c in cases]
    picked = [_pick(c, K, 152 + s)[0] for s, c in enumerate(cases)]
    picked = [dev(x) for x in picked]
    need = max([mla.decode_sparse_workspace_bytes(B, 1, H, K, kv)] +
               [mla.decode_shared_prefix_workspace_bytes(B, 1, H, prefix, c["max_len"], kv) for c in cases])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def sparse(i):
        c = cases[i]
        return mla.decode_sparse(c["q"], c["cache"], full[i], c["seq_lens"], picked[i], c["scale"], kv_dtype=kv,
                                 workspace=ws, num_blocks=c["num_blocks"])

    for call in (lambda i: _prefix(cases[i], workspace=ws), sparse):
        alone = []
        for i in range(2):
            torch.cuda.synchronize()
            ws.fill_(0xFF)
            torch.cuda.synchronize()
            alone.append(call(i))
            torch.cuda.synchronize()
        got = [call(i % 2) for i in range(20)]
        torch.cuda.synchronize()
        for i, (o, lse) in enumerate(got):
            assert torch.equal(o, alone[i % 2][0]) and torch.equal(lse, alone[i % 2][1]), i
        assert not torch.equal(alone[0][0], alone[1][0])


@pytest.mark.parametrize("H", [16, 128])
def test_lengths_and_tables_written_just_ahead(H):
    """Lengths and block tables that a kernel writes directly ahead of the calls, eager and in a graph."""
    import torch
    import mla_latent_kv_gb300 as mla
    cases = [paged_case([1 + (97 * b + 31 * s) % 900 for b in range(40)], 1, H, BF, seed=160 + s, extra_cols=4)
             for s in range(2)]
    cols, K = max(c["table"].shape[1] for c in cases), 6
    tables = [torch_pad(c["table"], cols) for c in cases]
    picked = [dev(_pick(c, K, 162 + s)[0]) for s, c in enumerate(cases)]
    blocks = max(c["num_blocks"] for c in cases)
    cache = torch.zeros((blocks, PAGE * 1152), dtype=torch.uint8, device="cuda")
    cache[:cases[0]["num_blocks"]] = cases[0]["cache"].view(-1, PAGE * 1152)
    q, table, lens, pages = cases[0]["q"], tables[0].clone(), cases[0]["seq_lens"].clone(), picked[0].clone()
    cache.view(torch.bfloat16).nan_to_num_(0.0)  # the second table's lengths reach rows that the first leaves unwritten
    max_len = cols * PAGE

    def calls(i):
        for dst, src in ((table, tables[i]), (pages, picked[i]), (lens, cases[i]["seq_lens"])):
            dst.copy_(src)
        sparse = mla.decode_sparse(q, cache, table, lens, pages, 0.07, num_blocks=blocks)
        lens.copy_(cases[i]["seq_lens"])
        return sparse + mla.decode_shared_prefix(q, cache, table, lens, max_len, 0, 0.07, num_blocks=blocks)

    alone = []
    for i in range(2):
        torch.cuda.synchronize()
        alone.append(calls(i))
    torch.cuda.synchronize()
    g, outs = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(g):
        outs = [calls(i % 2) for i in range(6)]
    g.replay()
    outs += [calls(i % 2) for i in range(6)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert all(torch.equal(x, y) for x, y in zip(out, alone[i % 2])), i
    assert not torch.equal(alone[0][0], alone[1][0])


def test_tensors_elsewhere_are_refused():
    """A tensor that the GPU cannot read is refused before anything is launched."""
    import torch
    import mla_latent_kv_gb300 as mla
    c = paged_case([200, 100], 1, 16, BF, seed=120)
    keys = torch.zeros((c["num_blocks"], D), dtype=torch.bfloat16, device="cuda")
    pages = torch.zeros((2, 1, 1), dtype=torch.int32, device="cuda")
    scores = torch.zeros((2, 1, 4), device="cuda")
    host = c["seq_lens"].cpu()
    st = torch.zeros(1, dtype=torch.int32)
    calls = [lambda lens, **kw: mla.decode_shared_prefix(c["q"], c["cache"], c["table"], lens, 200, 0, 0.1, **kw),
             lambda lens, **kw: mla.page_keys(c["cache"], c["table"], lens, 200, **kw),
             lambda lens, **kw: mla.page_scores(c["q"], keys, c["table"], lens, 200, 0.1, **kw),
             lambda lens, **kw: mla.select_pages(scores, lens, 2, **kw),
             lambda lens, **kw: mla.decode_sparse(c["q"], c["cache"], c["table"], lens, pages, 0.1, **kw)]
    for call in calls:
        with pytest.raises(ValueError):
            call(host)
        with pytest.raises(ValueError):
            call(c["seq_lens"], dev_status=st)
    for call in (calls[0], calls[4]):
        with pytest.raises(ValueError):
            call(c["seq_lens"], workspace=torch.empty(1 << 22, dtype=torch.uint8))
        with pytest.raises(ValueError):
            call(c["seq_lens"], workspace=torch.empty(1 << 22, dtype=torch.uint8, device="cuda")[::2])
    torch.cuda.synchronize()


_FIRST_CALL = """
import sys
import numpy as np, torch
sys.path.insert(0, "tests")
import mla_inputs
from longctx_util import attend, check_attention, paged_case
import mla_latent_kv_gb300 as mla
c = paged_case([640 + 1 + b for b in range(180)], 1, 16, mla_inputs.KV_BF16, seed=130, prefix=640)
keys = torch.zeros((c["num_blocks"], 576), dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
full = torch.from_numpy(c["full_table"]).cuda()
with torch.cuda.graph(g):
    o, lse = mla.decode_shared_prefix(c["q"], c["cache"], c["table"], c["seq_lens"], c["max_len"], 640, c["scale"],
                                      num_blocks=c["num_blocks"])
    mla.page_keys(c["cache"], full, c["seq_lens"], c["max_len"], page_keys=keys, num_blocks=c["num_blocks"])
    s = mla.page_scores(c["q"], keys, full, c["seq_lens"], c["max_len"], c["scale"])
    pages = mla.select_pages(s, c["seq_lens"], 4)
    o2, lse2 = mla.decode_sparse(c["q"], c["cache"], full, c["seq_lens"], pages, c["scale"], num_blocks=c["num_blocks"])
g.replay()
torch.cuda.synchronize()
check_attention(o, lse, attend(c))
picked = pages.cpu().numpy()
check_attention(o2, lse2, attend(c, [[[p for p in row if p >= 0] for row in req] for req in picked]))
print("same")
"""


def test_a_process_may_begin_with_a_capture():
    """The first calls of a process, captured into a graph: one-time set-up must not end the capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=root))
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
