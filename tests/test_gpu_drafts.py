"""Rotary positions, decode of drafted trees and the page pool, on the GPU, against their definitions in 64 bits."""
import math

import numpy as np
import pytest

import mla_inputs as mi
from drafts_util import accept_rule, attend_tree, fork_rule, random_pool, tree_case, tree_masks, turn64
from longctx_util import D, L, PAGE, bf16, check_attention, check_with_nan, dev

pytestmark = pytest.mark.gpu
BF, F8 = mi.KV_BF16, mi.KV_FP8
R = 64


def _status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _normal(rng, *shape):
    return bf16(mi.normal_bf16(rng, shape))


def _positions(rng, T, far):
    p = rng.integers(0, far, T).astype(np.int32)
    p[0] = far - 1
    if T > 2:
        p[1], p[2] = 0, -int(p[2])
    return dev(p)


# -------------------------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("adjacent", [True, False])
@pytest.mark.parametrize("T,N,far,mscale", [(1, 1, 10, 1.0), (7, 16, 4096, 1.0), (3, 33, 1 << 20, 0.7), (65, 5, 2 ** 31 - 1, 1.0),
                                            (2, 128, 163840, 1.2), (300, 31, 131072, 1.0)])
def test_rope(T, N, far, mscale, adjacent):
    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(T)
    freq = mla.rope_frequencies(10000.0, 40.0 if T % 2 else 1.0)
    x, pos = _normal(rng, T, N, R), _positions(rng, T, far)
    got = mla.rope(x, pos, freq, adjacent=adjacent, mscale=mscale)
    want, tol = turn64(x, pos, freq, adjacent, mscale)
    assert ((got.double() - want).abs() <= tol).all()


def test_rope_strides_in_place_and_neighbours():
    """The last 64 of each head's 192, in place and into the last 64 of 576; nothing else changes."""
    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(1)
    freq = mla.rope_frequencies()
    q, pos = _normal(rng, 9, 20, 192), _positions(rng, 9, 5000)
    absorbed = _normal(rng, 9, 20, D)
    before_q, before_a = q.clone(), absorbed.clone()
    want, tol = turn64(q[..., 128:], pos, freq, True)
    mla.rope(q[..., 128:], pos, freq, out=absorbed[..., L:])
    assert ((absorbed[..., L:].double() - want).abs() <= tol).all()
    assert bool((absorbed[..., :L] == before_a[..., :L]).all()) and bool((q == before_q).all())
    mla.rope(q[..., 128:], pos, freq, out=q[..., 128:])
    assert bool((q[..., 128:] == absorbed[..., L:]).all()) and bool((q[..., :128] == before_q[..., :128]).all())
    # head-major memory
    h = _normal(rng, 20, 9, R).transpose(0, 1)
    want, tol = turn64(h, pos, freq, False)
    assert ((mla.rope(h, pos, freq, adjacent=False).double() - want).abs() <= tol).all()
    assert mla.rope(h[:0], pos[:0], freq).shape == (0, 20, R)


def test_rope_far_positions_and_whole_turns():
    """At the largest positions angles are still those of the definition, here in exact arithmetic."""
    import torch
    from fractions import Fraction

    import mla_latent_kv_gb300 as mla
    freq = mla.rope_frequencies()
    pos = dev(np.array([2 ** 31 - 1, -2 ** 31, 1 << 30, 123456789], np.int32))
    x = torch.zeros((4, 1, R), dtype=torch.bfloat16, device="cuda")
    x[..., 0::2] = 1.0
    got = mla.rope(x, pos, freq).double().cpu()
    # 2 pi to 30 digits
    two_pi = Fraction(6283185307179586476925286766559, 10 ** 30)
    for t, m in enumerate(pos.tolist()):
        for i, w in enumerate(freq.tolist()):
            a = float(Fraction(w) * m / two_pi % 1 * two_pi)
            # w's step is its 64 bits' quotient by 2 pi (2^-53 relative): m w 2^-52 rad at most
            tol = 2.0 ** -8 + 2.0 ** -20 + abs(m) * w * 2.0 ** -52
            assert abs(got[t, 0, 2 * i] - math.cos(a)) <= tol and abs(got[t, 0, 2 * i + 1] - math.sin(a)) <= tol


@pytest.mark.parametrize("adjacent", [True, False])
def test_rope_gradient(adjacent):
    """Turning back by the same positions is the gradient: against autograd of the definition, and differences."""
    import torch

    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(5)
    freq = mla.rope_frequencies()
    x, g, pos = _normal(rng, 6, 3, R), _normal(rng, 6, 3, R), dev(rng.integers(0, 9000, 6).astype(np.int32))
    leaf = x.double().requires_grad_()
    (turn64(leaf, pos, freq, adjacent)[0] * g.double()).sum().backward()
    got = mla.rope(g, -pos, freq, adjacent=adjacent)
    tol = turn64(g, -pos, freq, adjacent)[1]
    assert ((got.double() - leaf.grad).abs() <= tol).all()
    # <g, rope(x + d) - rope(x)> = <rope^-1(g), d>; the map is linear, so a large d serves
    d = _normal(rng, 6, 3, R)
    moved = (x.float() + d.float()).to(torch.bfloat16)
    step = moved.double() - x.double()
    lhs = (g.double() * (mla.rope(moved, pos, freq, adjacent=adjacent).double() -
                         mla.rope(x, pos, freq, adjacent=adjacent).double())).sum()
    slack = (g.double().abs() * (turn64(moved, pos, freq, adjacent)[1] + turn64(x, pos, freq, adjacent)[1])).sum() + \
        (tol * step.abs()).sum()
    assert (lhs - (got.double() * step).sum()).abs() <= slack


def test_rope_nan_stays_in_its_pair():
    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(6)
    x, pos = _normal(rng, 4, 9, R), dev(np.array([0, 1, 77, 1000], np.int32))
    x[2, 3, 10] = float("nan")
    got = mla.rope(x, pos, mla.rope_frequencies())
    bad = got.isnan().nonzero().tolist()
    assert bad == [[2, 3, 10], [2, 3, 11]]
    bad = mla.rope(x, pos, mla.rope_frequencies(), adjacent=False).isnan().nonzero().tolist()
    assert bad == [[2, 3, 10], [2, 3, 42]]


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("adjacent", [True, False])
@pytest.mark.parametrize("T,H,kv_scale", [(1, 1, 0.0), (37, 16, 0.0), (130, 40, 0.02), (9, 128, 0.0)])
def test_rope_cache_write(T, H, kv_scale, adjacent, kv):
    """Equal to the separate calls where they round alike (bf16 rows, queries); FP8 rows within their step."""
    import torch

    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(T + H)
    freq = mla.rope_frequencies(10000.0, 40.0)
    kv_a, q = _normal(rng, T, D), _normal(rng, T, H, 192)
    pos = _positions(rng, T, 100000)
    nb = T // PAGE + 3
    slots = rng.permutation(nb * PAGE)[:T].astype(np.int64)
    if T > 5:
        slots[3] = -1
        kv_a[4] = 0
    slots = dev(slots)
    rb = mla.row_bytes(kv)
    fill = rng.integers(0, 256, (nb, PAGE * rb), dtype=np.uint8)
    cache, two, st = dev(fill), dev(fill), _status()
    absorbed = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    mla.rope_cache_write(kv_a[:, :L], kv_a[:, L:], pos, freq, slots, cache, kv_dtype=kv, adjacent=adjacent, kv_scale=kv_scale,
                         q_pe=q[..., 128:], q_out=absorbed[..., L:], dev_status=st)
    assert bool((absorbed[..., L:] == mla.rope(q[..., 128:], pos, freq, adjacent=adjacent)).all())
    assert bool((absorbed[..., :L] == 0).all()) and st.item() == 0
    k = mla.rope(kv_a[:, None, L:], pos, freq, adjacent=adjacent)[:, 0]
    mla.cache_write(kv_a[:, :L], k, slots, two, kv_dtype=kv, kv_scale=kv_scale)
    if kv == BF:
        assert bool((cache == two).all())
        return
    live = slots >= 0
    rows, untouched = cache.view(-1, rb), torch.ones(nb * PAGE, dtype=torch.bool, device="cuda")
    untouched[slots[live]] = False
    assert bool((rows[untouched] == dev(fill).view(-1, rb)[untouched]).all())
    got = rows[slots[live]]
    scale = got[:, D:].contiguous().view(torch.float32).double()
    exact, slack = turn64(kv_a[:, None, L:], pos, freq, adjacent)
    slack = slack - 2.0 ** -8 * exact.abs()  # the angle's part of the bound: nothing is rounded to bf16 here
    row = torch.cat([kv_a[:, :L].double(), exact[:, 0]], 1)[live]
    off = torch.cat([torch.zeros_like(kv_a[:, :L]).double(), slack[:, 0]], 1)[live]
    top = row.abs().amax(1)
    want = torch.full_like(top, kv_scale) if kv_scale else torch.where(top > 0, top / 448, torch.ones_like(top))
    assert bool((scale[:, 0] == scale[:, 1]).all())
    assert ((scale[:, 0] - want).abs() <= 2.0 ** -22 * want + off.amax(1) / 448).all()
    value = got[:, :D].contiguous().view(torch.float8_e4m3fn).double() * scale[:, :1]
    x = row.clamp(-448 * scale[:, :1], 448 * scale[:, :1])
    # half a step: 2^-4 of the value, or 2^-10 of the scale below 2^-6 of it
    bound = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * scale[:, :1]) * (1 + 2.0 ** -20) + 2 * off + 2.0 ** -22 * x.abs()
    assert ((value - x).abs() <= bound).all()


def test_rope_cache_write_bad_slots_and_rows_alone():
    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(9)
    kv_a, pos, st = _normal(rng, 4, D), dev(np.arange(4, dtype=np.int32)), _status()
    fill = rng.integers(0, 256, (3, PAGE * 1152), dtype=np.uint8)
    cache = dev(fill)
    slots = dev(np.array([5, 2 * PAGE, 10 ** 12, -7], np.int64))
    mla.rope_cache_write(kv_a[:, :L], kv_a[:, L:], pos, mla.rope_frequencies(), slots, cache, num_blocks=2, dev_status=st)
    assert st.item() == mla.DEV_BAD_SLOT
    want = fill.copy().reshape(3 * PAGE, 1152)
    k = mla.rope(kv_a[:, None, L:], pos, mla.rope_frequencies())[:, 0]
    want[5] = np.concatenate([x[0].view(__import__("torch").int16).cpu().numpy().view(np.uint8) for x in (kv_a[:, :L], k)])
    assert np.array_equal(cache.cpu().numpy().reshape(3 * PAGE, 1152), want)


# ------------------------------------------------------------------------------------------ trees
def _tree(c, o_dtype=None, status=None, max_len=None, **kw):
    import mla_latent_kv_gb300 as mla
    return mla.decode_tree(c["q"], c["cache"], c["table"], c["seq_lens"], c["masks"], max_len or max(c["max_len"], 1),
                           c["scale"], kv_dtype=c["kv"], o_dtype=o_dtype, dev_status=status, num_blocks=c["num_blocks"], **kw)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("Sq,H,lens", [
    (1, 1, [1]), (1, 16, [64, 65, 0]), (4, 16, [4, 68, 700]), (5, 3, [5, 6, 63, 64, 69, 70, 128, 133]),
    (64, 2, [64, 65, 127, 128, 190, 191]), (63, 1, [63, 126, 127, 2000]), (7, 128, [7, 900]), (33, 40, [700, 40]),
    (2, 128, [130, 129]), (3, 43, [2, 1, 0, 3, 200]), (64, 128, [64, 100]), (16, 17, [300 + i for i in range(40)]),
    (2, 16, [2, 65, 66, 129, 200]), (16, 2, [16, 79, 80, 81, 300]), (17, 1, [17, 20, 80]), (3, 11, [3, 130]), (32, 4, [40, 100, 33]),
])
def test_decode_tree(Sq, H, lens, kv):
    c = tree_case(lens, Sq, H, kv, seed=Sq * 1000 + H, scale_v=1.7 if kv == F8 else None)
    st = _status()
    want = attend_tree(c)
    check_attention(*_tree(c, status=st), want)
    import mla_latent_kv_gb300 as mla
    check_attention(*_tree(c, o_dtype=mla.DT_BF16), want, bf16_out=True)
    assert st.item() == 0


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("B,Sq,H,length,max_len", [(1, 4, 16, 9000, 9000), (3, 3, 128, 2500, 2500), (2, 9, 31, 3000, 40000),
                                                   (70, 2, 20, 500, 500), (1, 2, 9, 20000, 20000), (90, 2, 8, 700, 9000), (90, 4, 24, 700, 9000)])
def test_decode_tree_splits(B, Sq, H, length, max_len, kv):
    """Ranges of a request's pages joined by their log-sums; ranges behind a short request's end are empty."""
    import mla_latent_kv_gb300 as mla
    lens = [length] + [max(Sq, length * (b + 1) // (3 * B) - 17 * b) for b in range(1, B)]
    c = tree_case(lens, Sq, H, kv, seed=length, extra_cols=-(-max_len // PAGE) - -(-length // PAGE))
    assert B > 50 or mla.decode_tree_workspace_bytes(B, Sq, H, max_len, BF) > 0
    want = attend_tree(c)
    check_attention(*_tree(c, max_len=max_len), want)
    check_attention(*_tree(c, max_len=max_len, o_dtype=mla.DT_BF16), want, bf16_out=True)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("lens,Sq,H,max_len", [
    ([5000], 3, 128, 5000),                                          # one request in many parts, two tiles
    ([12800, 64, 12672], 2, 64, 12800),                              # cuts at and beside the edges of units
    ([0, 9000, 0, 7777, 1, 0], 6, 50, 9000),                         # empty slots first, between and last
    ([40, 129, 20000, 3, 64, 700, 128, 65] + [90] * 12, 2, 90, 20000),  # one long request among short ones
    ([0, 0, 0, 0], 2, 128, 20000),                                   # nothing at all
    ([2, 0, 1, 2], 2, 128, 20000),                                   # drafts alone, shares of no group
    ([300 + 97 * b for b in range(24)], 2, 120, 16000),              # far fewer tokens than the bound allows
    ([2000, 1500, 1700, 1999], 10, 128, 2000),                       # too little to be cut among seven clusters a tile
    ([9000, 1500], 10, 128, 9000),                                   # five tiles: 35 clusters
    ([9000], 20, 128, 9000),                                         # ten tiles, five at a time
    ([6000, 3001], 26, 128, 6000),                                   # thirteen, enough clusters for whole units
    ([20000], 26, 128, 20000),                                       # one at a time
    ([64 * (1 + b % 3) - b % 2 for b in range(112)], 2, 17, 30000),  # as many requests as are cut
    ([64 * (1 + b % 3) - b % 2 for b in range(113)], 2, 17, 30000),  # one more: whole units
])
def test_decode_tree_cut_requests(lens, Sq, H, max_len, kv):
    """Requests that are cut into shares wherever they end, and the merge of a request's parts."""
    import torch

    import mla_latent_kv_gb300 as mla
    c = tree_case(lens, Sq, H, kv, seed=sum(lens) + H, extra_cols=max(0, -(-max_len // PAGE) - -(-max(lens + [1]) // PAGE)))
    want, st = attend_tree(c), _status()
    o, lse = _tree(c, max_len=max_len, status=st)
    check_attention(o, lse, want)
    again = _tree(c, max_len=max_len)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    check_attention(*_tree(c, max_len=max_len, o_dtype=mla.DT_BF16), want, bf16_out=True)
    assert st.item() == 0
    if Sq * H > 32:  # partial states: the requests were cut
        assert (mla.decode_tree_workspace_bytes(len(lens), Sq, H, max_len, BF) > 0) == (len(lens) <= 112 and lens[0] not in (2000, 6000))


@pytest.mark.parametrize("kv", [BF, F8])
def test_decode_tree_cut_requests_replayed(kv):
    """The cuts follow the lengths on the device: a captured call with the lengths of another step, and back."""
    import torch
    c = tree_case([9000] * 6, 4, 60, kv, seed=5)
    g = torch.cuda.CUDAGraph()
    _tree(c)
    with torch.cuda.graph(g):
        o, lse = _tree(c)
    for lens in ([50, 9000, 4, 0, 8999, 64], [0, 0, 0, 0, 0, 3], [9000, 40, 6000, 3000, 9000, 100]):
        c["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check_attention(o, lse, attend_tree(dict(c, lens=lens)))


def _fill_rows(c, rows, value=None, inf=False):
    """Put NaN (or inf) into cache rows (block, place): every element for bf16, the scales for FP8."""
    import torch
    x = math.inf if inf else math.nan
    if c["kv"] == BF:
        view = c["cache"].view(torch.bfloat16).view(c["num_blocks"], PAGE, D)
        for blk, i in rows:
            view[blk, i] = x
    else:
        view = c["cache"].view(c["num_blocks"], PAGE, D + 8)[..., D:].view(torch.float32)
        for blk, i in rows:
            view[blk, i] = x


def _row(c, b, token):
    return int(c["full_table"][b, token // PAGE]), token % PAGE


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("inf", [False, True])
@pytest.mark.parametrize("H", [5, 21, 45])  # 30, 126 and 270 pairs: each of the kernels
def test_decode_tree_hidden_drafts_do_not_matter(H, kv, inf):
    """Drafts that no row sees, and whatever is behind the end, may hold anything."""
    Sq, lens = 6, [70, 134, 6, 200, 3]
    masks = tree_masks(5, Sq, 3)
    masks[:, :] &= ~(1 << 4)         # nobody sees draft 4
    masks[1, 2] = 0                  # sees the context alone
    masks[2, 1] = 0                  # sees nothing
    c = tree_case(lens, Sq, H, kv, 4, masks=masks)
    want = attend_tree(c)
    rows = [_row(c, b, n - Sq + 4) for b, n in enumerate(lens) if n - Sq + 4 >= 0]
    for b, n in enumerate(lens):
        rows += [(int(c["full_table"][b, (n - 1) // PAGE]), i) for i in range((n - 1) % PAGE + 1, PAGE)]
    _fill_rows(c, rows, inf=inf)
    o, lse = _tree(c)
    check_attention(o, lse, want)
    assert bool((lse[2, 1] == -math.inf).all()) and bool((o[2, 1] == 0).all())


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H", [4, 15, 20])
def test_decode_tree_nan_reaches_only_its_own_branch(H, kv):
    """A NaN draft is seen by its descendants alone; the others' results are as if it were not there."""
    Sq, lens = 8, [72, 130, 300]
    c = tree_case(lens, Sq, H, kv, 8)
    clean = attend_tree(c)
    _fill_rows(c, [_row(c, b, n - Sq + 2) for b, n in enumerate(lens)])
    sees = ((c["masks_host"] >> 2) & 1).astype(bool)
    assert sees.any() and not sees.all()
    o, lse = _tree(c)
    for b in range(3):
        for t in range(Sq):
            part = [x[b:b + 1, t:t + 1] for x in clean]
            if sees[b, t]:
                assert bool(o[b, t].isnan().all()) and bool(lse[b, t].isnan().all())
            else:
                check_attention(o[b:b + 1, t:t + 1], lse[b:b + 1, t:t + 1], part)


def test_decode_tree_cut_requests_with_nan():
    """A NaN token in one part of a request is all of its rows' result, and nobody else's."""
    c = tree_case([9000, 6000, 7001], 3, 60, BF, seed=21)
    _fill_rows(c, [_row(c, 1, 2500)])
    check_with_nan(*_tree(c), attend_tree(c))


@pytest.mark.parametrize("kv", [BF, F8])
def test_decode_tree_cut_requests_report_bad_blocks_and_lengths(kv):
    import mla_latent_kv_gb300 as mla
    c = tree_case([9000, 6000, 7001], 3, 60, kv, 22)
    want = attend_tree(c)
    table, st = c["table"].clone(), _status()
    table[1, 40] = c["num_blocks"]
    o, lse = _tree(dict(c, table=table), status=st)
    assert st.item() == mla.DEV_BAD_BLOCK_ID
    for b in (0, 2):
        check_attention(o[b:b + 1], lse[b:b + 1], [x[b:b + 1] for x in want])
    for n in (9001, -1):  # as the bound, as no token
        st, lens = _status(), c["seq_lens"].clone()
        lens[0] = n
        o, lse = _tree(dict(c, seq_lens=lens), status=st)
        assert st.item() == mla.DEV_SEQ_TOO_LONG
        check_attention(o[1:], lse[1:], [x[1:] for x in want])


@pytest.mark.parametrize("kv", [BF, F8])
def test_decode_tree_cut_requests_share_a_workspace(kv):
    """Calls one behind the other in one workspace, and two at once on two streams in their own."""
    import torch

    import mla_latent_kv_gb300 as mla
    cs = [tree_case(lens, 2, 100, kv, 30 + i) for i, lens in enumerate([[9000, 50, 4000], [300, 9000, 8000]])]
    wants = [attend_tree(c) for c in cs]
    size = mla.decode_tree_workspace_bytes(3, 2, 100, 9000, kv)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    results = [_tree(cs[i % 2], max_len=9000, workspace=ws[0]) for i in range(6)]
    for i, r in enumerate(results):
        check_attention(*r, wants[i % 2])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [(torch.empty((3, 2, 100, L), device="cuda"), torch.empty((3, 2, 100), device="cuda")) for _ in range(2)]
    for _ in range(4):
        for i in range(2):
            _tree(cs[i], max_len=9000, workspace=ws[i], o_latent=outs[i][0], lse=outs[i][1], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_attention(*outs[i], wants[i])


@pytest.mark.parametrize("H", [5, 16, 128])
def test_decode_tree_nan_in_the_context(H):
    c = tree_case([200, 100], 3, H, BF, 10)
    _fill_rows(c, [_row(c, 0, 50)])
    check_with_nan(*_tree(c), attend_tree(c))


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H", [9, 40, 100])
def test_decode_tree_empty_rows(H, kv):
    """Masks of no bits without a context, empty slots, and a bound of 0."""
    import torch
    masks = np.zeros((4, 3), np.int64)
    masks[1] = [1, 0, 5]
    c = tree_case([3, 3, 0, 67], 3, H, kv, 12, masks=masks)
    check_attention(*_tree(c), attend_tree(c))
    c["seq_lens"] = torch.zeros_like(c["seq_lens"])
    import mla_latent_kv_gb300 as mla
    o, lse = mla.decode_tree(c["q"], c["cache"], c["table"], c["seq_lens"], c["masks"], 0, c["scale"], kv_dtype=kv)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H", [6, 25, 128])
def test_decode_tree_with_a_causal_mask_is_decode(H, kv):
    """Bits from Sq on are not read, and the low t + 1 bits are mla_decode's order."""
    import mla_latent_kv_gb300 as mla
    Sq = 5
    masks = np.tile(np.array([(1 << t + 1) - 1 | -1 << Sq for t in range(Sq)], np.int64), (4, 1))
    c = tree_case([5, 64, 131, 2], Sq, H, kv, 14, masks=masks)
    o, lse = _tree(c)
    o1, lse1 = mla.decode(c["q"], c["cache"], c["table"], c["seq_lens"], c["max_len"], c["scale"], kv_dtype=kv, num_splits=1)
    o_ref, lse_ref, tol_o, tol_lse = attend_tree(c)
    assert ((o.double() - o1.double()).abs() <= 2 * tol_o).all()
    empty = torch_isinf(lse_ref)
    assert bool((lse[empty] == lse1[empty]).all())
    assert ((lse.double() - lse1.double()).abs()[~empty] <= 2 * tol_lse[~empty]).all()


def torch_isinf(x):
    import torch
    return torch.isinf(x)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H", [8, 16, 128])
def test_decode_tree_reports_bad_blocks_and_lengths(H, kv):
    import mla_latent_kv_gb300 as mla
    c = tree_case([200, 100], 3, H, kv, 16)
    for bad in (c["num_blocks"], -1, 2 ** 31 - 1):
        table, st = c["table"].clone(), _status()
        table[0, 1] = bad
        o, lse = mla.decode_tree(c["q"], c["cache"], table, c["seq_lens"], c["masks"], 200, c["scale"], kv_dtype=kv,
                                 num_blocks=c["num_blocks"], dev_status=st)
        assert st.item() == mla.DEV_BAD_BLOCK_ID
        part = [x[1:] for x in attend_tree(c)]
        check_attention(o[1:], lse[1:], part)
    for n in (201, -1):
        st, lens = _status(), c["seq_lens"].clone()
        lens[0] = n
        mla.decode_tree(c["q"], c["cache"], c["table"], lens, c["masks"], 200, c["scale"], kv_dtype=kv, num_blocks=c["num_blocks"],
                        dev_status=st)
        assert st.item() == mla.DEV_SEQ_TOO_LONG


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H", [8, 16, 65])
def test_decode_tree_replayed_with_other_inputs(H, kv):
    """A captured call reads lengths, tables, masks and cache anew, with a workspace that another call used."""
    import torch

    import mla_latent_kv_gb300 as mla
    a, b = tree_case([3000, 400], 4, H, kv, 18), tree_case([2900, 1400], 4, H, kv, 19)
    nb = max(a["num_blocks"], b["num_blocks"])
    width = max(a["table"].shape[1], b["table"].shape[1])

    def padded(c):
        cache = torch.zeros((nb, c["cache"].numel() // c["num_blocks"]), dtype=torch.uint8, device="cuda")
        cache[:c["num_blocks"]] = c["cache"].view(torch.uint8).view(c["num_blocks"], -1)
        table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
        table[:, :c["table"].shape[1]] = c["table"]
        return cache, table
    cache, table = padded(a)
    q, lens, masks = a["q"].clone(), a["seq_lens"].clone(), a["masks"].clone()
    ws = torch.empty(mla.decode_tree_workspace_bytes(2, 4, H, 3000, kv), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty((2, 4, H, L), device="cuda"), torch.empty((2, 4, H), device="cuda")
    call = lambda: mla.decode_tree(q, cache, table, lens, masks, 3000, a["scale"], kv_dtype=kv, workspace=ws, o_latent=o, lse=lse)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    for c in (b, a, b):
        new_cache, new_table = padded(c)
        cache.copy_(new_cache)
        table.copy_(new_table)
        q.copy_(c["q"])
        lens.copy_(c["seq_lens"])
        masks.copy_(c["masks"])
        ws.fill_(255)  # NaN
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check_attention(o, lse, attend_tree(c))


@pytest.mark.parametrize("kv", [BF, F8])
def test_decode_tree_of_many_requests(kv):
    """More requests than are sorted by length, several units a cluster, pages of every parity."""
    rng = np.random.default_rng(30)
    lens = rng.integers(0, 330, 530)
    c = tree_case(lens, 3, 44, kv, 31)
    check_attention(*_tree(c), attend_tree(c))


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H", [16, 60])
def test_decode_tree_calls_in_a_row(H, kv):
    """Calls that take turns on one workspace and one output without a wait between them."""
    import torch

    import mla_latent_kv_gb300 as mla
    cs = [tree_case([2500, 700, 66], 5, H, kv, 32), tree_case([64, 3000], 5, H, kv, 33)]
    need = max(mla.decode_tree_workspace_bytes(c["B"], 5, H, c["max_len"], kv) for c in cs)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [(torch.empty((c["B"], 5, H, L), device="cuda"), torch.empty((c["B"], 5, H), device="cuda")) for c in cs]
    for _ in range(4):
        for c, (o, lse) in zip(cs, outs):
            _tree(c, workspace=ws, o_latent=o, lse=lse)
    for c, (o, lse) in zip(cs, outs):
        check_attention(o, lse, attend_tree(c))


def test_decode_tree_on_two_streams():
    """Calls of two streams at once, each with its own workspace, also one made by the call."""
    import torch
    cs = [tree_case([5000, 300, 64], 6, H, kv, 20 + kv) for kv in (BF, F8) for H in (5, 16, 50)]
    want = [attend_tree(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [_tree(c, stream=s) for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        for (o, lse), w in zip(got, want):
            check_attention(o, lse, w)


# ---------------------------------------------------------------------------------- accepted drafts
@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("B,Sq,layers", [(1, 1, 1), (5, 4, 2), (9, 64, 3), (33, 17, 1)])
def test_accept_tokens(B, Sq, layers, kv):
    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(B * Sq)
    lens = rng.integers(0, 300, B).astype(np.int32)
    lens[0] = Sq
    pages = -(-lens // PAGE)
    nb = int(pages.sum()) + 3
    table = np.full((B, int(pages.max()) + 1), -1, np.int32)
    perm, at = rng.permutation(nb), 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    counts = rng.integers(0, Sq + 1, B).astype(np.int32)
    path = rng.integers(-5, Sq + 5, (B, Sq)).astype(np.int32)  # behind counts: anything
    for b in range(B):
        gone = max(0, Sq - int(lens[b]))
        counts[b] = min(counts[b], Sq - gone)
        path[b, :counts[b]] = np.sort(rng.choice(np.arange(gone, Sq), counts[b], replace=False))
    host = rng.integers(0, 256, (layers, nb, PAGE, mla.row_bytes(kv)), dtype=np.uint8)
    cache, st = dev(host.reshape(layers, nb, -1)), _status()
    new = mla.accept_tokens(cache, dev(table), dev(lens), dev(path), dev(counts), kv_dtype=kv, dev_status=st)
    want, want_lens, bad = accept_rule(host, table, lens, path, counts)
    assert not bad and st.item() == 0
    assert np.array_equal(new.cpu().numpy(), want_lens)
    assert np.array_equal(cache.cpu().numpy().reshape(host.shape), want)


def test_accept_tokens_bad_branches():
    """A branch ends before an entry out of order or out of range, and says so; bad blocks and lengths too."""
    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(2)
    Sq, nb = 5, 12
    table = np.arange(12, dtype=np.int32).reshape(6, 2)
    lens = np.array([70, 66, 5, 3, 100, 128], np.int32)
    path = np.array([[0, 2, 2, 3, 4], [1, 5, 0, 0, 0], [3, 1, 0, 0, 0], [1, 3, 4, 0, 0], [0, 1, 2, 3, 4], [-1, 0, 0, 0, 0]], np.int32)
    counts = np.array([4, 2, 2, 2, 6, 1], np.int32)
    host = rng.integers(0, 256, (1, nb, PAGE, 1152), dtype=np.uint8)
    want, want_lens, bad = accept_rule(host, table, lens, path, np.minimum(counts, Sq))
    assert bad and want_lens.tolist() == [67, 62, 1, 0, 100, 123]
    for b in range(6):  # each sets the bit by itself
        st = _status()
        mla.accept_tokens(dev(host.reshape(nb, -1)), dev(table[b:b + 1]), dev(lens[b:b + 1]), dev(path[b:b + 1]),
                          dev(counts[b:b + 1]), dev_status=st)
        assert st.item() == mla.DEV_BAD_BRANCH, b
    cache, st = dev(host.reshape(nb, -1)), _status()
    new = mla.accept_tokens(cache, dev(table), dev(lens), dev(path), dev(counts), dev_status=st)
    assert np.array_equal(new.cpu().numpy(), want_lens) and np.array_equal(cache.cpu().numpy().reshape(host.shape), want)
    table[0, 1], lens[1] = nb, 129
    cache, st = dev(host.reshape(nb, -1)), _status()
    mla.accept_tokens(cache, dev(table[:2]), dev(lens[:2]), dev(np.array([[1, 2, 0, 0, 0]] * 2, np.int32)),
                      dev(np.array([2, 2], np.int32)), dev_status=st)
    assert st.item() == mla.DEV_BAD_BLOCK_ID | mla.DEV_SEQ_TOO_LONG
    assert np.array_equal(cache.cpu().numpy().reshape(host.shape)[0, [0, 1]], host[0, [0, 1]])


# ---------------------------------------------------------------------------------------- page pool
def _fork(p, parents, room, kv, status=None, layers=None, **kw):
    import mla_latent_kv_gb300 as mla
    host = p["cache"]
    cache = dev(host.reshape(host.shape[0], host.shape[1], host.shape[2] * host.shape[3]))
    if layers == 0:
        cache = cache[:0]
    out = mla.fork_pages(cache, dev(p["table"]), dev(p["counts"]), dev(p["lens"]), dev(p["refs"]),
                         dev(np.asarray(parents, np.int32)), dev(np.asarray(room, np.int32)), kv_dtype=kv, dev_status=status, **kw)
    return cache, [x.cpu().numpy() for x in out]


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("B,B2,width,nb,layers,top", [(1, 1, 1, 4, 1, 60), (1, 7, 9, 40, 2, 500), (6, 6, 20, 300, 3, 1200),
                                                      (10, 3, 300, 700, 1, 5000), (40, 90, 7, 1100, 1, 300),
                                                      (3, 1100, 4, 3500, 1, 130), (12, 12, 40, 9000, 1, 2400)])
def test_fork_pages(B, B2, width, nb, layers, top, kv):
    for seed in range(3):
        rng = np.random.default_rng(seed)
        p = random_pool(B, width, nb, layers, kv, seed * 100 + B, min(top, width * PAGE))
        parents = rng.integers(-1, B, B2)
        own = np.where(parents >= 0, p["lens"][parents], 0)
        room = np.minimum(own + rng.integers(-3, 200, B2), width * PAGE)
        want = fork_rule(p["cache"], p["table"], p["counts"], p["lens"], p["refs"], parents, room)
        assert want is not None
        st = _status()
        cache, got = _fork(p, parents, room, kv, st)
        assert st.item() == 0
        for g, w in zip(got, want[1:]):
            assert np.array_equal(g, w)
        assert np.array_equal(cache.cpu().numpy().reshape(p["cache"].shape), want[0])


@pytest.mark.parametrize("case", ["pages", "parent", "parent_low", "room", "length", "count"])
def test_fork_pages_that_cannot_be_done(case):
    """All or nothing: every new row empty, the counts as they were, no cache row written."""
    import mla_latent_kv_gb300 as mla
    p = random_pool(5, 10, 60, 2, BF, 3, 400)
    parents, room = np.array([0, 1, 1, 4, -1]), np.array([100, 90, 500, 20, 64])
    bit = mla.DEV_SEQ_TOO_LONG
    if case == "pages":
        free = np.flatnonzero(p["refs"] == 0)
        p["refs"][free[:-2]] = 1
        bit = mla.DEV_NO_PAGES
    elif case == "parent":
        parents[3], bit = 5, mla.DEV_BAD_PARENT
    elif case == "parent_low":
        parents[3], bit = -2, mla.DEV_BAD_PARENT
    elif case == "room":
        room[0] = 10 * PAGE + 1
    elif case == "length":
        p["lens"][2] = int(p["counts"][2]) * PAGE + 1
    else:
        p["counts"][2] = 11
    st = _status()
    cache, (table, counts, lens, refs) = _fork(p, parents, room, BF, st)
    assert st.item() == bit
    assert (table == -1).all() and (counts == 0).all() and (lens == 0).all() and np.array_equal(refs, p["refs"])
    assert np.array_equal(cache.cpu().numpy().reshape(p["cache"].shape), p["cache"])


def test_fork_pages_bad_entries_are_not_counted():
    import mla_latent_kv_gb300 as mla
    p = random_pool(2, 6, 30, 1, BF, 5, 300)
    p["lens"][:], p["counts"][:] = [200, 10], [4, 1]
    p["table"][:] = -1
    p["table"][0, :4], p["table"][1, 0] = [3, 30, -5, 7], 9
    p["refs"][:] = 0
    p["refs"][[3, 7, 9]] = 1
    st = _status()
    _, (table, counts, lens, refs) = _fork(p, [0, 0], [200, 200], BF, st)
    assert st.item() == mla.DEV_BAD_BLOCK_ID
    assert table[0, :4].tolist() == [3, 30, -5, 7] and table[1, :4].tolist() == [3, 30, -5, 0]
    assert refs[3] == 2 and refs[7] == 1 and refs[0] == 1 and refs[9] == 0 and refs.sum() == 4


@pytest.mark.parametrize("kv", [BF, F8])
def test_fork_pages_with_much_room(kv):
    """Rows that hold many pages without tokens yet, some of them another holder's: kept, given back or replaced."""
    rng = np.random.default_rng(8)
    B, width, nb = 7, 400, 4000
    row = {BF: 1152, F8: 584}[kv]
    p = dict(cache=rng.integers(0, 256, (1, nb, PAGE, row), dtype=np.uint8), table=np.full((B, width), -1, np.int32),
             counts=np.array([400, 300, 9, 5, 4, 3, 0], np.int32), lens=np.array([100, 64 * 250, 64 * 4, 5, 0, 190, 0], np.int32),
             refs=np.zeros(nb, np.int32))
    perm, at = rng.permutation(nb), 0
    for b in range(B):
        n = int(p["counts"][b])
        p["table"][b, :n] = perm[at:at + n]
        p["refs"][perm[at:at + n]] = 1
        at += n
    p["refs"][p["table"][0, [1, 5, 77, 300]]] += 1   # the page held in part and some of the room behind it
    p["refs"][p["table"][1, 260:270]] += 1
    for parents, room in (([0, 0, 1, 2, 3, 4, 5], [400 * PAGE, 300, 64 * 299, 64 * 9, 64 * 5, 1, 0]),
                          ([1, 0, 6, 2], [0, 2000, 64 * 100, 64 * 300]), ([6, 5, 4, 3, 2, 1, 0], [1] * 7)):
        want = fork_rule(p["cache"], p["table"], p["counts"], p["lens"], p["refs"], parents, room)
        st = _status()
        cache, got = _fork(p, parents, room, kv, st)
        assert st.item() == 0
        for g, w in zip(got, want[1:]):
            assert np.array_equal(g, w)
        assert np.array_equal(cache.cpu().numpy().reshape(p["cache"].shape), want[0])


@pytest.mark.parametrize("nb,free", [(8192, [0, 8191]), (8193, [8192] + list(range(4000, 4030))), (70001, list(range(69000, 70001, 7))),
                                     (40000, [0, 1, 8191, 8192, 16383, 32767, 32768, 39999])])
@pytest.mark.parametrize("offset", [0, 1])
def test_fork_pages_in_large_pools(nb, free, offset):
    """Free pages far behind, at the borders of the search's steps, and counts that are not 16-byte aligned."""
    import torch

    import mla_latent_kv_gb300 as mla
    refs = np.ones(nb, np.int32)
    refs[free] = 0
    need = len(free) // 2 + 1
    parents, room = [-1, -1], [64 * need, 64 * (len(free) - need)]
    p = dict(cache=np.zeros((0, nb, 1, 1), np.uint8), table=np.full((1, 600), -1, np.int32), counts=np.zeros(1, np.int32),
             lens=np.zeros(1, np.int32), refs=refs)
    want = fork_rule(p["cache"], p["table"], p["counts"], p["lens"], refs, parents, room)
    buf = torch.zeros(nb + 4, dtype=torch.int32, device="cuda")
    at = buf[offset:offset + nb]
    at.copy_(dev(refs))
    cache = torch.zeros((0, nb, PAGE * 1152), dtype=torch.uint8, device="cuda")
    for extra in (0, 1):
        st = _status()
        got = mla.fork_pages(cache, dev(p["table"]), dev(p["counts"]), dev(p["lens"]), at, dev(np.array(parents, np.int32)),
                             dev(np.array(room, np.int32) + np.array([0, 64 * extra], np.int32)), dev_status=st)
        if extra:
            assert st.item() == mla.DEV_NO_PAGES
        else:
            assert st.item() == 0
            for g, w in zip(got, want[1:]):
                assert np.array_equal(g.cpu().numpy(), w)


def test_fork_pages_from_and_to_nothing():
    """A pool without rows, one that stays so, and one without pages."""
    import mla_latent_kv_gb300 as mla
    none = dict(cache=np.zeros((1, 9, PAGE, 1152), np.uint8), table=np.zeros((0, 5), np.int32), counts=np.zeros(0, np.int32),
                lens=np.zeros(0, np.int32), refs=np.array([0, 3, 0, 0, 1, 0, 0, 0, 0], np.int32))
    _, (table, counts, lens, refs) = _fork(none, [], [], BF)
    assert table.shape == (0, 5) and np.array_equal(refs, none["refs"])
    _, (table, counts, lens, refs) = _fork(none, [-1, -1], [100, -7], BF)
    assert table.tolist() == [[0, 2, -1, -1, -1], [-1] * 5] and counts.tolist() == [2, 0] and lens.tolist() == [0, 0]
    assert refs.tolist() == [1, 3, 1, 0, 1, 0, 0, 0, 0]
    empty = dict(none, cache=np.zeros((2, 0, PAGE, 1152), np.uint8), refs=np.zeros(0, np.int32))
    st = _status()
    _, (table, counts, lens, refs) = _fork(empty, [-1], [1], BF, st)
    assert st.item() == mla.DEV_NO_PAGES and counts.tolist() == [0] and refs.size == 0


@pytest.mark.parametrize("kv", [BF, F8])
def test_fork_pages_there_and_back(kv):
    """Two buffers of the state take turns over many random steps, captured or not, on a stream of their own."""
    import torch

    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(4)
    B, width, nb = 6, 6, 90
    p = random_pool(B, width, nb, 1, kv, 9, 200)
    cache = dev(p["cache"][0].reshape(nb, -1))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    a = tuple(dev(p[k]) for k in ("table", "counts", "lens", "refs"))
    b = (i32(B, width), i32(B), i32(B), i32(nb))
    parents, room, st = i32(B), i32(B), _status()
    ws = torch.empty(mla.fork_pages_workspace_bytes(B, B, nb), dtype=torch.uint8, device="cuda")

    def step():
        mla.fork_pages(cache, *a, parents, room, kv_dtype=kv, out=b, workspace=ws, dev_status=st)
        for x, y in zip(a, b):
            x.copy_(y)
    host = dict(p)
    side, graph = torch.cuda.Stream(), None
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for k in range(8):
            par = rng.integers(-1, B, B)
            own = np.where(par >= 0, host["lens"][par], 0)
            need = np.minimum(own + rng.integers(0, 100, B), width * PAGE)
            parents.copy_(dev(par.astype(np.int32)))
            room.copy_(dev(need.astype(np.int32)))
            ws.fill_(255)
            if k == 4:
                side.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step()
            graph.replay() if graph else step()
            side.synchronize()
            want = fork_rule(host["cache"], host["table"], host["counts"], host["lens"], host["refs"], par, need)
            assert want is not None and st.item() == 0
            host = dict(zip(("cache", "table", "counts", "lens", "refs"), want))
            for x, name in zip(a, ("table", "counts", "lens", "refs")):
                assert np.array_equal(x.cpu().numpy(), host[name]), (k, name)
            assert np.array_equal(cache.cpu().numpy().reshape(host["cache"][0].shape), host["cache"][0])
            # requests grow to the pages that they hold, as steps would make them
            grown = np.minimum(host["lens"] + rng.integers(0, 80, B), host["counts"] * PAGE).astype(np.int32)
            host["lens"] = grown
            a[2].copy_(dev(grown))


def test_fork_pages_tables_alone_and_no_rows():
    p = random_pool(4, 8, 50, 1, F8, 6, 300)
    want = fork_rule(p["cache"], p["table"], p["counts"], p["lens"], p["refs"], [3, 1], [0, 400])
    for g, w in zip(_fork(p, [3, 1], [0, 400], F8, layers=0)[1], want[1:]):
        assert np.array_equal(g, w)
    _, (table, counts, lens, refs) = _fork(p, [], [], F8)  # everything is given back
    assert table.shape == (0, 8) and np.array_equal(refs, fork_rule(p["cache"], p["table"], p["counts"], p["lens"], p["refs"], [], [])[4])


# -------------------------------------------------------------------------------------- a whole step
@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("captured", [False, True])
def test_steps_together(kv, captured):
    """Steps as a server makes them, all in a row on one stream: pages for the drafts, their rows turned and
    written, their queries absorbed, the tree's attention, the accepted branch moved up; forks and ends in
    between. Checked against the attention over the tokens that each row should hold by then."""
    import torch

    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(11)
    B, Sq, H, width, nb, steps = 5, 6, 16, 8, 80, 4
    freq, scale = mla.rope_frequencies(10000.0, 40.0), 1 / math.sqrt(192)
    w_uk_t, w_uv = _normal(rng, H, 128, L) * 0.05, _normal(rng, H, L, 128) * 0.05
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = torch.zeros((nb, PAGE * mla.row_bytes(kv)), dtype=torch.uint8, device="cuda")
    state = (torch.full((B, width), -1, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros(nb, **i32))
    other = tuple(torch.empty_like(x) for x in state)
    st = _status()
    # what each request should hold: its tokens' (kv_c, turned k_pe) as row values
    held = [[] for _ in range(B)]
    ins = dict(kv_a=torch.empty((B * Sq, D), dtype=torch.bfloat16, device="cuda"),
               q=torch.empty((B * Sq, H, 192), dtype=torch.bfloat16, device="cuda"),
               depth=torch.empty((B, Sq), **i32), masks=torch.empty((B, Sq), dtype=torch.int64, device="cuda"),
               parents=torch.empty(B, **i32), path=torch.empty((B, Sq), **i32), counts=torch.empty(B, **i32))
    absorbed = torch.empty((B * Sq, H, D), dtype=torch.bfloat16, device="cuda")
    outs = {}

    def step():
        """One step from `state` to `state` by way of `other`; every decision is in device memory."""
        table, pages, lens, refs = state
        before = torch.where(ins["parents"] >= 0, lens[ins["parents"].long().clamp_min(0)], torch.zeros_like(lens))
        mla.fork_pages(cache, table, pages, lens, refs, ins["parents"], before + Sq, kv_dtype=kv, out=other, dev_status=st)
        table, pages, lens, refs = other
        place = lens[:, None] + torch.arange(Sq, **i32)
        slots = (table.gather(1, (place // PAGE).long()).long() * PAGE + place % PAGE).view(-1)
        positions = (lens[:, None] + ins["depth"]).view(-1)
        mla.absorb_q(ins["q"][..., :128], None, w_uk_t, out=absorbed)
        mla.rope_cache_write(ins["kv_a"][:, :L], ins["kv_a"][:, L:], positions, freq, slots, cache, kv_dtype=kv,
                             q_pe=ins["q"][..., 128:], q_out=absorbed[..., L:], dev_status=st)
        full = lens + Sq
        o, lse = mla.decode_tree(absorbed.view(B, Sq, H, D), cache, table, full, ins["masks"], width * PAGE, scale, kv_dtype=kv,
                                 dev_status=st)
        outs["o"], outs["lse"] = o, lse
        outs["up"] = mla.out_proj(o.view(B * Sq, H, L), w_uv)
        new = mla.accept_tokens(cache, table, full, ins["path"], ins["counts"], kv_dtype=kv, dev_status=st)
        for x, y in zip(state, (table, pages, new, refs)):
            x.copy_(y)

    graph = None
    for k in range(steps):
        parents = np.arange(B) if k else np.full(B, -1)
        if k == 2:
            parents = np.array([1, 1, -1, 4, 1])  # forks, an end and a new one
        masks = tree_masks(B, Sq, 100 + k)
        depth = np.array([[bin(int(w) & (1 << 64) - 1).count("1") - 1 for w in row] for row in masks], np.int32)
        paths = []
        for b in range(B):
            leaf = int(rng.integers(0, Sq))
            paths.append([i for i in range(Sq) if int(masks[b, leaf]) >> i & 1])
        path = np.zeros((B, Sq), np.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = p
        for name, x in (("depth", depth), ("masks", masks), ("parents", parents.astype(np.int32)), ("path", path),
                        ("counts", np.array([len(p) for p in paths], np.int32))):
            ins[name].copy_(dev(x))
        ins["kv_a"].copy_(_normal(rng, B * Sq, D))
        ins["q"].copy_(_normal(rng, B * Sq, H, 192))
        held = [list(held[p]) if p >= 0 else [] for p in parents]
        starts = [len(h) for h in held]
        if not captured:
            step()
        else:
            if graph is None:
                copies = [x.clone() for x in state] + [cache.clone()]
                step()  # first calls outside the capture, then back to where it was
                torch.cuda.synchronize()
                for x, y in zip([*state, cache], copies):
                    x.copy_(y)
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        assert st.item() == 0
        # the definition, from this step's rows: bf16 values, or what e4m3 and a scale make of them
        pos = torch.tensor([starts[b] + int(depth[b, t]) for b in range(B) for t in range(Sq)], device="cuda")
        turned = mla.rope(ins["kv_a"][:, None, L:], pos.to(torch.int32), freq)[:, 0]
        rows = torch.cat([ins["kv_a"][:, :L], turned], 1).double()
        q_pe = mla.rope(ins["q"][..., 128:], pos.to(torch.int32), freq)
        q = torch.cat([torch.einsum("thp,hpl->thl", ins["q"][..., :128].double(), w_uk_t.double()), q_pe.double()], 2)
        for b in range(B):
            for t in range(Sq):
                keys = held[b] + [rows[b * Sq + i] for i in range(Sq) if int(masks[b, t]) >> i & 1]
                K = torch.stack(keys)
                x = q[b * Sq + t] @ K.t() * scale
                p = torch.softmax(x, 1)
                want, mag = p @ K[:, :L], p @ K[:, :L].abs()
                # relative steps of rows and query: bf16 2^-8 (q's rounding after absorption) in the scores, e4m3
                # 2^-4 of each value (or 2^-10 of 1/448 of the row's largest) in keys and values
                e = 2.0 ** -4 if kv == F8 else 0.0
                floor = (2.0 ** -10 / 448 * K.abs().amax(1, keepdim=True)) if kv == F8 else 0.0
                dk = e * K.abs() + floor
                ds = ((q[b * Sq + t].abs() @ dk.t()) * (1 + 2.0 ** -8) + 2.0 ** -8 * (q[b * Sq + t].abs() @ K.abs().t())) * scale
                # weights change by at most exp(2 ds) - 1 each; only of use where that is small
                grow = torch.expm1(2 * ds.amax(1, keepdim=True))
                dv = (dk[:, :L] if kv == F8 else torch.zeros_like(K[:, :L]))
                tol = grow * 2 * mag + p @ dv * (1 + grow) + 2.0 ** -7 * mag
                got = outs["o"][b, t].double()
                assert ((got - want).abs() <= tol).all(), (k, b, t)
            held[b] += [rows[b * Sq + i] for i in paths[b]]
        assert state[2].tolist() == [len(h) for h in held]
        # the cache holds the accepted rows in their places
        lens = state[2].tolist()
        for b in range(B):
            blocks = state[0][b, :-(-lens[b] // PAGE)].long()
            raw = cache[blocks].view(-1, mla.row_bytes(kv))[:lens[b]]
            K = torch.stack(held[b])
            if kv == BF:
                assert torch.equal(raw.contiguous().view(torch.bfloat16).double(), K)
            else:
                value = raw[:, :D].contiguous().view(torch.float8_e4m3fn).double() * raw[:, D:D + 4].contiguous().view(torch.float32).double()
                assert ((value - K).abs() <= (2.0 ** -4 + 2.0 ** -7) * K.abs() + 2.0 ** -10 / 447 * K.abs().amax(1, keepdim=True)).all()


# -------------------------------------------------------------------------------------- the binding
def test_what_the_library_refuses_is_raised_with_its_reason():
    """Arguments that only the C calls check, and buffers of the wrong size, type or place: nothing is launched."""
    import torch

    import mla_latent_kv_gb300 as mla
    freq = mla.rope_frequencies()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32
    with pytest.raises(mla.MlaError, match="mla_rope: 16-byte") as e:
        mla.rope(z(3, 2, 72)[..., 4:68], z(3, dtype=i32), freq)
    assert e.value.status == mla.ERR_UNSUPPORTED
    with pytest.raises(mla.MlaError, match="mscale"):
        mla.rope(z(3, 2, R), z(3, dtype=i32), freq, mscale=float("nan"))
    with pytest.raises(ValueError, match="inv_freq"):
        mla.rope(z(3, 2, R), z(3, dtype=i32), freq.cuda())
    with pytest.raises(ValueError, match="positions"):
        mla.rope(z(3, 2, R), z(3, dtype=torch.int64), freq)
    with pytest.raises(ValueError, match="one CUDA device"):
        mla.rope(z(3, 2, R), torch.zeros(3, dtype=i32), freq)
    c = tree_case([70, 90], 3, 16, BF, 1)
    args = (c["q"], c["cache"], c["table"], c["seq_lens"], c["masks"], 90)
    with pytest.raises(mla.MlaError, match="scale"):
        mla.decode_tree(*args, 0.0)
    with pytest.raises(mla.MlaError, match="workspace") as e:
        mla.fork_pages(z(4, PAGE * 576), z(2, 3, dtype=i32), z(2, dtype=i32), z(2, dtype=i32), z(4, dtype=i32), z(1, dtype=i32),
                       z(1, dtype=i32), workspace=z(8, dtype=torch.uint8))
    assert e.value.status == mla.ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(mla.MlaError, match="kv_dtype"):
        mla.decode_tree(*args, 0.07, kv_dtype=7)
    with pytest.raises(ValueError, match="o_latent"):
        mla.decode_tree(*args, 0.07, o_latent=z(2, 3, 16, 511))
    with pytest.raises(ValueError, match="lse"):
        mla.decode_tree(*args, 0.07, lse=z(2, 3, 16))
    with pytest.raises(ValueError, match="num_blocks"):
        mla.decode_tree(*args, 0.07, num_blocks=c["num_blocks"] + 1)
    many = tree_case([70], 2, 3, BF, 1)
    with pytest.raises(mla.MlaError, match="65 drafts"):
        mla.decode_tree(z(1, 65, 3, D), many["cache"], many["table"], many["seq_lens"], z(1, 65, dtype=torch.int64), 70, 0.07)
    lens = z(2, dtype=i32)
    with pytest.raises(mla.MlaError, match="seq_lens"):
        mla.accept_tokens(z(4, PAGE * 576), z(2, 3, dtype=i32), lens, z(2, 5, dtype=i32), z(2, dtype=i32), new_lens=lens)
    state = (z(2, 3, dtype=i32), z(2, dtype=i32), z(2, dtype=i32), z(4, dtype=i32))
    with pytest.raises(mla.MlaError, match="old one's buffers"):
        mla.fork_pages(z(4, PAGE * 576), *state, z(2, dtype=i32), z(2, dtype=i32), out=state)
    with pytest.raises(TypeError, match="tuple"):
        mla.fork_pages(z(4, PAGE * 576), *state, z(2, dtype=i32), z(2, dtype=i32), out=list(state))
    with pytest.raises(ValueError, match="pages of"):
        mla.fork_pages(z(4, PAGE * 500), *state, z(2, dtype=i32), z(2, dtype=i32))
    torch.cuda.synchronize()


def test_given_buffers_are_used_and_returned():
    import torch

    import mla_latent_kv_gb300 as mla
    c = tree_case([70, 90], 3, 16, F8, 2)
    o, lse = torch.zeros(2, 3, 16, L, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 3, 16, device="cuda")
    got = _tree(c, o_latent=o, lse=lse)
    assert got[0] is o and got[1] is lse
    check_attention(o, lse, attend_tree(c), bf16_out=True)
    x, pos = torch.ones(2, 3, R, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    assert mla.rope(x, pos, mla.rope_frequencies(), out=x) is x and bool((x == 1).all())
    assert mla.rope(x, pos, mla.rope_frequencies()).data_ptr() != x.data_ptr()
