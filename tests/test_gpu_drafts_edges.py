"""Calls of a step with drafted tokens that lie at the edge of what their documentation allows, on the GPU."""
import math
from fractions import Fraction

import numpy as np
import pytest

import mla_inputs as mi
from drafts_util import attend_tree, tree_case, tree_masks
from longctx_util import PAGE, check_attention, dev, paged_case

pytestmark = pytest.mark.gpu
BF, F8 = mi.KV_BF16, mi.KV_FP8
R = 64
TWO_PI = Fraction(62831853071795864769252867665590057684, 10 ** 37)


def _status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------------- page pool
@pytest.mark.parametrize("parents", [[0], [0, -1], [-1, 0], [0, 1], [1, 0], [0, 0], [1]])
@pytest.mark.parametrize("page", [0, 2, 3])
@pytest.mark.parametrize("bad", [30, -5, 2 ** 31 - 1])
def test_fork_pages_reports_every_bad_entry(parents, page, bad):
    """A row's entry outside the cache is reported whoever goes on from the row: its first child alone too, and
    in a page full of tokens too."""
    import mla_latent_kv_gb300 as mla
    table = np.array([[3, 4, 5, 6, -1], [9, -1, -1, -1, -1]], np.int32)
    table[0, page] = bad
    counts, lens = np.array([4, 1], np.int32), np.array([200, 10], np.int32)
    refs = np.zeros(30, np.int32)
    refs[[p for p in table.ravel() if 0 <= p < 30]] = 1
    host = np.random.default_rng(0).integers(0, 256, (30, PAGE * 1152), dtype=np.uint8)
    cache, st = dev(host), _status()
    room = [int(lens[p]) if p >= 0 else 0 for p in parents]
    got = mla.fork_pages(cache, dev(table), dev(counts), dev(lens), dev(refs), dev(np.array(parents, np.int32)),
                         dev(np.array(room, np.int32)), dev_status=st)
    assert st.item() == mla.DEV_BAD_BLOCK_ID
    new, new_counts, new_lens, new_refs = [x.cpu().numpy() for x in got]
    assert new_counts.tolist() == [-(-n // PAGE) for n in room] and new_lens.tolist() == room
    want = np.zeros(30, np.int32)
    for r, p in enumerate(parents):
        for j in range(new_counts[r]):
            if j < lens[p] // PAGE:
                assert new[r, j] == table[p, j]  # passed on
            if 0 <= new[r, j] < 30:
                want[new[r, j]] += 1
    assert np.array_equal(new_refs, want)        # and not counted
    before = np.flatnonzero(refs)
    assert np.array_equal(cache.cpu().numpy()[before], host[before])


# -------------------------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_rope_small_angles_at_far_positions(base, sign):
    """Positions near 2^31 that end within a few millionths of a whole turn: the sine has the angle's own relative
    accuracy in bf16, so that it shows the angle's absolute error.

    A pair's step is off by half of 2^-64 of a turn, 2^-34 turns after 2^31 positions, and the angle's leading 32 bits
    leave out less than 2^-32: together under 2^-31 turns, 2^-28.3 rad. Then sincospi and the products in fp32,
    2^-20 relative with room, and one rounding to bf16, 2^-8."""
    import torch

    import mla_latent_kv_gb300 as mla
    freq = mla.rope_frequencies(base)
    top = np.arange(2 ** 31 - 2 ** 22, 2 ** 31 - 1, dtype=np.uint64)
    positions = []
    for w in freq.tolist():
        step = np.uint64(round(Fraction(w) / TWO_PI * 2 ** 64) % 2 ** 64)
        off = (top * step).view(np.int64)
        size = np.abs(off.astype(np.float64))
        positions.append(sign * int(top[np.argmin(np.where(size > 2.0 ** 41, size, np.inf))]))
    x = np.zeros((32, 1, R), np.float32)
    x[..., 0::2] = 1.0
    got = mla.rope(torch.from_numpy(x).to(torch.bfloat16).cuda(), dev(np.array(positions, np.int32)), freq).double().cpu()
    for i, (m, w) in enumerate(zip(positions, freq.tolist())):
        turn = Fraction(w) * m / TWO_PI
        want = math.sin(float((turn - round(turn)) * TWO_PI))
        assert abs(want) < 0.02
        assert abs(got[i, 0, 2 * i + 1].item() - want) <= (2.0 ** -8 + 2.0 ** -20) * abs(want) + 2.0 ** -28.3, (i, m)


# ------------------------------------------------------------------------------------------ trees
@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("Sq,H", [(1, 1), (2, 16), (3, 11), (2, 64), (3, 43), (4, 128)])  # either side of 32 and 128 pairs
@pytest.mark.parametrize("B", [1, 90])
def test_decode_tree_with_a_bound_of_zero_needs_no_cache(B, Sq, H, kv):
    """Every row is an empty one, as in mla_decode, and a positive length is reported; the cache, the table and the
    workspace may be null though the cache is said to have blocks."""
    import torch

    import mla_latent_kv_gb300 as mla
    lib = mla.lib()
    q = torch.ones((B, Sq, H, 576), dtype=torch.bfloat16, device="cuda")
    masks = torch.full((B, Sq), -1, dtype=torch.int64, device="cuda")
    need = mla.decode_tree_workspace_bytes(B, Sq, H, 0, kv)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    for length in (0, 5):
        lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
        for max_blocks in (0, 4):
            o = torch.full((B, Sq, H, 512), 7.0, device="cuda")
            lse, st = torch.full((B, Sq, H), 7.0, device="cuda"), _status()
            p = lambda t: t.data_ptr()  # noqa: E731
            rc = lib.mla_decode_tree(p(q), None, kv, 8, None, max_blocks, p(lens), p(masks), 0, B, Sq, H, 0.07,
                                     p(ws) if need else None, need, p(o), mla.DT_F32, p(lse), p(st),
                                     torch.cuda.current_stream().cuda_stream)
            assert rc == mla.OK, lib.mla_last_error_detail()
            assert bool((o == 0).all()) and bool((lse == -math.inf).all())
            assert st.item() == (mla.DEV_SEQ_TOO_LONG if length else 0)


@pytest.mark.parametrize("Sq,H,kv", [(1, 33, BF), (3, 43, BF), (3, 43, F8), (2, 2, F8), (1, 40, F8)])
def test_decode_tree_of_more_requests_than_a_grid_is_high(Sq, H, kv):
    """70,000 requests of a page each, as mla_decode takes them; some of them checked in 64 bits."""
    import torch

    import mla_latent_kv_gb300 as mla
    B = 70000
    c = paged_case([PAGE] * 40, 1, 1, kv, 40)
    rng = np.random.default_rng(41)
    pages, lens = c["full_table"][rng.integers(0, 40, B), :1], rng.integers(0, PAGE + 1, B)
    masks = np.tile(tree_masks(50, Sq, 42), (B // 50, 1))
    q = torch.empty((B, Sq, H, 576), dtype=torch.bfloat16, device="cuda")
    q.normal_(generator=torch.Generator(device="cuda").manual_seed(43))
    st = _status()
    o, lse = mla.decode_tree(q, c["cache"], dev(pages), dev(lens.astype(np.int32)), dev(masks), PAGE, c["scale"], kv_dtype=kv,
                             o_dtype=mla.DT_BF16, dev_status=st, num_blocks=c["num_blocks"])
    assert st.item() == 0 and not bool(o.isnan().any())
    some = [0, 1, 32767, 65534, 65535, 65536, 65537, B - 2, B - 1]
    part = dict(c, B=len(some), Sq=Sq, H=H, lens=lens[some], full_table=pages[some], q=q[some], masks_host=masks[some])
    check_attention(o[some], lse[some], attend_tree(part), bf16_out=True)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("Sq,H,pages", [
    (27, 64, [10] * 9 + [9, 5, 4, 2, 0]),                        # seven tiles a request, 98 units for 36 clusters
    (28, 64, [13] * 9 + [12, 8, 3, 3, 1, 0, 0, 0]),
    (64, 128, [9, 9, 8, 0]),                                     # 32 tiles of four requests
    (16, 71, [11] * 7 + [10] * 6 + [8, 7, 7, 4, 4, 3, 2, 2, 1]),
    (12, 128, [20] * 8 + [19] * 8 + [18, 17, 16, 10, 8, 8, 5, 3, 2, 2, 1, 0]),
    (48, 128, [9, 9, 9, 9, 9, 8, 7, 7, 2, 0, 0]),                # 24 tiles: six units a cluster
    (24, 64, [31] * 3 + [30] * 6 + [29, 26, 26, 18, 14, 12, 9, 5, 2, 1, 0, 0]),
    (3, 60, [2] * 40 + [1] * 80 + [4] * 60),                     # five short units a cluster
])
def test_decode_tree_of_short_units_in_a_row(Sq, H, pages, kv):
    """Three and more short units a cluster: while the output CTAs finish one, the next one's weights wait to be sent and
    the third one's queries are loaded beside them. The same call over and over gives the same bits, and the right ones."""
    import torch

    import mla_latent_kv_gb300 as mla
    rng = np.random.default_rng(sum(pages))
    lens = [max(0, 64 * n - int(rng.integers(0, 64))) for n in pages]
    c = tree_case(lens, Sq, H, kv, 50 + len(pages), scale_v=1.7 if kv == F8 else None)
    st = _status()
    call = lambda: mla.decode_tree(c["q"], c["cache"], c["table"], c["seq_lens"], c["masks"], c["max_len"],  # noqa: E731
                                   c["scale"], kv_dtype=kv, num_blocks=c["num_blocks"], dev_status=st)
    o, lse = call()
    check_attention(o, lse, attend_tree(c))
    for _ in range(40):
        again = call()
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    assert st.item() == 0
