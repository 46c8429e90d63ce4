"""Refusals of the calls of a step with drafted tokens that their documentation implies: nothing is launched here."""
import ctypes

import pytest

from test_drafts_host import FREQ, P, P2
from test_longctx_host import _call, lib  # noqa: F401 (lib: a fixture)

mla = pytest.importorskip("mla_latent_kv_gb300")


def test_rope_cache_write_refuses_what_cache_write_does(lib):  # noqa: F811
    """A scale below 0 and a cache of more blocks than there can be, as mla_cache_write."""
    rope = dict(kv_c=P, st_c=512, k_pe=P, st_pe=64, q=None, qt=0, qh=0, out=None, ot=0, oh=0, pos=P, freq=FREQ, mscale=1.0,
                adjacent=1, slots=P, T=3, H=0, cache=P, kv=1, nb=4, kv_scale=0.0, st=None, s=None)
    plain = dict(kv_c=P, st_c=512, k_pe=P, st_pe=64, slots=P, T=3, cache=P, kv=1, nb=4, kv_scale=0.0, st=None, s=None)
    for bad, status in ((dict(kv_scale=-0.5), mla.ERR_INVALID_ARG), (dict(kv_scale=float("inf")), mla.ERR_INVALID_ARG),
                        (dict(kv_scale=float("nan")), mla.ERR_INVALID_ARG), (dict(nb=(1 << 40) + 1), mla.ERR_UNSUPPORTED)):
        assert _call(lib.mla_cache_write, plain, **bad) == status
        assert _call(lib.mla_rope_cache_write, rope, **bad) == status


def _at(x):
    return ctypes.c_void_p(x)


def test_accept_tokens_refuses_results_over_its_inputs(lib):  # noqa: F811
    """The blocks of every layer read the inputs while the first one's write new_lens: a buffer that overlaps any of
    them would change a branch for some layers."""
    d = dict(cache=P, kv=0, layers=2, nb=8, table=_at(0x10000), max_blocks=4, seq=_at(0x20000), path=_at(0x30000),
             counts=_at(0x40000), B=3, Sq=4, new=_at(0x50000), st=None, s=None)
    for base, n in ((0x10000, 12), (0x20000, 3), (0x30000, 12), (0x40000, 3)):
        for at in (base, base + 4 * (n - 1), base - 4 * 2):
            assert _call(lib.mla_accept_tokens, d, new=_at(at)) == mla.ERR_INVALID_ARG, hex(at)
            assert b"overlap" in lib.mla_last_error_detail()


def test_fork_pages_refuses_a_new_state_over_the_old(lib):  # noqa: F811
    d = dict(cache=P, kv=0, layers=1, nb=8, table=_at(0x10000), max_blocks=4, counts=_at(0x20000), lens=_at(0x30000),
             refs=_at(0x40000), B=2, parents=P, room=P, B2=3, new_table=_at(0x50000), new_counts=_at(0x60000),
             new_lens=_at(0x70000), new_refs=_at(0x80000), ws=None, ws_bytes=0, st=None, s=None)
    call = lambda **kw: _call(lib.mla_fork_pages, d, **kw)  # noqa: E731
    assert call() == mla.ERR_WORKSPACE_TOO_SMALL  # nothing else is wrong
    for name, size in (("new_table", 12), ("new_counts", 3), ("new_lens", 3), ("new_refs", 8)):
        for base, n in ((0x10000, 8), (0x20000, 2), (0x30000, 2), (0x40000, 8)):
            for at in (base, base + 4 * (n - 1), base - 4 * (size - 1)):
                assert call(**{name: _at(at)}) == mla.ERR_INVALID_ARG, (name, hex(at))
            for at in (base + 4 * n, base - 4 * size):
                assert call(**{name: _at(at)}) == mla.ERR_WORKSPACE_TOO_SMALL, (name, hex(at))
