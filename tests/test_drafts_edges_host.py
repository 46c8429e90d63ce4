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
