"""Argument checks and host arithmetic of the calls of a step with drafted tokens: nothing is launched here."""
import ctypes
import math
import types

import numpy as np
import pytest

from drafts_util import accept_rule, fork_rule
from test_longctx_host import _call, lib  # noqa: F401 (lib: a fixture)

mla = pytest.importorskip("mla_latent_kv_gb300")
P = ctypes.c_void_p(0x1000)      # never dereferenced: every call here is refused first
P2 = ctypes.c_void_p(0x2000)
ODD = ctypes.c_void_p(0x1008)    # not 16-byte aligned
FREQ = (ctypes.c_double * 32)(*[10000.0 ** (-i / 32) for i in range(32)])
ROPE = dict(x=P, xt=128, xn=64, pos=P, freq=FREQ, mscale=1.0, adjacent=1, out=P, ot=128, on=64, T=3, N=2, s=None)


def test_rope_refusals(lib):  # noqa: F811
    call = lambda **kw: _call(lib.mla_rope, ROPE, **kw)  # noqa: E731
    assert call(T=-1) == mla.ERR_INVALID_ARG and call(N=0) == mla.ERR_INVALID_ARG
    assert call(freq=None) == mla.ERR_INVALID_ARG and call(adjacent=2) == mla.ERR_INVALID_ARG
    for bad in (float("nan"), float("inf")):
        assert call(mscale=bad) == mla.ERR_INVALID_ARG
        assert call(freq=(ctypes.c_double * 32)(*[1.0] * 31, bad)) == mla.ERR_INVALID_ARG
    for name in ("x", "out", "pos"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG
    assert call(x=None, out=None) == mla.ERR_INVALID_ARG
    assert call(x=ODD) == mla.ERR_UNSUPPORTED and call(out=ODD) == mla.ERR_UNSUPPORTED
    for name in ("xt", "xn", "ot", "on"):
        assert call(**{name: 68}) == mla.ERR_UNSUPPORTED
    assert call(ot=0) == mla.ERR_INVALID_ARG and call(on=0) == mla.ERR_INVALID_ARG
    assert call(T=1 << 30, N=128) == mla.ERR_UNSUPPORTED
    assert b"mla_rope" in lib.mla_last_error_detail()
    assert call(T=0) == mla.OK and lib.mla_last_error_detail() == b""


def test_rope_cache_write_refusals(lib):  # noqa: F811
    d = dict(kv_c=P, st_c=512, k_pe=P, st_pe=64, q=P, qt=128, qh=64, out=P2, ot=128, oh=64, pos=P, freq=FREQ, mscale=1.0,
             adjacent=0, slots=P, T=3, H=2, cache=P, kv=0, nb=4, kv_scale=0.0, st=None, s=None)
    call = lambda **kw: _call(lib.mla_rope_cache_write, d, **kw)  # noqa: E731
    assert call(kv=5) == mla.ERR_INVALID_ARG and call(nb=-1) == mla.ERR_INVALID_ARG
    assert call(kv_scale=float("nan")) == mla.ERR_INVALID_ARG and call(T=-1) == mla.ERR_INVALID_ARG
    for name in ("kv_c", "k_pe", "pos", "freq", "slots", "cache", "q", "out"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG, name
    for name in ("kv_c", "k_pe", "cache", "q", "out"):
        assert call(**{name: ODD}) == mla.ERR_UNSUPPORTED, name
    for name in ("st_c", "st_pe", "qt", "oh"):
        assert call(**{name: 65}) == mla.ERR_UNSUPPORTED, name
    assert call(H=0) == mla.ERR_INVALID_ARG
    assert call(T=0) == mla.OK and call(T=0, q=None, out=None, H=0) == mla.OK


def test_decode_tree_refusals(lib):  # noqa: F811
    d = dict(q=P, cache=P, kv=0, nb=8, table=P, max_blocks=4, seq=P, mask=P, max_len=256, B=2, Sq=4, H=16, scale=0.07,
             ws=P, ws_bytes=1 << 40, o=P, o_dtype=0, lse=P, st=None, s=None)
    call = lambda **kw: _call(lib.mla_decode_tree, d, **kw)  # noqa: E731
    assert call(kv=9) == mla.ERR_INVALID_ARG and call(o_dtype=5) == mla.ERR_INVALID_ARG
    assert call(H=0) == mla.ERR_UNSUPPORTED and call(H=129) == mla.ERR_UNSUPPORTED
    assert call(B=-2) == mla.ERR_INVALID_ARG and call(Sq=0) == mla.ERR_INVALID_ARG
    assert call(Sq=65) == mla.ERR_UNSUPPORTED
    assert call(max_len=257) == mla.ERR_INVALID_ARG and call(max_len=-1) == mla.ERR_INVALID_ARG
    assert call(max_len=2 ** 31 - 1, max_blocks=2 ** 25) == mla.ERR_UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == mla.ERR_INVALID_ARG
    for name in ("q", "cache", "table", "seq", "mask", "o"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG, name
    for name in ("q", "cache", "o"):
        assert call(**{name: ODD}) == mla.ERR_UNSUPPORTED, name
    assert call(B=1 << 20, Sq=64) == mla.ERR_UNSUPPORTED
    assert call(B=0) == mla.OK
    for bad in (dict(kv=9), dict(Sq=65), dict(H=0), dict(B=0), dict(n=-1)):
        a = {**dict(kv=0, B=2, Sq=4, H=16, n=256), **bad}
        assert lib.mla_decode_tree_workspace_bytes(*a.values()) == 0


def test_accept_tokens_refusals(lib):  # noqa: F811
    d = dict(cache=P, kv=0, layers=2, nb=8, table=P, max_blocks=4, seq=P, path=P, counts=P, B=2, Sq=4, new=P2, st=None, s=None)
    call = lambda **kw: _call(lib.mla_accept_tokens, d, **kw)  # noqa: E731
    assert call(kv=3) == mla.ERR_INVALID_ARG and call(B=-1) == mla.ERR_INVALID_ARG and call(Sq=0) == mla.ERR_INVALID_ARG
    assert call(Sq=65) == mla.ERR_UNSUPPORTED and call(layers=0) == mla.ERR_INVALID_ARG
    assert call(nb=-1) == mla.ERR_INVALID_ARG and call(layers=-1) == mla.ERR_INVALID_ARG
    assert call(nb=1 << 40) == mla.ERR_UNSUPPORTED and call(max_blocks=1 << 30) == mla.ERR_UNSUPPORTED
    for name in ("cache", "table", "seq", "path", "counts", "new"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG, name
    assert call(new=P) == mla.ERR_INVALID_ARG  # seq_lens itself
    assert call(cache=ODD) == mla.ERR_UNSUPPORTED
    assert call(B=0) == mla.OK


def test_fork_pages_refusals(lib):  # noqa: F811
    d = dict(cache=P, kv=0, layers=1, nb=8, table=P, max_blocks=4, counts=P, lens=P, refs=P, B=2, parents=P, room=P, B2=3,
             new_table=P2, new_counts=P2, new_lens=P2, new_refs=P2, ws=P, ws_bytes=1 << 30, st=None, s=None)
    call = lambda **kw: _call(lib.mla_fork_pages, d, **kw)  # noqa: E731
    assert call(kv=3) == mla.ERR_INVALID_ARG and call(B=-1) == mla.ERR_INVALID_ARG and call(B2=-1) == mla.ERR_INVALID_ARG
    assert call(B=8193) == mla.ERR_UNSUPPORTED and call(B2=8193) == mla.ERR_UNSUPPORTED
    assert call(B=8192, max_blocks=1 << 19) == mla.ERR_UNSUPPORTED
    for name in ("cache", "table", "counts", "lens", "refs", "parents", "room", "new_table", "new_counts", "new_lens", "new_refs"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG, name
    for name in ("new_table", "new_counts", "new_lens", "new_refs"):
        assert call(**{name: P}) == mla.ERR_INVALID_ARG, name
    assert call(cache=ODD) == mla.ERR_UNSUPPORTED
    assert call(ws=None) == mla.ERR_WORKSPACE_TOO_SMALL and call(ws_bytes=64) == mla.ERR_WORKSPACE_TOO_SMALL
    assert call(ws=ctypes.c_void_p(0x1010)) == mla.ERR_UNSUPPORTED
    assert call(B=0, B2=0, nb=0) == mla.OK
    assert call(B2=0, new_table=None, new_counts=None, new_lens=None, parents=None, room=None, ws=None) == \
        mla.ERR_WORKSPACE_TOO_SMALL  # nothing else is missing then
    assert lib.mla_fork_pages_workspace_bytes(-1, 1, 1) == 0
    assert lib.mla_fork_pages_workspace_bytes(2, 3, 8) >= 256 + 3 * 32 + 2 * 4 + 8 * 4


def test_frequencies(lib):  # noqa: F811
    import torch
    plain = mla.rope_frequencies(10000.0)
    assert plain.dtype is torch.float64 and plain.device.type == "cpu"
    np.testing.assert_allclose(plain.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    # factor 40 over 4096 trained positions: pair 10 makes 36 turns there, pair 11 27, pair 22 1.2, pair 23 0.87
    got = mla.rope_frequencies(10000.0, 40.0, 4096, 32.0, 1.0)
    turns = 4096 * plain.numpy() / (2 * math.pi)
    assert turns[10] > 32 > turns[11] and turns[22] > 1 > turns[23]
    ramp = np.clip((np.arange(32) - 10) / 13, 0, 1)
    np.testing.assert_allclose(got.numpy(), plain.numpy() * (ramp / 40 + 1 - ramp), rtol=1e-14)
    for bad in (dict(base=1.0), dict(base=float("nan")), dict(factor=0.5), dict(factor=2.0, trained=0),
                dict(factor=2.0, beta_slow=0.0), dict(factor=2.0, beta_fast=0.5), dict(factor=float("inf"))):
        with pytest.raises(mla.MlaError):
            mla.rope_frequencies(**bad)
    assert lib.mla_rope_frequencies(10000.0, 1.0, 1, 1.0, 1.0, None) == mla.ERR_INVALID_ARG


def _args(torch):
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)  # noqa: E731
    i32, i64 = torch.int32, torch.int64
    freq = torch.ones(32, dtype=torch.float64)
    q, cache, table, lens = z(2, 3, 16, 576), z(8, 64 * 576), z(2, 4, dtype=i32), z(2, dtype=i32)
    return {
        "rope": dict(x=z(5, 2, 64), positions=z(5, dtype=i32), inv_freq=freq),
        "rope_cache_write": dict(kv_c=z(5, 512), k_pe=z(5, 64), positions=z(5, dtype=i32), inv_freq=freq,
                                 slot_mapping=z(5, dtype=i64), kv_cache=cache, q_pe=z(5, 2, 64), q_out=z(5, 2, 64)),
        "decode_tree": dict(q=q, kv_cache=cache, block_table=table, seq_lens=lens, tree_mask=z(2, 3, dtype=i64),
                            max_seq_len=200, scale=0.07),
        "accept_tokens": dict(kv_cache=cache, block_table=table, seq_lens=lens, path=z(2, 3, dtype=i32), counts=z(2, dtype=i32)),
        "fork_pages": dict(kv_cache=cache, block_table=table, page_counts=z(2, dtype=i32), seq_lens=lens, refs=z(8, dtype=i32),
                           parents=z(3, dtype=i32), room=z(3, dtype=i32)),
    }


@pytest.mark.parametrize("call", ["rope", "rope_cache_write", "decode_tree", "accept_tokens", "fork_pages"])
def test_binding_refuses_wrong_tensors(call, lib):  # noqa: F811
    torch = pytest.importorskip("torch")
    good = _args(torch)[call]
    for name, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        for bad in (t.to(torch.float16), t[:-1] if t.ndim == 1 else t[..., :-1], t[None]):
            if name == "kv_cache" and call in ("rope_cache_write", "decode_tree"):
                continue  # raw bytes: any element type that holds the pages
            if name == "kv_cache" and (bad.ndim == 3 or bad.dtype is torch.float16):
                continue  # one layer, or elements of the same size
            if name == "block_table" and bad.dtype is t.dtype and bad.ndim == 2:
                continue  # another max_blocks
            if name == "path" and bad.dtype is t.dtype and bad.ndim == 2:
                continue  # another number of drafts
            if name in ("refs", "parents") and bad.dtype is t.dtype and bad.ndim == 1 and call == "fork_pages" and name == "parents":
                with pytest.raises(ValueError):
                    getattr(mla, call)(**{**good, name: bad})  # room has another length
                continue
            with pytest.raises((ValueError, mla.MlaError)):
                getattr(mla, call)(**{**good, name: bad})
    with pytest.raises(ValueError, match="device"):
        getattr(mla, call)(**good)
    with pytest.raises(TypeError):
        getattr(mla, call)(**{**good, next(iter(good)): None})
    if call != "rope":
        with pytest.raises(ValueError, match="dev_status"):
            getattr(mla, call)(**good, dev_status=torch.zeros(1))


@pytest.mark.parametrize("call", ["rope", "decode_tree", "accept_tokens", "fork_pages"])
def test_buffers_are_made_on_the_stream_that_uses_them(call, monkeypatch):
    """As the other calls: what a call with stream= makes itself, it makes with that stream as the current one,
    and a call that is given every buffer goes to the stream as it is."""
    torch = pytest.importorskip("torch")
    here, native, used = [], [], []

    class OnStream:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            here.append(self.stream.name)

        def __exit__(self, *exc):
            here.pop()

    class Native:
        def __getattr__(self, name):
            def f(*args):
                native.append((here[-1] if here else "current", args[-2 if name == "decode_tree" else -1]))
                return (torch.zeros(2),) * (2 if name == "decode_tree" else 4) if name in ("decode_tree", "fork_pages") \
                    else torch.zeros(2)
            return f
    args = _args(torch)[call]
    monkeypatch.setattr(mla, "_native", Native)
    monkeypatch.setattr(torch.cuda, "stream", OnStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s: types.SimpleNamespace(device=0, name=s))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: used.append(s))
    side = types.SimpleNamespace(cuda_stream="side")
    getattr(mla, call)(**args)
    assert native == [("current", None)] and used == []
    out = getattr(mla, call)(**args, stream=side)
    assert native[1:] == [("side", None)]
    assert used == ["current"] * (len(out) if isinstance(out, tuple) else 1)  # kept while the caller's stream reads them
    ws = torch.zeros(4096, dtype=torch.uint8)
    bufs = {"rope": lambda: dict(out=out), "accept_tokens": lambda: dict(new_lens=out),
            "decode_tree": lambda: dict(o_latent=out[0], lse=out[1], workspace=ws),
            "fork_pages": lambda: dict(out=out, workspace=ws)}[call]()
    getattr(mla, call)(**args, **bufs, stream=side)
    assert native[2:] == [("current", "side")] and len(used) == (len(out) if isinstance(out, tuple) else 1)


def test_the_plain_rules():
    """The tests' own rules on cases worked by hand."""
    # one request of 70 tokens, 6 of them drafts (64..69, page 1): drafts 0, 2 and 5 accepted
    cache = np.arange(3 * 64, dtype=np.uint8).reshape(1, 3, 64, 1).copy()
    table = np.array([[2, 0]], np.int32)
    new, lens, bad = accept_rule(cache, table, [70], np.array([[0, 2, 5, 0, 0, 0]]), [3])
    assert lens.tolist() == [67] and not bad
    want = cache.copy()
    want[0, 0, 1], want[0, 0, 2] = cache[0, 0, 2], cache[0, 0, 5]
    assert np.array_equal(new, want)
    _, lens, bad = accept_rule(cache, table, [70], np.array([[0, 2, 2, 0, 0, 0]]), [3])
    assert lens.tolist() == [66] and bad
    # a row of 70 tokens in pages 5 and 1, forked in two; row 2 is new with room for 65 tokens
    refs = np.array([0, 1, 0, 0, 0, 1, 0], np.int32)
    cache = np.random.default_rng(0).integers(0, 256, (1, 7, 64, 2), dtype=np.uint8)
    got = fork_rule(cache, np.array([[5, 1, -1]], np.int32), [2], [70], refs, [0, 0, -1], [0, 129, 65])
    assert got[1].tolist() == [[5, 1, -1], [5, 0, 2], [3, 4, -1]]
    assert got[2].tolist() == [2, 3, 2] and got[3].tolist() == [70, 70, 0]
    assert got[4].tolist() == [1, 1, 1, 1, 1, 2, 0]
    assert np.array_equal(got[0][0, 0, :6], cache[0, 1, :6]) and np.array_equal(got[0][0, 0, 6:], cache[0, 0, 6:])
    assert fork_rule(cache, np.array([[5, 1, -1]], np.int32), [2], [70], refs, [0, -1], [0, 64 * 6]) is None
