"""Argument checks of the shared-prefix and selected-page calls: refused on the host, nothing launched."""
import ctypes
import types

import numpy as np
import pytest

from longctx_util import select_rule

mla = pytest.importorskip("mla_latent_kv_gb300")
P = ctypes.c_void_p(0x1000)      # never dereferenced: every call here is refused first
ODD = ctypes.c_void_p(0x1008)    # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    from mla_latent_kv_gb300 import build
    build.build()
    return mla.lib()


def _call(f, defaults, **kw):
    args = dict(defaults)
    assert set(kw) <= set(args)
    args.update(kw)
    return f(*args.values())


def test_page_keys_refusals(lib):
    d = dict(cache=P, kv=0, nb=8, table=P, max_blocks=4, start=None, seq=P, max_new=100, B=2, keys=P, st=None, s=None)
    call = lambda **kw: _call(lib.mla_page_keys, d, **kw)  # noqa: E731
    assert call(kv=3) == mla.ERR_INVALID_ARG
    assert call(B=-1) == mla.ERR_INVALID_ARG
    assert call(max_new=-1) == mla.ERR_INVALID_ARG
    assert call(max_new=4 * 64 + 1) == mla.ERR_INVALID_ARG
    assert call(nb=-1) == mla.ERR_INVALID_ARG
    assert call(nb=1 << 40) == mla.ERR_UNSUPPORTED
    for name in ("cache", "table", "seq", "keys"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG
    assert b"mla_page_keys" in lib.mla_last_error_detail()
    assert call(cache=ODD) == mla.ERR_UNSUPPORTED and call(keys=ODD) == mla.ERR_UNSUPPORTED
    assert call(B=0) == mla.OK and lib.mla_last_error_detail() == b""
    assert call(max_new=0) == mla.OK


def test_page_scores_refusals(lib):
    d = dict(q=P, keys=P, nb=8, table=P, max_blocks=4, seq=P, max_len=256, B=2, Sq=1, H=16, scale=0.07, scores=P,
             st=None, s=None)
    call = lambda **kw: _call(lib.mla_page_scores, d, **kw)  # noqa: E731
    assert call(H=0) == mla.ERR_UNSUPPORTED and call(H=129) == mla.ERR_UNSUPPORTED
    assert call(B=-1) == mla.ERR_INVALID_ARG and call(Sq=0) == mla.ERR_INVALID_ARG
    assert call(max_len=257) == mla.ERR_INVALID_ARG and call(max_len=-1) == mla.ERR_INVALID_ARG
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == mla.ERR_INVALID_ARG
    for name in ("q", "keys", "table", "seq", "scores"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG
    assert call(q=ODD) == mla.ERR_UNSUPPORTED and call(keys=ODD) == mla.ERR_UNSUPPORTED
    assert call(B=1 << 20, Sq=1 << 8) == mla.ERR_UNSUPPORTED
    assert call(B=0) == mla.OK and call(max_len=0) == mla.OK


def test_select_pages_refusals(lib):
    d = dict(scores=P, stride=100, n=100, seq=P, B=2, Sq=1, K=8, sink=1, local=1, pages=P, st=None, s=None)
    call = lambda **kw: _call(lib.mla_select_pages, d, **kw)  # noqa: E731
    assert call(K=0) == mla.ERR_INVALID_ARG and call(B=-1) == mla.ERR_INVALID_ARG and call(Sq=0) == mla.ERR_INVALID_ARG
    assert call(sink=-1) == mla.ERR_INVALID_ARG and call(local=-1) == mla.ERR_INVALID_ARG
    assert call(sink=4, local=5) == mla.ERR_INVALID_ARG
    assert call(sink=2147483647, local=2147483647) == mla.ERR_INVALID_ARG
    assert call(stride=99) == mla.ERR_INVALID_ARG and call(n=-1) == mla.ERR_INVALID_ARG
    assert call(n=32769, stride=32769) == mla.ERR_UNSUPPORTED
    for name in ("scores", "seq", "pages"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG
    assert call(B=0) == mla.OK


def test_decode_sparse_refusals(lib):
    d = dict(q=P, cache=P, kv=0, nb=8, table=P, max_blocks=4, seq=P, pages=P, K=4, B=2, Sq=1, H=16, scale=0.07, S=1,
             ws=P, ws_bytes=1 << 30, o=P, o_dtype=0, lse=P, st=None, s=None)
    call = lambda **kw: _call(lib.mla_decode_sparse, d, **kw)  # noqa: E731
    assert call(kv=9) == mla.ERR_INVALID_ARG and call(o_dtype=5) == mla.ERR_INVALID_ARG
    assert call(H=0) == mla.ERR_UNSUPPORTED and call(H=129) == mla.ERR_UNSUPPORTED
    assert call(B=-2) == mla.ERR_INVALID_ARG and call(Sq=0) == mla.ERR_INVALID_ARG
    assert call(K=0) == mla.ERR_INVALID_ARG and call(K=1 << 26) == mla.ERR_INVALID_ARG
    assert call(S=-3) == mla.ERR_INVALID_ARG and call(scale=float("nan")) == mla.ERR_INVALID_ARG
    assert call(max_blocks=1 << 26) == mla.ERR_UNSUPPORTED and call(nb=-1) == mla.ERR_INVALID_ARG
    for name in ("q", "cache", "table", "seq", "pages", "o"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG
    for name in ("q", "cache", "o"):
        assert call(**{name: ODD}) == mla.ERR_UNSUPPORTED
    assert call(ws=None) == mla.ERR_WORKSPACE_TOO_SMALL and call(ws_bytes=8) == mla.ERR_WORKSPACE_TOO_SMALL
    assert b"mla_decode_sparse" in lib.mla_last_error_detail()
    assert call(ws=ctypes.c_void_p(0x1010)) == mla.ERR_UNSUPPORTED
    assert call(B=0) == mla.OK


def test_decode_shared_prefix_refusals(lib):
    d = dict(q=P, cache=P, kv=0, nb=8, table=P, max_blocks=4, seq=P, max_len=256, prefix=128, B=2, Sq=1, H=16,
             scale=0.07, S=1, ws=P, ws_bytes=0, o=P, o_dtype=0, lse=P, st=None, s=None)
    call = lambda **kw: _call(lib.mla_decode_shared_prefix, d, **kw)  # noqa: E731
    assert call(prefix=100) == mla.ERR_INVALID_ARG and call(prefix=-64) == mla.ERR_INVALID_ARG
    assert call(prefix=5 * 64) == mla.ERR_INVALID_ARG
    assert call(max_len=257) == mla.ERR_INVALID_ARG
    assert call(kv=9) == mla.ERR_INVALID_ARG and call(o_dtype=5) == mla.ERR_INVALID_ARG
    assert call(H=0) == mla.ERR_UNSUPPORTED and call(H=129) == mla.ERR_UNSUPPORTED
    assert call(B=-2) == mla.ERR_INVALID_ARG and call(Sq=0) == mla.ERR_INVALID_ARG
    assert call(S=-3) == mla.ERR_INVALID_ARG and call(scale=-0.1) == mla.ERR_INVALID_ARG
    for name in ("q", "cache", "table", "seq", "o"):
        assert call(**{name: None}) == mla.ERR_INVALID_ARG
    for name in ("q", "cache", "o"):
        assert call(**{name: ODD}) == mla.ERR_UNSUPPORTED
    assert call(B=0) == mla.OK
    assert lib.mla_decode_shared_prefix_workspace_bytes(0, 2, 1, 16, 100, 1, 256) == 0
    assert lib.mla_decode_shared_prefix_workspace_bytes(7, 2, 1, 16, 64, 1, 256) == 0


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 1, 16, 576, dtype=torch.bfloat16)
    table, seq = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(8, 64 * 1152, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mla.decode_sparse(q, cache, table, seq.long(), torch.zeros(2, 1, 4, dtype=torch.int32), 0.07)
    with pytest.raises(ValueError):
        mla.decode_sparse(q, cache, table, seq, torch.zeros(2, 4, dtype=torch.int32), 0.07)
    with pytest.raises(ValueError):
        mla.decode_shared_prefix(q.float(), cache, table, seq, 100, 64, 0.07)
    with pytest.raises(ValueError):
        mla.decode_shared_prefix(q, cache, table, seq, 100, 64, 0.07, num_blocks=9)
    with pytest.raises(ValueError):
        mla.page_keys(cache, table.t(), seq, 100)
    with pytest.raises(ValueError):
        mla.page_scores(q, torch.zeros(8, 512, dtype=torch.bfloat16), table, seq, 100, 0.07)
    with pytest.raises(ValueError):
        mla.select_pages(torch.zeros(2, 1, 8).double(), seq, 4)
    with pytest.raises(ValueError):
        mla.select_pages(torch.zeros(2, 1, 8), seq, 4)  # not on the device


def test_binding_refuses_a_status_word_of_another_type():
    """The kernels OR bits into four bytes: one byte, another type or nothing at all is refused."""
    torch = pytest.importorskip("torch")
    i32, bf = torch.int32, torch.bfloat16
    q, cache = torch.zeros(2, 1, 16, 576, dtype=bf), torch.zeros(8, 64 * 1152, dtype=torch.uint8)
    table, seq = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32)
    keys, scores, pages = torch.zeros(8, 576, dtype=bf), torch.zeros(2, 1, 4), torch.zeros(2, 1, 2, dtype=i32)
    bufs = dict(o_latent=torch.zeros(2, 1, 16, 512), lse=torch.zeros(2, 1, 16), workspace=torch.zeros(4096, dtype=torch.uint8))
    for st in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64), torch.zeros(1), torch.zeros(0, dtype=i32)):
        for call in (lambda: mla.decode_shared_prefix(q, cache, table, seq, 100, 64, 0.07, dev_status=st, **bufs),
                     lambda: mla.page_keys(cache, table, seq, 100, page_keys=keys, dev_status=st),
                     lambda: mla.page_scores(q, keys, table, seq, 256, 0.07, scores=scores, dev_status=st),
                     lambda: mla.select_pages(scores, seq, 2, pages=pages, dev_status=st),
                     lambda: mla.decode_sparse(q, cache, table, seq, pages, 0.07, dev_status=st, **bufs)):
            with pytest.raises(ValueError, match="dev_status"):
                call()


class _FakeLib:
    """Stands for the native library: sizes are 4096 bytes, every call succeeds and launches nothing."""

    def __getattr__(self, name):
        if name == "mla_kv_row_bytes":
            return lambda kv: {0: 1152, 1: 584}[kv]
        if name == "mla_resolve_num_splits":
            return lambda *a: 2
        return lambda *a: 4096 if "workspace_bytes" in name else 0


@pytest.mark.parametrize("call", ["absorb_q", "decode", "decode_noalloc", "decode_varlen", "out_proj", "prefill",
                                  "decode_shared_prefix", "page_keys", "page_scores", "select_pages", "decode_sparse"])
def test_buffers_are_made_on_the_stream_that_uses_them(call, monkeypatch):
    """A call with stream= makes its outputs and workspace on that stream: from its pool, so that the memory
    is not given to other work while the call's kernels run, and filled there, so that they follow the fill."""
    torch = pytest.importorskip("torch")
    here, made, used, launched = [], [], [], []

    class OnStream:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            here.append(self.stream.name)

        def __exit__(self, *exc):
            here.pop()

    def recorded(make):
        def f(*a, **kw):
            made.append(here[-1] if here else "current")
            return make(*a, **kw)
        return f

    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)  # noqa: E731
    i32 = torch.int32
    q, cache, table, lens, starts = z(2, 1, 16, 576), z(8, 64 * 576), z(2, 4, dtype=i32), z(2, dtype=i32), z(3, dtype=i32)
    w_uk_t, w_uv = z(16, 128, 512), z(16, 512, 128)
    args = {
        "absorb_q": (z(2, 16, 128), z(2, 16, 64), w_uk_t),
        "decode": (q, cache, table, lens, 200, 0.07),
        "decode_noalloc": (q, cache, table, lens, 200, 0.07),
        "decode_varlen": (q[:, 0], cache, table, lens, starts, 200, 0.07),
        "out_proj": (z(2, 16, 512), w_uv),
        "prefill": (z(2, 16, 192), z(2, 512), z(2, 64), cache, table, lens, starts, w_uk_t, w_uv, 0.07),
        "decode_shared_prefix": (q, cache, table, lens, 200, 64, 0.07),
        "page_keys": (cache, table, lens, 200),
        "page_scores": (q, z(8, 576), table, lens, 200, 0.07),
        "select_pages": (z(2, 1, 4, dtype=torch.float32), lens, 2),
        "decode_sparse": (q, cache, table, lens, z(2, 1, 2, dtype=i32), 0.07),
    }[call]
    monkeypatch.setattr(mla, "lib", _FakeLib)
    monkeypatch.setattr(mla, "_stream", lambda *a: None)
    monkeypatch.setattr(mla, "_raw_stream", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "stream", OnStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s: types.SimpleNamespace(device=0, name=s))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: used.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    monkeypatch.setattr(torch, "zeros", recorded(torch.zeros))
    for given, where in (({}, "current"), ({"stream": types.SimpleNamespace(cuda_stream="side")}, "side")):
        made.clear()
        out = getattr(mla, call)(*args, **given)
        assert made and set(made) == {where}, (given, made)
        outs = out if isinstance(out, tuple) else (out,)
        assert used == [(t.data_ptr(), "current") for t in outs if given]  # kept while the caller's stream reads them
    # a call that is given every buffer makes none, and goes to the stream as it is
    made.clear()
    used.clear()
    monkeypatch.setattr(torch.cuda, "stream", None)
    monkeypatch.setattr(mla, "_stream", launched.append)
    monkeypatch.setattr(mla, "_raw_stream", lambda s, *t: launched.append(s))
    ws = z(4096, dtype=torch.uint8)
    names = {"absorb_q": ("out",), "out_proj": ("out",), "decode_noalloc": ("o_latent", "lse"), "prefill": ("o", "lse"),
             "page_keys": ("page_keys",), "page_scores": ("scores",), "select_pages": ("pages",)}
    given = dict(zip(names.get(call, ("o_latent", "lse")), outs), stream="side")
    if call in ("decode", "decode_varlen", "decode_shared_prefix", "decode_sparse", "prefill"):
        given["workspace"] = ws
    if call == "prefill":
        given.update(ctx_lens_host=lens, query_start_loc_host=starts)
    made.clear()
    getattr(mla, call)(*args, **given)
    assert made == [] and used == [] and launched == ["side"]


def test_the_plain_rule_of_the_choice():
    """The tests' own rule on cases worked by hand."""
    nan = float("nan")
    s = np.array([0.0, 5.0, 1.0, 5.0, nan, 2.0, 0.0])
    assert select_rule(s, 7 * 64, 7, 0, 0) == list(range(7))
    assert select_rule(s, 6 * 64 + 1, 3, 1, 1) == [0, 1, 6]
    assert select_rule(s, 6 * 64 + 1, 4, 1, 1) == [0, 1, 3, 6]
    assert select_rule(s, 6 * 64 + 1, 2, 0, 0) == [1, 3]
    assert select_rule(s, 5 * 64, 4, 0, 0) == [0, 1, 2, 3]
    assert select_rule(s, 0, 4, 1, 1) == []
