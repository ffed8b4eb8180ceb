"""Steps of the 8-bit K/V tile cache without a GPU: what the oracle does with
pending tokens and refused steps, and what is refused before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_attention_24_b200 as V
from tests.test_kv_cpu import FAKE, P, cache, make_oracle, refused


@pytest.mark.parametrize("bad", [2.0 ** 20, np.nan, np.inf])
def test_oracle_replaced_tokens_leave_nothing_behind(bad):
    rng = np.random.default_rng(1)
    first, last = (rng.standard_normal((1, n, 1, 64)) for n in (70, 9))
    wrong = rng.standard_normal((1, 30, 1, 64))
    wrong[0, 3, 0, 5] = bad
    a, e, dropped = make_oracle(), make_oracle(), make_oracle()
    for c in (a, e, dropped):
        c.append(first, -first, [70])
        c.advance(np.array([70]))
    held = [(c.k8[1, :6].copy(), c.k_scale[0, 0, 1]) for c in (e,)][0]
    for _ in range(2):
        for c in (a, dropped):
            c.append(wrong, wrong, [30])
            assert not c.k_scale[0, 0, 1] == held[1]
    dropped.append(wrong, wrong, [0])
    np.testing.assert_array_equal(dropped.k8[1, :6], held[0])
    assert dropped.k_scale[0, 0, 1] == held[1] and (dropped.k8[1, 6:] == 0).all()
    for c in (a, e, dropped):
        c.append(last, last, [9])
    for c in (a, dropped):
        for f in ("k8", "v8", "k_scale", "v_scale"):
            np.testing.assert_array_equal(getattr(c, f)[:2] if f[1:] == "8" else getattr(c, f)[0, 0, :2],
                                          getattr(e, f)[:2] if f[1:] == "8" else getattr(e, f)[0, 0, :2])


def test_oracle_taken_tokens_stay():
    """Once they are committed, what they did to the scale is not undone."""
    c = make_oracle()
    x = np.ones((1, 5, 1, 64))
    for size in (1.0, 2.0 ** 20, 1.0):
        c.append(x * size, x * size, [5])
        c.advance(np.array([5]))
    assert c.k_scale[0, 0, 0] == 2.0 ** 12 and c.len[0, 0] == 15
    assert (c.k8[0, :5] == 0).all() and (c.k8[0, 5:10] == 256).all() and (c.k8[0, 10:15] == 0).all()


def test_oracle_refuses_a_sequence_as_a_whole():
    c = make_oracle(B=2, hkv=2, nb=2)
    x = np.ones((2, 100, 2, 64))
    c.append(x, x, [100, 100])
    c.advance(np.array([100, 100]))
    c.len[0, 1] = 36                                    # a tile of this head has been evicted
    before = c.k8.copy()
    c.append(x, x, [50, 28])                            # 150 of 128; exactly full
    c.advance(np.array([50, 28]))
    assert c.len.tolist() == [[100, 36], [128, 128]] and c.next_pos.tolist() == [100, 128]
    np.testing.assert_array_equal(c.k8[:4], before[:4])


def test_append_pending_refusals():
    c, L, E = ctypes.byref(cache()), V._lib, V.VEDA_ERR_INVALID_ARG
    tail = lambda *p: ctypes.byref(V._KvTail(*p))
    ok = tail(FAKE, FAKE, FAKE)
    call = lambda t, k=FAKE, n=1, c=c: L.veda_kv_append_pending(c, t, P(k), None, P(FAKE), None, n, None, None)
    refused(call(tail(None, FAKE, FAKE)), E, "tail codes is NULL")
    refused(call(tail(FAKE, FAKE + 8, FAKE)), E, "tail key is not")
    refused(call(tail(FAKE, FAKE, None), n=0), E, "tail scale is NULL")
    refused(call(ok, k=None), E, "k is NULL")
    refused(call(ok, n=-1), E, "negative")
    refused(call(ok, c=None), E, "cache is NULL")
    assert call(None, n=0) == 0                         # nothing kept, nothing to do


def test_attention_that_fills_refuses_what_attention_does():
    def call(c=None, heads=6, n=2, window=0, o=FAKE):
        return V._lib.veda_kv_attn_fill(ctypes.byref(cache() if c is None else c), P(FAKE), None, heads, n, None, 1, 1,
                                        window, 0, 0.125, P(o), None, None, None, 1.0, P(FAKE), None)
    E = V.VEDA_ERR_INVALID_ARG
    refused(call(c=cache(pos=None)), E, "pos")
    refused(call(heads=4), E, "multiple of heads_kv")
    refused(call(window=-1), E, "window")
    refused(call(o=FAKE + 8), E, "o is not")
    assert call(n=0) == 0


def test_the_librarys_own_tensors_cannot_be_replaced():
    c = V.KVCache(1, 2, 64, 64, 4, "cpu")
    assert c.tail_codes.shape == (1, 2, 2, 64, 64) and not c.tail_key.any()
    for name in ("tail_codes", "tail_key", "tail_scale"):
        with pytest.raises(AttributeError, match="in place"):
            setattr(c, name, torch.zeros(1))


def test_stream_layer_refuses_tokens_that_do_not_match(monkeypatch):
    """Before the first kernel: k and v with more or fewer tokens than q (rows
    that nothing has written would be taken in, or surplus ones dropped)."""
    from block_sparse_attention_24_b200 import stream
    calls = []
    for name in ("veda_kv_append", "veda_kv_attn", "veda_kv_advance", "veda_kv_evict"):
        monkeypatch.setattr(stream, name, lambda *a, _n=name, **kw: calls.append(_n))
    layer = stream.VedaStream(2, 4, 2, 64, 64, 640, "cpu")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    q, k = bf(2, 5, 4, 64), bf(2, 5, 2, 64)
    for a, b, c in ((q, bf(2, 4, 2, 64), k), (q, k, bf(2, 6, 2, 64)), (q, k[:, :0], k[:, :0]), (q[:, :0], k, k),
                    (bf(2, 1, 4, 64), k, k)):
        with pytest.raises(ValueError, match="as many tokens"):
            layer.step(a, b, c)
    for a, b, c in ((bf(2, 5, 2, 64), k, k), (q, bf(2, 5, 4, 64), k), (q, k, bf(1, 5, 2, 64)), (q, k, bf(2, 5, 2, 128)),
                    (q[0], k, k), (q, k[0], k), (q, k, None)):
        with pytest.raises(ValueError, match="must be a"):
            layer.step(a, b, c)
    assert calls == []
    layer.step(q, k, k)
    layer.step(q[:, :0], k[:, :0], k[:, :0])
    assert calls == ["veda_kv_append", "veda_kv_attn", "veda_kv_advance"]


def test_stream_layer_refuses_a_step_past_the_capacity():
    from block_sparse_attention_24_b200.stream import VedaStream
    layer = VedaStream(1, 2, 2, 64, 64, 100, "cpu")         # two tiles
    step = lambda n, **kw: layer.step(*[torch.zeros((1, n, 2, 64), dtype=torch.bfloat16)] * 3, **kw)
    with pytest.raises(ValueError, match="129 tokens does not fit a cache of 128"):
        step(129)
    for call in (lambda: step(128), lambda: step(129, n_new=torch.tensor([100], dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):       # the padding does not have to fit
            call()


def test_a_cache_names_all_its_memory():
    """Every pointer that the kernels get is of one of tensors()."""
    c = V.KVCache(2, 3, 64, 64, 4, "cpu")
    spans = [(t.untyped_storage().data_ptr(), t.untyped_storage().data_ptr() + t.untyped_storage().nbytes())
             for t in c.tensors()]
    for struct in (c._c, c._tail):
        for name, kind in struct._fields_:
            if kind is ctypes.c_void_p:
                assert any(a <= getattr(struct, name) < b for a, b in spans), name
