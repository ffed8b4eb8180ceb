"""The 8-bit K/V tile cache without a GPU: refusals of the C ABI and of the
binding, which come before any CUDA call, and pins of the fp64 oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_24_b200 as V
from oracle import kv_oracle as O

P = ctypes.c_void_p
FAKE = 0x1000          # aligned, never dereferenced by a refused call


def cache(**over):
    f = dict(B=2, heads_kv=3, d=64, tile=64, n_slots=24, nb_cap=4)
    f.update({n: FAKE for n in ("k8", "v8", "table", "pos", "k_scale", "v_scale", "weight", "len", "next_pos",
                                "arrive", "dev_status")})
    f.update(over)
    return V._KvCache(*[f[n] for n, _ in V._KvCache._fields_])


def i64(*v):
    return (ctypes.c_int64 * 3)(*v)


def refused(rc, code, word):
    assert rc == code and word in V.veda_last_error(), (rc, V.veda_last_error())


BAD_CACHES = [
    (dict(B=0), V.VEDA_ERR_INVALID_ARG, "B="), (dict(B=70000), V.VEDA_ERR_INVALID_ARG, "B="),
    (dict(heads_kv=0), V.VEDA_ERR_INVALID_ARG, "heads_kv"), (dict(heads_kv=129), V.VEDA_ERR_INVALID_ARG, "heads_kv"),
    (dict(d=96), V.VEDA_ERR_UNSUPPORTED, "d="), (dict(tile=32), V.VEDA_ERR_UNSUPPORTED, "tile="),
    (dict(nb_cap=0), V.VEDA_ERR_INVALID_ARG, "nb_cap"), (dict(nb_cap=8193), V.VEDA_ERR_UNSUPPORTED, "nb_cap"),
    (dict(n_slots=0), V.VEDA_ERR_INVALID_ARG, "n_slots"), (dict(n_slots=1 << 26), V.VEDA_ERR_INVALID_ARG, "n_slots"),
    (dict(k8=None), V.VEDA_ERR_INVALID_ARG, "k8 is NULL"), (dict(v8=FAKE + 8), V.VEDA_ERR_INVALID_ARG, "v8 is not"),
    (dict(table=None), V.VEDA_ERR_INVALID_ARG, "table"), (dict(pos=FAKE + 4), V.VEDA_ERR_INVALID_ARG, "pos"),
    (dict(k_scale=None), V.VEDA_ERR_INVALID_ARG, "k_scale"), (dict(v_scale=None), V.VEDA_ERR_INVALID_ARG, "v_scale"),
    (dict(weight=FAKE + 4), V.VEDA_ERR_INVALID_ARG, "weight"), (dict(len=None), V.VEDA_ERR_INVALID_ARG, "len"),
    (dict(next_pos=None), V.VEDA_ERR_INVALID_ARG, "next_pos"), (dict(arrive=None), V.VEDA_ERR_INVALID_ARG, "arrive"),
]


@pytest.mark.parametrize("over,code,word", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(over, code, word):
    c = ctypes.byref(cache(**over))
    keep = (ctypes.c_int32 * 129)(*[4] * 129)
    L = V._lib
    refused(L.veda_kv_append(c, P(FAKE), None, P(FAKE), None, 1, None, None), code, word)
    refused(L.veda_kv_advance(c, 1, None, None), code, word)
    refused(L.veda_kv_attn(c, P(FAKE), None, 3, 1, None, 1, 1, 0, 0, 1.0, P(FAKE), None, None, None, 1.0, P(FAKE), None),
            code, word)
    assert L.veda_kv_attn_ws_bytes(c, 3, 1, 0) == 0
    refused(L.veda_kv_evict(c, keep, 1, 1, None, None), code, word)


def test_append_and_advance_refusals():
    c, L, E = ctypes.byref(cache()), V._lib, V.VEDA_ERR_INVALID_ARG
    refused(L.veda_kv_append(None, P(FAKE), None, P(FAKE), None, 1, None, None), E, "cache is NULL")
    refused(L.veda_kv_append(c, None, None, P(FAKE), None, 1, None, None), E, "k is NULL")
    refused(L.veda_kv_append(c, P(FAKE), None, P(FAKE + 2), None, 1, None, None), E, "v is not 16-byte")
    refused(L.veda_kv_append(c, P(FAKE), i64(64, 4, 64), P(FAKE), None, 1, None, None), E, "k: strides")
    refused(L.veda_kv_append(c, P(FAKE), None, P(FAKE), i64(64, 64, 1), 1, None, None), E, "v: strides")
    refused(L.veda_kv_append(c, P(FAKE), None, P(FAKE), None, -1, None, None), E, "negative")
    refused(L.veda_kv_append(c, P(FAKE), None, P(FAKE), None, 1 << 23, None, None), V.VEDA_ERR_UNSUPPORTED, "exceeds")
    refused(L.veda_kv_advance(c, -1, None, None), E, "negative")
    assert L.veda_kv_append(c, None, None, None, None, 0, None, None) == 0      # nothing to do
    assert L.veda_kv_advance(c, 0, None, None) == 0


def attn(c=None, q=FAKE, qs=None, heads=6, n=2, window=0, sinks=0, o=FAKE, os_=None, lse=None, weight=None, ws=FAKE):
    return V._lib.veda_kv_attn(ctypes.byref(cache() if c is None else c), P(q), qs, heads, n, None, 1, 1, window, sinks,
                               0.125, P(o), os_, P(lse), P(weight), 1.0, P(ws), None)


def test_attention_refusals():
    E = V.VEDA_ERR_INVALID_ARG
    refused(attn(heads=0), E, "heads=0")
    refused(attn(heads=4), E, "multiple of heads_kv")
    refused(attn(heads=4098), E, "heads=4098")
    refused(attn(n=-1), E, "n_q")
    refused(attn(n=1 << 23), V.VEDA_ERR_UNSUPPORTED, "n_q")
    refused(attn(n=1 << 22, heads=30), V.VEDA_ERR_UNSUPPORTED, "exceeds")
    refused(attn(window=-1), E, "window")
    refused(attn(sinks=-1), E, "sinks")
    refused(attn(q=None), E, "q is NULL")
    refused(attn(q=FAKE + 8), E, "q is not")
    refused(attn(qs=i64(0, 12, 64)), E, "q: strides")
    refused(attn(o=None), E, "o is NULL")
    refused(attn(os_=i64(768, 0, 64)), E, "overlap")
    refused(attn(os_=i64(0, 384, 64)), E, "overlap")
    refused(attn(lse=FAKE + 4), E, "lse")
    refused(attn(weight=FAKE + 8), E, "weight")
    refused(attn(ws=None), E, "ws is NULL")
    assert attn(n=0, q=None, o=None, ws=None) == 0
    L = V._lib
    assert L.veda_kv_attn_ws_bytes(ctypes.byref(cache()), 4, 2, 0) == 0
    less = L.veda_kv_attn_ws_bytes(ctypes.byref(cache()), 6, 2, 0)
    assert 0 < less < L.veda_kv_attn_ws_bytes(ctypes.byref(cache()), 6, 2, 1)


def test_evict_refusals():
    E, L = V.VEDA_ERR_INVALID_ARG, V._lib
    k3 = lambda *v: (ctypes.c_int32 * 3)(*v)

    def evict(c=None, keep=k3(4, 4, 4), sink=1, recent=1, out=None):
        return L.veda_kv_evict(ctypes.byref(cache() if c is None else c), keep, sink, recent,
                               None if out is None else ctypes.byref(out), None)

    refused(evict(c=cache(weight=None)), E, "weight is NULL")
    refused(evict(keep=None), E, "keep is NULL")
    refused(evict(sink=-1), E, "sink")
    refused(evict(recent=0), E, "recent")
    refused(evict(keep=k3(4, 1, 4)), E, "keep[1]")
    refused(evict(sink=0x7fffffff, recent=0x7fffffff), E, "keep[0]")
    apart = {n: 0x9000 + 0x100 * i for i, n in enumerate(("table", "pos", "k_scale", "v_scale", "weight", "len", "next_pos"))}
    here = {n: 0x5000 + 0x100 * i for i, n in enumerate(apart)}
    refused(evict(c=cache(**here), out=cache(**{**apart, "nb_cap": 5})), E, "another geometry")
    refused(evict(c=cache(**here), out=cache(**{**apart, "weight": None})), E, "out: weight")
    refused(evict(c=cache(**here), out=cache(**{**apart, "pos": here["pos"]})), E, "shares")
    refused(evict(c=cache(**here), out=cache(**{**apart, "pos": here["table"]})), E, "shares")


def test_status_refusals():
    refused(V._lib.veda_kv_check_status(None, None), V.VEDA_ERR_INVALID_ARG, "NULL")
    refused(V._lib.veda_kv_check_status(ctypes.byref(cache(dev_status=None)), None), V.VEDA_ERR_INVALID_ARG, "NULL")


def test_binding_checks_tensors():
    c = V.KVCache(2, 3, 64, 64, 4, "cpu")
    assert c.k8.shape == (24, 64, 64) and c.table.flatten().tolist() == list(range(24)) and c.len.sum() == 0
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    ok = bf(2, 5, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        V.veda_kv_append(c, ok, ok)
    for bad in (ok.float(), bf(2, 5, 3, 128), bf(1, 5, 3, 64), bf(2, 5, 3, 128)[..., ::2]):
        with pytest.raises(ValueError, match="k "if bad.dtype != torch.bfloat16 else "k"):
            V.veda_kv_append(c, bad, bad)
    with pytest.raises(ValueError, match="v must have shape"):
        V.veda_kv_append(c, ok, bf(2, 4, 3, 64))
    with pytest.raises(ValueError, match="n_new"):
        V.veda_kv_append(c, ok, ok, n_new=torch.zeros(2))
    with pytest.raises(ValueError, match="n_new"):
        V.veda_kv_advance(c, 5, n_new=torch.zeros(3, dtype=torch.int32))
    q = bf(2, 5, 6, 64)
    ws = torch.empty(V.veda_kv_attn_ws_bytes(c, 6, 5), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        V.veda_kv_attn(c, q, q.clone(), 0.125, ws)
    with pytest.raises(ValueError, match="bytes"):
        V.veda_kv_attn(c, q, q.clone(), 0.125, ws[:-1])
    with pytest.raises(ValueError, match="lse"):
        V.veda_kv_attn(c, q, q.clone(), 0.125, ws, lse=torch.zeros(2, 5, 6))
    with pytest.raises(ValueError, match="weight"):
        V.veda_kv_attn(c, q, q.clone(), 0.125, ws, weight=torch.zeros(2, 3, 5))
    with pytest.raises(ValueError, match="keep"):
        V.veda_kv_evict(c, [4, 4], 1, 1)
    with pytest.raises(ValueError, match="table"):
        V.KVCache(2, 3, 64, 64, 4, "cpu", table=torch.zeros((2, 3, 4)))
    with pytest.raises(ValueError, match="k8"):
        V.KVCache(2, 3, 64, 64, 4, "cpu", k8=torch.zeros((24, 64, 64), dtype=torch.uint8))
    with pytest.raises(ValueError, match="shape"):     # pools of one size
        V.KVCache(2, 3, 64, 64, 4, "cpu", k8=torch.zeros((24, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn),
                  v8=torch.zeros((25, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn))
    with pytest.raises(ValueError, match="needs a table"):
        V.KVCache(2, 3, 64, 64, 4, "cpu", k8=torch.zeros((9, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn),
                  v8=torch.zeros((9, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn))


def test_binding_refuses_numbers_past_32_bits():
    c = V.KVCache(1, 2, 64, 64, 4, "cpu")
    q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    ws = torch.empty(V.veda_kv_attn_ws_bytes(c, 2, 1), dtype=torch.uint8)
    for call in (lambda x: V.veda_kv_advance(c, x), lambda x: V.veda_kv_attn_ws_bytes(c, 2 * x, 1),
                 lambda x: V.veda_kv_attn_ws_bytes(c, 2, x), lambda x: V.veda_kv_attn(c, q, q.clone(), 1.0, ws, window=x),
                 lambda x: V.veda_kv_attn(c, q, q.clone(), 1.0, ws, sinks=x), lambda x: V.veda_kv_evict(c, [4, x], 1, 1),
                 lambda x: V.veda_kv_evict(c, [4, 4], x, 1), lambda x: V.veda_kv_evict(c, [4, 4], 1, x)):
        for x in (2 ** 31, 2 ** 32 + 4, -2 ** 31 - 1):
            with pytest.raises(ValueError, match="32 bits"):
                call(x)


def test_cache_tensors_cannot_be_replaced():
    c = V.KVCache(1, 2, 64, 64, 4, "cpu")
    held = c.len
    for name in ("len", "table", "k8", "weight", "nb_cap"):
        with pytest.raises(AttributeError, match="in place"):
            setattr(c, name, torch.zeros_like(c.len))
    c.len[0, 1] = 5
    assert c.len is held and held.tolist() == [[0, 5]]


def test_stream_layer_refusals():
    from block_sparse_attention_24_b200.stream import VedaStream
    make = lambda heads=4, **kw: VedaStream(1, heads, 2, 64, 64, 640, "cpu", **kw)
    assert make(keep=3, sink_tiles=1, recent_tiles=2).keep == [3, 3] and make(keep=[3, 4]).keep == [3, 4]
    with pytest.raises(ValueError, match="multiple"):
        make(heads=3)
    with pytest.raises(ValueError, match="window"):
        make(window=-1)
    with pytest.raises(ValueError, match="sinks"):
        make(sinks=-1)
    for bad in (dict(keep=[3]), dict(keep=[3, 1]), dict(keep=2, recent_tiles=2), dict(keep=2, recent_tiles=0),
                dict(keep=2, sink_tiles=-1)):
        with pytest.raises(ValueError, match="keep"):
            make(**bad)


def test_stream_layer_workspaces_are_few():
    from block_sparse_attention_24_b200.stream import VedaStream
    layer = VedaStream(1, 4, 2, 64, 64, 1280, "cpu")
    for n in range(1, 600):
        for weight in (False, True):
            assert layer.workspace(n, weight).numel() >= V.veda_kv_attn_ws_bytes(layer.cache, 4, n, weight)
    assert len(layer._ws) <= 30
    with pytest.raises(ValueError, match="limits"):
        layer.workspace(1 << 23, False)


def test_binding_defines_no_name_twice():
    import ast
    with open(V.__file__) as f:
        names = [n.name for n in ast.parse(f.read()).body if isinstance(n, (ast.FunctionDef, ast.ClassDef))]
    assert len(names) == len(set(names))


# ------------------------------------------------------------------ oracle

def test_oracle_codes_are_torchs():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(50000, generator=g) * torch.exp2(torch.randint(-12, 8, (50000,), generator=g).float())).clamp(-448, 448)
    np.testing.assert_array_equal(O.nearest_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    ties = (O.E4M3[1:] + O.E4M3[:-1]) / 2
    np.testing.assert_array_equal(O.nearest_e4m3(ties),
                                  torch.tensor(ties).float().to(torch.float8_e4m3fn).double().numpy())


def test_oracle_scale():
    assert O.scale_of(448.0) == 1.0 and O.scale_of(448.0000001) == 2.0 and O.scale_of(224.0) == 0.5
    assert O.scale_of(0.0) == 2.0 ** -40 and O.scale_of(448 * 2.0 ** 80) == 2.0 ** 80
    assert math.isnan(O.scale_of(449 * 2.0 ** 80)) and math.isnan(O.scale_of(math.inf)) and math.isnan(O.scale_of(math.nan))


def make_oracle(B=1, hkv=1, nb=4, d=64, tile=64):
    return O.Cache(tile, k8=np.zeros((B * hkv * nb, tile, d)), v8=np.zeros((B * hkv * nb, tile, d)),
                   table=np.arange(B * hkv * nb).reshape(B, hkv, nb), pos=np.zeros((B, hkv, nb)),
                   k_scale=np.zeros((B, hkv, nb)), v_scale=np.zeros((B, hkv, nb)), weight=np.zeros((B, hkv, nb)),
                   len=np.zeros((B, hkv)), next_pos=np.zeros(B))


def test_oracle_attention_equals_a_softmax_over_the_quantised_tokens():
    rng = np.random.default_rng(0)
    c = make_oracle()
    k, v = rng.standard_normal((1, 150, 1, 64)), rng.standard_normal((1, 150, 1, 64))
    c.append(k, v, [150])
    c.advance(np.array([150]))
    assert c.pos[0, 0, :3].tolist() == [0, 64, 128] and c.len[0, 0] == 150
    K, V_, at, _ = c.keys(0, 0, 150)
    assert np.abs(K - k[0, :, 0]).max() <= 2.0 ** -4 * np.abs(k).max() and at.tolist() == list(range(150))
    q = rng.standard_normal((1, 2, 2, 64))
    o, lse, w, *_ = c.attend(q, [2], 0.125, False, 0, 0, pending=False)
    s = q[0, 1, 1] @ K.T * 0.125
    p = np.exp(s - s.max())
    np.testing.assert_allclose(o[0, 1, 1], p @ V_ / p.sum(), rtol=1e-12)
    np.testing.assert_allclose(lse[0, 1, 1], np.log(np.exp(s).sum()), rtol=1e-12)
    np.testing.assert_allclose(w[0, 0].sum() if np.isfinite(w).all() else np.nansum(w), 4.0, rtol=1e-12)
    # window of 20 and 3 first tokens, from position 150
    o, *_ = c.attend(q, [2], 0.125, True, 20, 3, pending=False)
    see = [0, 1, 2] + list(range(131, 150))
    p = np.exp(q[0, 0, 0] @ K[see].T * 0.125)
    np.testing.assert_allclose(o[0, 0, 0], p @ V_[see] / p.sum(), rtol=1e-12)


def test_oracle_evict_keeps_the_heaviest():
    c = make_oracle(nb=6)
    c.len[:] = 5 * 64 + 10
    c.weight[0, 0] = [0, 3, 1, 3, 2, 9]
    c.pos[0, 0] = np.arange(6) * 64
    c.evict([4], 1, 1)
    assert c.table[0, 0].tolist() == [0, 1, 3, 5, 2, 4] and c.len[0, 0] == 3 * 64 + 10
    assert c.pos[0, 0, :4].tolist() == [0, 64, 192, 320]
