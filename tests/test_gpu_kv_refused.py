"""Steps that the 8-bit K/V tile cache cannot hold: refused whole, sequence by
sequence, and without a trace."""
import numpy as np
import pytest
import torch

import block_sparse_attention_24_b200 as V
from oracle.kv_oracle import Cache
from tests.test_gpu_kv_cache import (DEV, assert_same_state, bad_status, bf16, check_attention, host, oracle_of,
                                     random_cache, workspace)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,heads", [(100, 4), (3, 4)])
def test_a_sequence_is_refused_as_a_whole(n, heads):
    """One head of two is too full (eviction keeps more of its tiles). Were the
    other served, or the position moved on, the heads would disagree about
    where the next tokens stand."""
    hkv, d, tile = 2, 64, 64
    c = random_cache(1, 2, hkv, d, tile, 4, [254, 40])
    V.veda_kv_evict(c, [4, 2], 1, 1)
    assert c.len.tolist() == [[254, 126], [40, 40]]
    want, next_pos = oracle_of(c), c.next_pos.tolist()
    k, q = bf16(2, 2, n, hkv, d), bf16(3, 2, n, heads, d)
    o, lse = torch.full_like(q, 5.0), torch.full((2, heads, n), 5.0, device=DEV)
    V.veda_kv_append(c, k, k)
    bad_status(c)
    want.append(host(k), host(k), [n, n])
    assert_same_state(c, want)
    w = c.weight.clone()
    V.veda_kv_attn(c, q, o, 0.125, workspace(c, heads, n, True), lse=lse, weight=c.weight)
    bad_status(c)
    assert (o[0] == 5).all() and (lse[0] == 5).all() and torch.equal(c.weight[0], w[0])
    assert not (o[1] == 5).all(-1).any() and not (lse[1] == 5).any()
    V.veda_kv_advance(c, n)
    bad_status(c)
    assert c.len.tolist() == [[254, 126], [40 + n, 40 + n]]
    assert c.next_pos.tolist() == [next_pos[0], next_pos[1] + n]
    # with room made, the next tokens stand where the queries take them to be
    V.veda_kv_evict(c, [2, 2], 1, 1)
    V.veda_kv_append(c, k, k)
    for b in range(2):
        for h in range(hkv):
            held = int(c.len[b, h])
            assert int(c.pos[b, h, held // tile]) + held % tile == int(c.next_pos[b])
    check_attention(c, q, window=n // 2 + 1)
    check_attention(c, q, window=n + 5, sinks=3, causal=False)


def test_counts_of_all_heads_decide():
    """A head of many (more than a warp has lanes), first or last, without
    pending tokens as well."""
    hkv, d, tile = 100, 64, 64
    for head in (0, 31, 32, 99):
        c = random_cache(4, 1, hkv, d, tile, 2, [64])
        c.len[0, head] = 128
        k, q = bf16(5, 1, 30, hkv, d), bf16(6, 1, 30, hkv, d)
        before = {f: getattr(c, f).clone() for f in Cache.FIELDS}
        V.veda_kv_append(c, k, k)
        bad_status(c)
        V.veda_kv_advance(c, 30)
        bad_status(c)
        for f, t in before.items():
            assert torch.equal(t.view(torch.uint8), getattr(c, f).view(torch.uint8)), f
        for rows in (30, 1):
            o = torch.full_like(q, 5.0)[:, :rows].contiguous()
            V.veda_kv_attn(c, q[:, :rows].contiguous(), o, 0.125, workspace(c, hkv, rows, False))
            bad_status(c)
            assert (o == 5).all()
            V.veda_kv_attn(c, q[:, :rows].contiguous(), o, 0.125, workspace(c, hkv, rows, False), pending=False)
            V.veda_kv_check_status(c)
            assert not (o == 5).all(-1).any()                # no row is left as it was (a value may be 5)
        c.len[0, head] = -1
        o = torch.full_like(q, 5.0)
        V.veda_kv_attn(c, q, o, 0.125, workspace(c, hkv, 30, False), pending=False)
        bad_status(c)
        assert (o == 5).all()


@pytest.mark.parametrize("n", [1, 20])
def test_a_tile_without_a_slot_still_has_its_position(n):
    """Absent, but at its place in the stream: windows find the tiles around it
    by the positions, which ascend."""
    hkv, d, tile = 2, 64, 64
    c = V.KVCache(1, hkv, d, tile, 6, DEV)
    c.table[0, 0, 3], c.table[0, 1, 2] = -1, c.n_slots
    k, v, q = bf16(20, 1, 250, hkv, d), bf16(21, 1, 250, hkv, d), bf16(22, 1, n, 4, d)
    V.veda_kv_append(c, k, v)
    bad_status(c)
    V.veda_kv_advance(c, 250)
    assert c.pos[0, :, :4].tolist() == [[0, 64, 128, 192]] * 2
    for window, sinks in ((64, 0), (130, 0), (100, 64)):
        want = oracle_of(c).attend(host(q), [n], 0.125, True, window, sinks, pending=False)
        o, lse = torch.empty_like(q), torch.empty((1, 4, n), device=DEV)
        V.veda_kv_attn(c, q, o, 0.125, workspace(c, 4, n, False), window=window, sinks=sinks, pending=False, lse=lse)
        bad_status(c)
        # as in test_table_entries_outside_the_pool_are_absent_tiles: a value and its bf16 rounding, with room
        np.testing.assert_allclose(host(o), want[0], rtol=2.0 ** -7, atol=2.0 ** -6)
        np.testing.assert_allclose(host(lse), want[1], rtol=0, atol=2.0 ** -10)


@pytest.mark.parametrize("keep", [None, 2])
def test_a_step_past_the_capacity_returns_no_old_memory(keep):
    from block_sparse_attention_24_b200.stream import VedaStream
    n = 70
    layer = VedaStream(2, 4, 2, 64, 64, 128, DEV, keep=keep, sink_tiles=0)
    q, k = bf16(10, 2, n, 4, 64), bf16(11, 2, n, 2, 64)
    news = torch.tensor([n, 20], dtype=torch.int32, device=DEV)
    assert layer.step(q, k, k, n_new=news).shape == q.shape
    layer.check_status()
    for _ in range(2):
        junk = [torch.full_like(q, 7.0) for _ in range(4)]
        del junk
        o = layer.step(q, k, k, n_new=news)
        with pytest.raises(V.VedaError) as e:
            layer.check_status()
        assert e.value.code == V.VEDA_ERR_BAD_INDEX
        assert (o[0] == 0).all()                        # refused
        assert (o[1, 20:] == 0).all() and not (o[1, :20] == 0).all(-1).any()
    assert layer.cache.next_pos.tolist() == [70, 60]
    # what is given is left as it was
    o = torch.full_like(q, 7.0)
    assert layer.step(q, k, k, n_new=news, out=o) is o and (o[0] == 7).all() and (o[1, 20:] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,heads", [(1, 2), (3, 6), (8, 4), (20, 2), (70, 12), (600, 4)])
def test_rows_without_a_query_are_filled(n, heads, d):
    """Padded rows and those of refused sequences, by both kernels and with
    split heads; all others as without."""
    hkv, tile, nb = 2, 64, 20
    c = random_cache(30, 5, hkv, d, tile, nb, [600 + n] * 5)
    c.len.sub_(n)
    c.next_pos.sub_(n)
    c.len[3, 1] = nb * tile                             # full
    news = torch.tensor([n, n // 2, 0, n, n + 1], dtype=torch.int32, device=DEV)
    q, got = bf16(31, 5, n, heads, d), []
    for fill in (False, True):
        room = torch.full((5, heads, n + 2, d), 9.0, dtype=torch.bfloat16, device=DEV)
        o, lse, w = room.transpose(1, 2)[:, 1:n + 1], torch.full((5, heads, n), 9.0, device=DEV), c.weight.clone()
        V.veda_kv_attn(c, q, o, 0.125, workspace(c, heads, n, True), n_new=news, lse=lse, weight=w, fill=fill)
        bad_status(c)
        assert (room[:, :, 0] == 9).all() and (room[:, :, n + 1:] == 9).all()
        got.append((o, lse, w))
    (o, lse, w), (fo, flse, fw) = got
    assert torch.equal(w, fw)
    for b, m in enumerate((n, n // 2, 0, 0, 0)):
        assert torch.equal(o[b, :m], fo[b, :m]) and torch.equal(lse[b, :, :m], flse[b, :, :m])
        assert (o[b, m:] == 9).all() and (lse[b, :, m:] == 9).all()
        assert (fo[b, m:] == 0).all() and (flse[b, :, m:] == -float("inf")).all()
    V.veda_kv_attn(c, q, q, 0.125, workspace(c, heads, n, False), n_new=news, fill=True)     # over the query
    assert torch.equal(q, fo)


def test_evicted_tiles_of_a_shared_prefix():
    """Two sequences read one prefix, one of them drops some of it and goes on:
    with slots of its own in the entries that it gave up, the other's tokens
    stay as they are. (The slots: those that the prefix stands in for.)"""
    hkv, d, tile = 1, 64, 64
    c = random_cache(40, 2, hkv, d, tile, 6, [256, 256])
    own = c.table[1, 0, :3].clone()
    c.table[1, 0, :3] = c.table[0, 0, :3]
    c.len[0] = 100                                      # (fewer tiles than are kept: nothing leaves)
    c.next_pos[0] = 100
    c.weight[1, 0, :4] = torch.tensor([9.0, 1.0, 8.0, 1.0], device=DEV)
    V.veda_kv_evict(c, [3], 1, 1)
    shared = c.table[0, 0, :2].tolist()
    assert c.len.tolist() == [[100], [192]] and int(c.table[1, 0, 3]) == shared[1]
    c.table[1, 0, 3] = own[1]
    k, v, q = bf16(41, 2, 70, hkv, d), bf16(42, 2, 70, hkv, d), bf16(43, 2, 70, 2, d)
    nn = torch.tensor([0, 70], dtype=torch.int32, device=DEV)
    before = [t.view(torch.uint8)[shared].clone() for t in (c.k8, c.v8)]
    want = oracle_of(c)
    V.veda_kv_append(c, k, v, n_new=nn)
    want.append(host(k), host(v), [0, 70])
    assert_same_state(c, want)
    for x, t in zip(before, (c.k8, c.v8)):
        assert torch.equal(x, t.view(torch.uint8)[shared])
    check_attention(c, q, news=[0, 70])
    V.veda_kv_advance(c, 70, n_new=nn)
    check_attention(c, q, pending=False)
