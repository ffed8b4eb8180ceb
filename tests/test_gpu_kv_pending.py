"""Pending tokens of the 8-bit K/V tile cache: tokens that are replaced before
they are taken in leave nothing behind, in the codes and scales of the tail
tile that they shared with committed tokens least of all."""
import numpy as np
import pytest
import torch

import block_sparse_attention_24_b200 as V
from tests.test_gpu_kv_cache import DEV, assert_same_state, bf16, check_attention, oracle_of, random_cache, workspace

pytestmark = pytest.mark.gpu


def tokens(seed, B, n, hkv, d, kind=None):
    """K and V of a chunk; `kind`: what is wrong with a discarded one."""
    k, v = bf16(seed, B, n, hkv, d), bf16(seed + 1, B, n, hkv, d)
    if kind == "huge":
        k, v = k * 2.0 ** 18, v * 2.0 ** 18
    elif kind is not None:
        k[:, n // 2, :, 7] = kind
        v[:, n - 1, :, 0] = -kind
    return k, v


def held_state(c, b, h, total):
    """What counts of a head that holds `total` tokens, pending ones among them."""
    nb = -(-total // c.tile)
    slot = c.table[b, h, :nb].long()
    rows = lambda t: t.view(torch.uint8)[slot].reshape(nb * c.tile, c.d)
    return [rows(c.k8), rows(c.v8), slot, *(getattr(c, f)[b, h, :nb] for f in ("pos", "k_scale", "v_scale", "weight"))]


def assert_same_tokens(a, e, news):
    for b in range(a.B):
        for h in range(a.heads_kv):
            for x, y in zip(held_state(a, b, h, int(a.len[b, h]) + news[b]), held_state(e, b, h, int(e.len[b, h]) + news[b])):
                np.testing.assert_array_equal(x.cpu().numpy(), y.cpu().numpy(), err_msg=f"{b} {h}")


@pytest.mark.parametrize("d,tile", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("kind", ["huge", float("nan"), float("inf")])
def test_discarded_tokens_leave_nothing_behind(d, tile, kind):
    """Committed tokens, any number of chunks that are discarded, and the one
    that stays: bit for bit the cache that saw only the last."""
    B, hkv, lens = 4, 2, [5, tile - 1, tile + 3, tile]
    for discarded, n in (([40], 7), ([1, 2 * tile + 1], 40), ([tile, 1, 3], tile + 1)):
        a, e = (V.KVCache(B, hkv, d, tile, 5, DEV) for _ in range(2))
        first, nn = tokens(1, B, tile + 3, hkv, d), torch.tensor(lens, dtype=torch.int32, device=DEV)
        for c in (a, e):
            V.veda_kv_append(c, *first, n_new=nn)
            V.veda_kv_advance(c, tile + 3, n_new=nn)
        for i, m in enumerate(discarded):
            V.veda_kv_append(a, *tokens(10 + 2 * i, B, m, hkv, d, kind))
        last, q = tokens(30, B, n, hkv, d), bf16(40, B, n, 2 * hkv, d)
        outs = []
        for c in (a, e):
            V.veda_kv_append(c, *last)
            o, w = torch.empty_like(q), torch.zeros_like(c.weight)
            V.veda_kv_attn(c, q, o, d ** -0.5, workspace(c, 2 * hkv, n, True), weight=w, decay=0.0)
            outs.append((o, w))
        assert_same_tokens(a, e, [n] * B)
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        assert torch.isfinite(outs[0][0]).all()
        for c in (a, e):                                    # and in what follows
            V.veda_kv_advance(c, n)
            V.veda_kv_append(c, *tokens(50, B, 3, hkv, d))
            V.veda_kv_check_status(c)
        assert_same_tokens(a, e, [3] * B)


@pytest.mark.parametrize("kind", ["huge", float("nan")])
def test_no_tokens_take_the_place_of_pending_ones(kind):
    """A chunk that is dropped and not replaced: an append of none, for all
    sequences or some."""
    B, hkv, d, tile = 3, 2, 64, 64
    for some in (False, True):
        a, e = (random_cache(60, B, hkv, d, tile, 5, [70, 5, 128]) for _ in range(2))
        V.veda_kv_append(a, *tokens(61, B, 30, hkv, d, kind))
        if some:
            news = [0, 9, 0]
            nn = torch.tensor(news, dtype=torch.int32, device=DEV)
            for c in (a, e):
                V.veda_kv_append(c, *tokens(63, B, 9, hkv, d), n_new=nn)
        else:
            news = [0] * B
            V.veda_kv_append(a, *tokens(63, B, 0, hkv, d))
        V.veda_kv_check_status(a)
        for b in range(B):
            for h in range(hkv):
                total = int(a.len[b, h]) + news[b]
                for x, y in zip(held_state(a, b, h, total)[:2], held_state(e, b, h, total)[:2]):
                    np.testing.assert_array_equal(x[:total].cpu().numpy(), y[:total].cpu().numpy())
                for x, y in zip(held_state(a, b, h, total)[3:6], held_state(e, b, h, total)[3:6]):
                    np.testing.assert_array_equal(x.cpu().numpy(), y.cpu().numpy())
        check_attention(a, bf16(64, B, 4, 4, d), pending=False)


def test_tokens_set_in_place_are_not_undone():
    """The caller puts other contents in, with the same counts, between the
    append that raised the scale and the next: those are then the committed
    ones."""
    hkv, d, tile = 2, 64, 64
    for what in ("codes", "scale", "all"):
        a, e = (random_cache(70, 1, hkv, d, tile, 3, [70]) for _ in range(2))
        V.veda_kv_append(a, *tokens(71, 1, 20, hkv, d, "huge"))
        other = random_cache(72, 1, hkv, d, tile, 3, [70])
        if what == "all":
            for f in ("k8", "v8", "table", "pos", "k_scale", "v_scale", "weight", "len", "next_pos"):
                for c in (a, e):
                    getattr(c, f).copy_(getattr(other, f))
        else:
            for f in ("k8", "v8", "k_scale", "v_scale"):        # as the raising append left them
                getattr(e, f).copy_(getattr(a, f))
            for c in (a, e):
                if what == "codes":
                    c.k8.view(torch.uint8)[c.table[0, :, 1].long(), 2, 3] = 0x31
                    c.v8.view(torch.uint8)[c.table[0, :, 1].long(), 5, 60] = 0x31
                else:
                    c.k_scale[:, :, 1] *= 0.5
                    c.v_scale[:, :, 1] *= 4
        for c in (a, e):
            V.veda_kv_append(c, *tokens(74, 1, 9, hkv, d))
        assert_same_tokens(a, e, [9])


def test_any_order_of_calls_against_the_oracle():
    """Chunks of many sizes, discarded or taken in, and evictions between."""
    rng = np.random.default_rng(80)
    B, hkv, d, tile, keep = 2, 2, 64, 64, [3, 4]
    c = V.KVCache(B, hkv, d, tile, 7, DEV)
    want = oracle_of(c)
    for step in range(60):
        n = int(rng.integers(1, 90))
        news = [int(rng.integers(0, n + 1)), n]
        size = 2.0 ** float(rng.integers(-6, 7))
        k, v = bf16(1000 + 2 * step, B, n, hkv, d, size=size), bf16(1001 + 2 * step, B, n, hkv, d, size=1 / size)
        final = bool(rng.random() < 0.4) or step == 59
        if not final and rng.random() < 0.3:
            k[:, 0, 0, 0] = float("nan")
        nn = torch.tensor(news, dtype=torch.int32, device=DEV)
        V.veda_kv_append(c, k, v, n_new=nn)
        want.append(k.double().cpu().numpy(), v.double().cpu().numpy(), news)
        assert_same_state(c, want)
        if final:
            V.veda_kv_advance(c, n, n_new=nn)
            want.advance(np.array(news))
            V.veda_kv_evict(c, keep, 1, 1)
            want.evict(keep, 1, 1)
            assert_same_state(c, want)
    V.veda_kv_check_status(c)
    for b in range(B):
        for h in range(hkv):
            assert torch.isfinite(c.k_scale[b, h, :-(-int(c.len[b, h]) // tile)]).all()


def test_replaced_tokens_in_a_captured_step():
    """The append of a denoising step as a graph, replayed over chunks of which
    one is not finite."""
    hkv, d, tile, n = 2, 64, 64, 20
    a, e = (random_cache(90, 1, hkv, d, tile, 3, [70]) for _ in range(2))
    ins = [tokens(91, 1, n, hkv, d, float("nan")), tokens(93, 1, n, hkv, d, "huge"), tokens(95, 1, n, hkv, d)]
    k, v = (t.clone() for t in ins[0])
    V.veda_kv_append(random_cache(90, 1, hkv, d, tile, 3, [70]), k, v)      # loads the kernel before the capture
    gr, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(gr, stream=side):
        V.veda_kv_append(a, k, v)
    for x, y in ins:
        k.copy_(x), v.copy_(y)
        gr.replay()
    V.veda_kv_append(e, *ins[-1])
    torch.cuda.synchronize()
    assert_same_tokens(a, e, [n])


@pytest.mark.parametrize("n", [24, 96])
def test_stream_layer_forgets_what_it_denoised(n):
    """A chunk that is denoised in steps of which one went astray, and one that
    is committed at once: the same stream."""
    from block_sparse_attention_24_b200.stream import VedaStream
    make = lambda: VedaStream(1, 4, 2, 64, 64, 640, DEV, causal=False, window=400, sinks=64, keep=[4, 5], decay=0.9)
    a, e = make(), make()
    for chunk in range(6):
        q = bf16(200 + chunk, 1, n, 4, 64)
        for kind in ("huge", float("nan")):
            a.step(q, *tokens(300 + 10 * chunk, 1, n, 2, 64, kind), commit=False)
        got, want = (x.step(q, *tokens(310 + 10 * chunk, 1, n, 2, 64)) for x in (a, e))
        assert torch.equal(got, want) and torch.isfinite(got).all()
        assert_same_tokens(a.cache, e.cache, [0])
    a.check_status()
