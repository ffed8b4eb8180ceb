"""The 8-bit K/V tile cache against its fp64 oracle: append, attention,
advance and evict alone at the sizes and masks where each can go wrong, then
together as a stream uses them.

Tolerances of attention, per element. K and V are exact (codes times scales).
  logits  products of e4m3 values are exact in fp32; summing d of them (and
          two factors) costs at most d * 2^-23 of sum |q||k| =: S (the tensor
          core may truncate each partial sum, hence 2^-23), and the exponent's
          argument, at most 2 S in magnitude next to its reference, and ex2
          another 2^-22 * (1 + 4 S): D = 2^-16 * (1 + S) covers both for
          d <= 128.
  q       each row scaled so that its largest value is at 2^7 or above. In two
          e4m3 parts (more query rows per K/V head than FEW) what is left is
          half a step of e4m3's subnormals, 2^-10, at most: 2^-17 of max |q|,
          and D grows by 2^-17 * Q, Q = scale * max |q| * sum |k|. In four
          parts, each of 16 times what the last one left, it is 2^-29.
  P       relative to the largest p_j sv_j =: R of the row, which is at 2^7 or
          above. As fp16: 2^-11 of each weight, and 2^-25 where it is
          subnormal, 2^-32 R per key. In four e4m3 parts: 2^-16 of each, and
          2^-10 / 16^3 = 2^-22 where the last part is subnormal, 2^-29 R per
          key. Each times a code of up to 448 in any channel (that key's, so A,
          which may be small in that channel, does not bound it).
  O       with A = sum p |v|: (2^-11 + 4 D) * A + keys * (2^-32 or 2^-29) * 448
          * R before its own bf16 rounding of 2^-8 |O| (half a step).
  lse     D + 2^-22 * |lse|.
  weight  (4 D + 2^-20) of itself."""
import numpy as np
import pytest
import torch

import block_sparse_attention_24_b200 as V
from oracle.kv_oracle import Cache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FEW = 16          # query rows per K/V head up to which q and P are taken in four parts


def host(t):
    return t.detach().float().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def oracle_of(c: V.KVCache) -> Cache:
    return Cache(c.tile, **{f: host(getattr(c, f)) for f in Cache.FIELDS})


def random_cache(seed, B, hkv, d, tile, nb_cap, lens, spread=1.0, gaps=False, shuffle=True, n_slots=None):
    """A cache that holds lens[b] tokens per head, tile scales apart by a
    normal power of two of deviation `spread`; codes behind len are random
    bytes (NaN codes among them)."""
    g = torch.Generator().manual_seed(seed)
    n = n_slots or B * hkv * nb_cap
    order = torch.randperm(n, generator=g) if shuffle else torch.arange(n)
    c = V.KVCache(B, hkv, d, tile, nb_cap, DEV,
                  k8=torch.zeros((n, tile, d), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                  v8=torch.zeros((n, tile, d), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                  table=order[:B * hkv * nb_cap].to(torch.int32).view(B, hkv, nb_cap).to(DEV))
    for codes, scale in ((c.k8, c.k_scale), (c.v8, c.v_scale)):
        x = torch.randn((B, hkv, nb_cap, tile, d), generator=g) * 60
        u8 = x.to(torch.float8_e4m3fn).view(torch.uint8)
        behind = torch.arange(nb_cap * tile).view(1, nb_cap, tile) >= torch.tensor(lens).view(B, 1, 1)
        junk = torch.randint(0, 256, u8.shape, generator=g).to(torch.uint8)
        junk[..., ::5] = 0x7f
        u8 = torch.where(behind[:, None, :, :, None], junk, u8)
        codes.view(torch.uint8)[c.table.long()] = u8.to(DEV)
        e = torch.round(torch.randn((B, hkv, nb_cap), generator=g) * spread) - 6
        scale.copy_(torch.exp2(e))
    at = torch.arange(nb_cap) * tile
    skip = torch.zeros((B, hkv, nb_cap), dtype=torch.long)
    if gaps:
        skip = torch.randint(0, 3, (B, hkv, nb_cap), generator=g).cumsum(-1)
        last = (torch.tensor(lens) // tile).clamp(max=nb_cap - 1)
        for b in range(B):
            top = skip[b, :, last[b]].max()
            skip[b] = torch.minimum(skip[b], top)
            skip[b, :, last[b]:] = top
    c.pos.copy_((skip * tile + at).to(torch.int32))
    c.len.copy_(torch.tensor(lens, dtype=torch.int32).view(B, 1).expand(B, hkv))
    c.next_pos.copy_(torch.tensor([lens[b] + int(skip[b, 0, min(lens[b] // tile, nb_cap - 1)]) * tile for b in range(B)],
                                  dtype=torch.int32))
    c.weight.copy_(torch.rand((B, hkv, nb_cap), generator=g))
    return c


def assert_same_state(c: V.KVCache, want: Cache, codes=True):
    for f in Cache.FIELDS:
        if f in ("k8", "v8") and not codes:
            continue
        np.testing.assert_array_equal(host(getattr(c, f)), getattr(want, f), err_msg=f)


def workspace(c, heads, n, weight):
    size = V.veda_kv_attn_ws_bytes(c, heads, n, weight)
    assert size > 0
    return torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)   # NaN everywhere


def bf16(seed, *shape, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).to(torch.bfloat16).to(DEV)


def check_attention(c, q, news=None, causal=True, window=0, sinks=0, pending=True, weight=True, decay=0.5, scale=None,
                    o=None):
    B, n, heads, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    o = torch.full_like(q, 7.0) if o is None else o
    before = o.clone()
    lse = torch.full((B, heads, n), 7.0, device=DEV)
    w0 = host(c.weight)
    want_o, want_l, want_w, wrote, A, S, R, Q = oracle_of(c).attend(host(q), [n] * B if news is None else news, scale,
                                                                 causal, window, sinks, pending)
    nn = None if news is None else torch.tensor(news, dtype=torch.int32, device=DEV)
    V.veda_kv_attn(c, q, o, scale, workspace(c, heads, n, weight), causal=causal, window=window, sinks=sinks, n_new=nn,
                   pending=pending, lse=lse, weight=c.weight if weight else None, decay=decay)
    V.veda_kv_check_status(c)
    keys = c.nb_cap * c.tile
    few = n * heads // c.heads_kv <= FEW
    D = 2.0 ** -16 * (1 + S) + 2.0 ** (-29 if few else -17) * Q          # [B, heads, n]
    for b in range(B):
        m = n if news is None else news[b]
        # rows behind the sequence's own are left as they were
        np.testing.assert_array_equal(host(o[b, m:]), host(before[b, m:]))
        np.testing.assert_array_equal(host(lse[b, :, m:]), 7.0)
        go, gl = host(o[b, :m]), host(lse[b, :, :m])
        wo, wl, a, dd = want_o[b, :m], want_l[b, :, :m], A[b, :m], D[b, :, :m]
        np.testing.assert_array_equal(np.isnan(go), np.isnan(wo))
        np.testing.assert_array_equal(np.isnan(gl), np.isnan(wl))
        fin = np.isfinite(wl)
        np.testing.assert_array_equal(gl[~fin], wl[~fin])
        assert np.all(np.abs(gl[fin] - wl[fin]) <= (dd + 2.0 ** -22 * np.abs(wl))[fin])
        tol = ((2.0 ** -11 + 4 * dd.transpose(1, 0)[..., None]) * a + 2.0 ** -8 * np.abs(wo)
               + keys * 2.0 ** (-29 if few else -32) * 448 * R[b, :, :m].transpose(1, 0)[..., None])
        ok = np.isnan(wo) | (np.abs(go - wo) <= tol)
        assert ok.all(), f"batch {b}: {np.max((np.abs(go - wo) - tol)[~np.isnan(wo)])} over"
    if weight:
        gw, ww = host(c.weight), np.where(wrote, decay * w0 + want_w, w0)
        np.testing.assert_array_equal(np.isnan(gw), np.isnan(ww))
        fin = ~np.isnan(ww)
        rel = 4 * np.max(D, where=np.isfinite(D), initial=0.0) + 2.0 ** -20    # rows that see a NaN have no bound
        assert np.all(np.abs(gw - ww)[fin] <= rel * np.abs(ww)[fin] + 2.0 ** -40)
    else:
        np.testing.assert_array_equal(host(c.weight), w0)
    return o, lse


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("d,tile", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens,n,news", [
    ([0], 1, None), ([0, 5, 63], 1, None), ([0, 64, 128], 64, None), ([1, 127, 200], 129, [129, 0, 1]),
    ([130, 30], 300, [300, 171]),
])
def test_append_codes_scales_and_positions(d, tile, lens, n, news):
    B, hkv = len(lens), 3
    c = random_cache(1, B, hkv, d, tile, 8, lens, spread=2.0, gaps=True)
    want = oracle_of(c)
    size = torch.randint(-8, 9, (B, n, 1, 1), generator=torch.Generator().manual_seed(3)).float()
    k = bf16(2, B, n, hkv, d) * torch.exp2(size).to(DEV)
    v = bf16(4, B, n, hkv, d, size=1e-3)
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    nn = None if news is None else torch.tensor(news, dtype=torch.int32, device=DEV)
    V.veda_kv_append(c, k, v, n_new=nn)
    V.veda_kv_check_status(c)
    want.append(host(k), host(v), [n] * B if news is None else news)
    assert_same_state(c, want)
    V.veda_kv_advance(c, n, n_new=nn)
    want.advance(np.array([n] * B if news is None else news))
    assert_same_state(c, want)


def test_append_token_by_token_raises_the_scale_and_keeps_the_older_codes():
    c = V.KVCache(2, 2, 64, 64, 3, DEV)
    want = oracle_of(c)
    for i in range(70):
        size = 2.0 ** ((i * 5) % 13 - 6)
        k, v = bf16(100 + i, 2, 1, 2, 64, size=size), bf16(200 + i, 2, 1, 2, 64, size=1 / size)
        V.veda_kv_append(c, k, v)
        V.veda_kv_advance(c, 1)
        want.append(host(k), host(v), [1, 1])
        want.advance(np.array([1, 1]))
    V.veda_kv_check_status(c)
    assert_same_state(c, want)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38, 448.0 * 2 ** 80, 2.0 ** -133, 0.0,
                                   449.0, 448.0, 450.0])
def test_append_of_extreme_values(value):
    """Not finite, or beyond what the largest scale holds: the scale is NaN;
    all others by the formula (448 * 2^80 is the last that fits)."""
    c = V.KVCache(1, 2, 64, 64, 2, DEV)
    k = torch.zeros((1, 10, 2, 64), dtype=torch.bfloat16, device=DEV)
    k[0, 3, 1, 17] = value
    want = oracle_of(c)
    V.veda_kv_append(c, k, -k)
    want.append(host(k), -host(k), [10])
    assert_same_state(c, want)
    assert torch.isnan(c.k_scale[0, 1, 0]).item() == (not np.isfinite(value) or value > 448.0 * 2.0 ** 80)
    # a tile without a scale stays so while tokens join it
    V.veda_kv_advance(c, 10)
    want.advance(np.array([10]))
    V.veda_kv_append(c, torch.ones_like(k), k)
    want.append(np.ones(k.shape), host(k), [10])
    assert_same_state(c, want)


def test_append_again_replaces_the_pending_tokens():
    c = random_cache(5, 1, 2, 128, 64, 6, [70])
    want = oracle_of(c)
    for seed, n in ((1, 200), (2, 33)):
        k, v = bf16(seed, 1, n, 2, 128), bf16(seed + 10, 1, n, 2, 128)
        V.veda_kv_append(c, k, v)
        want.append(host(k), host(v), [n])
    # the second, shorter chunk touches tiles 1 only; the first chunk's other tiles are not looked at
    assert_same_state(c, want)


def test_append_reads_strided_rows():
    c, e = V.KVCache(2, 3, 64, 64, 4, DEV), V.KVCache(2, 3, 64, 64, 4, DEV)
    qkv = bf16(7, 2, 90, 3, 3, 64)                      # fused projections
    k, v = qkv[:, :, 1], qkv[:, :, 2].transpose(1, 2).contiguous().transpose(1, 2)
    assert not k.is_contiguous() and not v.is_contiguous()
    V.veda_kv_append(c, k, v)
    V.veda_kv_append(e, k.contiguous(), v.contiguous())
    for f in Cache.FIELDS:
        assert torch.equal(getattr(c, f).view(torch.uint8), getattr(e, f).view(torch.uint8)), f
    V.veda_kv_append(c, k[:, :1].expand(2, 5, 3, 64), v[:1].expand(2, 90, 3, 64)[:, :5])    # broadcast tokens, sequences
    V.veda_kv_append(e, k[:, :1].expand(2, 5, 3, 64).contiguous(), v[:1].expand(2, 90, 3, 64)[:, :5].contiguous())
    for f in Cache.FIELDS:
        assert torch.equal(getattr(c, f).view(torch.uint8), getattr(e, f).view(torch.uint8)), f


def bad_status(c):
    with pytest.raises(V.VedaError) as e:
        V.veda_kv_check_status(c)
    assert e.value.code == V.VEDA_ERR_BAD_INDEX
    V.veda_kv_check_status(c)                           # cleared


def test_full_cache_and_bad_counts_leave_the_sequence_alone():
    c = random_cache(8, 3, 2, 64, 64, 2, [100, 10, 0])
    want = oracle_of(c)
    k = bf16(9, 3, 30, 2, 64)
    news = [30, 31, 30]                                 # full; more than there are rows; fine
    nn = torch.tensor(news, dtype=torch.int32, device=DEV)
    V.veda_kv_append(c, k, k, n_new=nn)
    bad_status(c)
    want.append(host(k), host(k), [30, 0, 30])
    assert_same_state(c, want)
    q, o = bf16(10, 3, 30, 4, 64), torch.full((3, 30, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    V.veda_kv_attn(c, q, o, 0.125, workspace(c, 4, 30, True), n_new=nn, weight=c.weight)
    bad_status(c)
    assert (o[:2] == 5).all() and not (o[2] == 5).any()
    V.veda_kv_advance(c, 30, n_new=nn)
    bad_status(c)
    assert c.len.tolist() == [[100, 100], [10, 10], [30, 30]]
    for n_bad in ([-1, 0, 0], [0, 1 << 30, 0]):
        V.veda_kv_append(c, k, k, n_new=torch.tensor(n_bad, dtype=torch.int32, device=DEV))
        bad_status(c)


def test_table_entries_outside_the_pool_are_absent_tiles():
    c = random_cache(11, 1, 2, 64, 64, 5, [200], shuffle=False)
    c.table[0, 0, 1] = c.n_slots
    c.table[0, 1, 0] = -1
    q = bf16(12, 1, 3, 4, 64)
    want = oracle_of(c).attend(host(q), [3], 0.125, False, 0, 0, pending=False)
    o, w = torch.empty_like(q), torch.zeros_like(c.weight)
    V.veda_kv_attn(c, q, o, 0.125, workspace(c, 4, 3, True), causal=False, pending=False, weight=w)
    bad_status(c)
    np.testing.assert_allclose(host(o), want[0], rtol=2.0 ** -7, atol=2.0 ** -6)
    assert w[0, 0, 1] == 0 and w[0, 1, 0] == 0
    k = bf16(13, 1, 10, 2, 64)
    c.table[0, 0, 3] = c.n_slots + 5
    before = c.k8.view(torch.uint8).clone()
    V.veda_kv_append(c, k, k)
    bad_status(c)
    changed = (c.k8.view(torch.uint8) != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [8]                               # head 1's tail tile only


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("d,tile", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("heads,hkv,n", [(2, 2, 1), (8, 2, 1), (3, 1, 2), (16, 1, 1), (32, 1, 1), (10, 2, 5), (6, 3, 9),
                                         (4, 2, 40), (5, 1, 67), (2, 2, 131)])
def test_attention_of_few_and_of_many_rows(d, tile, heads, hkv, n):
    lens = [0, 1, 3 * tile - n % 7, 700]
    nb_cap = -(-(700 + n) // tile)
    c = random_cache(20 + n, 4, hkv, d, tile, nb_cap, [x + n for x in lens], gaps=False)
    c.len.sub_(n)                                       # the last n are pending
    c.next_pos.sub_(n)
    check_attention(c, bf16(21, 4, n, heads, d, size=2.0))
    check_attention(c, bf16(22, 4, n, heads, d), news=[n, max(0, n - 1), 0, (n + 1) // 2], causal=False, decay=0.0)


@pytest.mark.parametrize("n", [1, 4, 33, 150])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (64, 4), (200, 64), (129, 65), (5000, 3), (300, 10 ** 6)])
@pytest.mark.parametrize("causal", [True, False])
def test_window_and_first_tokens(n, window, sinks, causal):
    lens = [900, 130, 0]
    c = random_cache(30 + n, 3, 2, 64, 64, -(-(900 + n) // 64), [x + n for x in lens], gaps=True)
    c.len.sub_(n)
    c.next_pos.sub_(n)
    check_attention(c, bf16(31, 3, n, 6, 64, size=2.0), causal=causal, window=window, sinks=sinks)
    check_attention(c, bf16(32, 3, n, 6, 64), causal=causal, window=window, sinks=sinks, pending=False, weight=False)


@pytest.mark.parametrize("n", [1, 20, 200])
def test_queries_that_see_nothing(n):
    """No tokens held and none pending; a window that evicted tiles fill; all
    keys after the query."""
    c = random_cache(40, 2, 2, 128, 128, 4, [0, 300])
    o, lse = check_attention(c, bf16(41, 2, n, 4, 128), pending=False)
    assert (o[0] == 0).all() and torch.isinf(lse[0]).all() and (lse[0] < 0).all()
    c.next_pos[1] = 1 << 20
    o, lse = check_attention(c, bf16(42, 2, n, 4, 128), pending=False, window=50)
    assert (o == 0).all() and (lse == -float("inf")).all()
    c.next_pos[1] = -(1 << 20)
    o, lse = check_attention(c, bf16(43, 2, n, 4, 128), pending=False)
    assert (o == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("n", [1, 20, 200])
def test_window_behind_the_last_tile_leaves_the_first_tokens(n):
    """Positions far ahead of all tiles: only the first tokens are seen, and
    the last tile, which is not full, is none of theirs."""
    for held in (130, 64 * 6 + 1, 40):
        c = random_cache(45, 1, 2, 64, 64, 8, [held])
        c.next_pos.fill_(1 << 20)
        check_attention(c, bf16(46, 1, n, 4, 64), pending=False, window=50, sinks=100)


@pytest.mark.parametrize("n", [1, 3, 40, 300])
def test_long_cache_is_split(n):
    c = random_cache(50, 1, 1, 128, 128, 81, [10000 + n], spread=3.0)
    c.len.sub_(n)
    c.next_pos.sub_(n)
    check_attention(c, bf16(51, 1, n, 4, 128, size=1.5))


@pytest.mark.parametrize("B,hkv,d,tile,nb,n,window,sinks", [
    (5, 4, 128, 64, 59, 125, 1829, 831),
    (11, 1, 128, 64, 95, 188, 4332, 905),
    (9, 1, 64, 128, 65, 64, 7012, 478),
])
def test_a_window_needs_no_more_workspace(B, hkv, d, tile, nb, n, window, sinks):
    """The workspace is asked for without a window. These would be split into
    more parts by the steps that their window leaves than by all of them."""
    c = random_cache(52, B, hkv, d, tile, nb, [nb * tile - n - 7 * b for b in range(B)])
    q, size = bf16(53, B, n, hkv, d), V.veda_kv_attn_ws_bytes(c, hkv, n, True)
    buf = torch.full((size + (16 << 20),), 0xff, dtype=torch.uint8, device=DEV)
    for pending in (True, False):      # what is pending holds NaN codes, what is held does not
        o, w = torch.empty_like(q), c.weight.clone()
        V.veda_kv_attn(c, q, o, d ** -0.5, buf[:size], window=window, sinks=sinks, pending=pending, weight=w, decay=0.5)
        assert bool((buf[size:] == 0xff).all())
        got, _ = check_attention(c, q, window=window, sinks=sinks, pending=pending)
        assert torch.equal(o.view(torch.int16), got.view(torch.int16))
        assert torch.equal(w.view(torch.int32), c.weight.view(torch.int32))
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("n", [1, 40, 300])
def test_tile_scales_far_apart(n):
    """K scales that give one tile all the weight or none, V scales from one
    end of their range to the other."""
    c = random_cache(60, 1, 2, 64, 64, 16, [700 + n])
    c.len.sub_(n)
    c.next_pos.sub_(n)
    g = torch.Generator().manual_seed(61)
    c.v_scale.copy_(torch.exp2(torch.randint(-40, 81, c.v_scale.shape, generator=g).float()))
    check_attention(c, bf16(62, 1, n, 4, 64), weight=True)
    c.v_scale.fill_(2.0 ** -40)
    c.k_scale.copy_(torch.exp2(torch.randint(-12, 0, c.k_scale.shape, generator=g).float()))
    check_attention(c, bf16(63, 1, n, 4, 64, size=3.0))


@pytest.mark.parametrize("n", [1, 8, 40, 150])
def test_scales_that_are_no_powers_of_two(n):
    """Any positive scale reads right: log2 of a V scale and its inverse are
    then rounded, by 2^-22 each relative to 1 + |log2|, which D (2^-16) holds."""
    c = random_cache(65, 2, 2, 64, 128, 4, [300 + n, 100 + n])
    c.len.sub_(n)
    c.next_pos.sub_(n)
    g = torch.Generator().manual_seed(66)
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.rand(t.shape, generator=g) * 0.01 + 1e-4)
    check_attention(c, bf16(67, 2, n, 4, 64))


@pytest.mark.parametrize("n", [1, 20, 300])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30])
def test_any_softmax_scale(n, scale):
    c = random_cache(68, 1, 2, 64, 64, 10, [300 + n])
    c.len.sub_(n)
    c.next_pos.sub_(n)
    check_attention(c, bf16(69, 1, n, 4, 64), scale=scale)
    check_attention(c, torch.zeros((1, n, 4, 64), dtype=torch.bfloat16, device=DEV), window=100, sinks=5, scale=scale)


@pytest.mark.parametrize("n", [2, 40, 140])
def test_padded_queries_over_a_cache_without_pending_tokens(n):
    c = random_cache(73, 3, 2, 64, 64, 6, [300, 70, 0])
    check_attention(c, bf16(74, 3, n, 4, 64), news=[n - 1, 0, n], pending=False)
    check_attention(c, bf16(75, 3, n, 4, 64), news=[0, 0, 0], pending=False)


def test_output_may_be_the_query_itself():
    for n in (1, 30, 200, 700):
        c = random_cache(76, 2, 2, 64, 64, 20, [500 + n, 300 + n])
        c.len.sub_(n)
        c.next_pos.sub_(n)
        q = bf16(77, 2, n, 6, 64)
        o = torch.empty_like(q)
        V.veda_kv_attn(c, q, o, 0.125, workspace(c, 6, n, False))
        V.veda_kv_attn(c, q, q, 0.125, workspace(c, 6, n, False))
        assert torch.equal(q, o)


@pytest.mark.parametrize("B,hkv", [(40, 8), (3, 1), (1, 100)])
def test_more_and_fewer_heads_than_the_device_has_room_for(B, hkv):
    """One part per head, many parts per head."""
    lens = [(b * 37) % 400 for b in range(B)]
    c = random_cache(78, B, hkv, 64, 64, 7, [x + 1 for x in lens])
    c.len.sub_(1)
    c.next_pos.sub_(1)
    check_attention(c, bf16(79, B, 1, hkv, 64))


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -30, 2.0 ** 30, 2.0 ** 100])
@pytest.mark.parametrize("n", [1, 150])
def test_query_magnitudes_beyond_fp16(size, n):
    c = random_cache(70, 1, 2, 64, 64, 8, [300 + n])
    c.len.sub_(n)
    c.next_pos.sub_(n)
    q = bf16(71, 1, n, 2, 64) * size
    check_attention(c, q.to(torch.bfloat16), scale=0.125 / size)


@pytest.mark.parametrize("n", [1, 5, 40, 150])
def test_nan_tiles_reach_only_the_queries_that_see_them(n):
    c = random_cache(80, 1, 2, 64, 64, 12, [700], gaps=False)
    c.len.sub_(n)
    c.next_pos.sub_(n)
    c.k_scale[0, 0, 3] = float("nan")                   # outside the window of all
    c.v_scale[0, 1, 2] = float("nan")
    for codes, slot in ((c.k8, c.table[0, 0, 2]), (c.v8, c.table[0, 1, 1])):
        codes.view(torch.uint8)[slot.long()] = 0x7f     # NaN codes where no query looks
    o, _ = check_attention(c, bf16(81, 1, n, 4, 64), window=250, sinks=10)
    assert not torch.isnan(o).any()
    c.v_scale[0, 0, 11 - (60 + n) // 64] = float("nan")  # inside some queries' windows, behind others' if n is large
    c.k_scale[0, 1, 10] = float("nan")
    o, _ = check_attention(c, bf16(82, 1, n, 4, 64), window=30, sinks=10)
    o, _ = check_attention(c, bf16(83, 1, n, 4, 64), causal=False)
    assert torch.isnan(o).any()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_queries_that_are_not_finite_stay_alone(value):
    for n in (2, 160):
        c = random_cache(85, 1, 1, 64, 64, 6, [200 + n])
        c.len.sub_(n)
        c.next_pos.sub_(n)
        q = bf16(86, 1, n, 2, 64)
        clean = torch.empty_like(q)
        V.veda_kv_attn(c, q, clean, 0.125, workspace(c, 2, n, False))
        q[0, 1, 1, 5] = value
        o = torch.empty_like(q)
        V.veda_kv_attn(c, q, o, 0.125, workspace(c, 2, n, False))
        assert torch.isnan(o[0, 1, 1]).all()
        o[0, 1, 1] = clean[0, 1, 1]
        assert torch.equal(o, clean)


def test_attention_reads_and_writes_strided_rows():
    for n in (1, 70):
        c = random_cache(90, 2, 2, 64, 64, 5, [200 + n, 100 + n])
        c.len.sub_(n)
        c.next_pos.sub_(n)
        fused = bf16(91, 2, n, 3, 4, 64)
        room = torch.full((2, 4, n + 3, 64), 9.0, dtype=torch.bfloat16, device=DEV)
        o = room.transpose(1, 2)[:, 1:n + 1]
        check_attention(c, fused[:, :, 0], o=o)
        assert (room[:, :, 0] == 9).all() and (room[:, :, n + 1:] == 9).all()


@pytest.mark.parametrize("n", [1, 140])
def test_slots_past_two_gigabytes(n):
    """Code offsets that do not fit 31 bits."""
    tile, d = 128, 128
    n_slots = (1 << 31) // (tile * d) + 40
    k8 = torch.zeros((n_slots, tile, d), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    v8 = torch.zeros_like(k8.view(torch.uint8)).view(torch.float8_e4m3fn)
    table = torch.tensor([[n_slots - 1 - 7 * i for i in range(4)]], dtype=torch.int32, device=DEV).view(1, 1, 4)
    c = V.KVCache(1, 1, d, tile, 4, DEV, k8=k8, v8=v8, table=table)
    small = V.KVCache(1, 1, d, tile, 4, DEV)
    k, v, q = bf16(95, 1, 300 + n, 1, d), bf16(96, 1, 300 + n, 1, d), bf16(97, 1, n, 2, d)
    got = []
    for cache in (c, small):
        V.veda_kv_append(cache, k[:, :300], v[:, :300])
        V.veda_kv_advance(cache, 300)
        V.veda_kv_append(cache, k[:, 300:], v[:, 300:])
        o = torch.empty_like(q)
        V.veda_kv_attn(cache, q, o, 0.1, workspace(cache, 2, n, True), weight=cache.weight)
        got.append((o, cache.weight.clone()))
    V.veda_kv_check_status(c)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert (got[0][0] != 0).any()
    # a table near the end of the pool, rows of it read in place
    np.testing.assert_array_equal(host(c.k8[table.long().view(-1)]), host(small.k8))


def test_shared_slots():
    """Two sequences read one prefix."""
    for n in (1, 70):
        c = random_cache(98, 2, 1, 64, 64, 5, [256, 256])
        c.table[1, 0, :3] = c.table[0, 0, :3]
        check_attention(c, bf16(99, 2, n, 2, 64), pending=False)


def test_attention_is_repeatable():
    for n in (1, 90):
        c = random_cache(100, 2, 2, 128, 128, 20, [2000, 1500])
        q = bf16(101, 2, n, 8, 128)
        got = []
        for _ in range(3):
            o, w, l = torch.empty_like(q), torch.zeros_like(c.weight), torch.empty((2, 8, n), device=DEV)
            V.veda_kv_attn(c, q, o, 0.1, workspace(c, 8, n, True), pending=False, weight=w, lse=l)
            got.append((o, w, l))
        for x in got[1:]:
            assert all(torch.equal(a, b) for a, b in zip(x, got[0]))


# ------------------------------------------------------------------- evict

def evict_cache(seed, B, hkv, nb_cap, lens, weights):
    c = random_cache(seed, B, hkv, 64, 64, nb_cap, lens, gaps=True) if nb_cap < 100 else V.KVCache(
        B, hkv, 64, 64, nb_cap, DEV, k8=torch.zeros((B * hkv * nb_cap, 64, 64), dtype=torch.uint8, device=DEV).view(
            torch.float8_e4m3fn), v8=torch.zeros((B * hkv * nb_cap, 64, 64), dtype=torch.uint8, device=DEV).view(
                torch.float8_e4m3fn))
    c.len.copy_(torch.tensor(lens, dtype=torch.int32).view(B, 1).expand(B, hkv))
    c.weight.copy_(weights.to(DEV))
    if nb_cap >= 100:
        g = torch.Generator().manual_seed(seed)
        for t in (c.k_scale, c.v_scale):
            t.copy_(torch.rand(t.shape, generator=g))
        c.pos.copy_((torch.arange(nb_cap) * 64).to(torch.int32).expand_as(c.pos))
    return c


CASES = [
    # nb_cap, lens, keep, sink, recent
    (9, [9 * 64, 8 * 64 + 1, 300], [5, 6], 1, 2), (9, [576, 10, 0], [3, 9], 1, 2), (9, [576, 512, 511], [1, 2], 0, 1),
    (9, [576, 512, 511], [4, 8], 3, 1), (700, [700 * 64, 40000, 17001], [300, 513], 4, 100),
    (8192, [8192 * 64, 8191 * 64 + 1, 200000], [4000, 8191], 0, 1),
]


@pytest.mark.parametrize("nb_cap,lens,keep,sink,recent", CASES)
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
def test_evict_in_place_and_into_another(nb_cap, lens, keep, sink, recent, kind):
    g = torch.Generator().manual_seed(nb_cap)
    w = torch.rand((3, 2, nb_cap), generator=g) ** 8 * 1e3
    if kind == "ties":
        w = torch.randint(0, 3, w.shape, generator=g).float()
    elif kind == "odd":
        special = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -1.0, 1e-42, -1e-42, 3e38])
        w = torch.where(torch.rand(w.shape, generator=g) < 0.6, special[torch.randint(0, 9, w.shape, generator=g)], w)
    c = evict_cache(110, 3, 2, nb_cap, lens, w)
    meta = {f: getattr(c, f).clone() for f in ("table", "pos", "k_scale", "v_scale", "weight", "len", "next_pos")}
    out = V.KVCache(3, 2, 64, 64, nb_cap, DEV, k8=c.k8, v8=c.v8, **{f: t.clone().fill_(3) for f, t in meta.items()})
    want = oracle_of(c) if nb_cap < 100 else Cache(64, k8=np.zeros((1, 64, 64)), v8=np.zeros((1, 64, 64)),
                                                   **{f: host(t) for f, t in meta.items()})
    want.evict(keep, sink, recent)
    V.veda_kv_evict(c, keep, sink, recent, out=out)
    for f, t in meta.items():
        np.testing.assert_array_equal(host(getattr(c, f)), host(t), err_msg=f)     # as it was
    assert_same_state(out, want, codes=False)
    V.veda_kv_evict(c, keep, sink, recent)
    assert_same_state(c, want, codes=False)
    V.veda_kv_evict(c, keep, sink, recent)                                         # nothing more to drop
    assert_same_state(c, want, codes=False)
    V.veda_kv_check_status(c)


# ---------------------------------------------------------------- together

def stream_step(c, k, v, q, o, lse, ws, n_new=None, keep=None, causal=True, window=0, sinks=0):
    n = q.shape[1]
    V.veda_kv_append(c, k, v, n_new=n_new)
    V.veda_kv_attn(c, q, o, q.shape[-1] ** -0.5, ws, causal=causal, window=window, sinks=sinks, n_new=n_new, lse=lse,
                   weight=c.weight, decay=0.9)
    V.veda_kv_advance(c, n, n_new=n_new)
    if keep:
        V.veda_kv_evict(c, keep, 1, 2)


@pytest.mark.parametrize("n,d,tile,window", [(1, 64, 64, 0), (48, 64, 64, 0), (200, 128, 128, 300), (130, 128, 64, 0)])
def test_a_stream_of_steps(n, d, tile, window):
    """Append, attention, advance, evict, step after step, against the oracle
    that does the same: after eviction the heads hold different tiles."""
    B, hkv, heads, keep = 2, 2, 4, [4, 5]
    c = V.KVCache(B, hkv, d, tile, 6 + -(-n // tile), DEV)
    for step in range(8 if n > 1 else 3):
        k, v = bf16(300 + step, B, n, hkv, d), bf16(400 + step, B, n, hkv, d)
        q = bf16(500 + step, B, n, heads, d, size=2.0)
        news = [n, n if step % 3 else n // 2]
        want = oracle_of(c)
        nn = torch.tensor(news, dtype=torch.int32, device=DEV)
        V.veda_kv_append(c, k, v, n_new=nn)
        want.append(host(k), host(v), news)
        assert_same_state(c, want)
        check_attention(c, q, news=news, window=window, sinks=3, decay=0.9)
        want = oracle_of(c)
        V.veda_kv_advance(c, n, n_new=nn)
        want.advance(np.array(news))
        V.veda_kv_evict(c, keep, 1, 2)
        want.evict(keep, 1, 2)
        assert_same_state(c, want)


@pytest.mark.parametrize("n", [1, 70])
def test_captured_steps_equal_eager_ones(n):
    """One captured step, replayed over new inputs in the same buffers, and two
    captured graphs that share a workspace, replayed in turn."""
    B, hkv, heads, d, tile = 2, 2, 4, 64, 64
    ins = [(bf16(600 + s, B, n, hkv, d), bf16(610 + s, B, n, hkv, d), bf16(620 + s, B, n, heads, d)) for s in range(6)]
    make = lambda: V.KVCache(B, hkv, d, tile, 12, DEV)
    a, e = make(), make()
    ws = workspace(a, heads, n, True)
    k, v, q = (t.clone() for t in ins[0])
    o, lse = torch.zeros_like(q), torch.zeros((B, heads, n), device=DEV)
    first = make()                                      # loads every kernel before the capture
    stream_step(first, k, v, q, o, lse, ws, keep=[3, 3])
    graphs = []
    side = torch.cuda.Stream()
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(gr, stream=side):
            stream_step(a, k, v, q, o, lse, ws, keep=[3, 3])
        graphs.append(gr)
    eo, el = torch.zeros_like(q), torch.zeros_like(lse)
    for s, (k1, v1, q1) in enumerate(ins):
        k.copy_(k1), v.copy_(v1), q.copy_(q1)
        graphs[s % 2].replay()
        stream_step(e, k1, v1, q1, eo, el, ws.clone(), keep=[3, 3])
        torch.cuda.synchronize()
        assert torch.equal(o, eo) and torch.equal(lse, el)
        for f in Cache.FIELDS:
            assert torch.equal(getattr(a, f).view(torch.uint8), getattr(e, f).view(torch.uint8)), f
    V.veda_kv_check_status(a)


def test_steps_on_two_streams_at_once():
    B, hkv, heads, d, tile, n = 1, 2, 4, 128, 128, 64
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    caches = [V.KVCache(B, hkv, d, tile, 40, DEV) for _ in range(4)]
    ins = [(bf16(700 + s, B, n, hkv, d), bf16(710 + s, B, n, hkv, d), bf16(720 + s, B, n, heads, d)) for s in range(4)]
    outs = [torch.zeros((B, n, heads, d), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    wss = [workspace(caches[0], heads, n, True) for _ in range(4)]
    torch.cuda.synchronize()
    for step in range(4):
        for j, st in ((0, s1), (1, s2)):
            k, v, q = ins[(step + j) % 4]
            V.veda_kv_append(caches[j], k, v, stream=st)
            V.veda_kv_attn(caches[j], q, outs[j], 0.1, wss[j], weight=caches[j].weight, stream=st)
            V.veda_kv_advance(caches[j], n, stream=st)
    torch.cuda.synchronize()
    for step in range(4):
        for j in (0, 1):
            k, v, q = ins[(step + j) % 4]
            V.veda_kv_append(caches[2 + j], k, v)
            V.veda_kv_attn(caches[2 + j], q, outs[2 + j], 0.1, wss[2 + j], weight=caches[2 + j].weight)
            V.veda_kv_advance(caches[2 + j], n)
    torch.cuda.synchronize()
    for j in (0, 1):
        assert torch.equal(outs[j], outs[2 + j]) and torch.equal(caches[j].weight, caches[2 + j].weight)


def test_stream_layer_denoises_commits_and_evicts():
    """VedaStream: a chunk's keys are replaced while it is denoised and join
    the cache when it is committed; the heads are cut to their tiles."""
    from block_sparse_attention_24_b200.stream import VedaStream
    B, heads, hkv, d, tile, n = 1, 4, 2, 64, 64, 96
    layer = VedaStream(B, heads, hkv, d, tile, 640, DEV, causal=False, window=400, sinks=64, keep=[4, 5], decay=0.9)
    c = layer.cache
    for chunk in range(7):
        for t in range(3):
            k, v = bf16(800 + 10 * chunk + t, B, n, hkv, d), bf16(900 + 10 * chunk + t, B, n, hkv, d)
            q = bf16(1000 + 10 * chunk + t, B, n, heads, d)
            want = oracle_of(c)
            want.append(host(k), host(v), [n])
            o, lse, w, wrote, A, S, R, Q = want.attend(host(q), [n], d ** -0.5, False, 400, 64)
            got = layer.step(q, k, v, commit=t == 2)
            layer.check_status()
            D = (2.0 ** -16 * (1 + S) + 2.0 ** -17 * Q).transpose(0, 2, 1)[..., None]
            tol = (2.0 ** -11 + 4 * D) * A + 2.0 ** -8 * np.abs(o) + 640 * 2.0 ** -32 * 448 * R.transpose(0, 2, 1)[..., None]
            assert (np.abs(host(got) - o) <= tol).all()
            if t < 2:
                assert_same_state(c, want)
        want.weight = np.where(wrote, 0.9 * want.weight + w, want.weight)
        held = host(c.weight)
        want.advance(np.array([n]))
        # the same tiles go by the kernel's weights, which differ by rounding
        want.evict([4, 5], 1, 1)
        np.testing.assert_array_equal(host(c.len), want.len)
        np.testing.assert_array_equal(host(c.table), want.table)
        np.testing.assert_allclose(held, want.weight, rtol=1e-3)
        assert (host(c.len) <= np.array([4, 5]) * tile).all()
    assert int(c.next_pos[0]) == 7 * n
    layer.reset()
    assert int(c.len.sum()) == 0
    with pytest.raises(ValueError, match="multiple|limits"):
        VedaStream(1, 3, 2, 64, 64, 128, DEV).workspace(1, False)


def test_stream_layer_allocates_on_the_stream_of_the_step():
    """Memory that the current stream has freed may still be in use there."""
    from block_sparse_attention_24_b200.stream import VedaStream
    n = 1 << 13
    q, k, v = bf16(1100, 1, n, 2, 64), bf16(1101, 1, n, 2, 64), bf16(1102, 1, n, 2, 64)
    layers = [VedaStream(1, 2, 2, 64, 64, n, DEV, keep=5) for _ in range(2)]
    want = layers[0].step(q, k, v)
    torch.cuda.synchronize()
    freed = [torch.empty_like(q), torch.empty_like(layers[0].workspace(n, True))]
    held = [t.data_ptr() for t in freed]
    freed.clear()
    s = torch.cuda.Stream()
    got = layers[1].step(q, k, v, stream=s)
    assert got.data_ptr() not in held and layers[1].workspace(n, True).data_ptr() not in held
    s.synchronize()
    assert torch.equal(got, want)
    for f in ("k8", "v8"):
        assert torch.equal(getattr(layers[0].cache, f).view(torch.uint8), getattr(layers[1].cache, f).view(torch.uint8))
    for f in ("table", "pos", "k_scale", "v_scale", "weight", "len", "next_pos"):
        assert torch.equal(getattr(layers[0].cache, f), getattr(layers[1].cache, f))
    layers[1].reset(stream=s)
    s.synchronize()
    assert int(layers[1].cache.len.sum()) == 0 and int(layers[1].cache.next_pos[0]) == 0


@pytest.mark.parametrize("n,d,tile,heads,hkv", [(1, 64, 64, 8, 2), (1, 128, 128, 4, 4), (3, 128, 64, 12, 2), (40, 64, 64, 4, 1)])
def test_steps_back_to_back_equal_steps_one_at_a_time(n, d, tile, heads, hkv):
    """Kernels are set up while the one before them ends; each still sees all
    that those before it wrote, in both directions and between kernels of other
    kinds (the copies and fills here)."""
    B, steps, keep = 3, 40, 4
    got = []
    for alone in (True, False):
        c = V.KVCache(B, hkv, d, tile, keep + 2 + n // tile, DEV)
        ws = workspace(c, heads, n, True)
        news = torch.tensor([n, max(0, n - 1), n], dtype=torch.int32, device=DEV)
        x = [bf16(1200 + i, steps, B, n, heads if i == 0 else hkv, d) for i in range(3)]
        q = torch.empty((B, n, heads, d), dtype=torch.bfloat16, device=DEV)
        outs = []
        wait = torch.cuda.synchronize if alone else (lambda: None)
        wait()
        for t in range(steps):
            o, lse = torch.zeros_like(q), torch.zeros((B, heads, n), device=DEV)
            for call in (lambda: q.copy_(x[0][t]),
                         lambda: V.veda_kv_append(c, x[1][t], x[2][t], n_new=news),
                         lambda: V.veda_kv_attn(c, q, o, 0.1, ws, n_new=news, lse=lse, weight=c.weight, decay=0.9),
                         lambda: q.zero_(),
                         lambda: V.veda_kv_advance(c, n, n_new=news),
                         lambda: V.veda_kv_evict(c, [keep] * hkv, 1, 2)):
                call()
                wait()
            outs += [o, lse]
        V.veda_kv_check_status(c)
        got.append(outs + [c.k_scale, c.v_scale, c.table, c.pos, c.len, c.next_pos, c.weight])
    for a, b in zip(*got):
        assert torch.equal(a, b)
