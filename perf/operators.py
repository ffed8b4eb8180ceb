"""The operators of the 8-bit K/V tile cache, as cases that can be measured: their inputs, a plain form of each in
elementary torch operations, the library's own calls, and the values in 64 bits.

  append   new tokens' K and V are quantised into the cache (e4m3 codes, one power-of-two scale per tile and head)
  attend   queries attend to the cached tokens, under a causal, sliding-window and first-tokens mask
  evict    the tiles with the least accumulated attention weight leave the cache

A tile of the cache is `tile` consecutive tokens of one (sequence, K/V head): a row `slot` of the code pools
[n_slots, tile, d], found through table[b, h, i]. pos, k_scale, v_scale and weight are [b, h, i] too.
"""
import random

import torch

own = False

LOG2_E = 1.4426950408889634


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of four short conversations: the latency of the smallest call
        dict(name="append token", op="append", B=4, hkv=8, d=128, tile=128, n=1, len=1900, ragged=70),
        # one latent frame of 48 x 80 tokens joins a stream that holds seven
        dict(name="append frame", op="append", B=1, hkv=24, d=128, tile=128, n=3840, len=26900, ragged=0),
        # prompts of unequal length, padded to the longest, behind caches that end inside a tile
        dict(name="append ragged", op="append", B=6, hkv=4, d=64, tile=64, n=1111, len=517, ragged=90),
        # one query token over a short cache: latency
        dict(name="attend token", op="attend", B=1, heads=32, hkv=8, d=128, tile=128, n=1, len=1500, ragged=0,
             causal=True, window=0, sinks=0, weights=False),
        # a serving batch of unequal lengths, four query heads per K/V head, with the weights that eviction goes by
        dict(name="attend batch", op="attend", B=16, heads=32, hkv=8, d=128, tile=128, n=1, len=8190, ragged=50,
             causal=True, window=0, sinks=0, weights=True),
        # the longest cache: two streams of 21 frames, one K/V head per query head
        dict(name="attend long", op="attend", B=2, heads=24, hkv=24, d=128, tile=128, n=1, len=80639, ragged=0,
             causal=True, window=0, sinks=0, weights=False),
        # a sliding window with a few first tokens: most of the cache is not read
        dict(name="attend window", op="attend", B=32, heads=16, hkv=2, d=64, tile=64, n=2, len=16000, ragged=30,
             causal=True, window=2048, sinks=4, weights=False),
        # the queries of a whole new frame over eight cached ones and itself, no order inside the frame
        dict(name="attend frame", op="attend", B=1, heads=24, hkv=24, d=128, tile=128, n=3840, len=30720, ragged=0,
             causal=False, window=0, sinks=0, weights=False),
        # a prompt: queries over themselves, causal
        dict(name="attend prompt", op="attend", B=1, heads=32, hkv=8, d=128, tile=128, n=2048, len=0, ragged=0,
             causal=True, window=0, sinks=0, weights=True),
        # padded chunks of unequal sizes in the middle of a stream, windowed, small heads
        dict(name="attend chunk", op="attend", B=3, heads=12, hkv=4, d=64, tile=64, n=333, len=9000, ragged=60,
             causal=True, window=4096, sinks=64, weights=True),
        # one stream's heads drop a fifth of their tiles
        dict(name="evict stream", op="evict", B=1, hkv=24, d=128, tile=128, len=38300, ragged=0, keep=240, sink=1,
             recent=30),
        # a batch of long caches is halved
        dict(name="evict batch", op="evict", B=32, hkv=8, d=64, tile=64, len=131000, ragged=40, keep=1024, sink=2,
             recent=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    d, tile = rng.choice([64, 128]), rng.choice([64, 128])
    op = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "evict"])
    if op == "append":
        B = _log(rng, 1, 32)
        n = _log(rng, 1, 8000)
        hkv = _log(rng, 1, 40)
        while B * n * hkv * d > 3840 * 24 * 128:
            n, B = max(1, n // 2), max(1, B - 1)
        return dict(op=op, B=B, hkv=hkv, d=d, tile=tile, n=n, len=_log(rng, 1, 20000) - 1, ragged=rng.choice([0, 40, 95]))
    if op == "evict":
        n_tiles = _log(rng, 4, 2000)
        recent, sink = rng.randint(1, max(1, n_tiles // 8)), rng.randint(0, min(4, n_tiles // 4))
        return dict(op=op, B=_log(rng, 1, 32), hkv=_log(rng, 1, 24), d=64, tile=64, len=n_tiles * 64 - rng.randint(0, 63),
                    ragged=rng.choice([0, 30]), keep=max(sink + recent, int(n_tiles * rng.uniform(0.2, 1.1))), sink=sink,
                    recent=recent)
    hkv, group = _log(rng, 1, 24), rng.choice([1, 1, 2, 3, 4, 6, 8, 16])
    chunk = rng.random() < 0.4
    n = _log(rng, 17, 4000) if chunk else rng.choice([1, 1, 1, 2, 3, 5, 8])
    B, length = (_log(rng, 1, 4) if chunk else _log(rng, 1, 32)), _log(rng, 1, 80000) - 1
    while B * hkv * group * n * (length + n) > 24 * 3840 * 34560 or B * hkv * d * (length + n) > 2 * 24 * 128 * 80640:
        n, B, length = (n * 3 // 4 if n > 24 else n), max(1, B - 1), length * 3 // 4
    return dict(op=op, B=B, heads=hkv * group, hkv=hkv, d=d, tile=tile, n=n, len=length, ragged=rng.choice([0, 50, 90]),
                causal=rng.random() < 0.7, window=rng.choice([0, 0, _log(rng, 1, 20000)]), sinks=rng.choice([0, 4, 100]),
                weights=rng.random() < 0.5)


def _lengths(case):
    """Tokens that each sequence holds, and new ones (unequal where the case is ragged: some of its percent less)."""
    B, less = case["B"], case["ragged"]
    share = [(b * 7919 % B) / B * less / 100 for b in range(B)]
    n = case.get("n", 0)
    return [int(case["len"] * (1 - s)) for s in share], [max(0, n - int(n * s)) for s in share]


def _scale_of(amax):
    """The least power of two s with 448 s >= amax, kept within 2^-40 .. 2^80; NaN where there is none."""
    frac, exp = torch.frexp(amax)
    e = exp - 9 + (frac > 0.875).to(exp.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -40)).clamp(min=-40)
    s = torch.ldexp(torch.ones_like(amax), e)
    return torch.where(torch.isfinite(amax) & (e <= 80), s, torch.full_like(s, float("nan")))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    r = random.Random(seed)
    B, hkv, d, tile, op = case["B"], case["hkv"], case["d"], case["tile"], case["op"]
    lens, news = _lengths(case)
    n = case.get("n", 0)
    nb_cap = max(1, max(-(-(a + n) // tile) for a in lens))
    n_slots = B * hkv * nb_cap
    f32, i32 = dict(dtype=torch.float32, device=dev), dict(dtype=torch.int32, device=dev)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    st = dict(case=dict(case))
    # slots in the order in which a running server would have handed them out: none in particular
    st["table"] = torch.randperm(n_slots, generator=gen, device=dev).to(torch.int32).view(B, hkv, nb_cap)
    held = torch.tensor(lens, **i32)
    # some tokens have been evicted earlier: positions run ahead of the count, with gaps between tiles
    gaps = torch.randint(0, 3, (B, hkv, nb_cap), generator=gen, device=dev).cumsum(-1) * (op == "attend")
    gaps = gaps - gaps[..., :1]
    last = (held.view(B, 1, 1).expand(B, hkv, 1).long() // tile).clamp(max=nb_cap - 1)
    shift = gaps.gather(-1, last).amax(1, keepdim=True)             # the tail tile is the newest for every head
    at = torch.arange(nb_cap, device=dev)
    gaps = torch.where(at >= last, shift, torch.minimum(gaps, shift))
    st["pos"] = (gaps * tile + at * tile).to(torch.int32)
    st["next_pos"] = (held.long() + shift.view(B) * tile).to(torch.int32)
    st["len"] = held.view(B, 1).expand(B, hkv).contiguous()
    st["weight"] = torch.rand((B, hkv, nb_cap), generator=gen, device=dev) ** 4 * 100
    # tiles of the cache: normal values whose size differs from tile to tile by a few binary orders
    st["k8"] = torch.empty((n_slots, tile, d), dtype=torch.float8_e4m3fn, device=dev)
    st["v8"] = torch.empty_like(st["k8"])
    slots = st["table"].long().view(-1)
    for codes, scale in (("k8", "k_scale"), ("v8", "v_scale")):
        per_slot = torch.empty(n_slots, **f32)
        part = max(1, (1 << 27) // (tile * d)) if op != "evict" else n_slots
        for s0 in range(0, n_slots, part):
            c = min(part, n_slots - s0)
            if op == "evict":  # the codes are not touched: any will do
                st[codes].view(torch.uint8).fill_(0x30)
                per_slot.copy_(torch.ldexp(torch.ones(c, **f32), torch.randint(-12, -4, (c,), generator=gen, **i32)))
                break
            x = torch.randn((c, tile, d), generator=gen, **f32)
            x *= torch.exp2(torch.randn((c, 1, 1), generator=gen, **f32) * 0.5)
            per_slot[s0:s0 + c] = _scale_of(x.abs().amax((1, 2)))
            st[codes][s0:s0 + c] = (x / per_slot[s0:s0 + c].view(-1, 1, 1)).to(torch.float8_e4m3fn)
        st[scale] = per_slot[slots].view(B, hkv, nb_cap)
    st["n_new"] = torch.tensor(news, **i32)
    if op == "append":
        st["k"], st["v"] = normal(B, n, hkv, d), normal(B, n, hkv, d)
    elif op == "attend":
        st["q"] = normal(B, n, case["heads"], d)
        st["o"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((B, case["heads"], n), **f32)
    else:
        st["keep"] = [max(case["sink"] + case["recent"], case["keep"] - r.randint(0, 3)) for _ in range(hkv)]
    if own:
        import block_sparse_attention_24_b200 as V
        meta = ("table", "pos", "k_scale", "v_scale", "weight", "len", "next_pos")
        st["cache"] = V.KVCache(B, hkv, d, tile, nb_cap, device=dev, k8=st["k8"], v8=st["v8"],
                                **{m: st[m] for m in meta})
        if op == "attend":
            size = V.veda_kv_attn_ws_bytes(st["cache"], case["heads"], n, case["weights"])
            st["ws"] = torch.empty(max(16, size), dtype=torch.uint8, device=dev)
        elif op == "evict":
            st["out"] = V.KVCache(B, hkv, d, tile, nb_cap, device=dev, k8=st["k8"], v8=st["v8"],
                                  **{m: st[m].clone() for m in meta})
    return st


# ------------------------------------------------------------ plain forms

def _read(codes, slot):
    return codes.view(torch.uint8)[slot].view(torch.float8_e4m3fn).float()


def _append(st):
    """K and V of the new tokens into the tail tiles: [B, hkv, touched tiles, tile, d] at a time."""
    case, dev = st["case"], st["k"].device
    B, hkv, d, tile, n = (case[x] for x in ("B", "hkv", "d", "tile", "n"))
    nb_cap = st["table"].shape[-1]
    held, news = st["len"].long().view(B, hkv, 1, 1), st["n_new"].long().view(B, 1, 1, 1)
    touched = -(-n // tile) + 1
    block = held // tile + torch.arange(touched, device=dev).view(1, 1, -1, 1)          # [B, hkv, J, 1]
    token = block * tile + torch.arange(tile, device=dev) - held                         # [B, hkv, J, tile]
    new, old = (token >= 0) & (token < news), token < 0
    any_new, fresh = new.any(-1), token[..., 0] >= 0
    entry = block[..., 0].clamp(max=nb_cap - 1)
    b = torch.arange(B, device=dev).view(B, 1, 1, 1)
    h = torch.arange(hkv, device=dev).view(1, hkv, 1, 1)
    slot = st["table"].gather(-1, entry).long()
    for x, codes, scale in ((st["k"], st["k8"], st["k_scale"]), (st["v"], st["v8"], st["v_scale"])):
        x = x[b, token.clamp(0, n - 1), h].float()                                       # [B, hkv, J, tile, d]
        size = torch.where(new[..., None], x.abs(), torch.zeros_like(x)).amax((-1, -2))
        s_new, s_old = _scale_of(size), scale.gather(-1, entry)
        s = torch.where(fresh, s_new, torch.maximum(s_new, s_old))                       # NaN where either is
        fine = ~torch.isnan(s)[..., None, None]
        was = _read(codes, slot)
        moved = torch.where(fine & (s != s_old)[..., None, None],
                            (was * (s_old / s)[..., None, None]).to(codes.dtype).float(), was)
        x = torch.where(fine, (x / s[..., None, None]).to(codes.dtype).float(), torch.zeros_like(x))
        y = torch.where(new[..., None], x, torch.where(old[..., None], moved, torch.zeros_like(x))).to(codes.dtype)
        codes.view(torch.uint8)[slot[any_new]] = y.view(torch.uint8)[any_new]
        rows = (b[..., 0].expand_as(entry)[any_new], h[..., 0].expand_as(entry)[any_new], entry[any_new])
        scale[rows] = s[any_new]
    opened = any_new & fresh
    rows = (b[..., 0].expand_as(entry)[opened], h[..., 0].expand_as(entry)[opened], entry[opened])
    st["pos"][rows] = (st["next_pos"].view(B, 1, 1) + token[..., 0])[opened].to(torch.int32)
    st["weight"][rows] = 0.0


def _visible(st):
    """[B, hkv, queries, keys]: which cached keys each query sees, and which rows are queries."""
    case, dev = st["case"], st["q"].device
    B, hkv, tile, n = (case[x] for x in ("B", "hkv", "tile", "n"))
    nb_cap = st["table"].shape[-1]
    count = (st["len"] + st["n_new"].view(B, 1)).view(B, hkv, 1, 1)
    here = torch.arange(nb_cap * tile, device=dev) < count
    at = (st["pos"][..., None] + torch.arange(tile, device=dev, dtype=torch.int32)).view(B, hkv, 1, nb_cap * tile)
    t = (st["next_pos"].view(B, 1) + torch.arange(n, device=dev, dtype=torch.int32)).view(B, 1, n, 1)
    seen = here.expand(B, hkv, n, nb_cap * tile)
    if case["causal"]:
        seen = seen & (at <= t)
    if case["window"] > 0:
        seen = seen & ((at > t - case["window"]) | (at < case["sinks"]))
    return seen, torch.arange(n, device=dev) < st["n_new"].view(B, 1)


def _attend(st):
    case = st["case"]
    B, heads, hkv, d, tile, n = (case[x] for x in ("B", "heads", "hkv", "d", "tile", "n"))
    nb_cap, group = st["table"].shape[-1], heads // hkv
    slot = st["table"].long()
    k = (_read(st["k8"], slot) * st["k_scale"][..., None, None]).view(B, hkv, 1, nb_cap * tile, d)
    v = (_read(st["v8"], slot) * st["v_scale"][..., None, None]).view(B, hkv, 1, nb_cap * tile, d)
    q = st["q"].float().view(B, n, hkv, group, d).permute(0, 2, 3, 1, 4)
    seen, row = _visible(st)
    s = q @ k.transpose(-1, -2) * d ** -0.5
    s.masked_fill_(~seen[:, :, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    some = total > 0
    p = p.div_(torch.where(some, total, torch.ones_like(total)))
    o = (p @ v).permute(0, 3, 1, 2, 4).reshape(B, n, heads, d).to(st["o"].dtype)
    lse = (m + torch.log(total)).view(B, heads, n)
    st["o"] = torch.where(row[:, :, None, None], o, st["o"])
    st["lse"] = torch.where(row[:, None, :], lse, st["lse"])
    if case["weights"]:
        w = (p * row[:, None, None, :, None]).sum((2, 3)).view(B, hkv, nb_cap, tile).sum(-1)
        tiles = (st["len"] + st["n_new"].view(B, 1) + tile - 1) // tile
        used = (torch.arange(nb_cap, device=w.device) < tiles[..., None]) & (st["n_new"] > 0).view(B, 1, 1)
        st["weight"] = torch.where(used, w, st["weight"])


def _evict(st):
    case, dev = st["case"], st["len"].device
    tile, sink, recent = case["tile"], case["sink"], case["recent"]
    keep = torch.tensor(st["keep"], device=dev).view(1, -1, 1)
    tiles = ((st["len"].long() + tile - 1) // tile)[..., None]
    at = torch.arange(st["table"].shape[-1], device=dev)
    leaves = tiles > keep
    middle = (at >= sink) & (at < tiles - recent) & leaves
    key = torch.where(middle, st["weight"], torch.full_like(st["weight"], -1.0))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order).contiguous())
    gone = middle & (rank >= keep - sink - recent)
    stay = torch.where(gone, 1, torch.where(at < tiles, 0, 2))
    order = torch.sort(stay, dim=-1, stable=True).indices
    out = {x: st[x].gather(-1, order) for x in ("table", "pos", "k_scale", "v_scale", "weight")}
    out["len"] = (st["len"] - tile * gone.sum(-1)).to(torch.int32)
    return out


def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        import block_sparse_attention_24_b200 as V
        c = state["cache"]
        if op == "append":
            V.veda_kv_append(c, state["k"], state["v"], n_new=state["n_new"])
        elif op == "attend":
            V.veda_kv_attn(c, state["q"], state["o"], case["d"] ** -0.5, causal=case["causal"], window=case["window"],
                           sinks=case["sinks"], n_new=state["n_new"], lse=state["lse"],
                           weight=c.weight if case["weights"] else None, decay=0.0, ws=state["ws"])
        else:
            V.veda_kv_evict(c, state["keep"], case["sink"], case["recent"], out=state["out"])
            e = state["out"]
            return {x: getattr(e, x) for x in ("table", "pos", "k_scale", "v_scale", "weight", "len")}
    elif op == "append":
        _append(state)
    elif op == "attend":
        _attend(state)
    else:
        return _evict(state)
    if op == "append":
        return {x: state[x] for x in ("k8", "v8", "k_scale", "v_scale", "pos", "weight")}
    return {"o": state["o"], "lse": state["lse"], **({"weight": state["weight"]} if case["weights"] else {})}


# ------------------------------------------------------------------- work

def work(case):
    B, hkv, d, tile, n, op = case["B"], case["hkv"], case["d"], case["tile"], case.get("n", 0), case["op"]
    lens, news = _lengths(case)
    if op == "append":  # bf16 in, codes out
        return {"bytes": sum(news) * hkv * d * 2 * (2 + 1), "flops": 0}
    if op == "evict":   # five words of each entry in and out
        return {"bytes": sum(-(-a // tile) for a in lens) * hkv * 5 * 4 * 2, "flops": 0}
    nbytes = flops = 0
    for a, m in zip(lens, news):
        if not m:
            continue
        w, sinks = case["window"], case["sinks"]

        def pairs(i):       # keys that query i sees (evicted positions aside)
            hi = a + i + 1 if case["causal"] else a + m
            lo = max(0, a + i - w + 1) if w > 0 else 0
            return hi - lo + min(lo, sinks if w > 0 else 0)

        keys = a + m - (max(0, a - w + 1 - sinks) if w > 0 else 0)
        flops += 4 * d * case["heads"] * m * (pairs(0) + pairs(m - 1)) / 2
        nbytes += hkv * keys * d * 2 + m * case["heads"] * (d * 4 + 4)
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """From the definitions, one (sequence, head) at a time, in float64."""
    st = prepare(case, seed)
    op, tile, d = case["op"], case["tile"], case["d"]
    lens, news = _lengths(case)
    if op == "evict":
        return _exact_evict(case, st)
    if op == "append":
        return _exact_append(case, st, lens, news)
    B, heads, hkv = case["B"], case["heads"], case["hkv"]
    if 4.0 * d * B * heads * case["n"] * (case["len"] + case["n"]) > 1e13:
        return None
    o, lse, weight = st["o"].double(), st["lse"].double(), st["weight"].double()
    g = heads // hkv
    for b in range(B):
        m, total = news[b], lens[b] + news[b]
        if m == 0:
            continue
        for h in range(hkv):
            tiles = -(-total // tile)
            slot = st["table"][b, h, :tiles].long()
            keys = (st["k8"][slot].double() * st["k_scale"][b, h, :tiles, None, None].double()).reshape(-1, d)[:total]
            vals = (st["v8"][slot].double() * st["v_scale"][b, h, :tiles, None, None].double()).reshape(-1, d)[:total]
            at = (st["pos"][b, h, :tiles, None].long() + torch.arange(tile, device="cuda")).reshape(-1)[:total]
            w = torch.zeros(tiles * tile, dtype=torch.float64, device="cuda")
            for j in range(h * g, h * g + g):
                logits = st["q"][b, :m, j].double() @ keys.t() / d ** 0.5
                t = int(st["next_pos"][b]) + torch.arange(m, device="cuda")[:, None]
                hidden = torch.zeros_like(logits, dtype=torch.bool)
                if case["causal"]:
                    hidden |= at > t
                if case["window"] > 0:
                    hidden |= (at <= t - case["window"]) & (at >= case["sinks"])
                logits[hidden] = -float("inf")
                z = torch.logsumexp(logits, -1)
                prob = torch.where(hidden, 0.0, torch.exp(logits - torch.where(torch.isinf(z), 0.0, z)[:, None]))
                lse[b, j, :m] = z
                o[b, :m, j] = prob @ vals
                w[:total] += prob.sum(0)
            weight[b, h, :tiles] = w.view(tiles, tile).sum(-1)
    return {"o": o, "lse": lse, **({"weight": weight} if case["weights"] else {})}


_CODES = None


def _nearest_code(y):
    """The e4m3 value nearest to each of y (|y| <= 448), ties to the even code: by search among all of them."""
    global _CODES
    if _CODES is None:
        mags = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
        _CODES = torch.tensor(mags[:127], dtype=torch.float64, device="cuda")
    a = y.abs().contiguous()
    hi = torch.searchsorted(_CODES, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = _CODES[hi] - a, a - _CODES[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(_CODES[code], y)


def _exact_append(case, st, lens, news):
    tile, hkv = case["tile"], case["hkv"]
    if case["B"] * hkv * (case["n"] // tile + 2) > 20000:
        return None
    got = {"k8": st["k8"].double(), "v8": st["v8"].double(), "k_scale": st["k_scale"].double(),
           "v_scale": st["v_scale"].double(), "pos": st["pos"].clone(), "weight": st["weight"].double()}
    for b in range(case["B"]):
        first, end = lens[b], lens[b] + news[b]
        for i in range(first // tile, -(-end // tile) if news[b] else 0):
            lo, hi = max(first, i * tile), min(end, (i + 1) * tile)
            fresh = lo == i * tile
            slot = st["table"][b, :, i].long()
            for x, codes, scale in (("k", "k8", "k_scale"), ("v", "v8", "v_scale")):
                rows = st[x][b, lo - first:hi - first].double().transpose(0, 1)      # [hkv, rows, d]
                size = rows.abs().amax((1, 2))
                e = torch.ceil(torch.log2(torch.where(size > 0, size, torch.ones_like(size)) / 448)).long()
                e = torch.where(size > 0, e, -40).clamp(min=-40)
                s = 2.0 ** e.double()
                if not fresh:
                    was = got[scale][b, :, i]
                    s = torch.maximum(s, was)
                    keep = got[codes][slot, :lo - i * tile]
                    got[codes][slot, :lo - i * tile] = _nearest_code(keep * (was / s)[:, None, None])
                got[codes][slot, lo - i * tile:hi - i * tile] = _nearest_code(rows / s[:, None, None])
                got[codes][slot, hi - i * tile:] = 0.0
                got[scale][b, :, i] = s
            if fresh:
                got["pos"][b, :, i] = int(st["next_pos"][b]) + lo - first
                got["weight"][b, :, i] = 0.0
    return got


def _exact_evict(case, st):
    tile, sink, recent = case["tile"], case["sink"], case["recent"]
    host = {x: st[x].cpu() for x in ("table", "pos", "k_scale", "v_scale", "weight", "len")}
    got = {x: host[x].clone() for x in host}
    for b in range(case["B"]):
        for h in range(case["hkv"]):
            tiles, keep = -(-int(host["len"][b, h]) // tile), st["keep"][h]
            if tiles <= keep:
                continue
            w = host["weight"][b, h].tolist()
            best = sorted(range(sink, tiles - recent), key=lambda i: (-w[i], i))[:keep - sink - recent]
            stay = list(range(sink)) + sorted(best) + list(range(tiles - recent, tiles))
            kept = set(stay)
            order = stay + [i for i in range(tiles) if i not in kept] + list(range(tiles, len(w)))
            for x in ("table", "pos", "k_scale", "v_scale", "weight"):
                got[x][b, h] = host[x][b, h][order]
            got["len"][b, h] = host["len"][b, h] - tile * (tiles - keep)
    return {x: (got[x].double() if got[x].is_floating_point() else got[x]) for x in got}
