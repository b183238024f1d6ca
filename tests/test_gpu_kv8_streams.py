"""Attention over the 8-bit cache where a block of threads streams many tiles: error against the 64-bit
definition with a floor far below the smallest weight that counts, streams over several units and sequences,
long joins, summed weights."""
import math

import pytest
import torch

import bounded_ref as ref


@pytest.fixture(scope="module")
def mka():
    import route_kv_memory_b200 as m
    return m


def codes_of(x, scale, block):
    """e4m3 codes of x [B, H, L, dh] under scales [B, H, blocks]."""
    return (x / scale.repeat_interleave(block, 2)[:, :, :x.shape[2], None]).to(torch.float8_e4m3fn)


def value_of(codes, scale, block):
    """What the codes of one sequence and head stand for, in float64 on the CPU, and each position's scale."""
    s = scale.cpu().double().repeat_interleave(block)[:codes.shape[0]]
    return codes.cpu().double() * s[:, None], s


def attend(mka, c, cache, q, lens, weights=None):
    n = q.shape[1]
    out = torch.full_like(q, 7.0)
    ws = mka.buffer(mka.mka_kv8_attention_workspace_size(c, n, weights is not None))
    ws.fill_(255)
    mka.mka_kv8_attention(c, cache, q, lens, out, weights, ws)
    torch.cuda.synchronize()
    return out


def decode(q, k, v, vs, p, window, sinks, scale, bf16):
    """Query rows q [r, dh] at position p over k, v [L, dh] (float64; vs [L]: V's scales): out, weights [r, L] and the
    bounds of their errors.

    Scores are float32 sums of dh exact products (ds); 2^x is good to 2^-22 and its argument, below 2^7, to
    2^-17; a lane adds up a few hundred positions at most: 2^-15 covers both.  P is rounded to half, 2^-11 of
    itself or 2^-34 of the largest weight times V scale (float32 rows: 2^-22, 2^-45); the output once to its type."""
    j = torch.arange(k.shape[0], device=k.device)
    m = j <= p
    if window:
        m = m & ((j > p - window) | (j < sinks))
    k, v, vs = k[m], v[m], vs[m]
    s = q @ k.T * scale
    w = torch.softmax(s, -1)
    o = w @ v
    ds = (k.shape[1] + 8) * 2.0 ** -24 * (q.abs() @ k.abs().T).amax(-1, keepdim=True) * scale + 2.0 ** -15
    top = (w * vs).amax(-1, keepdim=True)
    e = (2 * ds + (2.0 ** -11 if bf16 else 2.0 ** -22)) * (w @ v.abs())
    e = e + (2.0 ** -34 if bf16 else 2.0 ** -45) * top * (v / vs[:, None]).abs().sum(0)
    e = e + (ref.BF16 if bf16 else 2.0 ** -23) * (o.abs() + e)
    full, bound = (torch.zeros(q.shape[0], len(j), dtype=torch.float64, device=k.device) for _ in range(2))
    full[:, m], bound[:, m] = w, 2 * ds * w
    return o, full, e, bound


def check(mka, c, cache, q, lens, out, units, w0=None, w1=None):
    """The outputs (and added weights) of these (sequence, KV head) pairs."""
    G, n = c.n_q_heads // c.n_kv_heads, q.shape[1]
    scale = c.attn_scale if c.attn_scale > 0 else 1 / math.sqrt(c.d_head)
    for b, g in units:
        L = lens[b]
        k, _ = value_of(cache.tensors[0][b, g, :L].view(torch.float8_e4m3fn), cache.tensors[2][b, g], c.block)
        v, vs = value_of(cache.tensors[1][b, g, :L].view(torch.float8_e4m3fn), cache.tensors[3][b, g], c.block)
        added, slack = torch.zeros(c.max_positions, dtype=torch.float64), torch.zeros(c.max_positions, dtype=torch.float64)
        for i in range(n):
            p = L - n + i
            got = out[b, i, g * G:(g + 1) * G].cpu().double()
            if p < 0:
                assert (got == 0).all()
                continue
            o, w, e, ew = decode(q[b, i, g * G:(g + 1) * G].cpu().double(), k, v, vs, p, c.window, c.sinks, scale,
                                 c.dtype == mka.MKA_BF16)
            assert ((got - o).abs() <= e).all(), f"({b}, {g}) {float(((got - o).abs() / e).max()):.3g} times its bound"
            added[:L] += w.sum(0)
            slack[:L] += ew.sum(0)
        if w0 is not None:
            total = w0[b, g].cpu().double() + added
            far = (w1[b, g].cpu().double() - total).abs()
            assert (far <= slack + 2.0 ** -23 * total.abs()).all(), (b, g)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,G", [(64, 2), (64, 12), (128, 2), (128, 12)])
def test_weights_far_below_the_largest(mka, dtype, dh, G):
    """One position takes all but 1e-5 of the weight, and its V is 0: the output is what the others give.  As many units as
    CTAs, so that a warp's stream is a quarter of a sequence."""
    B, H, L, block = 128, 4, 4096, 64
    c = mka.make_kv8_config(B, L, G * H, H, dh, block=block, dtype=dtype, attn_scale=1 / dh)
    g = torch.Generator("cuda").manual_seed(dh + G)
    ones = torch.ones(B, H, L // block, device="cuda")
    sk, sv = ones * 2.0 ** -8, ones * 2.0 ** -6
    k = 0.25 * torch.randn(B, H, L, dh, generator=g, device="cuda")
    v = torch.randn(B, H, L, dh, generator=g, device="cuda").abs() + 0.125
    k[:, :, 0], v[:, :, 0] = 1.0, 0.0
    cache = mka.kv8_cache(codes_of(k, sk, block), codes_of(v, sv, block), sk, sv)
    q = torch.full((B, 1, G * H, dh), math.log(1e5 * L), device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    out = attend(mka, c, cache, q, lens)
    check(mka, c, cache, q, [L] * B, out, [(0, 0), (1, 3), (63, 2), (127, 3)])
    assert mka.mka_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("L", [400, 70000])  # 400: a unit in a few blocks of threads; 70000: in several hundred
@pytest.mark.parametrize("what", ["query 0", "query 2", "last key"])
def test_summed_weights_beside_a_nan(mka, L, what):
    """A query whose scores are NaN gives NaN to the positions that it sees and nothing to the others: hidden positions
    keep their totals, and those that only other queries see get theirs."""
    B, H, G, dh, n, block, window, sinks = 1, 2, 2, 64, 3, 64, L - 250, 2
    c = mka.make_kv8_config(B, L, G * H, H, dh, block=block, window=window, sinks=sinks)
    g = torch.Generator("cuda").manual_seed(L)
    s = torch.full((B, H, -(-L // block)), 2.0 ** -6, device="cuda")
    cache = mka.kv8_cache(*(codes_of(torch.randn(B, H, L, dh, generator=g, device="cuda"), s, block) for _ in "kv"), s, s.clone())
    q = torch.randn(B, n, G * H, dh, generator=g, device="cuda").to(torch.bfloat16)
    bad = 2  # the query whose scores are NaN
    if what == "last key":
        cache.tensors[0].view(torch.uint8)[:, :, L - 1] = 0x7f
    else:
        bad = int(what[-1])
        q[0, bad] = math.nan
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    w0 = torch.rand(B, H, L, generator=g, device="cuda")
    w1 = w0.clone()
    out = attend(mka, c, cache, q, lens, w1)
    seen = torch.zeros(n, L, dtype=torch.bool)
    for i in range(n):
        p = L - n + i
        seen[i, p - window + 1:p + 1] = True
        seen[i, :sinks] = True
    w1, w0 = w1.cpu(), w0.cpu()
    for h in range(H):
        assert torch.equal(torch.isnan(w1[0, h]), seen[bad])
        assert torch.equal(w1[0, h, ~seen.any(0)], w0[0, h, ~seen.any(0)])
    finite = seen.any(0) & ~seen[bad]
    assert finite.any()
    good = [i for i in range(n) if i != bad]
    assert torch.isnan(out[0, bad]).all() and torch.isfinite(out[0, good]).all()
    # the positions that the NaN query does not see: what the others give
    for h in range(H):
        k, _ = value_of(cache.tensors[0][0, h], s[0, h], block)
        v, vs = value_of(cache.tensors[1][0, h], s[0, h], block)
        k = torch.nan_to_num(k)
        total, slack = w0[0, h].double(), torch.zeros(L, dtype=torch.float64)
        for i in good:
            _, w, _, ew = decode(q[0, i, h * G:(h + 1) * G].cpu().double(), k, v, vs, L - n + i, window, sinks, dh ** -0.5, True)
            total += w.sum(0)
            slack += ew.sum(0)
        far = (w1[0, h].double() - total).abs()
        assert (far <= slack + 2.0 ** -23 * total)[finite].all()
    assert mka.mka_status() == 0


def grown(kind, B, H, L, dh, block, g):
    """A cache's codes and scales.  "plain": blocks of different size; "rising": keys that grow along the sequence, so that
    the softmax's reference moves from tile to tile, and values that shrink; "falling": the other way round."""
    nb = -(-L // block)
    k, v = (torch.randn(B, H, L, dh, generator=g, device="cuda") for _ in "kv")
    at = torch.arange(nb, device="cuda") / nb
    step = {"plain": torch.zeros(nb, device="cuda"), "rising": at, "falling": 1 - at}[kind]
    jump = torch.randint(-1, 2, (2, B, H, nb), generator=g, device="cuda")
    sk = torch.exp2((-7 + torch.floor(3 * step)).expand(B, H, nb) + (jump[0] if kind == "plain" else 0))
    sv = torch.exp2((-7 - torch.floor(6 * step)).expand(B, H, nb) + jump[1])
    wide = lambda s: s.repeat_interleave(block, 2)[:, :, :L, None] * 2.0 ** 6  # noqa: E731
    sk, sv = sk.contiguous(), sv.contiguous()
    return codes_of(k * wide(sk), sk, block), codes_of(v * wide(sv), sv, block), sk, sv


STREAMS = [
    # B, L, Hq, H, dh, block, dtype, window, sinks, n, lens, kind, checked units (None: all)
    # sequences of every length, empty ones between: CTAs go on to the next unit and sequence
    (24, 3000, 16, 8, 128, 64, "bf16", 0, 0, 1, "spread", "plain", 30),
    (24, 3000, 16, 8, 64, 16, "f32", 0, 0, 2, "spread", "plain", 30),
    (24, 3000, 8, 8, 64, 128, "bf16", 0, 0, 3, "spread", "rising", 30),
    (24, 3000, 16, 8, 128, 32, "f32", 0, 0, 1, "spread", "falling", 30),
    # 21 query rows per KV head: two groups of rows, each a unit
    (12, 3000, 28, 4, 128, 64, "bf16", 0, 0, 3, "spread", "rising", 20),
    (24, 3000, 10, 5, 64, 64, "f32", 0, 0, 6, "spread", "plain", 20),
    # windows with sinks: lists of tiles with a gap
    (16, 6000, 16, 8, 64, 32, "bf16", 2500, 200, 3, "spread", "plain", 20),
    (20, 6000, 8, 4, 128, 64, "f32", 2500, 20, 2, "spread", "rising", 20),
    # as many units of a few tiles as CTAs of either residence: units that one CTA streams whole
    (111, 256, 8, 4, 64, 64, "bf16", 0, 0, 1, "near", "plain", 30),
    (37, 640, 24, 8, 128, 64, "bf16", 0, 0, 5, "near", "falling", 30),
    # one unit in more ranges than a CTA's warps join at once (32 records each), and one among many short ones
    (1, 40000, 2, 1, 64, 64, "bf16", 0, 0, 1, "full", "rising", None),
    (1, 40000, 12, 1, 128, 64, "f32", 0, 0, 1, "full", "plain", None),
    (70, 40000, 2, 1, 64, 64, "bf16", 0, 0, 1, "one", "falling", None),
    (70, 40000, 2, 1, 128, 64, "f32", 0, 0, 1, "one", "rising", None),
    (64, 5000, 4, 2, 64, 64, "bf16", 0, 0, 1, "one", "plain", None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("weighed", [False, True])
@pytest.mark.parametrize("case", STREAMS)
def test_streams(mka, case, weighed):
    B, L, Hq, H, dh, block, dtype, window, sinks, n, how, kind, units = case
    lens = {"spread": [0 if b % 5 == 3 else max(1, L - 211 * b % L) for b in range(B)],
            "near": [L - 3 * b % 100 for b in range(B)], "full": [L] * B,
            "one": [L if b == 30 else 1 + b % 2 for b in range(B)]}[how]
    c = mka.make_kv8_config(B, L, Hq, H, dh, block=block, dtype=dtype, window=window, sinks=sinks)
    g = torch.Generator("cuda").manual_seed(L + dh + B)
    cache = mka.kv8_cache(*grown(kind, B, H, L, dh, block, g))
    for b in range(B):  # rows behind a sequence's end hold NaN
        for t in cache.tensors[:2]:
            t.view(torch.uint8)[b, :, lens[b]:] = 0x7f
    q = torch.randn(B, n, Hq, dh, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w0 = torch.rand(B, H, L, generator=g, device="cuda") if weighed else None
    w1 = w0.clone() if weighed else None
    out = attend(mka, c, cache, q, at, w1)
    pairs = [(b, h) for b in range(B) for h in range(H)]
    if units:  # the longest and the last ones, and others spread over the batch
        pairs = pairs[::-(-len(pairs) // units)] + [pairs[-1]]
    check(mka, c, cache, q, lens, out, pairs, w0, w1)
    assert not torch.isnan(out).any()
    again = w0.clone() if weighed else None
    assert torch.equal(out, attend(mka, c, cache, q, at, again))  # sums in a fixed order
    assert not weighed or torch.equal(again, w1)
    assert mka.mka_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,L,keep", [(3, 1, 50001, 700), (1, 2, 32769, 32000), (2, 4, 16384, 16383), (9, 4, 131072, 999),
                                        (2, 1, 131073, 5000), (5, 30, 16385, 64)])
@pytest.mark.parametrize("ties", [False, True])
def test_kept_positions_of_every_cluster_size(mka, B, H, L, keep, ties):
    """One to eight blocks of threads a head, shares that end inside a warp's, more clusters than the card holds."""
    dh, first, recent = 64, 3, 21
    c, c2 = mka.make_kv8_config(B, L, H, H, dh), mka.make_kv8_config(B, keep, H, H, dh)
    empty = lambda n: mka.kv8_cache(*(torch.zeros(B, H, n, dh, dtype=torch.uint8, device="cuda") for _ in "kv"),  # noqa: E731
                                    *(torch.ones(B, H, -(-n // 64), device="cuda") for _ in "kv"))
    cache, d = empty(L), empty(keep)
    g = torch.Generator("cuda").manual_seed(L + keep)
    w = torch.rand(B, H, L, generator=g, device="cuda")
    if ties:
        w = torch.floor(4 * w) / 4
    lens = torch.tensor([L - 1201 * b % L for b in range(B)], dtype=torch.int32, device="cuda")
    lens2, kept = torch.zeros_like(lens), torch.full((B, H, keep), -7, dtype=torch.int32, device="cuda")
    w2 = torch.full((B, H, keep), -9.0, device="cuda")
    mka.mka_kv8_evict(c, cache, lens, w, keep, first, recent, c2, d, lens2, w2, kept,
                      mka.buffer(mka.mka_kv8_evict_workspace_size(c, keep)))
    assert mka.mka_status() == 0 and torch.equal(lens2, lens.clamp_max(keep))
    at = torch.arange(L, device="cuda")
    for b in range(B):
        n = int(lens[b])
        forced = (at < first) | (at >= n - recent)
        order = w[b].double().masked_fill(forced, math.inf).masked_fill(at >= n, -math.inf).sort(dim=-1, descending=True, stable=True)[1]
        want = order[:, :min(keep, n)].sort(-1)[0]
        assert torch.equal(kept[b, :, :want.shape[1]].long(), want) and (kept[b, :, want.shape[1]:] == -1).all()
        assert torch.equal(w2[b, :, :want.shape[1]], w[b].gather(1, want)) and (w2[b, :, want.shape[1]:] == -9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,n", [(1, 1), (1, 3), (2, 1)])
def test_strides_of_single_rows_do_not_matter(mka, B, n):
    """K and V that differ in nothing but the stride of a dimension of size 1 are rows of the same places."""
    H, dh = 2, 64
    c = mka.make_kv8_config(B, 40, 4, H, dh, block=16)
    g = torch.Generator("cuda").manual_seed(3)
    k = torch.randn(B, n, H, dh, generator=g, device="cuda").bfloat16()
    v = torch.randn(B, n, H, dh, generator=g, device="cuda").bfloat16()
    st = list(v.stride())
    if B == 1:
        st[0] += 4096
    if n == 1:
        st[1] += 512
    odd = v.as_strided(v.shape, st)
    assert odd.stride() != k.stride() and torch.equal(odd, v)
    got = []
    for x in (v, odd):
        cache = mka.kv8_cache(*(torch.zeros(B, H, 40, dh, dtype=torch.uint8, device="cuda") for _ in "kv"),
                              *(torch.ones(B, H, 3, device="cuda") for _ in "kv"))
        mka.mka_kv8_append(c, cache, k, x, torch.zeros(B, dtype=torch.int32, device="cuda"))
        ko, vo = torch.zeros_like(k), torch.zeros_like(k).as_strided(k.shape, st)
        mka.mka_kv8_read(c, cache, None, None, ko, vo)
        got.append([t.clone() for t in cache.tensors] + [ko, vo])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got[0][:4], got[1][:4]))
    assert torch.equal(got[0][4], got[1][4]) and torch.equal(got[0][5], got[1][5]) and bool(got[0][5].any())
    with pytest.raises(ValueError, match="same"):
        wide = torch.zeros(2, 3, 2 * H, dh, device="cuda").bfloat16()[:, :, :H]
        c2 = mka.make_kv8_config(2, 40, 4, H, dh, block=16)
        cache = mka.kv8_cache(*(torch.zeros(2, H, 40, dh, dtype=torch.uint8, device="cuda") for _ in "kv"),
                              *(torch.ones(2, H, 3, device="cuda") for _ in "kv"))
        mka.mka_kv8_append(c2, cache, wide, wide.contiguous(), torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert mka.mka_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** -114, 2.0 ** 112])
@pytest.mark.parametrize("L", [100, 3000, 70000])  # one tile, whole and split units
def test_values_near_the_ends_of_the_range(mka, dtype, size, L):
    """V whose block scales are near the smallest and the largest, under nearly equal weights: the factor of the whole row is
    then near the ends of float32's range too."""
    H, dh, block = 2, 64, 16
    c = mka.make_kv8_config(1, L, H, H, dh, block=block, dtype=dtype, attn_scale=2.0 ** -10)
    g = torch.Generator("cuda").manual_seed(L)
    nb = -(-L // block)
    k, v = (torch.randn(1, H, L, dh, generator=g, device="cuda") for _ in "kv")
    sk, sv = (torch.full((1, H, nb), 2.0 ** -6, device="cuda") for _ in "kv")
    kc, vc = codes_of(k, sk, block), codes_of(v.abs(), sv, block)
    cache = mka.kv8_cache(kc, vc, sk, sv * size)
    q = torch.randn(1, 1, H, dh, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    out = attend(mka, c, cache, q, torch.full((1,), L, dtype=torch.int32, device="cuda"))
    check(mka, c, cache, q, [L], out, [(0, h) for h in range(H)])
    assert mka.mka_status() == 0
