"""The 8-bit K/V cache on the GPU against its definition: appending (exact), reading, attention with
windows, drafts, float32 and bf16 rows and summed weights, eviction (exact), and a run of them together."""
import ctypes
import math

import pytest
import torch

import bounded_ref as ref


@pytest.fixture(scope="module")
def mka():
    import route_kv_memory_b200 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def new_cache(mka, c, fill=0x7f, dev="cuda"):
    """A cache whose unused codes are NaN and whose unused scales are NaN."""
    B, H, L, dh = c.batch, c.n_kv_heads, c.max_positions, c.d_head
    codes = [torch.full((B, H, L, dh), fill, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.full((B, H, -(-L // c.block)), float("nan"), device=dev) for _ in range(2)]
    return mka.kv8_cache(*codes, *scales)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def row_dtype(c, mka):
    return torch.bfloat16 if c.dtype == mka.MKA_BF16 else torch.float32


def read(mka, c, cache, lens, n=None, first=None):
    n = max(max(lens), 1) if n is None else n
    out = [torch.full((c.batch, n, c.n_kv_heads, c.d_head), 7.0, dtype=row_dtype(c, mka), device="cuda") for _ in range(2)]
    mka.mka_kv8_read(c, cache, None if first is None else ints(first), ints(lens), *out)
    torch.cuda.synchronize()
    return [x.cpu().double() for x in out]


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def check_cache(mka, c, cache, models, lens):
    """models[kv][b][g]: ref.Cache."""
    got = read(mka, c, cache, lens)
    for kv in range(2):
        for b in range(c.batch):
            for g in range(c.n_kv_heads):
                m, n = models[kv][b][g], lens[b]
                if n:
                    want = m.x[:n].to(row_dtype(c, mka)).double()
                    assert same(got[kv][b, :n, g], want), (kv, b, g)
                    sc = cache.tensors[2 + kv][b, g].cpu()
                    for tb in range(-(-n // c.block)):
                        assert float(sc[tb]) == m.scale[tb], (kv, b, g, tb)
            assert (got[kv][b, lens[b]:] == 7.0).all()


def models_of(c):
    return [[[ref.Cache(c.block) for _ in range(c.n_kv_heads)] for _ in range(c.batch)] for _ in range(2)]


def append(mka, c, cache, models, kn, vn, pos, count=None):
    mka.mka_kv8_append(c, cache, kn.cuda(), vn.cuda(), ints(pos), None if count is None else ints(count))
    for kv, x in enumerate((kn, vn)):
        for b in range(c.batch):
            n = x.shape[1] if count is None else count[b]
            for g in range(c.n_kv_heads):
                if n:
                    models[kv][b][g].append(pos[b], x[b, :n, g])


# ---------------------------------------------------------------- append and read
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,block", [(64, 16), (128, 32), (64, 128), (128, 64), (128, 128)])
def test_append_in_pieces(mka, dtype, dh, block):
    """Ragged pieces of growing and shrinking size of values: scales grow inside a block, codes are re-rounded."""
    B, H, L = 3, 2, 300
    c = mka.make_kv8_config(B, L, 4, H, dh, block=block, dtype=dtype)
    cache, models, g, pos = new_cache(mka, c), models_of(c), gen(dh + block), [0, 0, 0]
    for step, (n, count) in enumerate([(70, [70, 1, 33]), (1, None), (1, [1, 0, 1]), (130, [130, 64, 7]), (3, [0, 3, 2])]):
        x = [torch.randn(B, n, H, dh, generator=g) * 2.0 ** (3 * step - 4) for _ in range(2)]
        x = [t.to(row_dtype(c, mka)) for t in x]
        append(mka, c, cache, models, *x, pos, count)
        pos = [p + (n if count is None else count[b]) for b, p in enumerate(pos)]
        check_cache(mka, c, cache, models, pos)
    # going back inside a block: the rows behind are dropped, the scale of the rows in front stays
    back = [max(0, p - 5) for p in pos]
    x = [(torch.randn(B, 2, H, dh, generator=g) / 1024).to(row_dtype(c, mka)) for _ in range(2)]
    append(mka, c, cache, models, *x, back)
    check_cache(mka, c, cache, models, [p + 2 for p in back])
    assert mka.mka_status() == 0


@pytest.mark.gpu
def test_append_of_special_values(mka):
    """NaN and infinities are stored as NaN outside the scale; zeros, the smallest and the largest floats."""
    c = mka.make_kv8_config(1, 64, 1, 1, 64, block=16, dtype="f32")
    x = torch.randn(1, 64, 1, 64, generator=gen(1))
    x[0, 3, 0, 5], x[0, 4, 0, 6], x[0, 5, 0, 7] = math.nan, math.inf, -math.inf
    x[0, 16:32] = 0
    x[0, 32:48] *= 2.0 ** -140  # denormal
    x[0, 48:64] = torch.finfo(torch.float32).max * torch.sign(x[0, 48:64])
    cache, models = new_cache(mka, c), models_of(c)
    append(mka, c, cache, models, x, x.flip(1).contiguous(), [0])
    check_cache(mka, c, cache, models, [64])
    # values on rounding borders: halfway between codes, and at the edge of a scale (448 and the next float)
    y = torch.zeros(1, 16, 1, 64)
    y[0, 0, 0, :32] = torch.arange(32) / 16 + 1 / 32 + 16
    y[0, 0, 0, 32] = 448.0
    append(mka, c, cache, models, y, y * (1 + 2.0 ** -20), [0])
    check_cache(mka, c, cache, models, [16])
    assert mka.mka_status() == 0


@pytest.mark.gpu
def test_scales_that_jump(mka):
    """Codes re-rounded to scales 2^1 .. 2^60 as large on append, and 2^1 .. 2^18 as small on eviction."""
    c = mka.make_kv8_config(1, 64 * 16, 1, 1, 64, block=16, dtype="f32")
    c2 = mka.make_kv8_config(1, 15 * 64, 1, 1, 64, block=16, dtype="f32")
    g = gen(9)
    cache, models = new_cache(mka, c), models_of(c)
    for tb in range(64):  # 15 rows of codes of every size, then one row 2^tb times the block's scale
        x = torch.randn(1, 15, 1, 64, generator=g) * torch.exp2(torch.randint(-9, 1, (1, 15, 1, 64), generator=g) * 1.0)
        append(mka, c, cache, models, x, x.neg(), [16 * tb])
        check_cache(mka, c, cache, models, [16 * tb + 15])
        y = torch.randn(1, 1, 1, 64, generator=g) * 2.0 ** (tb if tb < 40 else tb - 40)
        append(mka, c, cache, models, y, y, [16 * tb + 15])
    check_cache(mka, c, cache, models, [64 * 16])
    w = torch.ones(1, 1, 64 * 16)
    w[0, 0, 15::16] = 0  # the large rows go
    check_evict(mka, c, models, [64 * 16], w, 15 * 64, 0, 0, c2, evict(mka, c, cache, [64 * 16], w, 15 * 64, 0, 0, c2))


@pytest.mark.gpu
def test_append_past_the_end_and_before_the_start(mka):
    c = mka.make_kv8_config(3, 40, 1, 1, 64, block=16)
    cache, models = new_cache(mka, c), models_of(c)
    x = torch.randn(3, 20, 1, 64, generator=gen(2)).to(torch.bfloat16)
    append(mka, c, cache, models, x, x, [0, 0, 0])
    before = [t.clone() for t in cache.tensors]
    mka.mka_kv8_append(c, cache, x.cuda(), x.cuda(), ints([21, -1, 5]), ints([20, 3, 0]))
    assert mka.mka_status() in (mka.MKA_ERR_CAPACITY, mka.MKA_ERR_DEVICE_BOUNDS)
    for t, s in zip(cache.tensors, before):
        assert torch.equal(t.view(torch.uint8), s.view(torch.uint8))
    mka.mka_kv8_append(c, cache, x.cuda(), x.cuda(), ints([21, 20, 20]), ints([20, 20, 20]))
    assert mka.mka_status() == mka.MKA_ERR_CAPACITY
    for b in (1, 2):
        for kv in range(2):
            models[kv][b][0].append(20, x[b, :, 0])
    check_cache(mka, c, cache, models, [20, 40, 40])
    out = [torch.full((3, 8, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    mka.mka_kv8_read(c, cache, ints([39, -1, 32]), ints([2, 1, 8]), *out)
    assert mka.mka_status() == mka.MKA_ERR_DEVICE_BOUNDS
    assert (out[0][:2] == 7.0).all() and torch.equal(out[0][2, :, 0].cpu().double(), models[0][2][0].x[32:40])


@pytest.mark.gpu
def test_strided_rows(mka):
    """K and V as column ranges of a packed tensor and as rows of a longer one, in and out."""
    B, n, H, dh = 2, 21, 2, 64
    c = mka.make_kv8_config(B, 64, 4, H, dh, block=16)
    packed = torch.randn(B, 50, 3, H * dh, generator=gen(3)).to(torch.bfloat16).cuda()
    k, v = packed[:, 5:5 + n, 0], packed[:, 5:5 + n, 2]
    cache, models = new_cache(mka, c), models_of(c)
    mka.mka_kv8_append(c, cache, k, v, ints([0, 0]))
    for kv, x in enumerate((k, v)):
        for b in range(B):
            for g in range(H):
                models[kv][b][g].append(0, x[b, :, g * dh:(g + 1) * dh].cpu())
    check_cache(mka, c, cache, models, [n, n])
    wide = torch.zeros(B, 30, 2, H * dh, dtype=torch.bfloat16, device="cuda")
    mka.mka_kv8_read(c, cache, ints([2, 0]), ints([19, 4]), wide[:, :, 0], wide[:, :, 1])
    for b, (a, m) in enumerate([(2, 19), (0, 4)]):
        for kv in range(2):
            got = wide[b, :m, kv].cpu().double()
            assert torch.equal(got, torch.cat([models[kv][b][g].x[a:a + m] for g in range(H)], -1))
    assert (wide[0, 19:] == 0).all() and (wide[1, 4:] == 0).all()


# ---------------------------------------------------------------- attention
def attend(mka, c, cache, models, q, lens, weights=None):
    out = torch.full_like(q, 7.0, device="cuda")
    n = q.shape[1]
    ws = mka.buffer(mka.mka_kv8_attention_workspace_size(c, n, weights is not None))
    ws.fill_(255)
    mka.mka_kv8_attention(c, cache, q.cuda(), ints(lens), out, weights, ws)
    torch.cuda.synchronize()
    return out.cpu()


def check_attention(mka, c, models, q, lens, out, w0=None, w1=None):
    G, bf = c.n_q_heads // c.n_kv_heads, c.dtype == mka.MKA_BF16
    scale = c.attn_scale if c.attn_scale > 0 else 1 / math.sqrt(c.d_head)
    for b in range(c.batch):
        for g in range(c.n_kv_heads):
            total = None if w0 is None else w0[b, g].double()
            for i in range(q.shape[1]):
                p = lens[b] - q.shape[1] + i
                got = out[b, i, g * G:(g + 1) * G].double()
                if p < 0:
                    assert (got == 0).all()
                    continue
                k, v = models[0][b][g].x[:lens[b]], models[1][b][g].x[:lens[b]]
                o, w, e = ref.decode(q[b, i, g * G:(g + 1) * G].double(), k, v, models[1][b][g].scales()[:lens[b]], p,
                                     c.window, c.sinks, scale, bf)
                assert ((got - o).abs() <= e).all(), f"{float(((got - o).abs() / e).max()):.3g} times its bound"
                if total is not None:
                    total[:lens[b]] += w.sum(0)
            if total is not None:
                # float32: weights of relative error 2 ds (see ref.decode) <= 2^-12, added up, and one rounding
                far = (w1[b, g].double() - total).abs()
                assert (far <= 2.0 ** -12 * (total - w0[b, g].double()).abs() + 2.0 ** -23 * total.abs()).all()


ATTN = [
    # B, Lmax, Hq, Hkv, dh, block, dtype, window, sinks, n, lens
    (1, 1, 1, 1, 64, 16, "bf16", 0, 0, 1, [1]),
    (2, 40, 4, 2, 64, 16, "f32", 0, 0, 1, [40, 0]),
    (1, 1000, 4, 2, 64, 32, "f32", 0, 0, 1, [1000]),
    (3, 700, 7, 1, 128, 64, "bf16", 0, 0, 1, [700, 129, 128]),
    (2, 515, 8, 2, 128, 128, "bf16", 0, 0, 4, [515, 3]),
    (2, 300, 28, 4, 128, 64, "bf16", 0, 0, 3, [300, 257]),
    (2, 300, 12, 1, 128, 32, "f32", 0, 0, 2, [299, 31]),
    (2, 600, 4, 2, 64, 16, "bf16", 100, 4, 1, [600, 90]),
    (2, 600, 4, 1, 128, 64, "f32", 130, 33, 5, [600, 250]),
    (1, 900, 32, 8, 128, 64, "bf16", 1, 0, 1, [900]),
    (2, 900, 4, 4, 64, 64, "bf16", 257, 140, 8, [900, 410]),
    (5, 260, 16, 2, 64, 16, "bf16", 0, 0, 1, [0, 260, 1, 17, 128]),
    (1, 2100, 6, 3, 128, 128, "bf16", 0, 0, 1, [2100]),
    (1, 300, 28, 4, 128, 64, "bf16", 0, 0, 20, [300]),    # 140 query rows per KV head
    (2, 200, 20, 1, 64, 32, "f32", 64, 2, 1, [200, 150]),  # 20 query heads on one KV head
    (150, 70, 2, 1, 64, 16, "bf16", 0, 0, 1, [(7 * i) % 71 for i in range(150)]),  # more sequences than threads
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ATTN)
@pytest.mark.parametrize("weighed", [False, True])
def test_attention_against_definition(mka, case, weighed):
    B, L, Hq, H, dh, block, dtype, window, sinks, n, lens = case
    c = mka.make_kv8_config(B, L, Hq, H, dh, block=block, dtype=dtype, window=window, sinks=sinks)
    g, cache, models = gen(L + dh), new_cache(mka, c), models_of(c)
    x = [torch.randn(B, max(lens), H, dh, generator=g) for _ in range(2)]
    for t in x:  # blocks of different size
        t *= torch.exp2(torch.randint(-3, 4, (B, max(lens), 1, 1), generator=g) // 2 * 1.0)
    append(mka, c, cache, models, *(t.to(row_dtype(c, mka)) for t in x), [0] * B, lens)
    q = torch.randn(B, n, Hq, dh, generator=g).to(row_dtype(c, mka))
    w0 = torch.rand(B, H, L, generator=g) if weighed else None
    w1 = w0.cuda() if weighed else None
    out = attend(mka, c, cache, models, q, lens, w1)
    check_attention(mka, c, models, q, lens, out, w0, w1.cpu() if weighed else None)
    assert torch.equal(out, attend(mka, c, cache, models, q, lens, w0.cuda() if weighed else None))
    assert mka.mka_status() == 0


@pytest.mark.gpu
def test_nan_in_hidden_and_in_seen_positions(mka):
    """NaN codes behind the window and past a query's position reach nothing; a seen NaN in one channel of V
    reaches that channel of the queries that see it, one in K every channel of them."""
    B, L, H, dh, n = 1, 400, 1, 64, 3
    c = mka.make_kv8_config(B, L, 2, H, dh, block=16, window=150, sinks=2)
    g, cache, models = gen(6), new_cache(mka, c), models_of(c)
    x = [torch.randn(B, L, H, dh, generator=g).to(torch.bfloat16) for _ in range(2)]
    for t in x:
        t[:, 2:200] = math.nan  # behind every window
    x[0][0, 399, 0, 3] = math.nan  # K of the last token: seen by the last query alone
    append(mka, c, cache, models, *x, [0])
    q = torch.randn(B, n, 2, dh, generator=g).to(torch.bfloat16)
    out = attend(mka, c, cache, models, q, [L])
    assert torch.isnan(out[0, 2]).all() and torch.isfinite(out[0, :2]).all()
    x[0][0, 399, 0, 3] = 1.0
    x[1][0, 398, 0, 5] = math.nan  # V of the last but one: channel 5 of the last two queries
    x[1][0, 399, 0, 63] = math.inf
    append(mka, c, cache, models, *x, [0])
    out = attend(mka, c, cache, models, q, [L])
    want = torch.zeros(n, 2, dh, dtype=torch.bool)
    want[1:, :, 5] = True
    want[2, :, 63] = True
    assert torch.equal(torch.isnan(out[0]), want)
    clean = [t.clone() for t in x]
    clean[1][0, 398, 0, 5] = clean[1][0, 399, 0, 63] = 0.0
    for t in clean:
        t[:, 2:200] = 0.0
    models2 = models_of(c)
    append(mka, c, cache, models2, *clean, [0])
    out2 = attend(mka, c, cache, models2, q, [L])
    check_attention(mka, c, models2, q, [L], out2)
    check_attention(mka, c, models2, q[:, :1], [L - 2], out[:, :1])


@pytest.mark.gpu
def test_block_scales_far_apart(mka):
    """V blocks whose scales differ by 2^40, the large ones at tokens of almost no weight and the other way round."""
    L, dh = 512, 64
    for big in (0, 1):
        c = mka.make_kv8_config(1, L, 2, 1, dh, block=32)
        g, cache, models = gen(big), new_cache(mka, c), models_of(c)
        k, v, q = torch.randn(1, L, 1, dh, generator=g), torch.randn(1, L, 1, dh, generator=g), torch.randn(1, 1, 2, dh, generator=g)
        v[0, 64:96] *= 2.0 ** 20
        v[0, 256:288] *= 2.0 ** -20
        k[0, 64:96] = (8 if big else -8) * q[0, 0, 0]
        q[0, 0, 1] = q[0, 0, 0] * 0.9
        k, v, q = (t.to(torch.bfloat16) for t in (k, v, q))
        append(mka, c, cache, models, k, v, [0])
        check_attention(mka, c, models, q, [L], attend(mka, c, cache, models, q, [L]))


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
def test_queries_of_any_size(mka, size):
    """Queries far outside the range of half precision."""
    c = mka.make_kv8_config(1, 200, 2, 1, 64, block=16, attn_scale=1 / (8 * size), dtype="f32")
    g, cache, models = gen(11), new_cache(mka, c), models_of(c)
    x = [torch.randn(1, 200, 1, 64, generator=g) for _ in range(2)]
    append(mka, c, cache, models, *x, [0])
    q = torch.randn(1, 1, 2, 64, generator=g) * size
    check_attention(mka, c, models, q, [200], attend(mka, c, cache, models, q, [200]))


# ---------------------------------------------------------------- eviction
def evict(mka, c, cache, lens, w, keep, first, recent, c2):
    d = new_cache(mka, c2)
    lens2, kept = ints([-5] * c.batch), torch.full((c.batch, c.n_kv_heads, keep), -7, dtype=torch.int32, device="cuda")
    w2 = torch.full((c.batch, c.n_kv_heads, c2.max_positions), -9.0, device="cuda")
    ws = mka.buffer(mka.mka_kv8_evict_workspace_size(c, keep))
    ws.fill_(255)
    mka.mka_kv8_evict(c, cache, ints(lens), w.cuda(), keep, first, recent, c2, d, lens2, w2, kept, ws)
    torch.cuda.synchronize()
    return d, lens2.tolist(), w2.cpu(), kept.cpu()


def check_evict(mka, c, models, lens, w, keep, first, recent, c2, got):
    d, lens2, w2, kept = got
    models2 = models_of(c2)
    assert lens2 == [min(n, keep) for n in lens]
    for b in range(c.batch):
        for g in range(c.n_kv_heads):
            pick = ref.keep_positions(w[b, g].tolist(), lens[b], keep, first, recent)
            assert kept[b, g].tolist() == pick + [-1] * (keep - len(pick))
            assert same(w2[b, g, :len(pick)].double(), w[b, g, pick].double()) and (w2[b, g, len(pick):] == -9).all()
            for kv in range(2):
                if pick:
                    models2[kv][b][g].append(0, models[kv][b][g].x[pick])
    check_cache(mka, c2, d, models2, lens2)
    return models2


@pytest.mark.gpu
@pytest.mark.parametrize("L,lens,keep,first,recent,block,block2,kind", [
    (300, [300, 100, 99, 0], 100, 4, 30, 16, 64, "random"), (300, [300, 101, 300, 1], 100, 0, 0, 64, 16, "ties"),
    (200, [200, 150, 3, 200], 64, 30, 34, 32, 32, "random"), (130, [130, 129, 130, 130], 129, 1, 100, 128, 128, "ties"),
    (2500, [2500, 1024, 1025, 2049], 1024, 4, 100, 64, 64, "few"), (90, [90, 88, 50, 2], 1, 0, 0, 16, 16, "special"),
    (90, [90, 88, 50, 2], 1, 1, 0, 16, 16, "random"), (3000, [3000, 2999, 5, 1500], 700, 2, 3, 64, 128, "special"),
])
def test_evict(mka, L, lens, keep, first, recent, block, block2, kind):
    B, H, dh = 4, 2, 64
    c = mka.make_kv8_config(B, L, 4, H, dh, block=block)
    c2 = mka.make_kv8_config(B, keep + 7, 4, H, dh, block=block2)
    g, cache, models = gen(L + keep), new_cache(mka, c), models_of(c)
    x = [(torch.randn(B, L, H, dh, generator=g) * torch.exp2(torch.randint(-6, 7, (B, L, 1, 1), generator=g) * 1.0)).to(
        torch.bfloat16) for _ in range(2)]
    append(mka, c, cache, models, *x, [0] * B, lens)
    w = torch.rand(B, H, L, generator=g)
    if kind == "ties":
        w = torch.randint(0, 3, (B, H, L), generator=g) * 0.5
    if kind == "few":
        w = torch.where(w < 0.9, 1e-30 * torch.ones(()), w)
    if kind == "special":
        w[..., ::3], w[..., 1::7], w[..., 2::11], w[..., 4::13] = 0.0, -0.0, math.inf, -1.0
        w[..., 5::17] = math.nan
    check_evict(mka, c, models, lens, w, keep, first, recent, c2, evict(mka, c, cache, lens, w, keep, first, recent, c2))
    assert mka.mka_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,keep", [(2, 9000, 8000), (1, 20000, 1234), (1, 70001, 40000), (1, 262144, 300),
                                      (1, 270000, 2000), (40, 9000, 60)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_long(mka, B, L, keep, ties):
    """Several CTAs per head, keys in few and many registers and read again; the order over warps and CTAs."""
    dh = 64
    c, c2 = mka.make_kv8_config(B, L, 1, 1, dh), mka.make_kv8_config(B, keep, 1, 1, dh)
    g = gen(L)
    codes = [torch.randint(0, 0x7f, (B, 1, L, dh), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    sc = [torch.exp2(torch.randint(-3, 4, (B, 1, -(-L // 64)), generator=g) * 1.0).cuda() for _ in range(2)]
    cache = mka.kv8_cache(*codes, *sc)
    w = torch.rand(B, 1, L, generator=g)
    if ties:
        w = torch.randint(0, 2, (B, 1, L), generator=g) * 0.25 + (torch.rand(B, 1, L, generator=g) < keep / L / 3)
    lens = [L - 37 * b for b in range(B)]
    d, lens2, w2, kept = evict(mka, c, cache, lens, w, keep, 3, 20, c2)
    assert lens2 == [keep] * B
    got = read(mka, c2, d, lens2)
    for b in range(B):
        pick = torch.tensor(ref.keep_positions(w[b, 0].tolist(), lens[b], keep, 3, 20))
        assert torch.equal(kept[b, 0].long(), pick) and torch.equal(w2[b, 0], w[b, 0, pick])
        for kv in range(2):
            x = codes[kv][b, 0].view(torch.float8_e4m3fn).cpu()[pick].double() * sc[kv][b, 0].cpu().double()[pick // 64, None]
            m = ref.Cache(64)
            m.append(0, x)
            assert torch.equal(got[kv][b, :, 0], m.x)


# ---------------------------------------------------------------- together
@pytest.mark.gpu
def test_prompt_decode_evict_decode(mka):
    """A ragged prompt goes in, tokens are decoded with their weights added up, the cache is thinned by them,
    and decoding goes on over the thinned cache -- eagerly, and with the decode step captured in a graph."""
    B, Hq, H, dh, n0 = 2, 4, 2, 64, 150
    g = gen(77)
    c = mka.make_kv8_config(B, 200, Hq, H, dh, block=32)
    c2 = mka.make_kv8_config(B, 96, Hq, H, dh, block=16, window=40, sinks=3)
    cache, models, lens = new_cache(mka, c), models_of(c), [150, 61]
    rows = lambda n, h: torch.randn(B, n, h, dh, generator=g).to(torch.bfloat16)  # noqa: E731
    append(mka, c, cache, models, rows(n0, H), rows(n0, H), [0] * B, lens)
    w = torch.zeros(B, H, 200, device="cuda")
    for _ in range(3):
        append(mka, c, cache, models, rows(1, H), rows(1, H), lens)
        lens = [n + 1 for n in lens]
        q, w0 = rows(1, Hq), w.cpu()
        out = attend(mka, c, cache, models, q, lens, w)
        check_attention(mka, c, models, q, lens, out, w0, w.cpu())
    got = evict(mka, c, cache, lens, w.cpu(), 80, 3, 20, c2)
    models, cache, lens = check_evict(mka, c, models, lens, w.cpu(), 80, 3, 20, c2, got), got[0], got[1]
    # one captured step: append a token, attend
    q, kn, vn = (torch.zeros(B, 1, h, dh, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H))
    out, pos, after = torch.empty_like(q), ints(lens), ints([n + 1 for n in lens])
    ws = mka.buffer(mka.mka_kv8_attention_workspace_size(c2, 1))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mka.mka_kv8_append(c2, cache, kn, vn, pos)
        mka.mka_kv8_attention(c2, cache, q, after, out, None, ws)
        pos.add_(1)
        after.add_(1)
    for _ in range(4):
        x = rows(1, H), rows(1, H), rows(1, Hq)
        kn.copy_(x[0]), vn.copy_(x[1]), q.copy_(x[2])
        graph.replay()
        torch.cuda.synchronize()
        for kv in range(2):
            for b in range(B):
                for h in range(H):
                    models[kv][b][h].append(lens[b], x[kv][b, :, h])
        lens = [n + 1 for n in lens]
        check_attention(mka, c2, models, x[2], lens, out.cpu())
    check_cache(mka, c2, cache, models, lens)
    assert mka.mka_status() == 0


# ---------------------------------------------------------------- refusals (host only)
def cfg(mka, **kw):
    c = mka.make_kv8_config(2, 300, 4, 2, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def fake(mka, at=0x1000):
    return mka.mka_kv8_cache(at, at + 0x1000, at + 0x2000, at + 0x3000)


@pytest.mark.parametrize("field,value,code", [
    ("batch", 0, "INVALID_ARG"), ("max_positions", 0, "INVALID_ARG"), ("n_kv_heads", 3, "INVALID_ARG"),
    ("d_head", 32, "UNSUPPORTED"), ("block", 48, "UNSUPPORTED"), ("block", 0, "UNSUPPORTED"), ("dtype", 2, "INVALID_ARG"),
    ("window", -1, "INVALID_ARG"), ("sinks", -2, "INVALID_ARG"), ("attn_scale", float("inf"), "INVALID_ARG"),
    ("batch", 65536, "UNSUPPORTED"), ("max_positions", 1 << 29, "UNSUPPORTED"),
])
def test_bad_configurations(mka, field, value, code):
    c, x, a, lib = cfg(mka, **{field: value}), fake(mka), ctypes.c_void_p(0x1000), mka._lib
    want = getattr(mka, "MKA_ERR_" + code)
    assert mka.mka_kv8_attention_workspace_size(c) == 0 and mka.mka_kv8_evict_workspace_size(c, 5) == 0
    assert lib.mka_kv8_append(c, x, a, a, 128, 1280, 10, a, None, None) == want
    assert lib.mka_kv8_read(c, x, None, None, 10, a, a, 128, 1280, None) == want
    assert lib.mka_kv8_attention(c, x, a, 1, a, a, None, a, 1 << 40, None) == want
    assert lib.mka_kv8_evict(c, x, a, a, 10, 0, 0, cfg(mka), fake(mka, 0x9000), ctypes.c_void_p(0x2000),
                             ctypes.c_void_p(0x3000), a, a, 1 << 20, None) == want


def test_bad_arguments(mka):
    c, x, a, odd, lib = cfg(mka), fake(mka), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), mka._lib
    bad, a2 = mka.MKA_ERR_INVALID_ARG, ctypes.c_void_p(0x1002)
    assert lib.mka_kv8_append(c, None, a, a, 128, 1280, 10, a, None, None) == bad
    assert lib.mka_kv8_append(c, x, odd, a, 128, 1280, 10, a, None, None) == bad
    assert lib.mka_kv8_append(c, x, a, None, 128, 1280, 10, a, None, None) == bad
    assert lib.mka_kv8_append(c, x, a, a, 120, 1280, 10, a, None, None) == bad
    assert lib.mka_kv8_append(c, x, a, a, 132, 1280, 10, a, None, None) == bad
    assert lib.mka_kv8_append(c, x, a, a, 128, -8, 10, a, None, None) == bad
    assert lib.mka_kv8_append(c, x, a, a, 128, 1280, 0, a, None, None) == bad
    assert lib.mka_kv8_append(c, x, a, a, 128, 1280, 10, None, None, None) == bad
    assert lib.mka_kv8_append(c, x, a, a, 128, 1280, 10, a, a2, None) == bad
    assert lib.mka_kv8_append(c, mka.mka_kv8_cache(0x1004, 0x2000, 0x3000, 0x4000), a, a, 128, 1280, 10, a, None, None) == bad
    assert lib.mka_kv8_append(c, mka.mka_kv8_cache(0x1000, 0x2000, None, 0x4000), a, a, 128, 1280, 10, a, None, None) == bad
    assert lib.mka_kv8_read(c, x, a2, None, 10, a, a, 128, 1280, None) == bad
    assert lib.mka_kv8_read(c, x, None, None, 10, a, odd, 128, 1280, None) == bad
    assert lib.mka_kv8_read(c, x, None, None, 10, a, a, 128, 0, None) == bad  # both sequences to the same rows
    assert lib.mka_kv8_attention(c, x, a, 0, a, a, None, a, 1 << 40, None) == bad
    assert lib.mka_kv8_attention(c, x, a, 1, None, a, None, a, 1 << 40, None) == bad
    assert lib.mka_kv8_attention(c, x, a, 1, a, a, a2, a, 1 << 40, None) == bad
    assert lib.mka_kv8_attention(c, x, a, 1, a, a, None, a, mka.mka_kv8_attention_workspace_size(c) - 1,
                                 None) == mka.MKA_ERR_WORKSPACE
    assert mka.mka_kv8_attention_workspace_size(c, 1, True) > mka.mka_kv8_attention_workspace_size(c, 1)
    y, l2, w2, crossed = fake(mka, 0x9000), ctypes.c_void_p(0x2000), ctypes.c_void_p(0x3000), fake(mka, 0x2000)
    crossed.k, crossed.v = x.v, x.k

    def ev(c2=None, cache=x, dst=y, lens=a, w=a, keep=10, first=2, recent=3, dl=l2, dw=w2, kept=a, ws=a, n=1 << 20):
        return lib.mka_kv8_evict(c, cache, lens, w, keep, first, recent, c2 or cfg(mka), dst, dl, dw, kept, ws, n, None)
    for kw in ({"dst": x}, {"dst": crossed}, {"dst": None}, {"lens": None}, {"w": None}, {"keep": 0}, {"first": -1}, {"recent": 9}, {"dl": None},
               {"dl": a}, {"dw": a}, {"kept": None}, {"ws": None}, {"keep": 301}, {"c2": cfg(mka, batch=3)},
               {"c2": cfg(mka, n_kv_heads=1)}, {"c2": cfg(mka, d_head=128)}, {"c2": cfg(mka, max_positions=9)}):
        assert ev(**kw) == bad, kw
    assert ev(n=1) == mka.MKA_ERR_WORKSPACE


def test_binding_refuses_shapes(mka):
    t = torch.zeros(2, 2, 300, 64, dtype=torch.uint8)
    s = torch.zeros(2, 2, 5)
    assert mka.kv8_cache(t, t.clone(), s, s.clone()).k == t.data_ptr()
    for bad in ((t, t[:1], s, s), (t, t.float(), s, s), (t, t, s.double(), s), (t.transpose(1, 2), t.transpose(1, 2), s, s),
                (t, t, s[0], s[0])):
        with pytest.raises(ValueError):
            mka.kv8_cache(*bad)
    x = mka.kv8_cache(t, t.clone(), s, s.clone())
    good, pos = torch.zeros(2, 3, 2, 64).bfloat16(), torch.zeros(2, dtype=torch.int32)
    q, ws = torch.zeros(2, 1, 4, 64).bfloat16(), torch.zeros(16, dtype=torch.uint8)
    for c in (cfg(mka, max_positions=301), cfg(mka, block=32), cfg(mka, batch=1)):
        with pytest.raises(ValueError, match="cache's"):
            mka.mka_kv8_append(c, x, good, good, pos)
    for bad in (torch.zeros(2, 3, 2, 64), torch.zeros(1, 3, 2, 64).bfloat16(), torch.zeros(2, 3, 2, 128).bfloat16()[..., ::2],
                torch.zeros(2, 3, 2, 128).bfloat16()[..., :64], torch.zeros(2, 128).bfloat16(), good.transpose(0, 1), None):
        with pytest.raises(ValueError, match="k_new"):
            mka.mka_kv8_append(cfg(mka), x, bad, bad, pos)
        with pytest.raises(ValueError, match="k_out"):
            mka.mka_kv8_read(cfg(mka), x, None, pos, bad, bad)
    with pytest.raises(ValueError, match="same"):
        mka.mka_kv8_append(cfg(mka), x, good, good[:, :2], pos)
    for p in (pos[:1], pos.long(), torch.zeros(4, dtype=torch.int32)[::2], 3):
        with pytest.raises(ValueError, match="pos"):
            mka.mka_kv8_append(cfg(mka), x, good, good, p)
        with pytest.raises(ValueError, match="lens"):
            mka.mka_kv8_attention(cfg(mka), x, q, p, q, None, ws)
    for p in (q.float(), q[:1], q[..., ::2], q[0]):
        with pytest.raises(ValueError, match="must be"):
            mka.mka_kv8_attention(cfg(mka), x, p, pos, q, None, ws)
    with pytest.raises(ValueError, match="weights"):
        mka.mka_kv8_attention(cfg(mka), x, q, pos, q, torch.zeros(2, 2, 299), ws)
    with pytest.raises(ValueError, match="structure"):
        mka.mka_kv8_append(mka.make_attn_config(1, 1, 1, 1, 64), x, good, good, pos)
    with pytest.raises(ValueError, match="kv8_cache|tensor"):
        y = fake(mka)
        y.tensors = (1, 2, 3, 4)
        mka.mka_kv8_append(cfg(mka), y, good, good, pos)
    with pytest.raises(AttributeError):
        mka.mka_kv8_append(cfg(mka), fake(mka), good, good, pos)
    with pytest.raises(TypeError):
        mka.mka_kv8_append(None, x, good, good, pos)
    with pytest.raises(ValueError, match="range|kept"):
        mka.mka_kv8_evict(cfg(mka), x, pos, torch.zeros(2, 2, 300), 1 << 40, 0, 0, cfg(mka), x, pos, None, pos, ws)
