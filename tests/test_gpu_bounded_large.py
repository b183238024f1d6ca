"""Bounded-memory operators at sizes whose offsets pass 32 bits and at the largest batches."""
import pytest
import torch

import bounded_ref as ref
import test_gpu_kv8_streams as streams


@pytest.fixture(scope="module")
def mka():
    import route_kv_memory_b200 as m
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,window,sinks,G", [("bf16", 0, 0, 1), ("f32", 5000, 7, 12)])
def test_cache_of_more_than_4_gb(mka, dtype, window, sinks, G):
    """Codes of 4.8 GB for K and for V: append, read, attention with weights and eviction in the last head."""
    B, H, L, dh, block, n = 1, 9, (1 << 22) + 77, 128, 64, 2
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    c = mka.make_kv8_config(B, L, G * H, H, dh, block=block, dtype=dtype, window=window, sinks=sinks)
    g = torch.Generator("cuda").manual_seed(4)
    nb = -(-L // block)
    one = torch.randn(1 << 20, dh, generator=g, device="cuda").mul_(64).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = []
    for kv in range(2):
        x = torch.empty(B, H, L, dh, dtype=torch.uint8, device="cuda")
        for h in range(H):
            for a in range(0, L, 1 << 20):
                x[0, h, a:a + (1 << 20)] = one.roll(131 * (h + 10 * kv) + a, 0)[:min(1 << 20, L - a)]
        codes.append(x)
    scales = [torch.full((B, H, nb), 2.0 ** -7, device="cuda") for _ in "kv"]
    cache = mka.kv8_cache(*codes, *scales)
    # new rows across the last full block's end
    pos, m = L - 20, 20
    new = [torch.randn(B, m, H, dh, generator=g, device="cuda").to(dt) for _ in "kv"]
    models = []
    for kv in range(2):
        y = ref.Cache(block)
        a = pos // block * block
        y.x = codes[kv][0, H - 1, a:pos].view(torch.float8_e4m3fn).cpu().double() * 2.0 ** -7
        y.scale = {0: 2.0 ** -7}
        y.append(pos - a, new[kv][0, :, H - 1].cpu())
        models.append(y)
    at = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    mka.mka_kv8_append(c, cache, *new, at(pos))
    out = [torch.zeros(B, 80, H, dh, dtype=dt, device="cuda") for _ in "kv"]
    first = pos // block * block
    mka.mka_kv8_read(c, cache, at(first), at(L - first), *out)
    for kv in range(2):
        assert torch.equal(out[kv][0, :L - first, H - 1].cpu().double(), models[kv].x.to(dt).double())
        assert (out[kv][0, L - first:] == 0).all()
    # attention, against 64 bits on the GPU
    q = torch.randn(B, n, G * H, dh, generator=g, device="cuda").to(dt)
    w0 = torch.rand(B, H, L, generator=g, device="cuda")
    w1 = w0.clone()
    got = streams.attend(mka, c, cache, q, at(L), w1)
    k, v = (codes[kv][0, H - 1].view(torch.float8_e4m3fn).double() * scales[kv][0, H - 1].double().repeat_interleave(block)[:L, None]
            for kv in range(2))
    vs = scales[1][0, H - 1].double().repeat_interleave(block)[:L]
    added, slack = torch.zeros(L, dtype=torch.float64, device="cuda"), torch.zeros(L, dtype=torch.float64, device="cuda")
    for i in range(n):
        o, w, e, ew = streams.decode(q[0, i, (H - 1) * G:].double(), k, v, vs, L - n + i, window, sinks, dh ** -0.5, dtype == "bf16")
        assert ((got[0, i, (H - 1) * G:].double() - o).abs() <= e).all()
        added += w.sum(0)
        slack += ew.sum(0)
    total = w0[0, H - 1].double() + added
    assert ((w1[0, H - 1].double() - total).abs() <= slack + 2.0 ** -23 * total).all()
    del k, v
    # eviction
    keep, lead, recent = 3000, 4, 100
    c2 = mka.make_kv8_config(B, keep, G * H, H, dh, block=block, dtype=dtype)
    d = mka.kv8_cache(*(torch.zeros(B, H, keep, dh, dtype=torch.uint8, device="cuda") for _ in "kv"),
                      *(torch.ones(B, H, -(-keep // block), device="cuda") for _ in "kv"))
    lens2, kept = at(0), torch.zeros(B, H, keep, dtype=torch.int32, device="cuda")
    mka.mka_kv8_evict(c, cache, at(L), w0, keep, lead, recent, c2, d, lens2, None, kept, mka.buffer(mka.mka_kv8_evict_workspace_size(c, keep)))
    w = w0[0, H - 1].clone()
    w[:lead] = w[L - recent:] = 2.0
    pick = w.sort(descending=True, stable=True)[1][:keep].sort()[0]
    assert torch.equal(kept[0, H - 1].long(), pick) and lens2.item() == keep
    for kv in range(2):
        x = (codes[kv][0, H - 1, pick].view(torch.float8_e4m3fn).double() * scales[kv][0, H - 1].double()[pick // block, None]).cpu()
        y = ref.Cache(block)
        y.append(0, x)
        have, _ = streams.value_of(d.tensors[kv][0, H - 1].view(torch.float8_e4m3fn), d.tensors[2 + kv][0, H - 1], block)
        assert torch.equal(have, y.x)
    assert mka.mka_status() == 0


@pytest.mark.gpu
def test_window_attention_of_more_than_4_gb(mka):
    """q, out and their gradients of 2.5e9 elements each: the last rows of the last head against 64 bits."""
    B, S, Hq, H, dh, window, sinks, last = 1, 600001, 32, 1, 128, 130, 2, 700
    g = torch.Generator("cuda").manual_seed(5)
    q, k, v, do = (torch.randn(B, S, h, dh, generator=g, device="cuda", dtype=torch.bfloat16) for h in (Hq, H, H, Hq))
    c = mka.make_attn_config(B, S, Hq, H, dh, window, sinks)
    out, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))
    lse, ws = mka.attention_lse(c), mka.buffer(mka.mka_window_attention_backward_workspace_size(c))
    mka.mka_window_attention(c, q, k, v, None, out, lse)
    mka.mka_window_attention_backward(c, q, k, v, out, lse, do, None, dq, dk, dv, ws)
    assert mka.mka_status() == 0
    # the sinks and the last rows as a sequence of their own: rows from `window` on see what they see in the whole one
    at = torch.cat([torch.arange(sinks), torch.arange(S - last, S)]).cuda()
    x = [t[0, at].cpu().double() for t in (q, k, v, do)]
    want = (ref.window_forward(*x[:3], window, sinks)[0], *ref.window_backward(*x, window, sinks))
    bound = ref.window_bounds(*x, window, sinks)
    for t, w, e in zip((out, dq, dk, dv), want, bound):
        have = t[0, at].cpu().double()[sinks + window:]
        assert ((have - w[sinks + window:]).abs() <= e[sinks + window:]).all()


@pytest.mark.gpu
def test_the_largest_batch_of_windows(mka):
    B, S, Hq, H, dh = 65535, 3, 2, 1, 64
    g = torch.Generator().manual_seed(6)
    q, k, v, do = (torch.randn(B, S, h, dh, generator=g).bfloat16() for h in (Hq, H, H, Hq))
    c = mka.make_attn_config(B, S, Hq, H, dh, 2, 1)
    lens = torch.randint(0, S + 1, (B,), generator=g, dtype=torch.int32)
    lens[-1] = S
    out, dq, dk, dv = (torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, q, k, v))
    lse, ws = mka.attention_lse(c), mka.buffer(mka.mka_window_attention_backward_workspace_size(c))
    d = [t.cuda() for t in (q, k, v, do, lens)]
    mka.mka_window_attention(c, *d[:3], d[4], out, lse)
    mka.mka_window_attention_backward(c, *d[:3], out, lse, d[3], d[4], dq, dk, dv, ws)
    assert mka.mka_status() == 0
    got = [t.cpu() for t in (out, dq, dk, dv)]
    for b in list(range(0, B, 1009)) + [B - 1]:
        n = int(lens[b])
        if n:
            x = [t[b, :n].double() for t in (q, k, v, do)]
            want = (ref.window_forward(*x[:3], 2, 1)[0], *ref.window_backward(*x, 2, 1))
            for t, w, e in zip(got, want, ref.window_bounds(*x, 2, 1)):
                assert ((t[b, :n].double() - w).abs() <= e).all()
    behind = torch.arange(S)[None] >= lens[:, None]
    assert all((t[behind] == 7.0).all() for t in got)


@pytest.mark.gpu
def test_the_largest_batch_of_caches(mka):
    B, L, Hq, H, dh, block = 65535, 5, 2, 1, 64, 16
    g = torch.Generator().manual_seed(7)
    c = mka.make_kv8_config(B, L, Hq, H, dh, block=block)
    cache = mka.kv8_cache(*(torch.zeros(B, H, L, dh, dtype=torch.uint8, device="cuda") for _ in "kv"),
                          *(torch.ones(B, H, 1, device="cuda") for _ in "kv"))
    lens = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
    lens[-1] = L
    x = [torch.randn(B, L, H, dh, generator=g).bfloat16().cuda() for _ in "kv"]
    at = lens.cuda()
    mka.mka_kv8_append(c, cache, *x, torch.zeros_like(at), at)
    q = torch.randn(B, 1, Hq, dh, generator=g).bfloat16().cuda()
    w1 = torch.zeros(B, H, L, device="cuda")
    out = streams.attend(mka, c, cache, q, at, w1)
    assert (out[at == 0] == 0).all()
    assert ((w1.sum(-1) - Hq * (at > 0)[:, None]).abs() < 1e-4).all()
    units = [(b, 0) for b in list(range(0, B, 1009)) + [B - 1] if int(lens[b])]
    streams.check(mka, c, cache, q, lens.tolist(), out, units, torch.zeros_like(w1), w1)
    keep = 2
    c2 = mka.make_kv8_config(B, keep, Hq, H, dh, block=block)
    d = mka.kv8_cache(*(torch.zeros(B, H, keep, dh, dtype=torch.uint8, device="cuda") for _ in "kv"),
                      *(torch.ones(B, H, 1, device="cuda") for _ in "kv"))
    lens2, kept = torch.zeros_like(at), torch.zeros(B, H, keep, dtype=torch.int32, device="cuda")
    mka.mka_kv8_evict(c, cache, at, w1, keep, 0, 1, c2, d, lens2, None, kept, mka.buffer(256))
    assert torch.equal(lens2, at.clamp_max(keep))
    for b in list(range(0, B, 1009)) + [B - 1]:
        n = int(lens[b])
        pick = ref.keep_positions(w1[b, 0].tolist(), n, keep, 0, 1)
        assert kept[b, 0].tolist() == pick + [-1] * (keep - len(pick))
    assert mka.mka_status() == 0
