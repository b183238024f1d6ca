"""Window attention with sinks on the GPU against its float64 definition: forward, gradients, padded
batches, strides, refusals."""
import ctypes

import pytest
import torch

import bounded_ref as ref


@pytest.fixture(scope="module")
def mka():
    import route_kv_memory_b200 as m
    return m


def draw(B, S, Hq, Hkv, dh, seed, x=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    return n(B, S, Hq, dh) * x, n(B, S, Hkv, dh) * x, n(B, S, Hkv, dh), n(B, S, Hq, dh)


def test_formula_against_differences():
    """The gradient formula the GPU is held to, against central differences of the definition."""
    g = torch.Generator().manual_seed(3)
    q, do = (torch.randn(9, 4, 8, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(9, 2, 8, generator=g, dtype=torch.float64) for _ in range(2))
    grads = ref.window_backward(q, k, v, do, 3, 2)
    for i, x in enumerate((q, k, v)):
        for _ in range(20):
            at = tuple(int(torch.randint(n, (), generator=g)) for n in x.shape)
            old, h, f = float(x[at]), 1e-5, []
            for step in (h, -h):
                x[at] = old + step
                f.append(float((ref.window_forward(q, k, v, 3, 2)[0] * do).sum()))
            x[at] = old
            assert abs((f[0] - f[1]) / (2 * h) - float(grads[i][at])) < 1e-8


def run(mka, q, k, v, do, window, sinks, lens=None, dev="cuda", fill=7.0):
    B, S, Hq, dh = q.shape
    c = mka.make_attn_config(B, S, Hq, k.shape[2], dh, window, sinks)
    q, k, v, do = (x.to(dev) if not x.is_cuda else x for x in (q, k, v, do))
    out = torch.full((B, S, Hq, dh), fill, dtype=torch.bfloat16, device=dev)
    dq, dk, dv = (torch.full(x.shape, fill, dtype=torch.bfloat16, device=dev) for x in (q, k, v))
    lse = mka.attention_lse(c).fill_(float("nan"))
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    ws = mka.buffer(mka.mka_window_attention_backward_workspace_size(c))
    ws.fill_(255)  # NaN patterns: nothing may be read before it is written
    mka.mka_window_attention(c, q, k, v, ln, out, lse)
    mka.mka_window_attention_backward(c, q, k, v, out, lse, do, ln, dq, dk, dv, ws)
    torch.cuda.synchronize()
    assert mka.mka_status() == 0
    return [x.cpu() for x in (out, dq, dk, dv)] + [lse.cpu()]


def check(got, q, k, v, do, window, sinks, lens=None, fill=7.0):
    for b in range(q.shape[0]):
        n = q.shape[1] if lens is None else lens[b]
        x = [t[b, :n].double() for t in (q, k, v, do)]
        if n:
            out, _, lse = ref.window_forward(*x[:3], window, sinks)
            want = (out, *ref.window_backward(*x, window, sinks))
            for name, y, w, e in zip(("out", "dq", "dk", "dv"), got, want, ref.window_bounds(*x, window, sinks)):
                far = (y[b, :n].double() - w).abs()
                assert (far <= e).all(), f"{name}: {float((far / e.clamp_min(1e-300)).max()):.3g} times its bound"
            # log2 normalisers: float32 scores of magnitude <= 2^5 and a float32 sum
            assert (got[4][b, :, :n].double() - lse).abs().max() < 2.0 ** -12
        for y in got[:4]:
            assert (y[b, n:] == fill).all(), "rows behind the sequence were written"


CASES = [
    # B, S, Hq, Hkv, dh, window, sinks
    (1, 1, 1, 1, 64, 1, 0), (2, 5, 4, 2, 64, 2, 1), (1, 127, 2, 1, 128, 1, 1), (1, 128, 2, 2, 128, 128, 0),
    (1, 129, 7, 1, 128, 64, 4), (1, 255, 4, 2, 64, 64, 4), (2, 256, 4, 1, 128, 129, 3), (1, 300, 4, 2, 64, 0, 5),
    (1, 300, 4, 2, 128, 300, 0), (1, 385, 2, 1, 64, 127, 130), (1, 513, 4, 4, 128, 100, 128), (1, 640, 3, 1, 64, 1, 300),
    (1, 1400, 4, 2, 64, 1024, 4), (1, 1300, 3, 1, 128, 1100, 140), (2, 1200, 2, 1, 128, 1025, 0),
    (3, 390, 4, 2, 64, 255, 4), (1, 1100, 8, 2, 128, 256, 4), (1, 1537, 2, 1, 64, 5, 2), (2, 200, 5, 1, 64, 60, 2),
    # more query tiles than SMs: two of them in an item, with odd groups also two of different rows
    (1, 700, 28, 4, 128, 200, 3), (2, 1300, 9, 3, 64, 1030, 2), (1, 1000, 24, 8, 128, 0, 0), (1, 641, 32, 8, 64, 90, 140),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_against_definition(mka, case):
    B, S, Hq, Hkv, dh, window, sinks = case
    x = draw(B, S, Hq, Hkv, dh, sum(case))
    check(run(mka, *x, window, sinks), *x, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("case,lens", [
    ((3, 300, 4, 2, 64, 70, 4), [300, 0, 129]), ((4, 260, 2, 1, 128, 128, 1), [1, 256, 257, 128]),
    ((2, 700, 4, 2, 128, 64, 140), [700, 333]), ((2, 1300, 2, 1, 64, 1030, 3), [1300, 1153]), ((3, 513, 2, 2, 64, 0, 0), [513, 384, 2]),
    ((3, 700, 10, 2, 64, 130, 5), [700, 0, 401]), ((2, 1300, 7, 1, 128, 1040, 1), [640, 1300]),
])
def test_padded_batch(mka, case, lens):
    """Padding rows hold NaN and infinities: they reach nothing, and nothing is written there."""
    B, S, Hq, Hkv, dh, window, sinks = case
    x = draw(B, S, Hq, Hkv, dh, 17)
    for t in x:
        for b, n in enumerate(lens):
            t[b, n:] = float("nan")
            t[b, n::3] = float("inf")
    check(run(mka, *x, window, sinks, lens), *x, window, sinks, lens)


@pytest.mark.gpu
def test_many_short_sequences(mka):
    """More sequences than the forward keeps a table of, most of them shorter than the padding."""
    B, S = 530, 150
    x = draw(B, S, 2, 1, 64, 6)
    lens = [(37 * b) % (S + 1) for b in range(B)]
    check(run(mka, *x, 40, 2, lens), *x, 40, 2, lens)


@pytest.mark.gpu
def test_sequence_end_does_not_read_the_next_sequence(mka):
    """S is not a multiple of a tile: the tile's last rows belong to the next sequence, here all NaN there."""
    x = draw(2, 200, 2, 1, 64, 5)
    for t in x:
        t[1] = float("nan")
    got = run(mka, *x, 50, 2)
    check([g[:1] for g in got], *(t[:1] for t in x), 50, 2)


@pytest.mark.gpu
def test_large_scores_move_the_maximum(mka):
    """Keys grow along the sequence, so later tiles beat earlier maxima by far more than the lazy threshold."""
    q, k, v, do = draw(1, 600, 2, 1, 64, 9)
    k = (k * torch.linspace(1, 4, 600)[None, :, None, None]).to(torch.bfloat16)
    got = run(mka, q, k, v, do, 300, 4)
    check(got, q, k, v, do, 300, 4)


@pytest.mark.gpu
def test_lens_past_the_end_and_negative_are_clamped(mka):
    x = draw(2, 150, 2, 1, 64, 8)
    got = run(mka, *x, 40, 1, [1000, -3])
    check(got, *x, 40, 1, [150, 0])


@pytest.mark.gpu
def test_strided_rows_of_a_packed_projection(mka):
    B, S, Hq, Hkv, dh = 2, 333, 4, 2, 64
    g = torch.Generator().manual_seed(2)
    packed = torch.randn(B, S, (Hq + 2 * Hkv) * dh + 8, generator=g).to(torch.bfloat16).cuda()
    q, k, v = packed[..., :Hq * dh], packed[..., Hq * dh:(Hq + Hkv) * dh], packed[..., (Hq + Hkv) * dh:(Hq + 2 * Hkv) * dh]
    wide = torch.zeros(B, S, 2 * Hq * dh, dtype=torch.bfloat16, device="cuda")
    out = wide[..., Hq * dh:]
    do = torch.randn(B, S, 2, Hq * dh, generator=g).to(torch.bfloat16).cuda()[:, :, 1]
    c = mka.make_attn_config(B, S, Hq, Hkv, dh, 100, 4)
    lse = mka.attention_lse(c)
    dq, dk, dv = (torch.empty(B, S, h, dh, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    mka.mka_window_attention(c, q, k, v, None, out, lse)
    ws = mka.buffer(mka.mka_window_attention_backward_workspace_size(c))
    mka.mka_window_attention_backward(c, q, k, v, out, lse, do, None, dq, dk, dv, ws)
    dense = [x.reshape(B, S, -1, dh).cpu() for x in (q, k, v, do)]
    check([x.reshape(B, S, -1, dh).cpu() for x in (out, dq, dk, dv)] + [lse.cpu()], *dense, 100, 4)
    assert (wide[..., :Hq * dh] == 0).all()


@pytest.mark.gpu
def test_same_call_twice_gives_the_same_bits(mka):
    x = draw(2, 900, 4, 2, 128, 21)
    a, b = run(mka, *x, 200, 4, [900, 555], fill=0.0), run(mka, *x, 200, 4, [900, 555], fill=0.0)
    for y, z in zip(a[:4], b[:4]):
        assert torch.equal(y, z)


@pytest.mark.gpu
def test_captured_replayed_and_on_another_stream(mka):
    B, S, Hq, Hkv, dh = 1, 400, 4, 2, 64
    x = draw(B, S, Hq, Hkv, dh, 4)
    c = mka.make_attn_config(B, S, Hq, Hkv, dh, 90, 3)
    q, k, v, do = (t.cuda() for t in x)
    out, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))
    lse, ws = mka.attention_lse(c), mka.buffer(mka.mka_window_attention_backward_workspace_size(c))
    lens = torch.tensor([S], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mka.mka_window_attention(c, q, k, v, lens, out, lse)
        mka.mka_window_attention_backward(c, q, k, v, out, lse, do, lens, dq, dk, dv, ws)
    y = draw(B, S, Hq, Hkv, dh, 40)
    for t, z in zip((q, k, v, do), y):
        t.copy_(z)
    lens.fill_(310)
    for t in (out, dq, dk, dv):
        t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    check([t.cpu() for t in (out, dq, dk, dv, lse)], *y, 90, 3, [310])
    side.wait_stream(torch.cuda.current_stream())
    out2 = torch.full_like(out, 7.0)
    side.wait_stream(torch.cuda.current_stream())
    mka.mka_window_attention(c, q, k, v, lens, out2, None, side)
    side.synchronize()
    assert torch.equal(out2, out)


# ---------------------------------------------------------------- refusals (host only)
def cfg(mka, **kw):
    c = mka.make_attn_config(2, 300, 4, 2, 64, 50, 4)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("field,value,code", [
    ("batch", 0, "INVALID_ARG"), ("seq", 0, "INVALID_ARG"), ("n_kv_heads", 3, "INVALID_ARG"), ("n_q_heads", 0, "INVALID_ARG"),
    ("d_head", 96, "UNSUPPORTED"), ("dtype", 0, "UNSUPPORTED"), ("dtype", 5, "INVALID_ARG"), ("window", -1, "INVALID_ARG"),
    ("sinks", -1, "INVALID_ARG"), ("attn_scale", float("nan"), "INVALID_ARG"), ("seq", 1 << 30, "UNSUPPORTED"),
    ("batch", 70000, "UNSUPPORTED"),
])
def test_bad_configurations(mka, field, value, code):
    c, a = cfg(mka, **{field: value}), ctypes.c_void_p(0x1000)
    assert mka.mka_window_attention_backward_workspace_size(c) == 0
    want = getattr(mka, "MKA_ERR_" + code)
    assert mka._lib.mka_window_attention(c, None, a, a, a, None, a, None, None) == want
    assert mka._lib.mka_window_attention_backward(c, None, a, a, a, a, a, a, None, a, a, a, a, 1 << 40, None) == want


def test_bad_pointers_strides_and_workspace(mka):
    c, a, odd, lib = cfg(mka), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), mka._lib
    bad = mka.MKA_ERR_INVALID_ARG
    assert lib.mka_window_attention(None, None, a, a, a, None, a, None, None) == bad
    for i in range(5):  # q, k, v, out NULL or misaligned; lse misaligned
        p = [a, a, a, None, a, None]
        at = [0, 1, 2, 4, 5][i]
        p[at] = odd
        assert lib.mka_window_attention(c, None, *p, None) == bad
        if at != 5:
            p[at] = None
            assert lib.mka_window_attention(c, None, *p, None) == bad
    assert lib.mka_window_attention(c, None, a, a, a, ctypes.c_void_p(0x1002), a, None, None) == bad
    for ld in (mka.mka_attn_strides(255, 0, 0, 0, 0), mka.mka_attn_strides(0, 120, 0, 0, 0), mka.mka_attn_strides(0, 0, 0, 260, 0),
               mka.mka_attn_strides(0, 0, -128, 0, 0)):
        assert lib.mka_window_attention(c, ld, a, a, a, None, a, None, None) == bad
    need = mka.mka_window_attention_backward_workspace_size(c)
    assert need >= 2 * 4 * 384 * 4
    assert lib.mka_window_attention_backward(c, None, a, a, a, a, a, a, None, a, a, a, a, need - 1,
                                             None) == mka.MKA_ERR_WORKSPACE
    assert lib.mka_window_attention_backward(c, None, a, a, a, a, None, a, None, a, a, a, a, need, None) == bad


@pytest.mark.gpu
def test_binding_refuses_shapes_types_and_devices(mka):
    c = cfg(mka)
    q, k = (torch.zeros(2, 300, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    out = torch.zeros_like(q)
    with pytest.raises(ValueError):
        mka.mka_window_attention(c, q[:, :299], k, k, None, out)
    with pytest.raises(ValueError):
        mka.mka_window_attention(c, q.float(), k, k, None, out)
    with pytest.raises(ValueError, match="current CUDA device"):
        mka.mka_window_attention(c, q.cpu(), k, k, None, out)
    with pytest.raises(ValueError, match="lens"):
        mka.mka_window_attention(c, q, k, k, [300, 300], out)
    with pytest.raises(ValueError):
        mka.mka_window_attention(c, q, k, k, torch.zeros(3, dtype=torch.int32, device="cuda"), out)
    with pytest.raises(ValueError):
        mka.mka_window_attention(c, q, k, k, torch.zeros(2, device="cuda"), out)
    with pytest.raises(ValueError):  # heads not next to each other
        mka.mka_window_attention(c, torch.zeros(2, 300, 4, 128, dtype=torch.bfloat16, device="cuda")[..., ::2], k, k, None, out)
    with pytest.raises(mka.MKAError):
        mka.mka_window_attention(cfg(mka, window=-1), q, k, k, None, out)
