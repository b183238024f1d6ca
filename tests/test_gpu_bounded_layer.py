"""The 8-bit cache behind the layer: a prompt's fused K/V taken from its decode state, attended, thinned and
attended again; and the timeout path of the bounded-memory kernels."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import bounded_ref as ref
from fastmka_inputs import CONFIGS, FastMKAConfig, make_inputs
from gpu_util import gpu_weights


@pytest.fixture(scope="module")
def mka():
    import route_kv_memory_b200 as m
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_prompt_into_the_8_bit_cache(mka, dtype):
    B, S, L = 2, 300, 340
    cfg = FastMKAConfig("kv8_layer", B, S, 256, 4, 2, 64, 64, 0.9, 32, 2, 16, dtype, 31)
    inp = make_inputs(cfg)
    layer = mka.FastMKALayer(cfg, gpu_weights(inp))
    state = layer.new_state(L)
    out = torch.empty(B, S, cfg.dq, dtype=inp.x.dtype, device="cuda")
    layer.prefill(inp.x.cuda(), out, state=state, max_positions=L)
    k, v = layer.fused_kv(state, L)
    assert k.shape == (B, L, 2, 64) and k.dtype == inp.x.dtype
    cache = mka.KV8Cache(B, 512, 4, 2, 64, block=32, dtype=dtype, weights=True)
    cache.append(k[:, :S], v[:, :S])
    assert cache.lens.tolist() == [S, S]
    models = [[[ref.Cache(32) for _ in range(2)] for _ in range(B)] for _ in range(2)]
    for kv, t in enumerate((k, v)):
        for b in range(B):
            for g in range(2):
                models[kv][b][g].append(0, t[b, :S, g].cpu())
    got = cache.read(S)
    for kv in range(2):
        for b in range(B):
            for g in range(2):
                assert torch.equal(got[kv][b, :, g].cpu().double(), models[kv][b][g].x)

    def attend(c, models, n):
        q = torch.randn(B, 1, 4, 64, generator=torch.Generator().manual_seed(n)).to(inp.x.dtype)
        o = c.attend(q.cuda(), torch.empty_like(q, device="cuda")).cpu()
        for b in range(B):
            for g in range(2):
                want, w, e = ref.decode(q[b, 0, 2 * g:2 * g + 2].double(), models[0][b][g].x, models[1][b][g].x,
                                        models[1][b][g].scales(), n - 1, 0, 0, 0.125, dtype == "bf16")
                assert ((o[b, 0, 2 * g:2 * g + 2].double() - want).abs() <= e).all()

    attend(cache, models, S)
    assert abs(float(cache.weights.sum()) - 4 * B) < 1e-3  # every query row's weights sum to 1
    w = cache.weights.cpu()
    small, kept = cache.evict(100, 4, 30, 128)
    thin = [[[ref.Cache(32) for _ in range(2)] for _ in range(B)] for _ in range(2)]
    for b in range(B):
        for g in range(2):
            pick = ref.keep_positions(w[b, g, :S].tolist(), S, 100, 4, 30)
            assert kept[b, g].tolist() == pick
            for kv in range(2):
                thin[kv][b][g].append(0, models[kv][b][g].x[pick])
    attend(small, thin, 100)
    # a cache that is full keeps what it has
    row = torch.zeros(B, 60, 2, 64, dtype=inp.x.dtype, device="cuda")
    small.append(row, row)
    assert mka.mka_status() == mka.MKA_ERR_CAPACITY and small.lens.tolist() == [100, 100]
    small.append(row[:, :28], row[:, :28], torch.tensor([28, 0], dtype=torch.int32, device="cuda"))
    assert small.lens.tolist() == [128, 100] and mka.mka_status() == 0


def test_fused_kv_refusals(mka):
    c = mka.make_config(CONFIGS["qwen7b_4k"])
    lib, a, bad = mka._lib, ctypes.c_void_p(0x1000), mka.MKA_ERR_INVALID_ARG
    k, v = ctypes.c_void_p(), ctypes.c_void_p()
    n = mka.mka_state_size(c, 100)
    assert lib.mka_state_kv(ctypes.byref(c), 100, a, n, ctypes.byref(k), ctypes.byref(v)) == mka.MKA_OK
    assert 0x1000 < k.value < v.value < 0x1000 + n
    assert lib.mka_state_kv(ctypes.byref(c), 100, a, n - 1, ctypes.byref(k), ctypes.byref(v)) == mka.MKA_ERR_WORKSPACE
    assert lib.mka_state_kv(ctypes.byref(c), 0, a, n, ctypes.byref(k), ctypes.byref(v)) == bad
    assert lib.mka_state_kv(ctypes.byref(c), 100, None, n, ctypes.byref(k), ctypes.byref(v)) == bad
    assert lib.mka_state_kv(ctypes.byref(c), 100, a, n, None, ctypes.byref(v)) == bad


def limited(mka, fn):
    """fn() with a 1 ns limit on the pipeline waits; returns the status that it leaves."""
    assert mka.mka_status() == 0
    mka.mka_set_wait_limit(1, mka.MKA_WAIT_PIPELINE)
    try:
        fn()
        torch.cuda.synchronize()
        return mka.mka_status()
    finally:
        mka.mka_set_wait_limit(0, 0)


@pytest.mark.gpu
def test_window_attention_waits_run_out_and_it_recovers(mka):
    B, S, Hq, Hkv, dh = 2, 700, 4, 2, 128
    c = mka.make_attn_config(B, S, Hq, Hkv, dh, 100, 3)
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(B, S, h, dh, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv, Hq))
    lse, ws = mka.attention_lse(c), mka.buffer(mka.mka_window_attention_backward_workspace_size(c))

    def step():
        out, dq, dk, dv = (torch.zeros_like(t) for t in (q, q, k, v))
        mka.mka_window_attention(c, q, k, v, None, out, lse)
        mka.mka_window_attention_backward(c, q, k, v, out, lse, do, None, dq, dk, dv, ws)
        torch.cuda.synchronize()
        return out, dq, dk, dv

    want = step()
    assert limited(mka, step) == mka.MKA_ERR_DEVICE_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(step(), want)) and mka.mka_status() == 0


CAPTURED_FIRST = """
import sys, torch
sys.path[:0] = [%r, %r]
import route_kv_memory_b200 as mka
import test_gpu_window_attention as w
import bounded_ref as ref
B, S, Hq, Hkv, dh = 1, 200, 4, 2, 128
x = w.draw(B, S, Hq, Hkv, dh, 4)
c = mka.make_attn_config(B, S, Hq, Hkv, dh, 90, 3)
q, k, v, do = (t.cuda() for t in x)
out, dq, dk, dv = (torch.zeros_like(t) for t in (q, q, k, v))
lse, ws = mka.attention_lse(c), mka.buffer(mka.mka_window_attention_backward_workspace_size(c))
cache = mka.KV8Cache(B, S, Hq, Hkv, dh, weights=True)
one, new = torch.zeros(B, 1, Hq, dh, dtype=torch.bfloat16, device="cuda"), mka.KV8Cache(B, 64, Hq, Hkv, dh, weights=True)
o1, kept = torch.empty_like(one), torch.empty(B, Hkv, 64, dtype=torch.int32, device="cuda")
ws1, ws2 = (mka.buffer(n) for n in (mka.mka_kv8_attention_workspace_size(cache.c, 1, True), mka.mka_kv8_evict_workspace_size(cache.c, 64)))
pos, lens = (torch.tensor([n], dtype=torch.int32, device="cuda") for n in (0, S))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    mka.mka_window_attention(c, q, k, v, None, out, lse)
    mka.mka_window_attention_backward(c, q, k, v, out, lse, do, None, dq, dk, dv, ws)
    mka.mka_kv8_append(cache.c, cache.cache, k, v, pos)
    mka.mka_kv8_attention(cache.c, cache.cache, one, lens, o1, cache.weights, ws1)
    mka.mka_kv8_evict(cache.c, cache.cache, lens, cache.weights, 64, 4, 10, new.c, new.cache, new.lens, new.weights, kept, ws2)
g.replay()
torch.cuda.synchronize()
assert mka.mka_status() == 0
w.check([t.cpu() for t in (out, dq, dk, dv, lse)], *x, 90, 3)
# a query of zeros weighs all values alike
m = [ref.Cache(64) for _ in range(Hkv)]
for h in range(Hkv):
    m[h].append(0, x[2][0, :, h])
    assert (o1[0, 0, 2 * h].cpu().double() - m[h].x.mean(0)).abs().max() < 2 ** -8
assert new.lens.tolist() == [64] and kept[0, 0, :4].tolist() == [0, 1, 2, 3] and kept[0, 0, -1].item() == S - 1
print("captured first: ok")
"""


def steps_on(mka, seed, dh, stream):
    """Training steps of window attention and steps of an 8-bit cache that is thinned, all on `stream`: the results."""
    g, B, S, Hq, H, keep = torch.Generator().manual_seed(seed), 2, 300, 6, 2, 100

    def rnd(*s):
        return torch.randn(*s, generator=g).bfloat16().cuda()

    def zeros(*s, dtype=torch.bfloat16):
        return torch.zeros(*s, dtype=dtype, device="cuda")
    c = mka.make_attn_config(B, S, Hq, H, dh, window=70, sinks=2)
    q, k, v, do, q4 = rnd(B, S, Hq, dh), rnd(B, S, H, dh), rnd(B, S, H, dh), rnd(B, S, Hq, dh), rnd(B, 4, Hq, dh)
    out, dq, dk, dv, lse = zeros(B, S, Hq, dh), zeros(B, S, Hq, dh), zeros(B, S, H, dh), zeros(B, S, H, dh), mka.attention_lse(c)
    lens = torch.tensor([S, 211], dtype=torch.int32, device="cuda")
    ws = mka.buffer(mka.mka_window_attention_backward_workspace_size(c))
    c8, d8 = mka.make_kv8_config(B, S + 8, Hq, H, dh), mka.make_kv8_config(B, keep, Hq, H, dh)
    a, d = (mka.kv8_cache(*[zeros(B, H, n, dh, dtype=torch.uint8) for _ in "kv"],
                          *[zeros(B, H, -(-n // 64), dtype=torch.float32) for _ in "kv"]) for n in (S + 8, keep))
    at, l2, kept = zeros(B, dtype=torch.int32), zeros(B, dtype=torch.int32), zeros(B, H, keep, dtype=torch.int32)
    w, w2, o8 = zeros(B, H, S + 8, dtype=torch.float32), zeros(B, H, keep, dtype=torch.float32), zeros(B, 4, Hq, dh)
    ko, vo = zeros(B, keep, H, dh), zeros(B, keep, H, dh)
    ws8 = mka.buffer(mka.mka_kv8_attention_workspace_size(c8, 4, True))
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(stream):
            w.zero_()
        mka.mka_window_attention(c, q, k, v, lens, out, lse, stream=stream)
        mka.mka_window_attention_backward(c, q, k, v, out, lse, do, lens, dq, dk, dv, ws, stream=stream)
        mka.mka_kv8_append(c8, a, k, v, at, stream=stream)
        mka.mka_kv8_attention(c8, a, q4, lens, o8, w, ws8, stream=stream)
        mka.mka_kv8_evict(c8, a, lens, w, keep, 3, 20, d8, d, l2, w2, kept, ws8, stream=stream)
        mka.mka_kv8_read(d8, d, None, l2, ko, vo, stream=stream)
    stream.synchronize()
    return [t.cpu() for t in (out, dq, dk, dv, o8, w, kept, w2, ko, vo)]


@pytest.mark.gpu
@pytest.mark.parametrize("dh", [64, 128])
def test_two_threads_on_two_streams(mka, dh):
    """Calls of two threads at once, each on a stream and with buffers of its own, give what they give alone."""
    alone = [steps_on(mka, seed, dh, torch.cuda.current_stream()) for seed in (1, 2)]
    got = [None, None]

    def work(i, stream):
        got[i] = steps_on(mka, i + 1, dh, stream)
    threads = [threading.Thread(target=work, args=(i, torch.cuda.Stream())) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert got[i] is not None
        for x, y in zip(alone[i], got[i]):
            assert torch.equal(x, y)
    assert mka.mka_status() == 0


@pytest.mark.gpu
def test_first_calls_of_a_process_may_be_captured():
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", CAPTURED_FIRST % (os.path.dirname(here), here)], capture_output=True, text=True)
    assert r.returncode == 0 and "captured first: ok" in r.stdout, r.stderr[-2000:]
