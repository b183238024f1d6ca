"""Operands of the bounded-memory operators that overlap an output are refused on the host (no call here reaches a GPU but
the last, whose operands do not overlap)."""
import ctypes

import pytest
import torch

import bounded_ref as ref


@pytest.fixture(scope="module")
def mka():
    import route_kv_memory_b200 as m
    return m


MB = 1 << 20


class Call:
    """A call, and addresses of its operands that lie 16 MB apart."""

    def __init__(self, fn, order):
        self.fn = fn
        self.at = {n: (16 * i + 16) * MB for i, n in enumerate(order)}


def refused(mka, call, a, b, at=16):
    """With operand a moved into b, `at` bytes behind its start."""
    rc = call.fn({**call.at, a: call.at[b] + at})
    text = mka._lib.mka_last_error().decode()
    assert rc == mka.MKA_ERR_INVALID_ARG and "overlap" in text, (a, b, rc, text)


def p(x):
    return ctypes.c_void_p(x)


def cache(mka, at, pre=""):
    return mka.mka_kv8_cache(at[pre + "k"], at[pre + "v"], at[pre + "ks"], at[pre + "vs"])


def pairs(outs, ins):
    return [(a, b) for i, a in enumerate(outs) for b in outs[:i] + ins]


def test_evict(mka):
    B, H, L, dh, keep = 300, 2, 100, 64, 50
    c, d = mka.make_kv8_config(B, L, 4, H, dh), mka.make_kv8_config(B, keep + 3, 4, H, dh)
    outs, ins = ["dk", "dv", "dks", "dvs", "lens2", "w2", "kept"], ["k", "v", "ks", "vs", "lens", "w"]
    call = Call(lambda t: mka._lib.mka_kv8_evict(c, cache(mka, t), p(t["lens"]), p(t["w"]), keep, 3, 4, d, cache(mka, t, "d"),
                                                 p(t["lens2"]), p(t["w2"]), p(t["kept"]), p(t["ws"]), 1 << 20, None),
                outs + ins + ["ws"])
    for a, b in pairs(outs, ins):
        refused(mka, call, a, b)
    refused(mka, call, "lens", "kept", B * H * keep * 4 - 16)  # the last bytes


def test_attention(mka):
    c = mka.make_kv8_config(300, 100, 4, 2, 64)
    ws = mka.mka_kv8_attention_workspace_size(c, 3, True)
    assert ws < 16 * 16 * MB
    outs, ins = ["out", "w", "ws"], ["k", "v", "ks", "vs", "lens", "q"]
    call = Call(lambda t: mka._lib.mka_kv8_attention(c, cache(mka, t), p(t["q"]), 3, p(t["lens"]), p(t["out"]), p(t["w"]),
                                                     p(t["ws"]), ws, None), ["out", "w"] + ins + ["ws"])
    for a, b in pairs(outs, ins):
        refused(mka, call, a, b)


def test_append_and_read(mka):
    c = mka.make_kv8_config(300, 100, 4, 2, 64)
    outs, ins = ["k", "v", "ks", "vs"], ["pos", "count"]
    call = Call(lambda t: mka._lib.mka_kv8_append(c, cache(mka, t), p(t["kn"]), p(t["vn"]), 128, 1280, 10, p(t["pos"]),
                                                  p(t["count"]), None), outs + ins + ["kn", "vn"])
    for a, b in pairs(outs, ins):
        refused(mka, call, a, b)
    x, lib = mka.mka_kv8_cache(16 * MB, 32 * MB, 48 * MB, 64 * MB), mka._lib
    for k, v, bs in ((80 * MB, 80 * MB, 1280), (80 * MB, 80 * MB + 128, 1280), (80 * MB, 112 * MB, 120)):
        assert lib.mka_kv8_read(c, x, None, None, 10, p(k), p(v), 128, bs, None) == mka.MKA_ERR_INVALID_ARG
        text = lib.mka_last_error().decode()
        assert "overlap" in text or "same rows" in text


def test_window(mka):
    B, S, Hq, H, dh = 5, 200, 4, 2, 64
    c = mka.make_attn_config(B, S, Hq, H, dh, 50, 4)
    ins = ["q", "k", "v", "lens"]
    call = Call(lambda t: mka._lib.mka_window_attention(c, None, p(t["q"]), p(t["k"]), p(t["v"]), p(t["lens"]), p(t["out"]),
                                                        p(t["lse"]), None), ["out", "lse"] + ins)
    for a, b in [("out", x) for x in ins] + [("out", "lse"), ("lse", "lens")]:
        refused(mka, call, a, b)
    refused(mka, call, "out", "q", 0)
    need = mka.mka_window_attention_backward_workspace_size(c)
    outs, ins = ["dq", "dk", "dv", "ws"], ["q", "k", "v", "out", "lse", "dout", "lens"]
    call = Call(lambda t: mka._lib.mka_window_attention_backward(
        c, None, p(t["q"]), p(t["k"]), p(t["v"]), p(t["out"]), p(t["lse"]), p(t["dout"]), p(t["lens"]), p(t["dq"]), p(t["dk"]),
        p(t["dv"]), p(t["ws"]), need, None), outs + ins)
    for a, b in pairs(["dq", "dk", "dv"], ["q", "k", "v", "out", "lse", "dout", "lens"]) + [("ws", x) for x in ("dq", "dk", "lse")]:
        refused(mka, call, a, b)
    # columns of one array that overlap by the last 16 bytes of a row, and different strides
    row = (Hq + H) * dh
    for st, k in ((mka.mka_attn_strides(row, row, 0, row, 0), 2 * Hq * dh - 16), (mka.mka_attn_strides(row, row + 8, 0, row, 0), 2 * Hq * dh)):
        a = 16 * MB
        assert mka._lib.mka_window_attention(c, st, p(80 * MB), p(a + k), p(96 * MB), None, p(a), None, None) == mka.MKA_ERR_INVALID_ARG
        assert "overlap" in mka._lib.mka_last_error().decode()


@pytest.mark.gpu
def test_columns_of_one_array_do_not_overlap(mka):
    """q, k, v, out and dout as columns of one array."""
    B, S, Hq, H, dh, window, sinks = 2, 150, 4, 2, 64, 40, 2
    g = torch.Generator().manual_seed(9)
    wide = torch.randn(B, S, (3 * Hq + 2 * H) * dh, generator=g).bfloat16().cuda()
    cols, at = [], 0
    for h in (Hq, H, H, Hq, Hq):
        cols.append(wide[..., at * dh:(at + h) * dh])
        at += h
    q, k, v, out, dout = cols
    x = [t.clone().cpu().view(B, S, -1, dh) for t in (q, k, v, dout)]
    c = mka.make_attn_config(B, S, Hq, H, dh, window, sinks)
    lse, ws = mka.attention_lse(c), mka.buffer(mka.mka_window_attention_backward_workspace_size(c))
    dq, dk, dv = (torch.zeros(B, S, h, dh, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H))
    mka.mka_window_attention(c, q, k, v, None, out, lse)
    mka.mka_window_attention_backward(c, q, k, v, out, lse, dout, None, dq, dk, dv, ws)
    got = [out.cpu().view(B, S, Hq, dh), dq.cpu(), dk.cpu(), dv.cpu()]
    for b in range(B):
        y = [t[b].double() for t in x]
        want = (ref.window_forward(*y[:3], window, sinks)[0], *ref.window_backward(*y, window, sinks))
        for t, w, e in zip(got, want, ref.window_bounds(*y, window, sinks)):
            assert ((t[b].double() - w).abs() <= e).all()
    for t, s in zip((q, k, v, dout), x):
        assert torch.equal(t.cpu().view_as(s), s)
    assert mka.mka_status() == 0
