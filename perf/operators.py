"""Workloads and plain forms of the bounded-memory attention operators.

Four operators that keep a long context's attention within a bounded memory:

* window  causal GQA attention in which a token sees the last `window` positions and the first
          `sinks` ones, forward and (training) with its gradients;
* decode  attention of new tokens over a K/V cache held in 8 bits (e4m3 codes, one power-of-two
          scale per block of tokens and head), optionally adding every cached token's attention
          weight to a running total;
* append  quantising new K/V rows into that cache, and reading rows back as values;
* evict   keeping, per sequence and KV head, the first, the last and the heaviest tokens.

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, by the
library's entry points.  `exact` is their definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 64  # tokens that share a scale in the listed caches
QWEN = {"hq": 28, "hkv": 4, "dh": 128}
LLAMA = {"hq": 32, "hkv": 8, "dh": 128}
TINY = {"hq": 4, "hkv": 2, "dh": 64}


def listed():
    return [
        # one short document through a small layer: the latency of a call
        {"name": "window 1x255 tiny", "op": "window", "b": 1, "s": 255, **TINY, "window": 64, "sinks": 4,
         "train": False, "ragged": False},
        # a long prompt, each token reading its last 4096 positions
        {"name": "window 1x32768 llama", "op": "window", "b": 1, "s": 32768, **LLAMA, "window": 4096, "sinks": 4,
         "train": False, "ragged": False},
        # a training step on one odd-length sample of a small layer
        {"name": "window train 1x777 tiny", "op": "window", "b": 1, "s": 777, **TINY, "window": 100, "sinks": 3,
         "train": True, "ragged": False},
        # a training step on a padded batch of the 7B layer
        {"name": "window train 2x4096 qwen", "op": "window", "b": 2, "s": 4096, **QWEN, "window": 1024, "sinks": 4,
         "train": True, "ragged": True},
        # the first tokens of an answer in a float32 layer: latency
        {"name": "decode 1x1000 tiny f32", "op": "decode", "b": 1, "l": 1000, "n": 1, **TINY, "window": 0, "sinks": 0,
         "dtype": "f32", "weights": False, "ragged": False, "block": 32},
        # one token of one long conversation
        {"name": "decode 1x131072 qwen", "op": "decode", "b": 1, "l": 131072, "n": 1, **QWEN, "window": 0, "sinks": 0,
         "dtype": "bf16", "weights": False, "ragged": False, "block": BLOCK},
        # four drafted tokens checked at once in a batch of conversations of different lengths
        {"name": "decode 16x32768 llama draft", "op": "decode", "b": 16, "l": 32768, "n": 4, **LLAMA, "window": 0,
         "sinks": 0, "dtype": "bf16", "weights": False, "ragged": True, "block": BLOCK},
        # a batch whose cache is about to be thinned: every token's weight is added up
        {"name": "decode 8x16384 qwen weights", "op": "decode", "b": 8, "l": 16384, "n": 1, **QWEN, "window": 0,
         "sinks": 0, "dtype": "bf16", "weights": True, "ragged": True, "block": BLOCK},
        # two prompts' rows into an empty cache, and back as values
        {"name": "append 2x4096 qwen", "op": "append", "b": 2, "l": 4096, "n": 4096, **QWEN, "dtype": "bf16",
         "ragged": False, "block": BLOCK},
        # one new token of each of 64 conversations, inside blocks that hold older ones
        {"name": "append 64x1 llama", "op": "append", "b": 64, "l": 2048, "n": 1, **LLAMA, "dtype": "bf16",
         "ragged": True, "block": BLOCK},
        # a batch thinned to a quarter; a sequence that is short enough keeps all it has
        {"name": "evict 4x16384 qwen", "op": "evict", "b": 4, "l": 16384, **QWEN, "keep": 4096, "first": 4,
         "recent": 1024, "ragged": True, "block": BLOCK},
        # one long prompt's cache thinned before the answer
        {"name": "evict 1x131072 llama", "op": "evict", "b": 1, "l": 131072, **LLAMA, "keep": 8192, "first": 4,
         "recent": 2048, "ragged": False, "block": BLOCK},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads = dict(rng.choice([QWEN, LLAMA, TINY, {"hq": 8, "hkv": 8, "dh": 64}, {"hq": 12, "hkv": 1, "dh": 128}]))
    op = rng.choice(["window", "decode", "append", "evict"])
    if op == "window":
        train = rng.random() < 0.5
        b = rng.randint(1, 4)
        s = _spread(rng, 1, (6000 if train else 20000) // b)
        return {"op": op, "b": b, "s": s, **heads, "window": _spread(rng, 1, 2048), "sinks": rng.choice([0, 1, 4, 20, 130]),
                "train": train, "ragged": rng.random() < 0.5}
    block = rng.choice([16, 32, 64, 128])
    if op == "decode":
        b = _spread(rng, 1, 32)
        windowed = rng.random() < 0.4
        return {"op": op, "b": b, "l": _spread(rng, 1, 200000 // b), "n": rng.choice([1, 1, 1, 2, 3, 5, 8]), **heads,
                "window": _spread(rng, 1, 4096) if windowed else 0, "sinks": rng.choice([0, 4, 33]) if windowed else 0,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "weights": rng.random() < 0.4, "ragged": rng.random() < 0.7,
                "block": block}
    if op == "append":
        b = _spread(rng, 1, 64)
        n = _spread(rng, 1, 12000 // b)
        return {"op": op, "b": b, "l": n + rng.randint(0, 1000), "n": n, **heads, "dtype": rng.choice(["bf16", "f32"]),
                "ragged": rng.random() < 0.7, "block": block}
    b = _spread(rng, 1, 16)
    length = _spread(rng, 2, 130000 // b)
    keep = rng.randint(1, length)
    first = rng.randint(0, min(4, keep))
    return {"op": op, "b": b, "l": length, **heads, "keep": keep, "first": first,
            "recent": rng.randint(0, keep - first), "ragged": rng.random() < 0.7, "block": block}


# ---------------------------------------------------------------- inputs
def _lens(c, g, most, least=0):
    """Rows in use per sequence: all of them, or spread with the longest full."""
    if not c["ragged"]:
        return torch.full((c["b"],), most, dtype=torch.int32, device="cuda")
    x = torch.randint(least, most + 1, (c["b"],), generator=g, device="cuda", dtype=torch.int32)
    x[0] = most
    return x


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (448: the largest e4m3 value), at least 2^-120."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8).clamp(-120, 120))


def _codes(x, scale):
    return (x / scale).to(torch.float8_e4m3fn)


def _filled(c, g, length):
    """Codes and scales of `length` random rows per sequence and head: [B, H, L, dh], [B, H, L / block]."""
    nb = -(-length // c["block"])
    x = torch.randn(c["b"], c["hkv"], nb, c["block"], c["dh"], generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(c["b"], c["hkv"], nb, 1, 1, generator=g, device="cuda"))  # blocks differ in size
    sc = _pow2_scale(x.abs().amax((3, 4)))
    codes = _codes(x, sc[..., None, None]).reshape(c["b"], c["hkv"], nb * c["block"], c["dh"])
    return codes[:, :, :length].contiguous(), sc


def prepare(case, seed):
    c, g = case, torch.Generator("cuda").manual_seed(seed)
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16

    def rows(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    def zeros(*shape, dtype=dt):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    st = {"case": c}
    B, H, dh = c["b"], c["hkv"], c["dh"]
    if c["op"] == "window":
        for n, h in (("q", c["hq"]), ("k", H), ("v", H)):
            st[n] = rows(B, c["s"], h, dh)
        st["lens"] = _lens(c, g, c["s"])
        st["out"] = torch.zeros_like(st["q"])
        if c["train"]:
            st["dout"] = rows(B, c["s"], c["hq"], dh)
            st["dq"], st["dk"], st["dv"] = (torch.zeros_like(st[n]) for n in ("q", "k", "v"))
        return st
    if c["op"] == "append":
        st["pos"] = _lens(c, g, c["l"] - c["n"])
        st["count"] = _lens(c, g, c["n"], 1)
        st["k"], st["ks"] = _filled(c, g, c["l"])
        st["v"], st["vs"] = _filled(c, g, c["l"])
        st["kn"], st["vn"] = 2 * rows(B, c["n"], H, dh), 2 * rows(B, c["n"], H, dh)
        # what is read back: from the start of the first touched block
        st["first"] = st["pos"] // c["block"] * c["block"]
        st["rows"] = st["pos"] + st["count"] - st["first"]
        m = c["n"] + c["block"] - 1
        st["k_out"], st["v_out"] = zeros(B, m, H, dh), zeros(B, m, H, dh)
        return st
    st["lens"] = _lens(c, g, c["l"])
    st["k"], st["ks"] = _filled(c, g, c["l"])
    st["v"], st["vs"] = _filled(c, g, c["l"])
    if c["op"] == "decode":
        st["q"] = rows(B, c["n"], c["hq"], dh)
        st["out"] = torch.zeros_like(st["q"])
        if c["weights"]:  # totals of earlier steps; the pass adds to a copy, as a step of its own would to the total
            st["total"] = torch.rand(B, H, c["l"], generator=g, device="cuda")
            st["weights"] = torch.empty_like(st["total"])
        return st
    # totals of attention weight: a few heavy tokens, many equal light ones
    w = torch.exp(2 * torch.randn(B, H, c["l"], generator=g, device="cuda"))
    st["weights"] = torch.where(w < 0.2, torch.full_like(w, 0.125), w)
    nk = -(-c["keep"] // c["block"])
    for n in ("k", "v"):
        st[n + "2"] = zeros(B, H, c["keep"], dh, dtype=torch.float8_e4m3fn)
        st[n + "s2"] = zeros(B, H, nk, dtype=torch.float32)
        st[n + "_out"] = zeros(B, c["keep"], H, dh, dtype=torch.bfloat16)
    st["lens2"] = zeros(B, dtype=torch.int32)
    st["zero"] = zeros(B, dtype=torch.int32)
    st["weights2"] = zeros(B, H, c["keep"], dtype=torch.float32)
    st["kept"] = zeros(B, H, c["keep"], dtype=torch.int32)
    return st


# ---------------------------------------------------------------- plain forms
def _sees(t, j, window, sinks):
    """Whether the token at position t sees the one at position j."""
    m = j <= t
    return m & ((j > t - window) | (j < sinks)) if window else m


def _softmax_rows(q, k, mask):
    """P [B, H, G, n, m] of q [B, n, H, G, dh] (already scaled) over k [B, m, H, dh]; rows that see nothing are 0."""
    B, n, H, G, dh = q.shape
    s = q.permute(0, 2, 3, 1, 4).reshape(B, H, G * n, dh) @ k.permute(0, 2, 3, 1)
    s = s.view(B, H, G, n, -1).masked_fill_(~mask[:, None, None], -math.inf)
    s -= s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = s.exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(torch.where(total > 0, total, 1))


def _times_v(p, v):
    """sum_m P V: [B, n, H, G, dh]."""
    B, H, G, n, m = p.shape
    return (p.reshape(B, H, G * n, m) @ v.permute(0, 2, 1, 3)).view(B, H, G, n, -1).permute(0, 3, 1, 2, 4)


def _plain_window(st):
    c = st["case"]
    B, S, Hq, dh = st["q"].shape
    H, G, scale = c["hkv"], c["hq"] // c["hkv"], 1 / math.sqrt(dh)
    q, k, v = (st[n].float() for n in ("q", "k", "v"))
    q = q.view(B, S, H, G, dh)
    if c["train"]:
        do = st["dout"].float().view(B, S, H, G, dh)
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    at = torch.arange(S, device="cuda")
    step = 1024  # query rows at a time: the scores of all rows at once would not fit the card
    for t0 in range(0, S, step):
        t = at[t0:t0 + step]
        lo = max(0, t0 - c["window"] + 1) if c["window"] else 0
        j = torch.cat([at[:min(c["sinks"], lo)], at[lo:t0 + len(t)]])
        mask = _sees(t[:, None], j[None], c["window"], c["sinks"])[None] & (t[None, :, None] < st["lens"].view(B, 1, 1))
        kj, vj, qt = k[:, j], v[:, j], q[:, t]
        p = _softmax_rows(qt * scale, kj, mask)
        o = _times_v(p, vj)
        st["out"][:, t] = o.reshape(B, len(t), Hq, dh).to(st["out"].dtype)
        if c["train"]:
            dot = do[:, t]
            dp = (dot.permute(0, 2, 3, 1, 4).reshape(B, H, -1, dh) @ vj.permute(0, 2, 3, 1)).view_as(p)
            ds = p * (dp - (dot * o).sum(-1).permute(0, 2, 3, 1)[..., None]) * scale
            st["dq"][:, t] = _times_v(ds, kj).reshape(B, len(t), Hq, dh).to(st["dq"].dtype)
            ds, p = ds.view(B, H, -1, len(j)), p.view(B, H, -1, len(j))
            dk.index_add_(1, j, (ds.mT @ qt.permute(0, 2, 3, 1, 4).reshape(B, H, -1, dh)).permute(0, 2, 1, 3))
            dv.index_add_(1, j, (p.mT @ dot.permute(0, 2, 3, 1, 4).reshape(B, H, -1, dh)).permute(0, 2, 1, 3))
    if c["train"]:
        st["dk"].copy_(dk)
        st["dv"].copy_(dv)


def _values(codes, scale, block):
    """What the codes stand for: [B, H, L, dh] in 32 bits."""
    return codes.float() * scale.repeat_interleave(block, 2)[:, :, :codes.shape[2], None]


def _plain_decode(st):
    c = st["case"]
    B, n, Hq, dh = st["q"].shape
    H, G = c["hkv"], c["hq"] // c["hkv"]
    k = _values(st["k"], st["ks"], c["block"]).permute(0, 2, 1, 3)
    v = _values(st["v"], st["vs"], c["block"]).permute(0, 2, 1, 3)
    t = st["lens"][:, None] - n + torch.arange(n, device="cuda")
    j = torch.arange(c["l"], device="cuda")
    mask = _sees(t[:, :, None], j, c["window"], c["sinks"])
    p = _softmax_rows(st["q"].float().view(B, n, H, G, dh) / math.sqrt(dh), k, mask)
    st["out"].copy_(_times_v(p, v).reshape(B, n, Hq, dh))
    if c["weights"]:
        torch.add(st["total"], p.sum((2, 3)), out=st["weights"])


def _plain_append(st):
    c = st["case"]
    B, H, dh, n, blk = c["b"], c["hkv"], c["dh"], c["n"], c["block"]
    nb = -(-(n + blk - 1) // blk)  # blocks that the new rows may touch
    b = torch.arange(B, device="cuda")[:, None]
    row = st["first"][:, None] + torch.arange(nb * blk, device="cuda")     # positions of the touched blocks
    new = row - st["pos"][:, None]                                         # rank among the new rows
    is_new = (new >= 0) & (new < st["count"][:, None])
    is_old = new < 0
    block = row.view(B, nb, blk)[:, :, 0] // blk
    live = is_new.view(B, nb, blk).any(-1)
    had = is_old.view(B, nb, blk).any(-1)                                  # blocks that hold older rows
    for codes, scales, x, out in ((st["k"], st["ks"], st["kn"], st["k_out"]), (st["v"], st["vs"], st["vn"], st["v_out"])):
        inside, at = row < c["l"], row.clamp_max(c["l"] - 1)
        old = codes[b, :, at].float()                                      # [B, rows, H, dh]
        bi = block.clamp_max(scales.shape[2] - 1)
        old_scale = scales[b, :, bi]                                       # [B, nb, H]
        xn = x.float()[b, new.clamp(0, n - 1)] * is_new[..., None, None]
        amax = xn.abs().amax(-1).view(B, nb, blk, H).amax(2)
        scale = torch.maximum(_pow2_scale(amax), torch.where(had[..., None], old_scale, 0))
        wide = scale.repeat_interleave(blk, 1)[..., None]
        was = old_scale.repeat_interleave(blk, 1)[..., None]
        got = _codes(torch.where(is_new[..., None, None], xn, old * was), wide)
        write = ((is_new | is_old) & inside)[..., None, None].expand_as(got)
        bb, hh, dd = b[:, :, None, None], torch.arange(H, device="cuda")[:, None], torch.arange(dh, device="cuda")
        codes.view(torch.uint8)[bb.expand_as(got)[write], hh.expand_as(got)[write], at[..., None, None].expand_as(got)[write],
                                dd.expand_as(got)[write]] = got.view(torch.uint8)[write]
        bs, hs = b[:, :, None].expand_as(scale)[live], torch.arange(H, device="cuda").expand_as(scale)[live]
        scales[bs, hs, bi[..., None].expand_as(scale)[live]] = scale[live]
        m = out.shape[1]
        seen = (torch.arange(m, device="cuda") < st["rows"][:, None])[..., None, None]
        out.copy_(torch.where(seen, (got.float() * wide)[:, :m], 0))


def _plain_evict(st):
    c = st["case"]
    B, H, keep, blk, L = c["b"], c["hkv"], c["keep"], c["block"], c["l"]
    j = torch.arange(L, device="cuda")
    n = st["lens"].view(B, 1, 1)
    w = st["weights"].masked_fill((j < c["first"]) | (j >= n - c["recent"]), math.inf).masked_fill(j >= n, -math.inf)
    kept = w.sort(dim=-1, descending=True, stable=True)[1][..., :keep]          # ties: the lowest index first
    left = torch.arange(keep, device="cuda") < n                           # a short sequence keeps all it has
    kept = torch.where(left, kept, L).sort(-1)[0]
    at = kept.clamp_max(L - 1)
    st["kept"].copy_(torch.where(left, kept, -1))
    st["lens2"].copy_(st["lens"].clamp_max(keep))
    st["weights2"].copy_(torch.where(left, st["weights"].gather(2, at), 0))
    nk = -(-keep // blk)
    for name in ("k", "v"):
        x = _values(st[name], st[name + "s"], blk).gather(2, at[..., None].expand(-1, -1, -1, c["dh"]))
        x = torch.where(left[..., None], x, 0)
        x = torch.nn.functional.pad(x, (0, 0, 0, nk * blk - keep)).view(B, H, nk, blk, -1)
        scale = _pow2_scale(x.abs().amax((3, 4)))
        codes = _codes(x, scale[..., None, None])
        st[name + "2"].copy_(codes.view(B, H, nk * blk, -1)[:, :, :keep])
        st[name + "s2"].copy_(scale)
        x = (codes.float() * scale[..., None, None]).view(B, H, nk * blk, -1)[:, :, :keep]
        st[name + "_out"].copy_(x.permute(0, 2, 1, 3))


# ---------------------------------------------------------------- the library's entry points
def _plan(st):
    """The configuration, views and scratch that a user's program keeps from call to call."""
    import route_kv_memory_b200 as mka
    c = st["case"]
    if c["op"] == "window":
        cfg = mka.make_attn_config(c["b"], c["s"], c["hq"], c["hkv"], c["dh"], window=c["window"], sinks=c["sinks"])
        if not c["train"]:
            return mka, cfg, None, None
        return mka, cfg, mka.attention_lse(cfg), mka.buffer(mka.mka_window_attention_backward_workspace_size(cfg))
    cfg = mka.make_kv8_config(c["b"], c["l"], c["hq"], c["hkv"], c["dh"], block=c["block"], dtype=c.get("dtype", "bf16"),
                              window=c.get("window", 0), sinks=c.get("sinks", 0))
    cache = mka.kv8_cache(st["k"], st["v"], st["ks"], st["vs"])
    if c["op"] == "decode":
        return mka, cfg, cache, mka.buffer(mka.mka_kv8_attention_workspace_size(cfg, c["n"], c["weights"]))
    if c["op"] == "append":
        return mka, cfg, cache, None
    cfg2 = mka.make_kv8_config(c["b"], c["keep"], c["hq"], c["hkv"], c["dh"], block=c["block"])
    cache2 = mka.kv8_cache(st["k2"], st["v2"], st["ks2"], st["vs2"])
    return mka, cfg, cache, mka.buffer(mka.mka_kv8_evict_workspace_size(cfg, c["keep"])), cfg2, cache2


def _call(st):
    if "plan" not in st:
        st["plan"] = _plan(st)
    c = st["case"]
    mka, cfg, x, ws = st["plan"][:4]
    if c["op"] == "window":
        mka.mka_window_attention(cfg, st["q"], st["k"], st["v"], st["lens"], st["out"], x)
        if c["train"]:
            mka.mka_window_attention_backward(cfg, st["q"], st["k"], st["v"], st["out"], x, st["dout"], st["lens"],
                                              st["dq"], st["dk"], st["dv"], ws)
    elif c["op"] == "decode":
        if c["weights"]:
            st["weights"].copy_(st["total"])
        mka.mka_kv8_attention(cfg, x, st["q"], st["lens"], st["out"], st.get("weights"), ws)
    elif c["op"] == "append":
        mka.mka_kv8_append(cfg, x, st["kn"], st["vn"], st["pos"], st["count"])
        mka.mka_kv8_read(cfg, x, st["first"], st["rows"], st["k_out"], st["v_out"])
    else:
        cfg2, x2 = st["plan"][4:]
        mka.mka_kv8_evict(cfg, x, st["lens"], st["weights"], c["keep"], c["first"], c["recent"], cfg2, x2, st["lens2"],
                          st["weights2"], st["kept"], ws)
        mka.mka_kv8_read(cfg2, x2, st["zero"], st["lens2"], st["k_out"], st["v_out"])


def run(state):
    st, c = state, state["case"]
    if own:
        _call(st)
    else:
        {"window": _plain_window, "decode": _plain_decode, "append": _plain_append, "evict": _plain_evict}[c["op"]](st)
    if c["op"] == "window":
        return {n: st[n] for n in (("out", "dq", "dk", "dv") if c["train"] else ("out",))}
    if c["op"] == "decode":
        return {n: st[n] for n in (("out", "weights") if c["weights"] else ("out",))}
    if c["op"] == "append":
        return {n: st[n] for n in ("k_out", "v_out", "ks", "vs")}
    return {n: st[n] for n in ("kept", "lens2", "weights2", "k_out", "v_out")}


def work(case):
    c = case
    row = c["hkv"] * c["dh"]
    e = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "window":
        w, s, extra = min(c["window"] or c["s"], c["s"]), c["s"], 0
        pairs = w * (w + 1) // 2 + (s - w) * w
        if c["sinks"] and s > w:  # sinks that the window has left behind
            x = min(c["sinks"], s - w)
            extra = x * (x + 1) // 2 + (s - w - x) * x
        full = (c["b"] + 1) / 2 if c["ragged"] else c["b"]                  # sequences' worth of rows in use
        pairs = full * (pairs + extra)
        moved = full * s * c["dh"] * 2 * (c["hq"] + c["hkv"])               # half of q, k, v in, o out
        if not c["train"]:
            return {"bytes": 2 * moved, "flops": 4 * c["dh"] * c["hq"] * pairs}
        # dO in, dq, dk, dv out; five products behind the forward's two
        return {"bytes": 2 * moved + full * s * c["dh"] * 2 * (2 * c["hq"] + 2 * c["hkv"]),
                "flops": 14 * c["dh"] * c["hq"] * pairs}
    if c["op"] == "decode":
        seen = min(c["l"], c["window"] + c["sinks"] + c["n"] - 1) if c["window"] else c["l"]
        mean = (c["l"] + seen * (c["b"] - 1) / 2) / c["b"] if c["ragged"] and not c["window"] else seen
        io = 2 * c["b"] * c["n"] * c["hq"] * c["dh"] * e
        more = 8 * c["b"] * c["hkv"] * mean if c["weights"] else 0
        return {"bytes": 2 * c["b"] * mean * row + io + more, "flops": 4 * c["dh"] * c["hq"] * c["n"] * c["b"] * mean}
    if c["op"] == "append":  # rows in, codes out and in, values out
        mean = (c["n"] + c["n"] * (c["b"] - 1) / 2) / c["b"] if c["ragged"] else c["n"]
        return {"bytes": 2 * c["b"] * mean * row * (e + 1 + 1 + e), "flops": 0}
    # weights in; kept rows in, out, in again and out as values
    mean = (c["l"] + c["l"] * (c["b"] - 1) / 2) / c["b"] if c["ragged"] else c["l"]
    return {"bytes": c["b"] * (4 * mean * c["hkv"] + 2 * min(mean, c["keep"]) * row * (1 + 1 + 1 + 2)), "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits
def _e4m3_64(x):
    """x rounded to the nearest e4m3 value, ties to even: 3 fraction bits down to the exponent -6."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _scale_64(amax):
    """Powers of two s, tried from below, until amax <= 448 s."""
    x = torch.floor(torch.log2((amax / 448).clamp_min(2.0 ** -140))).clamp_min(-120) - 1
    x = torch.where(448 * torch.exp2(x) < amax, x + 1, x)
    x = torch.where(448 * torch.exp2(x) < amax, x + 1, x)
    return torch.exp2(x.clamp_min(-120))


def _exact_window(st, c):
    """Row blocks of one head at a time, gradients by differentiating the definition."""
    B, S, dh, G = c["b"], c["s"], c["dh"], c["hq"] // c["hkv"]
    x = {n: st[n].double() for n in ("q", "k", "v")}
    out = torch.zeros_like(x["q"])
    grads = {n: torch.zeros_like(x[n]) for n in x} if c["train"] else {}
    for b in range(B):
        n = int(st["lens"][b])
        for h in range(c["hq"]):
            for t0 in range(0, n, 4096):
                t1 = min(n, t0 + 4096)
                lo = max(0, t0 - c["window"] + 1) if c["window"] else 0
                head = min(c["sinks"], lo)
                pos = torch.cat([torch.arange(head), torch.arange(lo, t1)]).cuda()
                part = [x["q"][b, t0:t1, h].clone(), x["k"][b, pos, h // G].clone(), x["v"][b, pos, h // G].clone()]
                with torch.set_grad_enabled(c["train"]):
                    for p in part:
                        p.requires_grad_(c["train"])
                    far = torch.arange(t0, t1, device="cuda")[:, None] - pos[None]
                    hidden = far < 0
                    if c["window"]:
                        hidden = hidden | ((far >= c["window"]) & (pos[None] >= c["sinks"]))
                    o = torch.softmax((part[0] @ part[1].T / math.sqrt(dh)).masked_fill(hidden, -math.inf), -1) @ part[2]
                    out[b, t0:t1, h] = o.detach()
                    if c["train"]:
                        dq, dk, dv = torch.autograd.grad(o, part, st["dout"][b, t0:t1, h].double())
                        grads["q"][b, t0:t1, h] = dq
                        grads["k"][b, :, h // G].index_add_(0, pos, dk)
                        grads["v"][b, :, h // G].index_add_(0, pos, dv)
    return {"out": out, **{"d" + n: g for n, g in grads.items()}}


def _exact_decode(st, c):
    G, n, L = c["hq"] // c["hkv"], c["n"], c["l"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    total = st["total"].double() if c["weights"] else None
    of = torch.arange(L, device="cuda")
    for b in range(c["b"]):
        for g in range(c["hkv"]):
            k = st["k"][b, g].double() * st["ks"][b, g, of // c["block"], None].double()
            v = st["v"][b, g].double() * st["vs"][b, g, of // c["block"], None].double()
            for i in range(n):
                t = int(st["lens"][b]) - n + i
                see = [j for j in ([(0, t + 1)] if not c["window"] or t + 1 <= c["window"] else
                                   [(0, min(c["sinks"], t + 1 - c["window"])), (t + 1 - c["window"], t + 1)]) if j[1] > j[0]]
                if not see:
                    continue
                j = torch.cat([of[a:z] for a, z in see])
                w = torch.softmax(st["q"][b, i, g * G:(g + 1) * G].double() @ k[j].T / math.sqrt(c["dh"]), -1)
                out[b, i, g * G:(g + 1) * G] = w @ v[j]
                if total is not None:
                    total[b, g, j] += w.sum(0)
    return {"out": out, **({"weights": total} if c["weights"] else {})}


def _exact_append(st, c):
    got = {"ks": st["ks"].double(), "vs": st["vs"].double()}
    blk = c["block"]
    for codes, sc, x, o in (("k", "ks", "kn", "k_out"), ("v", "vs", "vn", "v_out")):
        got[o] = torch.zeros(st[o].shape, dtype=torch.float64, device="cuda")
        for b in range(c["b"]):
            p, n = int(st["pos"][b]), int(st["count"][b])
            a = p // blk * blk
            old = st[codes][b, :, a:p].double() * st[sc][b, :, a // blk, None, None].double()
            rows = torch.cat([old, st[x][b, :n].double().permute(1, 0, 2)], 1)              # [H, rows, dh]
            nb = -(-rows.shape[1] // blk)
            pad = torch.nn.functional.pad(rows, (0, 0, 0, nb * blk - rows.shape[1]))
            fresh = pad.clone()
            fresh[:, :p - a] = 0
            s = _scale_64(fresh.view(c["hkv"], nb, blk, -1).abs().amax((2, 3)))
            if p > a:
                s[:, 0] = torch.maximum(s[:, 0], st[sc][b, :, a // blk].double())
            got[sc][b, :, a // blk:a // blk + nb] = s
            wide = s.repeat_interleave(blk, 1)[..., None]
            got[o][b, :rows.shape[1]] = (_e4m3_64(pad / wide) * wide)[:, :rows.shape[1]].permute(1, 0, 2)
    return got


def _exact_evict(st, c):
    keep, blk = c["keep"], c["block"]
    kept = torch.full((c["b"], c["hkv"], keep), -1, dtype=torch.int64)
    w2 = torch.zeros(c["b"], c["hkv"], keep, dtype=torch.float64, device="cuda")
    kv = {n: torch.zeros(c["b"], keep, c["hkv"], c["dh"], dtype=torch.float64, device="cuda") for n in "kv"}
    for b in range(c["b"]):
        n = int(st["lens"][b])
        for g in range(c["hkv"]):
            if n <= keep:
                pick = torch.arange(n, device="cuda")
            else:  # the rest of the budget, heaviest first, by (weight down, index up)
                mid = torch.arange(c["first"], n - c["recent"], device="cuda")
                order = torch.sort(-st["weights"][b, g, mid].double(), stable=True)[1][:keep - c["first"] - c["recent"]]
                pick = torch.cat([torch.arange(c["first"], device="cuda"), mid[order].sort()[0],
                                  torch.arange(n - c["recent"], n, device="cuda")])
            m = len(pick)
            kept[b, g, :m] = pick.cpu()
            w2[b, g, :m] = st["weights"][b, g, pick].double()
            for name in "kv":
                x = st[name][b, g, pick].double() * st[name + "s"][b, g, pick // blk, None].double()
                for a in range(0, m, blk):
                    s = _scale_64(x[a:a + blk].abs().max())
                    kv[name][b, a:a + blk, g][:m - a] = _e4m3_64(x[a:a + blk] / s) * s
    return {"kept": kept, "lens2": st["lens"].clamp_max(keep), "weights2": w2, "k_out": kv["k"], "v_out": kv["v"]}


def exact(case, seed):
    st = prepare(case, seed)
    return {"window": _exact_window, "decode": _exact_decode, "append": _exact_append, "evict": _exact_evict}[case["op"]](st, case)
