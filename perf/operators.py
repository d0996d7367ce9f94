"""The library's operators around its causal attention, as measured cases: attention under
a key span per query row (documents, windows, prefixes, padding; capped scores, distance
bias) with its gradients, one-token attention over a paged cache of unequal sequences, and
the per-head norm and rotary positions of queries and keys, for training and for appending
new tokens to the paged cache.

`run` computes a case in plain torch operations in 32 bits (angles in 64), or, where `own`
is true, by the package's calls; `exact` computes it in 64 bits, head by head.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ESIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # training on packed documents at long context: each token sees its own
        # document up to itself (the largest case)
        dict(name="train_documents_8k", op="train", dtype="bf16", B=1, Hq=32, Hkv=8, Sq=8192,
             Skv=8192, d=128, mask="documents", span=2048, mask_seed=1, softcap=0.0, alibi=False),
        # a small model's training step with a sliding window and a distance bias
        dict(name="train_window_alibi", op="train", dtype="bf16", B=8, Hq=12, Hkv=12, Sq=1024,
             Skv=1024, d=64, mask="window", span=256, mask_seed=2, softcap=0.0, alibi=True),
        # a padded batch of odd length (rows past each sequence see nothing), capped scores
        dict(name="train_padded_softcap", op="train", dtype="fp16", B=3, Hq=8, Hkv=2, Sq=1537,
             Skv=1537, d=128, mask="padded", span=700, mask_seed=3, softcap=30.0, alibi=False),
        # a chunk of queries at the end of a longer context whose first part every row sees
        dict(name="prefill_prefix_softcap", op="prefill", dtype="bf16", B=1, Hq=32, Hkv=8,
             Sq=2048, Skv=8192, d=128, mask="prefix", span=7000, mask_seed=4, softcap=50.0,
             alibi=False),
        # a short prompt: latency of one forward call
        dict(name="prefill_short", op="prefill", dtype="fp16", B=1, Hq=12, Hkv=12, Sq=77,
             Skv=77, d=64, mask="prefix", span=20, mask_seed=5, softcap=0.0, alibi=True),
        # a serving step: one new token of each of 16 sequences of unequal length
        dict(name="decode_ragged_8k", op="decode", dtype="bf16", B=16, Hq=32, Hkv=8, Sq=1,
             d=128, block=64, min_len=1, max_len=8192, len_seed=6, window=0, softcap=0.0,
             alibi=False),
        # one short stream: latency of one decoding call
        dict(name="decode_one_stream", op="decode", dtype="fp16", B=1, Hq=12, Hkv=12, Sq=1,
             d=64, block=16, min_len=500, max_len=501, len_seed=7, window=0, softcap=0.0,
             alibi=True),
        # four speculated tokens a sequence over long caches, capped scores
        dict(name="decode_spec_32k", op="decode", dtype="bf16", B=2, Hq=32, Hkv=8, Sq=4,
             d=128, block=128, min_len=20000, max_len=32768, len_seed=8, window=0,
             softcap=50.0, alibi=False),
        # queries and keys of a training batch: norm and rotation, forward and backward
        dict(name="heads_train", op="heads", dtype="bf16", B=4, Hq=32, Hkv=8, S=2048, d=128,
             rope_dim=128, interleaved=False, norm=True, packed=True, far=0),
        # rotation of part of the head, interleaved, fp32, far positions
        dict(name="heads_train_partial", op="heads", dtype="fp32", B=1, Hq=12, Hkv=12, S=1999,
             d=64, rope_dim=32, interleaved=True, norm=False, packed=False, far=500000),
        # a serving step's new token of each sequence into the paged cache
        dict(name="append_step", op="append", dtype="bf16", B=16, Hq=32, Hkv=8, Sq=1, d=128,
             block=64, min_len=1, max_len=8192, len_seed=9, rope_dim=128, interleaved=False,
             norm=True),
        # prompts of odd length into the paged cache
        dict(name="append_prompt", op="append", dtype="fp16", B=3, Hq=16, Hkv=4, Sq=1025,
             d=64, block=16, min_len=1025, max_len=3000, len_seed=10, rope_dim=64,
             interleaved=False, norm=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    Hkv = rng.choice([1, 2, 3, 4, 8, 12])
    G = rng.choice([1, 1, 2, 4, 8]) if Hkv < 12 else 1
    return Hkv * G, Hkv


def draw(rng):
    op = rng.choice(["train", "train", "prefill", "decode", "decode", "heads", "append"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), d=rng.choice([64, 128]))
    c["Hq"], c["Hkv"] = _heads(rng)
    if op in ("train", "prefill"):
        c["Sq"] = _log_int(rng, 33, 6000)
        c["Skv"] = c["Sq"] + (rng.choice([0, _log_int(rng, 1, 4000)]) if op == "prefill" else 0)
        while 14 * c["d"] * c["Hq"] * c["Sq"] * c["Skv"] > 4.2e11:
            c["Sq"], c["Skv"] = c["Sq"] * 2 // 3, c["Skv"] - c["Sq"] + c["Sq"] * 2 // 3
        fit = int(4.2e11 / (14.0 * c["d"] * c["Hq"] * c["Sq"] * c["Skv"]))
        c["B"] = max(1, min(rng.choice([1, 1, 2, 3, 5, 8]), fit))
        c["mask"] = rng.choice(["documents", "window", "prefix", "padded"])
        c["span"] = _log_int(rng, 24, max(24, c["Skv"]))
        c["mask_seed"] = rng.randrange(1 << 20)
        c["softcap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
        c["alibi"] = rng.random() < 0.3
    elif op == "decode":
        c["Sq"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        c["max_len"] = _log_int(rng, 40, 32768)
        c["min_len"] = rng.choice([1, c["max_len"] // 2 + 1])
        fit = 16 * 8 * 8192 * 128 // (c["Hkv"] * c["max_len"] * c["d"])
        c["B"] = max(1, min(_log_int(rng, 1, 96), fit))
        c["block"] = rng.choice([16, 32, 64, 128, 256])
        c["len_seed"] = rng.randrange(1 << 20)
        c["window"] = rng.choice([0, 0, _log_int(rng, 32, c["max_len"])])
        c["softcap"] = rng.choice([0.0, 0.0, 30.0])
        c["alibi"] = rng.random() < 0.3
    else:
        c["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
        c["rope_dim"] = rng.choice([16, 32, 48, c["d"], c["d"], c["d"]])
        c["interleaved"] = rng.random() < 0.5
        c["norm"] = rng.random() < 0.7
        if op == "heads":
            c["S"] = _log_int(rng, 1, 8000)
            c["B"] = max(1, min(rng.choice([1, 2, 3, 4]), 4 * 2048 * 32 // (c["S"] * c["Hq"])))
            c["packed"] = rng.random() < 0.5
            c["far"] = rng.choice([0, 0, 100000, 1000000])
        else:
            c["Sq"] = rng.choice([1, 1, 4, _log_int(rng, 1, 1500)])
            c["max_len"] = c["Sq"] + _log_int(rng, 1, 4000)
            c["min_len"] = c["Sq"]
            c["B"] = max(1, min(_log_int(rng, 1, 64), 40000 // c["max_len"]))
            c["block"] = rng.choice([16, 32, 64, 256])
            c["len_seed"] = rng.randrange(1 << 20)
    return c


# --------------------------------------------------------- what a case fixes --
def _spans(c):
    """int32 [B, Sq] arrays key_begin, key_end: row i sees keys key_begin <= j < key_end.
    Row i stands at position i + Skv - Sq."""
    rng = random.Random(c["mask_seed"])
    B, Sq, Skv, n = c["B"], c["Sq"], c["Skv"], c["span"]
    pos = np.arange(Sq) + (Skv - Sq)
    lo, hi = np.zeros((B, Sq), np.int32), np.zeros((B, Sq), np.int32)
    for b in range(B):
        hi[b] = pos + 1
        if c["mask"] == "documents":         # packed documents, `span` tokens at most
            start = np.zeros(Skv, np.int64)
            at = 0
            while at < Skv:
                m = _log_int(rng, max(1, n // 16), n)
                start[at: at + m] = at
                at += m
            lo[b] = start[pos]
        elif c["mask"] == "window":          # the last `span` keys
            lo[b] = np.maximum(pos + 1 - n, 0)
        elif c["mask"] == "prefix":          # a prefix that every row sees, then causal
            m = rng.randint(1, min(n, Skv))
            hi[b] = np.maximum(pos + 1, m)
        else:                                # padded: rows past the sequence see nothing
            m = rng.randint(min(n, Skv), Skv)
            hi[b] = np.where(pos < m, pos + 1, 0)
    return lo, hi


def _lens(c):
    rng = random.Random(c["len_seed"])
    lens = [rng.randint(c["min_len"], c["max_len"]) for _ in range(c["B"])]
    lens[rng.randrange(c["B"])] = c["max_len"]
    return lens


def _inv_freq(c):
    """Rotary frequencies of the first rope_dim elements of a head (base 10000), the slower
    ones stretched four times, as for contexts longer than the trained one."""
    f = 10000.0 ** (-np.arange(0, c["rope_dim"], 2, dtype=np.float64) / c["rope_dim"])
    ramp = np.clip((f * 8192 / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
    return f * (ramp + (1.0 - ramp) / 4.0)


def _turns(inv_freq):
    """Turns a position, in units of 2^-64 (the table that the calls take)."""
    out = np.array([int(round(float(f) / (2 * math.pi) * 2.0 ** 64)) % (1 << 64)
                    for f in inv_freq], dtype=np.uint64)
    return torch.from_numpy(out.view(np.int64).copy())


def _slopes(c):
    h = np.arange(1, c["Hq"] + 1, dtype=np.float64)
    return torch.from_numpy((2.0 ** (-8.0 * h / c["Hq"])).astype(np.float32)).to(DEV)


def work(c):
    op, d, e = c["op"], c["d"], ESIZE[c["dtype"]]
    if op in ("train", "prefill"):
        lo, hi = _spans(c)
        pairs = float(np.maximum(hi.astype(np.int64) - lo, 0).sum()) * c["Hq"]
        nq, nk = c["B"] * c["Hq"] * c["Sq"], c["B"] * c["Hkv"] * c["Skv"]
        n = (2 * nq + 2 * nk) * d * e + nq * 4 + 8 * c["B"] * c["Sq"]
        if op == "prefill":
            return {"bytes": n, "flops": 4 * d * pairs}
        return {"bytes": n + (2 * nq + 2 * nk) * d * e, "flops": 14 * d * pairs}
    if op == "decode":
        keys = pairs = 0
        for L in _lens(c):
            first = max(0, L - c["Sq"] + 1 - c["window"]) if c["window"] else 0
            keys += L - first
            for s in range(c["Sq"]):
                p = L - c["Sq"] + s
                pairs += max(0, min(p + 1, c["window"] or p + 1))
        n = 2 * keys * c["Hkv"] * d * e + c["B"] * c["Hq"] * c["Sq"] * (2 * d * e + 4)
        return {"bytes": n, "flops": 4 * d * pairs * c["Hq"]}
    if op == "heads":
        n = c["B"] * c["S"] * (c["Hq"] + c["Hkv"]) * d
        # forward reads and writes once; backward reads the gradient (and, under the
        # norm, the input again) and writes a gradient
        return {"bytes": (5 if c["norm"] else 4) * n * e + 8 * c["B"] * c["S"],
                "flops": (25 if c["norm"] else 6) * n}
    n = c["B"] * c["Sq"] * d
    return {"bytes": 2 * n * (c["Hq"] + 2 * c["Hkv"]) * e,
            "flops": (10 if c["norm"] else 3) * n * (c["Hq"] + c["Hkv"])}


# ----------------------------------------------------------------- prepare --
def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dt)

    st = dict(c)
    d = c["d"]
    if c["op"] in ("train", "prefill"):
        # capped scores are those of a model that needs the cap: larger than 1
        st["q"] = randn(c["B"], c["Hq"], c["Sq"], d, scale=3.0 if c["softcap"] else 1.0)
        st["k"] = randn(c["B"], c["Hkv"], c["Skv"], d)
        st["v"] = randn(c["B"], c["Hkv"], c["Skv"], d)
        if c["op"] == "train":
            st["dout"] = randn(c["B"], c["Hq"], c["Sq"], d)
        lo, hi = _spans(c)
        st["key_begin"], st["key_end"] = (torch.from_numpy(x).to(DEV) for x in (lo, hi))
        st["slopes"] = _slopes(c) if c["alibi"] else None
        return st
    if c["op"] == "heads":
        B, S, Hq, Hkv = c["B"], c["S"], c["Hq"], c["Hkv"]
        if c["packed"]:              # views of one projection's rows [q | k | v]
            x = randn(B, S, Hq + 2 * Hkv, d)
            st["q"], st["k"] = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
        else:
            st["q"] = randn(B, S, Hq, d).transpose(1, 2)
            st["k"] = randn(B, S, Hkv, d).transpose(1, 2)
        st["dq_out"], st["dk_out"] = randn(B, Hq, S, d), randn(B, Hkv, S, d)
        st["positions"] = (torch.arange(S, dtype=torch.int32, device=DEV)[None, :]
                           + c["far"] * torch.arange(1, B + 1, dtype=torch.int32, device=DEV)[:, None]
                           ).contiguous()
    else:
        lens = _lens(c)
        B, bs = c["B"], c["block"]
        per = [-(-L // bs) for L in lens]
        n_blocks = sum(per) + 3
        perm = torch.randperm(n_blocks, generator=g, device=DEV)[: sum(per)].to(torch.int32)
        table = torch.full((B, max(per)), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = perm[at: at + n]
            at += n
        st["block_table"] = table
        st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["k_cache"] = randn(n_blocks, c["Hkv"], bs, d)
        st["v_cache"] = randn(n_blocks, c["Hkv"], bs, d)
        if c["op"] == "decode":
            st["q"] = randn(B, c["Hq"], c["Sq"], d, scale=3.0 if c["softcap"] else 1.0)
            st["slopes"] = _slopes(c) if c["alibi"] else None
            return st
        x = randn(B, c["Sq"], c["Hq"] + 2 * c["Hkv"], d)
        st["q"], st["k"], st["v"] = (t.transpose(1, 2) for t in
                                     x.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2))
    f = _inv_freq(c)
    st["inv_freq"] = torch.from_numpy(f).to(DEV)
    st["turns"] = _turns(f).to(DEV)
    st["q_weight"] = (1 + 0.2 * randn(d).float()).to(dt) if c["norm"] else None
    st["k_weight"] = (1 + 0.2 * randn(d).float()).to(dt) if c["norm"] else None
    return st


EPS = 1e-6


# ------------------------------------------------------------------- plain --
def _grouped(q, Hkv):
    """[B, Hq, S, d] -> [B, Hkv, G * S, d]: the query heads of one key/value head together."""
    B, Hq, S, d = q.shape
    return q.reshape(B, Hkv, Hq // Hkv * S, d)


def _scores(st, q, k, visible, distance):
    """Scaled, capped, biased and masked scores [B, Hkv, G * Sq, Skv] and the derivative of
    the cap (None without one). visible, distance: [B, Sq, Skv]."""
    B, Hq, Sq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    s = torch.matmul(_grouped(q, Hkv), k.transpose(2, 3)) / math.sqrt(d)
    slope = None
    if st["softcap"]:
        t = torch.tanh(s / st["softcap"])
        s, slope = st["softcap"] * t, 1 - t * t
    s = s.view(B, Hkv, G, Sq, -1)
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, Hkv, G, 1, 1) * distance[:, None, None].float()
    s = torch.where(visible[:, None, None], s, -math.inf).view(B, Hkv, G * Sq, -1)
    return s, slope


def _softmax(s):
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(dim=-1, keepdim=True)
    return p / torch.where(l == 0, torch.ones_like(l), l), (m + torch.log(l)).squeeze(-1)


def _plain_attention(st, k, v, visible, distance, dout=None):
    q = st["q"].float()
    B, Hq, Sq, d = q.shape
    Hkv, dt = k.shape[1], st["q"].dtype
    s, slope = _scores(st, q, k, visible, distance)
    p, lse = _softmax(s)
    del s
    out = torch.matmul(p, v)
    res = {"out": out.view(B, Hq, Sq, d).to(dt), "lse": lse.view(B, Hq, Sq)}
    if dout is None:
        return res
    do = _grouped(dout.float(), Hkv)
    res["dv"] = torch.matmul(p.transpose(2, 3), do).to(dt)
    ds = torch.matmul(do, v.transpose(2, 3))
    ds = p * (ds - (do * out).sum(dim=-1, keepdim=True))
    if slope is not None:
        ds = ds * slope
    ds = ds / math.sqrt(d)
    res["dq"] = torch.matmul(ds, k).view(B, Hq, Sq, d).to(dt)
    res["dk"] = torch.matmul(ds.transpose(2, 3), _grouped(q, Hkv)).to(dt)
    return res


def _plain_spans(st):
    j = torch.arange(st["Skv"], device=DEV)
    pos = torch.arange(st["Sq"], device=DEV) + (st["Skv"] - st["Sq"])
    visible = (j >= st["key_begin"][:, :, None]) & (j < st["key_end"][:, :, None])
    distance = (pos[:, None] - j).abs()[None]
    return _plain_attention(st, st["k"].float(), st["v"].float(), visible, distance,
                            st.get("dout"))


def _plain_decode(st):
    n = st["block_table"].shape[1] * st["block"]
    B, Hkv, d = st["B"], st["Hkv"], st["d"]
    at = st["block_table"].clamp(min=0).long()
    k, v = (st[x][at].transpose(1, 2).reshape(B, Hkv, n, d) for x in ("k_cache", "v_cache"))
    lens = st["seq_lens"]
    j = torch.arange(n, device=DEV)
    pos = lens[:, None] - st["Sq"] + torch.arange(st["Sq"], device=DEV)
    distance = pos[:, :, None] - j
    visible = distance >= 0
    if st["window"]:
        visible = visible & (distance < st["window"])
    # the last page's rows past the sequence belong to nobody
    v = torch.where((j < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
    return _plain_attention(st, k.float(), v.float(), visible, distance)


def _cos_sin(st, positions):
    a = positions.double()[:, None, :, None] * st["inv_freq"]
    return torch.cos(a).float(), torch.sin(a).float()          # [B, 1, S, rope_dim / 2]


def _rotate(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    y, rest = x[..., :r], x[..., r:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = y[..., : r // 2], y[..., r // 2:]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((y, rest), dim=-1)


def _norm_rotate(x, w, cos, sin, interleaved):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w.float()
    return _rotate(x, cos, sin, interleaved)


def _norm_rotate_backward(dy, x, w, cos, sin, interleaved):
    dz = _rotate(dy.float(), cos, -sin, interleaved)
    if w is None:
        return dz.to(x.dtype), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
    gx = dz * w.float()
    dx = r * (gx - x * (r * r) * (gx * x).mean(dim=-1, keepdim=True))
    return dx.to(dy.dtype), (dz * x * r).sum(dim=(0, 1, 2))


def _plain_heads(st):
    cos, sin = _cos_sin(st, st["positions"])
    il, dt, res = st["interleaved"], st["q"].dtype, {}
    for n in ("q", "k"):
        w = st[n + "_weight"]
        res[n + "_out"] = _norm_rotate(st[n], w, cos, sin, il).to(dt)
        res["d" + n], dw = _norm_rotate_backward(st["d%s_out" % n], st[n], w, cos, sin, il)
        if dw is not None:
            res["d%s_weight" % n] = dw
    return res


def _plain_append(st):
    bs, Sq, dt = st["block"], st["Sq"], st["q"].dtype
    pos = st["seq_lens"][:, None] - Sq + torch.arange(Sq, device=DEV)
    cos, sin = _cos_sin(st, pos)
    il = st["interleaved"]
    q = _norm_rotate(st["q"], st["q_weight"], cos, sin, il).to(dt)
    k = _norm_rotate(st["k"], st["k_weight"], cos, sin, il).to(dt)
    page = torch.gather(st["block_table"].long(), 1, pos.long() // bs)
    row = pos.long() % bs
    st["k_cache"][page, :, row] = k.transpose(1, 2)
    st["v_cache"][page, :, row] = st["v"].transpose(1, 2)
    return {"q_out": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def run(state):
    st = state
    op = st["op"]
    if not own:
        return {"train": _plain_spans, "prefill": _plain_spans, "decode": _plain_decode,
                "heads": _plain_heads, "append": _plain_append}[op](st)
    import causal_flash_attention_gb300 as fa
    if op in ("train", "prefill"):
        mods = dict(softcap=st["softcap"], slopes=st["slopes"])
        q, k, v, lo, hi = st["q"], st["k"], st["v"], st["key_begin"], st["key_end"]
        out, lse = fa.attention_span_forward(q, k, v, lo, hi, **mods)
        if op == "prefill":
            return {"out": out, "lse": lse}
        dq, dk, dv = fa.attention_span_backward(q, k, v, out, st["dout"], lse, lo, hi, **mods)
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if op == "decode":
        out, lse = fa.decode_forward_ragged(st["q"], st["k_cache"], st["v_cache"],
                                            st["block_table"], st["seq_lens"],
                                            window=st["window"], softcap=st["softcap"],
                                            slopes=st["slopes"])
        return {"out": out, "lse": lse}
    rot = dict(turns=st["turns"], interleaved=st["interleaved"], q_weight=st["q_weight"],
               k_weight=st["k_weight"], eps=EPS)
    if op == "heads":
        q_out, k_out = fa.qk_norm_rope_forward(st["q"], st["k"], positions=st["positions"], **rot)
        dq, dk, dwq, dwk = fa.qk_norm_rope_backward(st["dq_out"], st["dk_out"], st["q"], st["k"],
                                                    positions=st["positions"], **rot)
        res = {"q_out": q_out, "k_out": k_out, "dq": dq, "dk": dk}
        if dwq is not None:
            res["dq_weight"], res["dk_weight"] = dwq, dwk
        return res
    q_out = fa.qk_norm_rope_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                                   st["block_table"], st["seq_lens"], **rot)
    return {"q_out": q_out, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


# ------------------------------------------------------------------- exact --
def _exact_head(st, q, k, v, ok, dist, slope, dout=None):
    """One query head of one sequence in 64 bits: q [Sq, d], k, v [n, d], ok, dist [Sq, n]."""
    scale = 1.0 / math.sqrt(q.shape[-1])
    s = (q @ k.T).mul_(scale)
    cap = st["softcap"]
    u = torch.tanh(s / cap) if cap else None
    if cap:
        s = cap * u
    if slope is not None:
        s = s - slope * dist
    s.masked_fill_(~ok, -math.inf)
    lse = torch.logsumexp(s, dim=1)
    p = torch.exp(s - lse[:, None]).masked_fill_(~ok, 0.0)
    out = p @ v
    if dout is None:
        return out, lse
    dv = p.T @ dout
    ds = p.mul_(dout @ v.T - (dout * out).sum(1, keepdim=True)).mul_(scale)
    if cap:
        ds = ds * (1 - u * u)
    return out, lse, ds @ k, ds.T @ q, dv


def _exact_attention(st):
    Hq, Hkv, Sq, d = st["Hq"], st["Hkv"], st["Sq"], st["d"]
    G = Hq // Hkv
    train = st["op"] == "train"
    D = torch.float64
    out = torch.empty(st["B"], Hq, Sq, d, dtype=D, device=DEV)
    lse = torch.empty(st["B"], Hq, Sq, dtype=D, device=DEV)
    if train:
        dq = torch.empty_like(out)
        dk = torch.zeros(st["B"], Hkv, st["Skv"], d, dtype=D, device=DEV)
        dv = torch.zeros_like(dk)
    for b in range(st["B"]):
        if st["op"] == "decode":
            n = int(st["seq_lens"][b])
            pages = st["block_table"][b, : -(-n // st["block"])].long()
            K, V = (torch.cat(list(st[x][pages]), dim=1)[:, :n].to(D)
                    for x in ("k_cache", "v_cache"))
            at = torch.arange(n - Sq, n, device=DEV)[:, None] - torch.arange(n, device=DEV)
            ok = (at >= 0) & (at < (st["window"] or n + 1))
        else:
            K, V = st["k"][b].to(D), st["v"][b].to(D)
            i = torch.arange(st["Skv"] - Sq, st["Skv"], device=DEV)[:, None]
            j = torch.arange(st["Skv"], device=DEV)
            at = i - j
            ok = (st["key_begin"][b][:, None] <= j) & (st["key_end"][b][:, None] > j)
        dist = at.abs().to(D)
        for h in range(Hq):
            slope = None if st["slopes"] is None else float(st["slopes"][h])
            do = st["dout"][b, h].to(D) if train else None
            got = _exact_head(st, st["q"][b, h].to(D), K[h // G], V[h // G], ok, dist, slope, do)
            out[b, h], lse[b, h] = got[:2]
            if train:
                dq[b, h] = got[2]
                dk[b, h // G] += got[3]
                dv[b, h // G] += got[4]
    res = {"out": out, "lse": lse}
    if train:
        res.update(dq=dq, dk=dk, dv=dv)
    return res


def _exact_turned(x, ang, interleaved, sign=1.0):
    """x [B, H, S, d] in 64 bits, each pair as one complex number times e^(i ang)."""
    r = 2 * ang.shape[-1]
    y = x.clone()
    a, b = ((x[..., 0:r:2], x[..., 1:r:2]) if interleaved
            else (x[..., : r // 2], x[..., r // 2: r]))
    z = torch.complex(a.contiguous(), b.contiguous()) * torch.polar(torch.ones_like(ang), sign * ang)
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        y[..., : r // 2], y[..., r // 2: r] = z.real, z.imag
    return y


def _exact_heads(st, positions):
    D = torch.float64
    ang = positions.to(D)[:, None, :, None] * st["inv_freq"]
    res = {}
    for n in ("q", "k"):
        x, w = st[n].to(D), st[n + "_weight"]
        rms = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / st["d"] + EPS)
        y = x / rms * w.to(D) if w is not None else x
        res[n + "_out"] = _exact_turned(y, ang, st["interleaved"])
        if st["op"] == "heads":
            dz = _exact_turned(st["d%s_out" % n].to(D), ang, st["interleaved"], -1.0)
            if w is None:
                res["d" + n] = dz
            else:
                gw = dz * w.to(D)
                xn = x / rms
                res["d" + n] = (gw - xn * (gw * xn).sum(-1, keepdim=True) / st["d"]) / rms
                res["d%s_weight" % n] = (dz * xn).sum((0, 1, 2))
    return res


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] in ("train", "prefill", "decode"):
        return _exact_attention(st)
    if st["op"] == "heads":
        return _exact_heads(st, st["positions"])
    lens, Sq, bs = st["seq_lens"].tolist(), st["Sq"], st["block"]
    pos = torch.tensor([[L - Sq + s for s in range(Sq)] for L in lens], device=DEV)
    got = _exact_heads(st, pos)
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    for b in range(st["B"]):
        at = pos[b]
        page = st["block_table"][b].long()[at // bs]
        kc[page, :, at % bs] = got["k_out"][b].transpose(0, 1)
        vc[page, :, at % bs] = st["v"][b].double().transpose(0, 1)
    return {"q_out": got["q_out"], "k_cache": kc, "v_cache": vc}
