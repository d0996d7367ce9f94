"""The library's latent attention as measured cases: attention whose keys and values all come
from one latent vector a token, with a rotated part of the key that the heads share. Training
and prompts run on keys and values expanded from the latents (with gradients); serving runs on
the latents themselves, kept in a paged cache to which new tokens are appended.

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
ROPE = 64          # rotated elements of a key, and of a query
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # training at a context of 4096, causal (the largest case)
        dict(name="train_4k", op="train", dtype="bf16", B=1, H=32, Sq=4096, Skv=4096, d=128,
             mask="causal", span=0, mask_seed=1),
        # packed documents at an odd length
        dict(name="train_documents", op="train", dtype="fp16", B=2, H=16, Sq=2999, Skv=2999,
             d=128, mask="documents", span=1200, mask_seed=2),
        # a small model's padded batch: rows past each sequence see nothing
        dict(name="train_padded_small", op="train", dtype="bf16", B=4, H=12, Sq=1000, Skv=1000,
             d=64, mask="padded", span=500, mask_seed=3),
        # a chunk of a long prompt over the context before it
        dict(name="prefill_chunk", op="prefill", dtype="bf16", B=1, H=32, Sq=1024, Skv=8192,
             d=128, mask="causal", span=0, mask_seed=4),
        # a short prompt: latency of one call
        dict(name="prefill_short", op="prefill", dtype="bf16", B=1, H=16, Sq=61, Skv=61, d=128,
             mask="causal", span=0, mask_seed=5),
        # a serving step, many heads: one new token of each of 16 sequences of unequal length
        dict(name="decode_128_heads", op="decode", dtype="bf16", B=16, H=128, Sq=1, rank=512,
             block=64, min_len=1, max_len=8192, len_seed=6, window=0, tree=False),
        # the same step of a model with few heads, or of one shard of the heads
        dict(name="decode_16_heads", op="decode", dtype="bf16", B=16, H=16, Sq=1, rank=512,
             block=64, min_len=1, max_len=8192, len_seed=7, window=0, tree=False),
        # one short stream: latency of one decoding call
        dict(name="decode_one_stream", op="decode", dtype="fp16", B=1, H=16, Sq=1, rank=512,
             block=16, min_len=500, max_len=501, len_seed=8, window=0, tree=False),
        # a tree of 8 drafted tokens a sequence over long caches
        dict(name="decode_tree_20k", op="decode", dtype="bf16", B=3, H=16, Sq=8, rank=512,
             block=128, min_len=9000, max_len=20001, len_seed=9, window=0, tree=True),
        # a small model, many short sequences, sliding window
        dict(name="decode_small_window", op="decode", dtype="fp16", B=60, H=8, Sq=1, rank=256,
             block=32, min_len=1, max_len=1500, len_seed=10, window=512, tree=False),
        # a serving step's new token of each sequence into the paged cache
        dict(name="append_step", op="append", dtype="bf16", B=16, H=128, Sq=1, rank=512, block=64,
             min_len=1, max_len=8192, len_seed=11, norm=True, interleaved=True, tree=False),
        # prompts of odd length into the paged cache
        dict(name="append_prompt", op="append", dtype="fp16", B=3, H=16, Sq=1025, rank=512,
             block=16, min_len=1025, max_len=3000, len_seed=12, norm=True, interleaved=False,
             tree=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["train", "train", "prefill", "decode", "decode", "decode", "append"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]))
    if op in ("train", "prefill"):
        c["d"] = rng.choice([64, 128, 128])
        c["H"] = rng.choice([1, 2, 3, 5, 8, 12, 16, 24, 32])
        c["Sq"] = _log_int(rng, 33, 6000)
        c["Skv"] = c["Sq"] + (rng.choice([0, _log_int(rng, 1, 8000)]) if op == "prefill" else 0)
        limit = 4096 * 4096 * 32 * 128
        while c["d"] * c["H"] * c["Sq"] * c["Skv"] > limit:
            c["Sq"], c["Skv"] = c["Sq"] * 2 // 3, c["Skv"] - c["Sq"] + c["Sq"] * 2 // 3
        fit = limit // (c["d"] * c["H"] * c["Sq"] * c["Skv"])
        c["B"] = max(1, min(rng.choice([1, 1, 2, 3, 5, 8]), fit))
        c["mask"] = rng.choice(["causal", "causal", "documents", "window", "prefix", "padded"])
        c["span"] = _log_int(rng, 24, max(24, c["Skv"]))
        c["mask_seed"] = rng.randrange(1 << 20)
        return c
    c["rank"] = rng.choice([256, 512, 512])
    c["H"] = rng.choice([1, 2, 4, 8, 12, 16, 20, 32, 40, 64, 128])
    c["len_seed"] = rng.randrange(1 << 20)
    if op == "decode":
        c["Sq"] = rng.choice([1, 1, 1, 2, 3, 4, 8])
        c["tree"] = c["Sq"] > 1 and rng.random() < 0.5
        c["max_len"] = c["Sq"] + _log_int(rng, 30, 32768)
        c["min_len"] = rng.choice([c["Sq"], c["max_len"] // 2 + 1, c["max_len"]])
        fit = 16 * 8192 * 128 * 512 // (c["max_len"] * c["rank"] * c["H"] * c["Sq"])
        c["B"] = max(1, min(_log_int(rng, 1, 96), fit))
        c["block"] = rng.choice([16, 32, 64, 128, 256])
        c["window"] = 0 if c["tree"] else rng.choice([0, 0, _log_int(rng, 32, c["max_len"])])
        return c
    c["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
    c["Sq"] = rng.choice([1, 1, 4, _log_int(rng, 1, 1500)])
    c["tree"] = c["Sq"] == 4
    c["max_len"] = c["Sq"] + _log_int(rng, 1, 4000)
    c["min_len"] = c["Sq"]
    c["B"] = max(1, min(_log_int(rng, 1, 64), 40000 // c["max_len"]))
    c["block"] = rng.choice([16, 32, 64, 256])
    c["norm"] = rng.random() < 0.7
    c["interleaved"] = rng.random() < 0.5
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
        elif c["mask"] == "padded":          # rows past the sequence see nothing
            m = rng.randint(min(n, Skv), Skv)
            hi[b] = np.where(pos < m, pos + 1, 0)
    return lo, hi


def _lens(c):
    rng = random.Random(c["len_seed"])
    lens = [rng.randint(c["min_len"], c["max_len"]) for _ in range(c["B"])]
    lens[rng.randrange(c["B"])] = c["max_len"]
    return lens


def _parents(c):
    """The tree of drafted tokens of each sequence: token t > 0 hangs below an earlier one."""
    rng = random.Random(c["len_seed"] + 1)
    return [[-1] + [rng.randrange(t) for t in range(1, c["Sq"])] for _ in range(c["B"])]


def _tree(c):
    """(masks, depths) as numpy [B, Sq]: bit t of masks[b, s] set where token t is token s or
    above it; depth 0 at the root."""
    masks = np.zeros((c["B"], c["Sq"]), np.int64)
    depths = np.zeros((c["B"], c["Sq"]), np.int64)
    for b, parents in enumerate(_parents(c)):
        for s, up in enumerate(parents):
            masks[b, s] = (1 << s) | (masks[b, up] if up >= 0 else 0)
            depths[b, s] = depths[b, up] + 1 if up >= 0 else 0
    return masks, depths


def _inv_freq():
    """Rotary frequencies of the rotated elements (base 10000), the slower ones stretched four
    times, as for contexts longer than the trained one."""
    f = 10000.0 ** (-np.arange(0, ROPE, 2, dtype=np.float64) / ROPE)
    ramp = np.clip((f * 8192 / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
    return f * (ramp + (1.0 - ramp) / 4.0)


def _turns(inv_freq):
    """Turns a position, in units of 2^-64 (the table that the rotary calls take)."""
    out = np.array([int(round(float(f) / (2 * math.pi) * 2.0 ** 64)) % (1 << 64)
                    for f in inv_freq], dtype=np.uint64)
    return torch.from_numpy(out.view(np.int64).copy())


def _scale(c):
    """One over the root of a query's elements before any absorption (128 + 64 when serving)."""
    return 1.0 / math.sqrt((c["d"] if "d" in c else 128) + ROPE)


def work(c):
    op, e, H = c["op"], ESIZE[c["dtype"]], c["H"]
    if op in ("train", "prefill"):
        d = c["d"]
        lo, hi = _spans(c)
        pairs = float(np.maximum(hi.astype(np.int64) - lo, 0).sum()) * H
        nq, nk = c["B"] * H * c["Sq"], c["B"] * H * c["Skv"]
        q, k, v, o = nq * (d + ROPE), nk * d + c["B"] * c["Skv"] * ROPE, nk * d, nq * d
        n = (q + k + v + o) * e + nq * 4 + (0 if c["mask"] == "causal" else 8 * c["B"] * c["Sq"])
        forward = 2 * (2 * d + ROPE) * pairs
        if op == "prefill":
            return {"bytes": n, "flops": forward}
        return {"bytes": n + (q + k + v + o) * e,
                "flops": forward + 2 * (3 * (d + ROPE) + 2 * d) * pairs}
    Sq, r = c["Sq"], c["rank"]
    if op == "decode":
        keys = pairs = 0
        masks = _tree(c)[0] if c["tree"] else None
        for b, L in enumerate(_lens(c)):
            first = max(0, L - Sq + 1 - c["window"]) if c["window"] else 0
            keys += L - first
            for s in range(Sq):
                p = L - Sq + s
                pairs += (L - Sq + bin(int(masks[b, s])).count("1") if c["tree"] else
                          max(0, min(p + 1, c["window"] or p + 1)))
        rows = c["B"] * H * Sq
        return {"bytes": keys * (r + ROPE) * e + rows * ((2 * r + ROPE) * e + 4),
                "flops": 2 * (2 * r + ROPE) * pairs * H}
    n = c["B"] * Sq
    return {"bytes": 2 * n * (r + ROPE + H * ROPE) * e,
            "flops": n * ((4 * r if c["norm"] else 0) + 3 * ROPE * (H + 1))}


# ----------------------------------------------------------------- prepare --
def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dt)

    st = dict(c)
    B, H, Sq = c["B"], c["H"], c["Sq"]
    if c["op"] in ("train", "prefill"):
        d, Skv = c["d"], c["Skv"]
        # as the projections leave them: tokens first, keys and values in one tensor
        st["q"] = randn(B, Sq, H, d + ROPE).transpose(1, 2)
        kv = randn(B, Skv, H, 2 * d).transpose(1, 2)
        st["k"], st["v"] = kv[..., :d], kv[..., d:]
        st["k_rope"] = randn(B, Skv, ROPE)
        st["key_begin"] = st["key_end"] = None
        if c["mask"] != "causal":
            lo, hi = _spans(c)
            st["key_begin"], st["key_end"] = (torch.from_numpy(x).to(DEV) for x in (lo, hi))
        if c["op"] == "train":
            st["dout"] = randn(B, Sq, H, d).transpose(1, 2)
        return st
    lens, bs, r = _lens(c), c["block"], c["rank"]
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
    st["cache"] = randn(n_blocks, bs, r + ROPE)
    if c["tree"]:
        masks, depths = _tree(c)
        st["tree_masks"] = torch.from_numpy(masks).to(DEV)
        pos = np.array(lens)[:, None] - Sq + depths
        st["positions"] = torch.from_numpy(pos.astype(np.int32)).to(DEV)
    else:
        st["tree_masks"] = st["positions"] = None
    if c["op"] == "decode":
        # absorbed queries; scores of about unit variance
        q = randn(B, H, Sq, r + ROPE)
        q[..., :r] *= 0.5 * math.sqrt(512 / r)
        st["q"] = q
        return st
    f = _inv_freq()
    st["inv_freq"] = torch.from_numpy(f).to(DEV)
    st["turns"] = _turns(f).to(DEV)
    down = randn(B, Sq, r + ROPE)               # one projection gives latent and shared key part
    st["latent"], st["new_k_rope"] = down[..., :r], down[..., r:]
    st["q_rope"] = randn(B, Sq, H, 128 + ROPE)[..., 128:].transpose(1, 2)
    st["weight"] = (1 + 0.2 * randn(r).float()).to(dt) if c["norm"] else None
    return st


# ------------------------------------------------------------------- plain --
def _softmax(s):
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(dim=-1, keepdim=True)
    return p / torch.where(l == 0, torch.ones_like(l), l), (m + torch.log(l)).squeeze(-1)


def _plain_expanded(st):
    d, dt, scale = st["d"], st["q"].dtype, _scale(st)
    q, v = st["q"].float(), st["v"].float()
    kr = st["k_rope"].float()[:, None].expand(-1, st["H"], -1, -1)
    k = torch.cat((st["k"].float(), kr), dim=-1)
    j = torch.arange(st["Skv"], device=DEV)
    if st["key_begin"] is None:
        visible = (j <= torch.arange(st["Sq"], device=DEV)[:, None] + (st["Skv"] - st["Sq"]))[None]
    else:
        visible = (j >= st["key_begin"][:, :, None]) & (j < st["key_end"][:, :, None])
    s = torch.matmul(q, k.transpose(2, 3)) * scale
    p, lse = _softmax(torch.where(visible[:, None], s, -math.inf))
    del s
    out = torch.matmul(p, v)
    res = {"out": out.to(dt), "lse": lse}
    if st["op"] == "prefill":
        return res
    do = st["dout"].float()
    res["dv"] = torch.matmul(p.transpose(2, 3), do).to(dt)
    ds = torch.matmul(do, v.transpose(2, 3))
    ds = p * (ds - (do * out).sum(dim=-1, keepdim=True)) * scale
    res["dq"] = torch.matmul(ds, k).to(dt)
    dk = torch.matmul(ds.transpose(2, 3), q)
    res["dk"] = dk[..., :d].to(dt)
    res["dk_rope"] = dk[..., d:].sum(dim=1).to(dt)
    return res


def _plain_decode(st):
    B, H, Sq, r, dt = st["B"], st["H"], st["Sq"], st["rank"], st["q"].dtype
    n = st["block_table"].shape[1] * st["block"]
    at = st["block_table"].clamp(min=0).long()
    lens = st["seq_lens"].long()
    j = torch.arange(n, device=DEV)
    keys = st["cache"][at].reshape(B, n, r + ROPE)
    # rows of the last page past the sequence belong to nobody
    keys = torch.where((j < lens[:, None])[..., None], keys, torch.zeros_like(keys)).float()
    first = lens - Sq                              # position of the first new token
    if st["tree_masks"] is not None:
        t = j - first[:, None]                     # [B, n] index among the drafted tokens
        bit = (st["tree_masks"][:, :, None] >> t.clamp(0, Sq - 1)[:, None]) & 1
        visible = (t < 0)[:, None] | ((t < Sq)[:, None] & (bit == 1))
    else:
        ahead = (first[:, None] + torch.arange(Sq, device=DEV))[:, :, None] - j
        visible = ahead >= 0
        if st["window"]:
            visible = visible & (ahead < st["window"])
    q = st["q"].float().reshape(B, H * Sq, r + ROPE)
    s = (torch.matmul(q, keys.transpose(1, 2)) * _scale(st)).view(B, H, Sq, n)
    p, lse = _softmax(torch.where(visible[:, None], s, -math.inf))
    out = torch.matmul(p.view(B, H * Sq, n), keys[..., :r])
    return {"out": out.view(B, H, Sq, r).to(dt), "lse": lse}


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    a, b = x[..., : ROPE // 2], x[..., ROPE // 2:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)


def _plain_append(st):
    bs, Sq, r, dt = st["block"], st["Sq"], st["rank"], st["cache"].dtype
    row = st["seq_lens"].long()[:, None] - Sq + torch.arange(Sq, device=DEV)
    pos = row if st["positions"] is None else st["positions"]
    angle = pos.double()[..., None] * st["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()          # [B, Sq, ROPE / 2]
    x = st["latent"].float()
    if st["weight"] is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * st["weight"].float()
    page = torch.gather(st["block_table"].long(), 1, row // bs)
    st["cache"][page, row % bs, :r] = x.to(dt)
    st["cache"][page, row % bs, r:] = _rotate(st["new_k_rope"].float(), cos, sin,
                                              st["interleaved"]).to(dt)
    q = _rotate(st["q_rope"].float(), cos[:, None], sin[:, None], st["interleaved"]).to(dt)
    return {"q_out": q, "cache": st["cache"]}


def run(state):
    st = state
    op = st["op"]
    if not own:
        return {"train": _plain_expanded, "prefill": _plain_expanded, "decode": _plain_decode,
                "append": _plain_append}[op](st)
    import causal_flash_attention_gb300 as fa
    if op in ("train", "prefill"):
        q, k, kr, v = st["q"], st["k"], st["k_rope"], st["v"]
        lo, hi, scale = st["key_begin"], st["key_end"], _scale(st)
        out, lse = fa.attention_latent_forward(q, k, kr, v, lo, hi, scale=scale)
        if op == "prefill":
            return {"out": out, "lse": lse}
        dq, dk, dkr, dv = fa.attention_latent_backward(q, k, kr, v, out, st["dout"], lse, lo, hi,
                                                       scale=scale)
        return {"out": out, "lse": lse, "dv": dv, "dq": dq, "dk": dk, "dk_rope": dkr}
    if op == "decode":
        out, lse = fa.decode_latent_paged(st["q"], st["cache"], st["block_table"], st["seq_lens"],
                                          scale=_scale(st), window=st["window"],
                                          tree_masks=st["tree_masks"])
        return {"out": out, "lse": lse}
    q_out = fa.latent_append(st["latent"], st["new_k_rope"], st["q_rope"], st["cache"],
                             st["block_table"], st["seq_lens"], st["turns"], weight=st["weight"],
                             eps=EPS, positions=st["positions"], interleaved=st["interleaved"])
    return {"q_out": q_out, "cache": st["cache"]}


# ------------------------------------------------------------------- exact --
def _exact_row_softmax(s, ok):
    s = s.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, dim=1)
    return torch.exp(s - lse[:, None]).masked_fill_(~ok, 0.0), lse


def _exact_expanded(st):
    D = torch.float64
    B, H, Sq, Skv, d, scale = st["B"], st["H"], st["Sq"], st["Skv"], st["d"], _scale(st)
    train = st["op"] == "train"
    out = torch.empty(B, H, Sq, d, dtype=D, device=DEV)
    lse = torch.empty(B, H, Sq, dtype=D, device=DEV)
    res = {"out": out, "lse": lse}
    if train:
        res["dv"] = torch.empty(B, H, Skv, d, dtype=D, device=DEV)
        res["dq"] = torch.empty(B, H, Sq, d + ROPE, dtype=D, device=DEV)
        res["dk"] = torch.empty_like(res["dv"])
        res["dk_rope"] = torch.zeros(B, Skv, ROPE, dtype=D, device=DEV)
    lo, hi = (torch.from_numpy(x).to(DEV) for x in _spans(st))
    j = torch.arange(Skv, device=DEV)
    for b in range(B):
        ok = (lo[b][:, None] <= j) & (hi[b][:, None] > j)
        kr = st["k_rope"][b].to(D)
        for h in range(H):
            q, k, v = (st[x][b, h].to(D) for x in ("q", "k", "v"))
            p, lse[b, h] = _exact_row_softmax((q[:, :d] @ k.T + q[:, d:] @ kr.T).mul_(scale), ok)
            o = p @ v
            out[b, h] = o
            if train:
                do = st["dout"][b, h].to(D)
                res["dv"][b, h] = p.T @ do
                ds = p.mul_(do @ v.T - (do * o).sum(1, keepdim=True)).mul_(scale)
                res["dq"][b, h, :, :d] = ds @ k
                res["dq"][b, h, :, d:] = ds @ kr
                res["dk"][b, h] = ds.T @ q[:, :d]
                res["dk_rope"][b] += ds.T @ q[:, d:]
    return res


def _exact_decode(st):
    D = torch.float64
    B, H, Sq, r, bs = st["B"], st["H"], st["Sq"], st["rank"], st["block"]
    out = torch.empty(B, H, Sq, r, dtype=D, device=DEV)
    lse = torch.empty(B, H, Sq, dtype=D, device=DEV)
    for b, n in enumerate(_lens(st)):
        pages = st["block_table"][b, : -(-n // bs)].long()
        keys = torch.cat(list(st["cache"][pages]))[:n].to(D)
        ok = torch.zeros(Sq, n, dtype=torch.bool, device=DEV)
        for s in range(Sq):
            if st["tree"]:
                ok[s, : n - Sq] = True
                t = s
                while t >= 0:                      # up the tree
                    ok[s, n - Sq + t] = True
                    t = _parents(st)[b][t]
            else:
                p = n - Sq + s
                ok[s, max(0, p + 1 - st["window"]) if st["window"] else 0: p + 1] = True
        for h in range(H):
            p, lse[b, h] = _exact_row_softmax((st["q"][b, h].to(D) @ keys.T) * _scale(st), ok)
            out[b, h] = p @ keys[:, :r]
    return {"out": out, "lse": lse}


def _exact_turned(x, angle, interleaved):
    """x [..., ROPE] in 64 bits, each pair as one complex number times e^(i angle)."""
    y = torch.empty_like(x)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, dim=-1)
    z = torch.complex(a.contiguous(), b.contiguous()) * torch.polar(torch.ones_like(angle), angle)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = z.real, z.imag
    else:
        y[..., : ROPE // 2], y[..., ROPE // 2:] = z.real, z.imag
    return y


def _exact_append(st):
    D = torch.float64
    Sq, r, bs = st["Sq"], st["rank"], st["block"]
    cache, q_out = st["cache"].to(D), torch.empty(st["q_rope"].shape, dtype=D, device=DEV)
    depths = _tree(st)[1] if st["tree"] else None
    for b, n in enumerate(_lens(st)):
        rows = torch.arange(n - Sq, n, device=DEV)
        pos = n - Sq + torch.from_numpy(depths[b]).to(DEV) if st["tree"] else rows
        angle = pos.to(D)[:, None] * st["inv_freq"]
        x = st["latent"][b].to(D)
        if st["weight"] is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / r + EPS) * st["weight"].to(D)
        page = st["block_table"][b].long()[rows // bs]
        cache[page, rows % bs] = torch.cat(
            (x, _exact_turned(st["new_k_rope"][b].to(D), angle, st["interleaved"])), dim=-1)
        q_out[b] = _exact_turned(st["q_rope"][b].to(D), angle.expand(st["H"], -1, -1),
                                 st["interleaved"])
    return {"q_out": q_out, "cache": cache}


def exact(case, seed):
    st = prepare(case, seed)
    return {"train": _exact_expanded, "prefill": _exact_expanded, "decode": _exact_decode,
            "append": _exact_append}[st["op"]](st)
