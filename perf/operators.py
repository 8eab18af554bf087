"""Measured cases of the serving operators around the KV cache.

Six entry points of ``lightning_indexer_top_relu_b200.indexcache``:

* ``prefix_attn``       attention of a batch whose sequences share one long prefix;
* ``attn_mass``         the attention weight each cached position received, summed over query
                        rows and heads, added to a running fp32 total per position;
* ``attn_mass_sparse``  the same over the positions of an index cache;
* ``evict_select`` and ``cache_gather``  the positions a cache keeps under a budget (most
                        accumulated weight, first and latest positions protected) and the
                        compaction of the caches to them.

With ``own`` false every operator runs in its plain form in torch, 32 bits and one rounding.
"""
import math

import numpy as np
import torch

own = False

OPS = ("prefix_attn", "attn_mass", "attn_mass_sparse", "evict")


def listed():
    return [
        # Four chats over a 1K system prompt, a few dozen tokens in: the smallest call, latency.
        dict(name="prefix_small", op="prefix_attn", B=4, Lq=1, P=1024, S=64, Hq=8, Hkv=1, d=64),
        # One decode step of 32 sequences behind a shared 32K document, answers up to 2K tokens.
        dict(name="prefix_decode_32k", op="prefix_attn", B=32, Lq=1, P=32768, S=2048, Hq=16, Hkv=1, d=128),
        # Drafted tokens checked five at a time, two K/V heads, odd prefix and cache sizes.
        dict(name="prefix_drafts_8k", op="prefix_attn", B=24, Lq=5, P=8191, S=777, Hq=16, Hkv=2, d=128),
        # Many rollouts of one prompt: 256 sequences, 64K shared, 1K of their own.
        dict(name="prefix_rollouts_64k", op="prefix_attn", B=256, Lq=1, P=65536, S=1024, Hq=16, Hkv=1, d=128),
        # Decode: one token's dense attention weight over each of 32 caches of up to 32K.
        dict(name="mass_decode_32k", op="attn_mass", B=32, Lq=1, Lk=32768, ragged=True, Hq=16, Hkv=1, d=128),
        # The last 64 prompt tokens vote on which of 64K positions stay.
        dict(name="mass_window_64k", op="attn_mass", B=1, Lq=64, Lk=65536, ragged=False, Hq=16, Hkv=1, d=128),
        # Every row of an 8K prefill votes (causal).
        dict(name="mass_prefill_8k", op="attn_mass", B=1, Lq=8192, Lk=8192, ragged=False, Hq=16, Hkv=1, d=128),
        # Decode over an index cache: 2048 selected positions of 32K, 32 sequences.
        dict(name="sparse_mass_decode_32k", op="attn_mass_sparse", B=32, Lq=1, Lk=32768, k=2048, Hq=16, d=128),
        # A 500-row prefill chunk over its index rows, in the middle of a 16K context.
        dict(name="sparse_mass_chunk_16k", op="attn_mass_sparse", B=1, Lq=500, Lk=16001, k=1024, Hq=8, d=128),
        # Four short caches of 1000 halved: latency.
        dict(name="evict_small", op="evict", B=4, Lk=1000, n_keep=500, n_sink=4, n_recent=64, ragged=False, d=64, d_I=64),
        # 32 caches of up to 32K cut to 16K, K, V and indexer keys moved.
        dict(name="evict_32k", op="evict", B=32, Lk=32768, n_keep=16384, n_sink=4, n_recent=1024, ragged=True, d=128, d_I=128),
        # Two half-million-token caches cut to 64K.
        dict(name="evict_long", op="evict", B=2, Lk=500000, n_keep=65536, n_sink=16, n_recent=4096, ragged=False, d=128, d_I=128),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(OPS)
    d = rng.choice((64, 128))
    if op == "prefix_attn":
        Hkv = rng.choice((1, 1, 2, 4))
        Hq = Hkv * rng.choice((1, 3, 4, 8, 16) if Hkv > 1 else (8, 16))
        Lq = rng.choice((1, 1, 1, 2, 4, 7))
        P = _log(rng, 200, 65536)
        S = _log(rng, Lq + 1, 2048)
        B = _log(rng, 1, 256)
        # no more than 4096 query rows of one head against 64K, nor more cache than the largest case
        B = max(1, min(B, int(4000 * 65536 // (Lq * Hq * P)), (256 * 1024) // (S * Hkv)))
        return dict(op=op, B=B, Lq=Lq, P=P, S=S, Hq=Hq, Hkv=Hkv, d=d)
    if op == "attn_mass":
        Hq = rng.choice((8, 16))
        Hkv = rng.choice((1, 1, 2))
        if rng.random() < 0.5:                      # decode
            Lq, Lk, B = rng.choice((1, 1, 2, 5)), _log(rng, 100, 65536), _log(rng, 1, 32)
            B = max(1, min(B, (32 * 32768) // (Lk * Hkv)))
            return dict(op=op, B=B, Lq=Lq, Lk=Lk, ragged=True, Hq=Hq, Hkv=Hkv, d=d)
        Lk = _log(rng, 300, 65536)                   # a window or all rows of a prefill
        Lq = max(1, min(_log(rng, 16, 8192), Lk, 8192 * 4096 // Lk))
        return dict(op=op, B=1, Lq=Lq, Lk=Lk, ragged=False, Hq=Hq, Hkv=Hkv, d=d)
    if op == "attn_mass_sparse":
        Hq = rng.choice((8, 16))
        Lk = _log(rng, 300, 32768)
        k = min(_log(rng, 32, 2048), Lk)
        if rng.random() < 0.5:
            return dict(op=op, B=_log(rng, 1, 32), Lq=1, Lk=Lk, k=k, Hq=Hq, d=d)
        Lq = min(_log(rng, 2, 500), Lk)
        k = min(k, 1024)
        return dict(op=op, B=1, Lq=Lq, Lk=Lk, k=k, Hq=Hq, d=d)
    Lk = _log(rng, 500, 500000)
    B = max(1, min(_log(rng, 1, 32), (28 * 32768) // Lk))
    n_keep = max(100, min(int(Lk * rng.uniform(0.1, 0.7)), (28 * 16384) // B))
    return dict(op=op, B=B, Lk=Lk, n_keep=n_keep, n_sink=rng.choice((0, 4, 16)),
                n_recent=rng.randrange(0, n_keep // 4), ragged=rng.random() < 0.5, d=d,
                d_I=rng.choice((64, 128)))


# ------------------------------------------------------------------------------------ inputs


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _keys(g, *shape):
    """Keys of unit variance; one in 64 is three times as long, as a few tokens of a text draw
    most of the attention."""
    k = _randn(g, *shape)
    heavy = torch.rand(shape[:-2], generator=g, device="cuda") < 1 / 64
    return (k * torch.where(heavy, 3.0, 1.0)[..., None, None]).bfloat16()


def _lens(g, B, lo, hi):
    return torch.randint(lo, hi + 1, (B,), generator=g, device="cuda", dtype=torch.int32)


def _limits(s):
    """Positions each query row sees of its own cache, [B, Lq]."""
    B, Lq, Lk = s["q"].shape[0], s["q"].shape[1], s["k"].shape[1]
    i = torch.arange(Lq, device="cuda")
    if s.get("lens") is not None:
        lim = s["lens"].long()[:, None] - Lq + i[None] + 1
    else:
        lim = (s["q_offset"] + i + 1)[None].expand(B, Lq)
    return lim.clamp(0, Lk)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = dict(case)
    s = {"case": c}
    if own:
        from lightning_indexer_top_relu_b200 import indexcache
        s["ic"] = indexcache
    if c["op"] == "prefix_attn":
        B, Lq, P, S, Hq, Hkv, d = (c[n] for n in ("B", "Lq", "P", "S", "Hq", "Hkv", "d"))
        s["q"] = _randn(g, B, Lq, Hq, d).bfloat16()
        s["k_prefix"], s["v_prefix"] = _keys(g, P, Hkv, d), _randn(g, P, Hkv, d).bfloat16()
        s["k"], s["v"] = _keys(g, B, S, Hkv, d), _randn(g, B, S, Hkv, d).bfloat16()
        s["lens"] = _lens(g, B, Lq, S)
        if own:
            # what a decode loop keeps over its steps
            n = s["ic"].prefix_attn_workspace_bytes(B, Lq, P, S, Hq, Hkv, d)
            s["ws"] = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)
    elif c["op"] == "attn_mass":
        B, Lq, Lk, Hq, Hkv, d = (c[n] for n in ("B", "Lq", "Lk", "Hq", "Hkv", "d"))
        s["q"], s["k"] = _randn(g, B, Lq, Hq, d).bfloat16(), _keys(g, B, Lk, Hkv, d)
        s["lens"] = _lens(g, B, max(Lq, Lk // 2), Lk) if c["ragged"] else None
        s["q_offset"] = Lk - Lq
        s["mass"] = torch.rand(B, Lk, generator=g, device="cuda") * (Lq * Hq / Lk)
        s["lse"] = torch.empty(B, Lq, Hq, device="cuda")
        lim = _limits(s)
        at = torch.arange(Lk, device="cuda")
        G = Hq // Hkv
        for b in range(B):
            for h in range(Hq):
                z = (s["q"][b, :, h] @ s["k"][b, :, h // G].T).float() / math.sqrt(d)
                z.masked_fill_(at[None] >= lim[b][:, None], -math.inf)
                s["lse"][b, :, h] = torch.logsumexp(z, -1)
    elif c["op"] == "attn_mass_sparse":
        B, Lq, Lk, k, Hq, d = (c[n] for n in ("B", "Lq", "Lk", "k", "Hq", "d"))
        s["q"], s["k"] = _randn(g, B, Lq, Hq, d).bfloat16(), _keys(g, B, Lk, 1, d)
        s["q_offset"] = Lk - Lq
        t = s["q_offset"] + torch.arange(Lq, device="cuda")
        pick = torch.rand(B, Lq, Lk, generator=g, device="cuda")
        pick.masked_fill_(torch.arange(Lk, device="cuda")[None, None] > t[None, :, None], -1.0)
        s["idx"] = torch.topk(pick, k, dim=-1).indices.sort(-1).values
        s["idx"] = torch.where(s["idx"] <= t[None, :, None], s["idx"], -1).int()
        s["mass"] = torch.rand(B, Lk, generator=g, device="cuda") * (Lq * Hq / Lk)
        s["lse"] = torch.logsumexp(_slot_logits(s), -1).transpose(1, 2).contiguous()
        if own:
            n = s["ic"].attn_mass_sparse_workspace_bytes(B, Lq, Lk)
            s["ws"] = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)
    else:
        B, Lk, n_keep, d, d_I = (c[n] for n in ("B", "Lk", "n_keep", "d", "d_I"))
        # weights that a few positions hold most of, as attention gives them
        s["mass"] = torch.exp(2.0 * _randn(g, B, Lk)) / Lk
        s["lens"] = _lens(g, B, n_keep // 2, Lk) if c["ragged"] else None
        s["src"] = [_randn(g, B, Lk, 1, d).bfloat16(), _randn(g, B, Lk, 1, d).bfloat16(),
                    _randn(g, B, Lk, d_I).bfloat16(), s["mass"]]
        s["dst"] = [torch.zeros((B, n_keep + 64) + t.shape[2:], device="cuda", dtype=t.dtype)
                    for t in s["src"]]
        s["keep"] = torch.empty(B, n_keep, device="cuda", dtype=torch.int32)
        s["new_lens"] = torch.empty(B, device="cuda", dtype=torch.int32)
    return s


# ------------------------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if own:
        ic = s["ic"]
        if op == "prefix_attn":
            return ic.prefix_attn(s["q"], s["k_prefix"], s["v_prefix"], s["k"], s["v"], s["lens"], ws=s["ws"])
        if op == "attn_mass":
            return ic.attn_mass(s["q"], s["k"], s["lse"], s["mass"], lens=s["lens"], q_offset=s["q_offset"])
        if op == "attn_mass_sparse":
            return ic.attn_mass_sparse(s["q"], s["k"], s["idx"], s["lse"], s["mass"], q_offset=s["q_offset"], ws=s["ws"])
        c = s["case"]
        keep, new_lens = ic.evict_select(s["mass"], c["n_keep"], lens=s["lens"], n_sink=c["n_sink"],
                                         n_recent=c["n_recent"], keep=s["keep"], new_lens=s["new_lens"])
        ic.cache_gather(keep, s["src"], s["dst"])
        return [keep, new_lens] + s["dst"]
    if op == "prefix_attn":
        return _prefix_attn(s)
    if op == "attn_mass":
        return _attn_mass(s)
    if op == "attn_mass_sparse":
        w = torch.exp(_slot_logits(s) - s["lse"].transpose(1, 2)[..., None]).sum(1)   # [B, Lq, k]
        add = torch.zeros(s["mass"].shape[0], s["mass"].shape[1] + 1, device="cuda", dtype=torch.float64)
        add.scatter_add_(1, (s["idx"].long() + 1).flatten(1), w.double().flatten(1))
        s["mass"] += add[:, 1:].float()
        return s["mass"]
    return _evict(s)


def _prefix_attn(s):
    c = s["case"]
    B, Lq, Hq, Hkv, d, S = c["B"], c["Lq"], c["Hq"], c["Hkv"], c["d"], c["S"]
    G = Hq // Hkv
    q = s["q"].float().reshape(B, Lq, Hkv, G, d).permute(2, 0, 1, 3, 4) / math.sqrt(d)   # [Hkv,B,Lq,G,d]
    kp, vp = s["k_prefix"].float().transpose(0, 1), s["v_prefix"].float().transpose(0, 1)
    k, v = (s[n].float().permute(2, 0, 1, 3) for n in ("k", "v"))                        # [Hkv,B,S,d]
    zp = q.reshape(Hkv, -1, d) @ kp.transpose(1, 2)                                       # [Hkv,rows,P]
    zo = (q.reshape(Hkv, B, Lq * G, d) @ k.transpose(2, 3)).reshape(Hkv, B, Lq, G, S)
    seen = torch.arange(S, device="cuda")[None, None] < _limits(s)[..., None]             # [B,Lq,S]
    zo = zo.masked_fill(~seen[None, :, :, None], -math.inf).reshape(Hkv, -1, S)
    m = torch.maximum(zp.amax(-1), zo.amax(-1))
    zp, zo = torch.exp(zp - m[..., None]), torch.exp(zo - m[..., None])
    den = zp.sum(-1) + zo.sum(-1)
    o = zp @ vp + (zo.reshape(Hkv, B, Lq * G, S) @ v).reshape(Hkv, -1, d)
    o, lse = o / den[..., None], m + torch.log(den)
    o = o.reshape(Hkv, B, Lq, G, d).permute(1, 2, 0, 3, 4).reshape(B, Lq, Hq, d)
    return o.bfloat16(), lse.reshape(Hkv, B, Lq, G).permute(1, 2, 0, 3).reshape(B, Lq, Hq)


def _attn_mass(s):
    B, Lq, Hq, d = s["q"].shape
    Lk, Hkv = s["k"].shape[1], s["k"].shape[2]
    G = Hq // Hkv
    q = s["q"].float().reshape(B, Lq, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, Lq * G, d) / math.sqrt(d)
    z = (q @ s["k"].float().permute(0, 2, 3, 1)).reshape(B, Hkv, Lq, G, Lk)
    z -= s["lse"].reshape(B, Lq, Hkv, G).transpose(1, 2)[..., None]
    seen = torch.arange(Lk, device="cuda")[None, None] < _limits(s)[..., None]
    s["mass"] += z.masked_fill_(~seen[:, None, :, None], -math.inf).exp_().sum((1, 2, 3))
    return s["mass"]


def _slot_logits(s):
    """Logits of every head over the slots of each row, [B, Hq, Lq, k]; -inf at empty slots."""
    idx = s["idx"].long()
    B, Lq, k = idx.shape
    rows = s["k"][:, :, 0].float()[torch.arange(B, device="cuda")[:, None, None], idx.clamp(min=0)]
    z = torch.einsum("blhd,blkd->bhlk", s["q"].float() / math.sqrt(s["q"].shape[-1]), rows)
    return z.masked_fill(idx[:, None] < 0, -math.inf)


def _evict(s):
    c = s["case"]
    B, Lk, n_keep = c["B"], c["Lk"], c["n_keep"]
    n = s["lens"].long() if s["lens"] is not None else torch.full((B,), Lk, device="cuda")
    at = torch.arange(Lk, device="cuda")[None]
    safe = (at < c["n_sink"]) | (at >= n[:, None] - c["n_recent"])
    w = torch.where(safe, math.inf, s["mass"]).masked_fill(at >= n[:, None], -math.inf)
    first = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :n_keep].sort(1).values
    slot = torch.arange(n_keep, device="cuda")[None]
    some = slot < n[:, None]
    s["keep"].copy_(torch.where(some, first, -1))
    s["new_lens"].copy_(n.clamp(max=n_keep))
    row = torch.arange(B, device="cuda")[:, None]
    to = torch.where(some, slot, n_keep + 63)         # rows without a source end in the last, unused one
    for src, dst in zip(s["src"], s["dst"]):
        dst[row, to] = src[row, first.clamp(max=Lk - 1)]
        dst[:, n_keep + 63] = 0
    return [s["keep"], s["new_lens"]] + s["dst"]


# ------------------------------------------------------------------------------------ work


def work(c):
    if c["op"] == "prefix_attn":
        rows, S = c["B"] * c["Lq"], (c["S"] + c["Lq"]) / 2       # the caches are filled evenly from Lq to S
        kv = c["P"] * c["Hkv"] + c["B"] * S * c["Hkv"]
        return {"bytes": kv * c["d"] * 4 + rows * c["Hq"] * (c["d"] * 4 + 4),
                "flops": 4 * rows * c["Hq"] * c["d"] * (c["P"] + S)}
    if c["op"] == "attn_mass":
        Lk = c["Lk"] * (0.75 if c["ragged"] else 1.0)
        pairs = c["Lq"] * Lk if c["ragged"] else c["Lq"] * (Lk - (c["Lq"] - 1) / 2)
        return {"bytes": c["B"] * (Lk * (c["Hkv"] * c["d"] * 2 + 8) + c["Lq"] * c["Hq"] * (c["d"] * 2 + 4)),
                "flops": 2 * c["B"] * c["Hq"] * c["d"] * pairs}
    if c["op"] == "attn_mass_sparse":
        slots = c["B"] * c["Lq"] * c["k"]
        distinct = c["B"] * min(c["Lk"], c["Lq"] * c["k"])
        return {"bytes": distinct * (c["d"] * 2 + 8) + slots * 4 + c["B"] * c["Lq"] * c["Hq"] * (c["d"] * 2 + 4),
                "flops": 2 * slots * c["Hq"] * c["d"]}
    Lk, kept = c["Lk"], c["n_keep"]
    if c["ragged"]:                                # lengths spread evenly from n_keep / 2 to Lk
        low = (Lk - kept) / (Lk - kept / 2)        # the share of them above n_keep
        Lk, kept = (Lk + kept / 2) / 2, kept * (low + (1 - low) * 0.75)
    return {"bytes": c["B"] * (4 * Lk + c["n_keep"] * 4 + kept * 2 * (c["d"] * 4 + c["d_I"] * 2 + 4)),
            "flops": c["B"] * Lk}


# ------------------------------------------------------------------------------------ 64 bits


def exact(case, seed):
    """What one pass returns, from the definitions, row by row of the batch in 64 bits."""
    s = prepare(case, seed)
    c = s["case"]
    f8 = torch.float64
    if c["op"] == "prefix_attn":
        B, Lq, Hq, d, S, P = c["B"], c["Lq"], c["Hq"], c["d"], c["S"], c["P"]
        G = Hq // c["Hkv"]
        out, lse = torch.empty(B, Lq, Hq, d, device="cuda", dtype=f8), torch.empty(B, Lq, Hq, device="cuda", dtype=f8)
        lens = s["lens"].tolist()
        kp, vp = s["k_prefix"].to(f8), s["v_prefix"].to(f8)
        for b in range(B):
            for j in range(c["Hkv"]):
                h = slice(j * G, (j + 1) * G)
                keys = torch.cat([kp[:, j], s["k"][b, :lens[b], j].to(f8)])
                vals = torch.cat([vp[:, j], s["v"][b, :lens[b], j].to(f8)])
                z = torch.einsum("ihd,sd->his", s["q"][b, :, h].to(f8), keys) * d ** -0.5
                for i in range(Lq):
                    z[:, i, P + max(0, lens[b] - Lq + i + 1):] = -math.inf
                out[b, :, h] = torch.einsum("his,sd->ihd", torch.softmax(z, -1), vals)
                lse[b, :, h] = torch.logsumexp(z, -1).T
        return out, lse
    if c["op"] in ("attn_mass", "attn_mass_sparse"):
        mass = s["mass"].to(f8)
        B, Lq, Lk, Hq, d = c["B"], c["Lq"], c["Lk"], c["Hq"], c["d"]
        if c["op"] == "attn_mass_sparse":
            for b in range(B):
                for i in range(Lq):
                    at = s["idx"][b, i][s["idx"][b, i] >= 0].long()
                    z = s["q"][b, i].to(f8) @ s["k"][b, at, 0].to(f8).T * d ** -0.5
                    mass[b].index_add_(0, at, torch.exp(z - s["lse"][b, i].to(f8)[:, None]).sum(0))
            return mass
        G = Hq // c["Hkv"]
        i = torch.arange(Lq, device="cuda")[:, None]
        for b in range(B):
            n = Lk if s["lens"] is None else int(s["lens"][b])
            t = n - Lq + i                             # q_offset is Lk - Lq
            for h in range(Hq):
                z = s["q"][b, :, h].to(f8) @ s["k"][b, :n, h // G].to(f8).T * d ** -0.5
                p = torch.exp(z - s["lse"][b, :, h].to(f8)[:, None])
                mass[b, :n] += torch.where(torch.arange(n, device="cuda")[None] <= t, p, 0.0).sum(0)
        return mass
    B, Lk, n_keep = c["B"], c["Lk"], c["n_keep"]
    keep = np.full((B, n_keep), -1, np.int32)
    lens = [Lk] * B if s["lens"] is None else s["lens"].tolist()
    w = s["mass"].cpu().numpy().astype(np.float64)
    for b, n in enumerate(lens):
        rank = w[b, :n].copy()
        rank[:c["n_sink"]] = rank[max(0, n - c["n_recent"]):] = np.inf
        kept = np.sort(np.argsort(-rank, kind="stable")[:n_keep])
        keep[b, :len(kept)] = kept
        for src, dst in zip(s["src"], s["dst"]):
            dst[b, :len(kept)] = src[b][torch.from_numpy(kept).cuda()]
    return [torch.from_numpy(keep), torch.tensor([min(n, n_keep) for n in lens], dtype=torch.int32)] + [t.to(f8) for t in s["dst"]]
