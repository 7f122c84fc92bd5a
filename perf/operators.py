"""The attention half of a decode or prefill step over a paged key/value cache: what is measured.

Three operators, each beside the MLP operators the library has had so far:

* ``rope``: rotary positions applied to the queries and keys of a fused QKV row;
* ``rope_append``: the same with the rotated keys and the values written into the cache's pages;
* ``attention``: each sequence's new tokens (one when decoding, a chunk when a prompt is read)
  attend over the sequence's pages, causally, optionally with a sliding window and with scores
  capped by a tanh.

``run`` computes them in plain torch operations (in 32 bits, angles in 64) where ``own`` is
false, and through the library's entry points where it is true. ``exact`` is the definition in
64 bits, sequence by sequence.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------ cases


def listed():
    """32 query and 8 key/value heads of 128 are the attention of the 4096-wide layer whose MLP
    the benchmark times (its QKV product has 6144 = 32 * 128 + 2 * 8 * 128 outputs)."""
    return [
        # one new token of one chat: only latency counts
        dict(name="rope 1 token", op="rope", tokens=1, hq=32, hk=8, d=128, rot=128,
             interleaved=False, scaling="none", far=8000),
        # a long prompt, a part of each head rotated, interleaved pairs, positions far out
        dict(name="rope 8191 tokens partial", op="rope", tokens=8191, hq=32, hk=8, d=128, rot=64,
             interleaved=True, scaling="ramp", far=1000000),
        # one decode step of 64 sequences with long contexts
        dict(name="append decode 64", op="append", batch=64, q=1, ragged_q=False, kv=40000,
             ragged_kv=True, hq=32, hk=8, d=128, page=16, head_major=False, rot=128,
             interleaved=False, scaling="banded"),
        # five prompts of different lengths written at once
        dict(name="append prompts 5x1639", op="append", batch=5, q=1639, ragged_q=True, kv=2100,
             ragged_kv=True, hq=32, hk=8, d=128, page=64, head_major=True, rot=128,
             interleaved=False, scaling="none"),
        # one chat, a few thousand tokens in
        dict(name="decode 1 of 4097", op="attention", batch=1, q=1, ragged_q=False, kv=4097,
             ragged_kv=False, hq=32, hk=8, d=128, page=16, head_major=False, window=0, cap=0.0),
        # a served batch with contexts of every length
        dict(name="decode 64 up to 8192", op="attention", batch=64, q=1, ragged_q=False, kv=8192,
             ragged_kv=True, hq=32, hk=8, d=128, page=16, head_major=True, window=0, cap=0.0),
        # two long documents
        dict(name="decode 2 of 131072", op="attention", batch=2, q=1, ragged_q=False, kv=131072,
             ragged_kv=False, hq=32, hk=8, d=128, page=64, head_major=False, window=0, cap=0.0),
        # a few guessed tokens of 16 sequences checked at once
        dict(name="verify 16x8 of 6000", op="attention", batch=16, q=8, ragged_q=True, kv=6000,
             ragged_kv=True, hq=32, hk=8, d=128, page=32, head_major=False, window=0, cap=0.0),
        # a chunk of a long prompt: the prompt is read in pieces between decode steps
        dict(name="chunk 512 of 16500", op="attention", batch=1, q=512, ragged_q=False, kv=16500,
             ragged_kv=False, hq=32, hk=8, d=128, page=16, head_major=False, window=0, cap=0.0),
        # narrow heads, seven queries to a key head, capped scores and a window
        dict(name="windowed capped prompts", op="attention", batch=3, q=2500, ragged_q=True,
             kv=2500, ragged_kv=False, hq=28, hk=4, d=64, page=16, head_major=True, window=512,
             cap=30.0),
        # a whole prompt at once: the largest
        dict(name="prompt 8192", op="attention", batch=1, q=8192, ragged_q=False, kv=8192,
             ragged_kv=False, hq=32, hk=8, d=128, page=128, head_major=False, window=0, cap=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: every layout, head grouping, page size and option of the
    listed ones in any combination, lengths from one token up."""
    while True:
        op = rng.choice(["rope", "append", "attention", "attention", "attention"])
        hk = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 128, 128])
        hq = hk * rng.choice([1, 2, 3, 4, 5, 7, 8])
        c = dict(op=op, hq=hq, hk=hk, d=d)
        if op in ("rope", "append"):
            c.update(rot=rng.choice([d // 4, d // 2, d, d]), interleaved=rng.random() < 0.5,
                     scaling=rng.choice(["none", "linear", "banded", "ramp"]))
        if op == "rope":
            c.update(tokens=_log(rng, 1, 8192), far=_log(rng, 100, 1000000))
            return c
        c.update(page=rng.choice([16, 16, 32, 64, 128]), head_major=rng.random() < 0.5,
                 ragged_q=rng.random() < 0.5, ragged_kv=rng.random() < 0.5)
        kind = rng.choice(["decode", "decode", "verify", "chunk", "prompt"])
        if kind == "decode":
            c.update(batch=_log(rng, 1, 128), q=1, kv=_log(rng, 16, 100000))
        elif kind == "verify":
            c.update(batch=_log(rng, 1, 64), q=rng.randint(2, 16), kv=_log(rng, 100, 20000))
        elif kind == "chunk":
            q = _log(rng, 17, 1500)
            c.update(batch=_log(rng, 1, 4), q=q, kv=q + _log(rng, 1, 20000))
        else:
            q = _log(rng, 100, 6000)
            c.update(batch=_log(rng, 1, 4), q=q, kv=q)
        if op == "attention":
            c.update(window=rng.choice([0, 0, 0, _log(rng, 32, 4096)]),
                     cap=rng.choice([0.0, 0.0, 0.0, 30.0]))
        # no larger than the listed ones: tokens in the cache, and scores of one pass
        if c["batch"] * c["kv"] <= 262144 and c["batch"] * hq * c["q"] * c["kv"] <= 32 * 8192 * 8192:
            return c


def _lengths(case):
    """(new tokens, tokens in the cache with them) of every sequence; a function of the case."""
    rng = random.Random(7919 * case["batch"] + 31 * case["q"] + case["kv"])
    q, kv = [], []
    for b in range(case["batch"]):
        n = rng.randint(max(1, case["q"] // 4), case["q"]) if case["ragged_q"] and b else case["q"]
        t = rng.randint(max(n, case["kv"] // 16), case["kv"]) if case["ragged_kv"] and b else case["kv"]
        q.append(n)
        kv.append(max(n, t))
    return q, kv


def _inv_freq(rot, scaling):
    """The rotary frequencies in 64 bits and the factor on cosine and sine: a base of 500000, and
    the usual ways to stretch a trained context of 8192 by 8."""
    f = [500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    m, stretch, trained = 1.0, 8.0, 8192.0
    if scaling == "linear":
        f = [x / stretch for x in f]
    elif scaling == "banded":  # long wavelengths stretched, short ones kept, blended between
        lo, hi = 1.0, 4.0
        out = []
        for x in f:
            turns = trained * x / (2 * math.pi)
            s = min(1.0, max(0.0, (turns - lo) / (hi - lo)))
            out.append(x / stretch * (1 - s) + x * s)
        f = out
    elif scaling == "ramp":  # the blend linear in the pair's index
        at = [rot * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(500000.0)) for n in (32.0, 1.0)]
        lo, hi = max(0.0, math.floor(at[0])), min(rot - 1.0, math.ceil(at[1]))
        out = []
        for i, x in enumerate(f):
            s = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            out.append(x / stretch * s + x * (1 - s))
        f, m = out, 0.1 * math.log(stretch) + 1.0
    return f, m


# ------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    """The tensors a serving program holds before the call: activations, the cache's pages and
    the batch's index tensors; with the library, the scratch it keeps too."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        return t.normal_(0.0, std, generator=g)

    hq, hk, d = case["hq"], case["hk"], case["d"]
    s = {"case": case}
    if case["op"] in ("rope", "append"):
        f, s["m"] = _inv_freq(case["rot"], case["scaling"])
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    if case["op"] == "rope":
        n = case["tokens"]
        qkv = normal(n, (hq + 2 * hk) * d)
        first = int(torch.randint(0, case["far"], (1,), device=DEV, generator=g))
        s["positions"] = torch.arange(first, first + n, dtype=torch.int32, device=DEV)
    else:
        ql, kl = _lengths(case)
        n, page = sum(ql), case["page"]
        counts = [(t + page - 1) // page for t in kl]
        pages = sum(counts) + 3
        # pages are handed out as sequences grow, so a sequence's pages lie anywhere
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        row = torch.arange(max(counts), device=DEV)[None, :]
        c = torch.tensor(counts, device=DEV)
        at = (torch.cumsum(c, 0) - c)[:, None] + row
        s["block_table"] = torch.where(row < c[:, None], order[at.clamp(max=pages - 1)],
                                       torch.full_like(order[:1], -1)).contiguous()
        s["q_start"] = torch.tensor([sum(ql[:i]) for i in range(len(ql) + 1)], dtype=torch.int32, device=DEV)
        s["kv_len"] = torch.tensor(kl, dtype=torch.int32, device=DEV)
        s["max_q"] = max(ql)
        if case["head_major"]:
            s["k_cache"], s["v_cache"] = (normal(pages, hk, page, d).transpose(1, 2) for _ in range(2))
        else:
            s["k_cache"], s["v_cache"] = (normal(pages, page, hk, d) for _ in range(2))
        if case["op"] == "append":
            qkv = normal(n, (hq + 2 * hk) * d)
        else:
            s["q"] = normal(n, hq, d, std=2.0)
            if own:
                import memory_bound_decode_fd_gb300 as fd

                s["scratch"] = fd.paged_attention_scratch(len(ql), n, hq, hk, d, s["max_q"], DEV)
    if case["op"] != "attention":
        s["q"] = qkv[:, :hq * d].view(n, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
        s["v"] = qkv[:, (hq + hk) * d:].view(n, hk, d)
    return s


# --------------------------------------------------------------------------------- the passes


def run(s):
    c = s["case"]
    if own:
        import memory_bound_decode_fd_gb300 as fd

        if c["op"] == "rope":
            return fd.rope(s["q"], s["k"], s["positions"], s["inv_freq"],
                           interleaved=c["interleaved"], scale=s["m"])
        if c["op"] == "append":
            q = fd.rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["q_start"],
                               s["kv_len"], s["block_table"], s["inv_freq"],
                               interleaved=c["interleaved"], scale=s["m"])
            return q, s["k_cache"], s["v_cache"]
        return fd.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["q_start"], s["kv_len"],
                                  s["block_table"], s["max_q"], s["scratch"], window=c["window"],
                                  softcap=c["cap"])
    if c["op"] == "rope":
        return (_rotate(s["q"], s["positions"], s), _rotate(s["k"], s["positions"], s))
    if c["op"] == "append":
        return _append(s)
    return _attention(s)


def _rotate(x, positions, s):
    c, r = s["case"], s["case"]["rot"]
    angle = positions.double()[:, None] * s["inv_freq"][None, :]
    cos, sin = (torch.cos(angle) * s["m"]).float()[:, None], (torch.sin(angle) * s["m"]).float()[:, None]
    y = x.float()
    if c["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, y[..., r:]), -1).to(x.dtype)


def _places(s):
    """(sequence, position in the sequence) of every new token."""
    n = s["q"].shape[0]
    token = torch.arange(n, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"], token, right=True) - 1
    new = s["q_start"][1:] - s["q_start"][:-1]
    return seq, token - s["q_start"][seq] + (s["kv_len"] - new)[seq]


def _append(s):
    page = s["case"]["page"]
    seq, pos = _places(s)
    where = s["block_table"][seq, pos // page].long(), (pos % page).long()
    s["k_cache"][where] = _rotate(s["k"], pos, s)
    s["v_cache"][where] = s["v"]
    return _rotate(s["q"], pos, s), s["k_cache"], s["v_cache"]


def _attention(s):
    """All sequences at once, padded to the longest."""
    c = s["case"]
    hq, hk, d = c["hq"], c["hk"], c["d"]
    batch, n = c["batch"], s["q"].shape[0]
    seq, pos = _places(s)
    new = s["q_start"][1:] - s["q_start"][:-1]
    row = torch.arange(n, device=DEV) - s["q_start"][seq]
    q = torch.zeros(batch, s["max_q"], hq, d, device=DEV)
    q[seq, row] = s["q"].float()
    q = q.view(batch, s["max_q"], hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    q = q.reshape(batch, hk, -1, d)                                   # [B, Hk, G * Q, D]
    table = s["block_table"].clamp(min=0).long()
    k = s["k_cache"][table].flatten(1, 2).float().permute(0, 2, 3, 1)  # [B, Hk, D, T]
    v = s["v_cache"][table].flatten(1, 2).float().transpose(1, 2)      # [B, Hk, T, D]
    x = torch.matmul(q, k)
    x *= 1.0 / math.sqrt(d)
    if c["cap"]:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    last = torch.arange(s["max_q"], device=DEV)[None] + (s["kv_len"] - new)[:, None]  # [B, Q]
    key = torch.arange(k.shape[-1], device=DEV)
    hidden = (key > last[..., None]) | (key >= s["kv_len"][:, None, None])
    if c["window"]:
        hidden |= key <= last[..., None] - c["window"]
    x = x.view(batch, hk, hq // hk, s["max_q"], -1)
    x.masked_fill_(hidden[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top.masked_fill_(top == -math.inf, 0.0)
    x -= top
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(batch, hk, -1, x.shape[-1]), v).view(batch, hk, hq // hk, s["max_q"], d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(0, 3, 1, 2, 4).reshape(batch, s["max_q"], hq, d)[seq, row].to(s["q"].dtype)


# ------------------------------------------------------------------------------- what it costs


def work(case):
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "rope":
        n = case["tokens"]
        return {"bytes": 4 * n * (hq + hk) * d + 4 * n + 4 * case["rot"], "flops": 6 * n * (hq + hk) * case["rot"] // 2}
    ql, kl = _lengths(case)
    n, page = sum(ql), case["page"]
    index = 4 * (2 * len(ql) + 1) + 4 * sum((t + page - 1) // page for t in kl)
    if case["op"] == "append":
        new_pages = sum((t - 1) // page - (t - m) // page + 1 for m, t in zip(ql, kl))
        return {"bytes": 4 * n * (hq + 2 * hk) * d + 4 * case["rot"] + 8 * len(ql) + 4 * new_pages,
                "flops": 6 * n * (hq + hk) * case["rot"] // 2}
    w = case["window"] or max(kl)
    read, pairs = 0, 0
    for m, t in zip(ql, kl):
        read += t - max(0, t - m + 1 - w)
        pairs += sum(min(w, t - m + 1 + i) for i in range(m))
    return {"bytes": 4 * read * hk * d + 4 * n * hq * d + index, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------- in 64 bits


def _turned64(x, at, s):
    """Each pair of a head as a complex number, multiplied by m * exp(i * angle)."""
    c = s["case"]
    half = c["rot"] // 2
    i = torch.arange(half, device=DEV)
    one, two = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    a = at.to(torch.float64).view(-1, 1, 1) * s["inv_freq"].view(1, 1, -1)
    x = x.to(torch.float64)
    z = torch.complex(x[:, :, one], x[:, :, two]) * torch.polar(torch.full_like(a, s["m"]), a)
    y = x.clone()
    y[:, :, one], y[:, :, two] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned64(s["q"], s["positions"], s), _turned64(s["k"], s["positions"], s)
    ql, kl = _lengths(case)
    page = case["page"]
    table = s["block_table"].tolist()
    if case["op"] == "append":
        at = torch.cat([torch.arange(t - m, t) for m, t in zip(ql, kl)]).to(DEV)
        q, k = _turned64(s["q"], at, s), _turned64(s["k"], at, s)
        kc, vc = s["k_cache"].to(torch.float64), s["v_cache"].to(torch.float64)
        first = 0
        for m, t, pages in zip(ql, kl, table):
            slot = torch.tensor([pages[p // page] * page + p % page for p in range(t - m, t)], device=DEV)
            kc[slot // page, slot % page] = k[first:first + m]
            vc[slot // page, slot % page] = s["v"][first:first + m].to(torch.float64)
            first += m
        return q, kc, vc
    hq, hk, d = case["hq"], case["hk"], case["d"]
    out = torch.zeros(sum(ql), hq, d, dtype=torch.float64, device=DEV)
    first = 0
    for m, t, pages in zip(ql, kl, table):
        used = torch.tensor(pages[:(t + page - 1) // page], device=DEV)
        place = torch.arange(t - m, t, device=DEV).view(-1, 1)
        key = torch.arange(t, device=DEV).view(1, -1)
        seen = key <= place
        if case["window"]:
            seen &= key > place - case["window"]
        for h in range(hk):
            k = s["k_cache"][used, :, h].reshape(-1, d)[:t].to(torch.float64)
            v = s["v_cache"][used, :, h].reshape(-1, d)[:t].to(torch.float64)
            for e in range(h * (hq // hk), (h + 1) * (hq // hk)):
                x = s["q"][first:first + m, e].to(torch.float64) @ k.T / math.sqrt(d)
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                out[first:first + m, e] = torch.softmax(x, -1) @ v
        first += m
    return out
