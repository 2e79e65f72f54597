"""Serving operators of a transformer's attention, as cases to be measured.

Three operators that a decoder runs one after the other:

append   rotate the new tokens' queries and keys by their positions, and put
         keys and values into a paged cache;
packed   attention over whole prompts of different lengths, packed one behind
         the other, with grouped heads;
decode   attention of one new token of each sequence over the paged cache.

`run` computes a case in its plain form (torch operations in 32 bits, angles
in 64), or through the library when `own` is true.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One step of a few conversations: the call's own cost is all there is.
        dict(name="append_step_8", op="append", seqs=8, tokens=8, heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, page=16, start=1500, dtype="bf16"),
        # One step of a full server.
        dict(name="append_step_256", op="append", seqs=256, tokens=256, heads=64, kv_heads=8,
             dim=128, rot=128, interleaved=False, page=64, start=2000, dtype="bf16"),
        # A whole batch of prompts goes into the cache; half of each head turns, in pairs of
        # neighbours, and far positions follow a long shared prefix.
        dict(name="append_prompts_16k", op="append", seqs=11, tokens=16001, heads=32, kv_heads=8,
             dim=128, rot=64, interleaved=True, page=32, start=100000, dtype="f16"),
        # One short conversation: latency.
        dict(name="decode_1x700", op="decode", batch=1, heads=32, kv_heads=8, dim=128, page=16,
             longest=700, ragged=False, padded=0, dtype="bf16"),
        # A server's batch with conversations of all lengths, and a few unused places in it.
        dict(name="decode_64_ragged_8k", op="decode", batch=64, heads=32, kv_heads=8, dim=128,
             page=16, longest=8192, ragged=True, padded=3, dtype="bf16"),
        # Many short conversations, a cached head for each query head, small heads.
        dict(name="decode_200x1000_d64", op="decode", batch=200, heads=16, kv_heads=16, dim=64,
             page=32, longest=1000, ragged=False, padded=0, dtype="f16"),
        # A few long documents, many query heads to a cached head.
        dict(name="decode_4x131072", op="decode", batch=4, heads=64, kv_heads=8, dim=128, page=64,
             longest=131072, ragged=False, padded=0, dtype="bf16"),
        # A short question: latency.
        dict(name="packed_1x90", op="packed", seqs=1, heads=32, kv_heads=8, dim=128, longest=90,
             ragged=False, context=0, causal=True, fused=False, dtype="bf16"),
        # Prompts of all lengths, q, k and v parts of one projection's output.
        dict(name="packed_16_ragged_4k", op="packed", seqs=16, heads=32, kv_heads=8, dim=128,
             longest=4096, ragged=True, context=0, causal=True, fused=True, dtype="bf16"),
        # A later part of a prompt, behind what its sequences hold already.
        dict(name="packed_2x500_after_8000", op="packed", seqs=2, heads=32, kv_heads=8, dim=128,
             longest=500, ragged=False, context=8000, causal=True, fused=False, dtype="bf16"),
        # An encoder's batch: every key, a key head for each query head, small heads.
        dict(name="packed_24x513_d64_full", op="packed", seqs=24, heads=12, kv_heads=12, dim=64,
             longest=513, ragged=False, context=0, causal=False, fused=True, dtype="f16"),
        # One long document.
        dict(name="packed_1x16384", op="packed", seqs=1, heads=16, kv_heads=2, dim=128,
             longest=16384, ragged=False, context=0, causal=True, fused=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8, 16] if kv_heads <= 4 else [1, 2, 3, 4])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    op = rng.choice(["append", "decode", "packed"])
    if op == "append":
        step = rng.random() < 0.5
        tokens = _log(rng, 1, 256 if step else 16001)
        return dict(op=op, seqs=tokens if step else max(1, min(tokens, _log(rng, 1, 40))),
                    tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]),
                    interleaved=rng.random() < 0.5, page=page,
                    start=_log(rng, 1, 2000 if step else 200000), dtype=dtype)
    if op == "decode":
        batch = _log(rng, 1, 256)
        most = 4 * 131072 * 8 * 128 // (batch * kv_heads * dim)
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    longest=_log(rng, 1, min(131072, most)), ragged=rng.random() < 0.6,
                    padded=rng.choice([0, 0, min(2, batch - 1)]), dtype=dtype)
    seqs = _log(rng, 1, 32)
    context = rng.choice([0, 0, _log(rng, 1, 8000)])
    most = int(math.sqrt(16384 * 16384 * 16 / 2 / (seqs * heads) + context * context)) - context
    return dict(op=op, seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim,
                longest=_log(rng, 1, max(1, min(8192, most))), ragged=rng.random() < 0.6,
                context=context, causal=rng.random() < 0.75,
                fused=context == 0 and rng.random() < 0.5, dtype=dtype)


def _lengths(case):
    """Lengths of a case's sequences: of the case alone, the same for every seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "append":
        if case["tokens"] == case["seqs"]:
            return [1] * case["seqs"]
        cuts = sorted(rng.sample(range(1, case["tokens"]), case["seqs"] - 1))
        return [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]
    n = case["batch"] - case["padded"] if case["op"] == "decode" else case["seqs"]
    top = case["longest"]
    if case["ragged"]:
        got = [top] + [_log(rng, max(1, top // 64), top) for _ in range(n - 1)]
    else:
        got = [top] + [rng.randint(max(1, top - top // 16), top) for _ in range(n - 1)]
    rng.shuffle(got)
    return got + [0] * case.get("padded", 0)


def _starts(case):
    """Where the new tokens of an append's sequences begin: of the case alone."""
    rng = random.Random(case["start"] + 7 * case["tokens"])
    return [rng.randrange(case["start"]) for _ in range(case["seqs"])]


# ------------------------------------------------------------------ inputs
def _table(starts, ends, page, rng, device):
    """A page table with pages in no order for places [start, end) of each sequence (0 where
    nothing is read or written), and how many pages there are."""
    low, high = [a // page for a in starts], [-(-b // page) for b in ends]
    need = [max(0, b - a) for a, b in zip(low, high)]
    pages = torch.randperm(sum(need) + 1, generator=rng, device=device, dtype=torch.int64)
    first, low, need = (torch.tensor(x, device=device)[:, None] for x in
                        ([sum(need[:i]) for i in range(len(need))], low, need))
    at = torch.arange(max(1, max(high)), device=device)[None] - low
    held = (at >= 0) & (at < need)
    table = torch.where(held, pages[torch.where(held, at + first, 0)], 0)
    return table.to(torch.int32), pages.numel()


def prepare(case, seed):
    device = "cuda"
    rng = torch.Generator(device=device)
    rng.manual_seed(seed)
    kind, d, hk, h = TYPES[case["dtype"]], case["dim"], case["kv_heads"], case["heads"]
    lengths = _lengths(case)

    def normal(*shape, by=1.0):
        return torch.empty(shape, device=device, dtype=kind).normal_(0.0, by, generator=rng)

    s = {"op": case["op"]}
    if case["op"] == "append":
        n, page = case["tokens"], case["page"]
        starts = _starts(case)
        s["table"], pages = _table(starts, [a + m for a, m in zip(starts, lengths)], page, rng,
                                   device)
        start, count = (torch.tensor(x, device=device) for x in (starts, lengths))
        ids = torch.repeat_interleave(torch.arange(case["seqs"], device=device), count)
        within = torch.arange(n, device=device) - (torch.cumsum(count, 0) - count)[ids]
        s["positions"] = (start[ids] + within).to(torch.int32)
        s["ids"] = ids.to(torch.int32)
        width = (h + 2 * hk) * d                       # q, k and v: one projection's output
        qkv = normal(n, width)
        s["q"] = qkv[:, :h * d].view(n, h, d)
        s["k"] = qkv[:, h * d:(h + hk) * d].view(n, hk, d)
        s["v"] = qkv[:, (h + hk) * d:].view(n, hk, d)
        s["k_cache"] = normal(pages, page, hk, d)
        s["v_cache"] = normal(pages, page, hk, d)
        half = case["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, device=device, dtype=torch.float64) / half)
        s["interleaved"] = case["interleaved"]
    elif case["op"] == "decode":
        page = case["page"]
        s["table"], pages = _table([0] * len(lengths), lengths, page, rng, device)
        s["lengths"] = torch.tensor(lengths, device=device, dtype=torch.int32)
        s["q"] = normal(case["batch"], h, d, by=2.0)
        s["k_cache"] = normal(pages, page, hk, d)
        s["v_cache"] = normal(pages, page, hk, d)
    else:
        keys = [m + case["context"] for m in lengths]
        total = sum(lengths)
        if case["fused"]:
            qkv = normal(total, (h + 2 * hk) * d)
            s["q"] = qkv[:, :h * d].mul_(2.0).view(total, h, d)
            s["k"] = qkv[:, h * d:(h + hk) * d].view(total, hk, d)
            s["v"] = qkv[:, (h + hk) * d:].view(total, hk, d)
        else:
            s["q"] = normal(total, h, d, by=2.0)
            s["k"] = normal(sum(keys), hk, d)
            s["v"] = normal(sum(keys), hk, d)
        s["cu_q"] = torch.tensor([0] + lengths, device=device).cumsum(0).to(torch.int32)
        s["cu_k"] = torch.tensor([0] + keys, device=device).cumsum(0).to(torch.int32)
        s["longest_q"], s["longest_k"] = max(lengths), max(keys)
        s["causal"] = case["causal"]
    return s


# --------------------------------------------------------------- plain forms
def _turned(x, positions, inv_freq, interleaved):
    """x [tokens, heads, dim] with its first 2 * len(inv_freq) elements turned."""
    half = inv_freq.numel()
    angle = positions.to(torch.float64)[:, None] * inv_freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y = x.float()
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1).to(x.dtype)


def _append(s):
    page = s["k_cache"].shape[1]
    places, ids = s["positions"].long(), s["ids"].long()
    at = s["table"][ids, places // page].long()
    q = _turned(s["q"], s["positions"], s["inv_freq"], s["interleaved"])
    s["k_cache"][at, places % page] = _turned(s["k"], s["positions"], s["inv_freq"],
                                              s["interleaved"])
    s["v_cache"][at, places % page] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _softmax_times(scores, v):
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    return torch.matmul(p, v) / p.sum(-1, keepdim=True)


def _decode(s):
    q, table = s["q"], s["table"].long()
    b, h, d = q.shape
    hk = s["k_cache"].shape[2]
    k = s["k_cache"][table].flatten(1, 2).transpose(1, 2).float()       # [b, hk, n, d]
    v = s["v_cache"][table].flatten(1, 2).transpose(1, 2).float()
    scores = torch.matmul(q.float().view(b, hk, h // hk, d), k.transpose(-1, -2)) / math.sqrt(d)
    past = torch.arange(k.shape[2], device=q.device)[None] >= s["lengths"][:, None]
    scores.masked_fill_(past[:, None, None], -math.inf)
    return _softmax_times(scores, v).view(b, h, d).to(q.dtype)


def _packed(s):
    q, device = s["q"], s["q"].device
    h, d = q.shape[1:]
    hk = s["k"].shape[1]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    n_q, n_k = cu_q.diff(), cu_k.diff()
    i, j = (torch.arange(s[n], device=device) for n in ("longest_q", "longest_k"))
    at_q = torch.clamp(cu_q[:-1, None] + i, max=q.shape[0] - 1)
    at_k = torch.clamp(cu_k[:-1, None] + j, max=s["k"].shape[0] - 1)
    b = at_q.shape[0]
    qp = q[at_q].float().view(b, -1, hk, h // hk, d).permute(0, 2, 3, 1, 4)   # [b, hk, g, nq, d]
    kp = s["k"][at_k].float().permute(0, 2, 3, 1)[:, :, None]                 # [b, hk, 1, d, nk]
    vp = s["v"][at_k].float().permute(0, 2, 1, 3)[:, :, None]                 # [b, hk, 1, nk, d]
    scores = torch.matmul(qp, kp).div_(math.sqrt(d))
    seen = (j[None] < n_k[:, None])[:, None]
    if s["causal"]:
        seen = seen & (j[None, None] <= (i[None] + (n_k - n_q)[:, None])[..., None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    out = _softmax_times(scores, vp).permute(0, 3, 1, 2, 4).flatten(2, 3)     # [b, nq, h, d]
    token = torch.arange(q.shape[0], device=device)
    row = torch.searchsorted(cu_q, token, right=True) - 1
    return out[row, token - cu_q[row]].to(q.dtype)


def run(state):
    s = state
    if own:
        import row_wise_softmax_gb300 as rws
        if s["op"] == "append":
            q = rws.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"],
                              s["positions"], seq_ids=s["ids"], q=s["q"],
                              inv_freq=s["inv_freq"], interleaved=s["interleaved"])
            return q, s["k_cache"], s["v_cache"]
        if s["op"] == "decode":
            return rws.attention_decode(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                        s["lengths"])
        return rws.attention_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"],
                                    causal=s["causal"])
    return {"append": _append, "decode": _decode, "packed": _packed}[s["op"]](s)


# ---------------------------------------------------------------- definition
def _exact_append(s):
    n, h, d = s["q"].shape
    half = s["inv_freq"].numel()
    first = list(range(0, 2 * half, 2)) if s["interleaved"] else list(range(half))
    second = [a + 1 for a in first] if s["interleaved"] else [a + half for a in first]
    turn = torch.polar(torch.ones(n, 1, half, dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None, None] * s["inv_freq"])

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    page = k_cache.shape[1]
    slot = torch.gather(s["table"].long()[s["ids"].long()], 1,
                        torch.div(s["positions"].long(), page, rounding_mode="floor")[:, None])
    slot = slot[:, 0] * page + torch.remainder(s["positions"].long(), page)
    k_cache.flatten(0, 1).index_copy_(0, slot, turned(s["k"]))
    v_cache.flatten(0, 1).index_copy_(0, slot, s["v"].double())
    return turned(s["q"]), k_cache, v_cache


def _exact_head(q, k, v, seen):
    """softmax(q k^T / sqrt(d)) v of one head in 64 bits, over the keys that are seen."""
    z = torch.einsum("qd,kd->qk", q.double(), k.double()) * q.shape[-1] ** -0.5
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    return torch.einsum("qk,kd->qd", torch.softmax(z, -1), v.double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    if case["op"] == "decode":
        page = case["page"]
        for b, n in enumerate(_lengths(case)):
            if n == 0:
                out[b] = math.nan
                continue
            rows = s["table"][b, :-(-n // page)].long()
            k = s["k_cache"][rows].flatten(0, 1)[:n].double()
            v = s["v_cache"][rows].flatten(0, 1)[:n].double()
            z = torch.einsum("hgd,nhd->hgn", s["q"][b].double().view(-1, group, case["dim"]), k)
            p = torch.softmax(z * case["dim"] ** -0.5, -1)
            out[b] = torch.einsum("hgn,nhd->hgd", p, v).reshape(out[b].shape)
        return out
    a = c = 0
    for n in _lengths(case):
        m = n + case["context"]
        for t in range(0, n, 2048):                     # queries, a block at a time
            e = min(n, t + 2048)
            last = m if not case["causal"] else e + m - n
            i = torch.arange(t, e, device="cuda")[:, None] + (m - n if case["causal"] else m)
            seen = torch.arange(last, device="cuda")[None] <= i
            for h in range(case["heads"]):
                out[a + t:a + e, h] = _exact_head(s["q"][a + t:a + e, h],
                                                  s["k"][c:c + last, h // group],
                                                  s["v"][c:c + last, h // group], seen)
        a, c = a + n, c + m
    return out


# ---------------------------------------------------------------------- work
def work(case):
    d, h, hk, lengths = case["dim"], case["heads"], case["kv_heads"], _lengths(case)
    if case["op"] == "append":
        n = case["tokens"]
        return {"bytes": n * (2 * h + 4 * hk) * d * 2 + 12 * n + 4 * case["rot"],
                "flops": 3.0 * n * (h + hk) * case["rot"]}
    if case["op"] == "decode":
        tokens = sum(lengths)
        return {"bytes": tokens * hk * d * 4 + case["batch"] * (h * d * 4 + 4)
                + 4 * sum(-(-n // case["page"]) for n in lengths),
                "flops": 4.0 * tokens * h * d}
    keys = [n + case["context"] for n in lengths]
    pairs = sum(n * (m - n) + n * (n + 1) // 2 if case["causal"] else n * m
                for n, m in zip(lengths, keys))
    return {"bytes": sum(lengths) * h * d * 4 + sum(keys) * hk * d * 4 + 8 * (len(lengths) + 1),
            "flops": 4.0 * pairs * h * d}
