"""The paged 16-bit cache and the attention over packed prompts: cases, plain forms and timings' work.

Four operators that a server uses together:
  packed   causal attention of packed prompts of different lengths
  paged    attention of each request's new tokens (one, or a chunk) over its cache pages
  assign   block tables, slot map and positions of a step from the requests' lengths
  append   the step's keys and values into the pages by the slot map
``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is set,
through the package's entry points.  Lengths follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a few short prompts of a small model: launch and latency
        {"name": "packed small", "op": "packed", "dtype": "bf16", "batch": 3, "tokens": 97,
         "hq": 4, "hkv": 2, "dim": 64, "mix": 1},
        # a batch of prompts of mixed lengths, one key head per query head
        {"name": "packed ragged mha fp16", "op": "packed", "dtype": "fp16", "batch": 13,
         "tokens": 8111, "hq": 32, "hkv": 32, "dim": 128, "mix": 2},
        # one long prompt with grouped heads
        {"name": "packed long gqa", "op": "packed", "dtype": "bf16", "batch": 1, "tokens": 16384,
         "hq": 32, "hkv": 8, "dim": 128, "mix": 3},
        # one request's next token, a short context
        {"name": "decode small", "op": "paged", "dtype": "bf16", "batch": 1, "chunks": 0,
         "chunk": 1, "context": 513, "page": 16, "hq": 4, "hkv": 2, "dim": 64, "mix": 4},
        # a decode step of one layer, contexts up to 8K
        {"name": "decode gqa 8k", "op": "paged", "dtype": "bf16", "batch": 16, "chunks": 0,
         "chunk": 1, "context": 8192, "page": 64, "hq": 32, "hkv": 8, "dim": 128, "mix": 5},
        # the same with one key head per query head and small pages
        {"name": "decode mha fp16 4k", "op": "paged", "dtype": "fp16", "batch": 8, "chunks": 0,
         "chunk": 1, "context": 4096, "page": 16, "hq": 32, "hkv": 32, "dim": 128, "mix": 6},
        # a mixed step: two prompts' chunks beside decoding requests
        {"name": "mixed step", "op": "paged", "dtype": "bf16", "batch": 32, "chunks": 2,
         "chunk": 509, "context": 4096, "page": 32, "hq": 32, "hkv": 8, "dim": 128, "mix": 7},
        # the last chunk of a long prompt
        {"name": "chunk of long prompt", "op": "paged", "dtype": "bf16", "batch": 1, "chunks": 1,
         "chunk": 1024, "context": 32768, "page": 128, "hq": 32, "hkv": 8, "dim": 128, "mix": 8},
        # bookkeeping of a decode step
        {"name": "assign decode step", "op": "assign", "batch": 16, "tokens": 16, "context": 8192,
         "page": 64, "mix": 9},
        # bookkeeping of a large step with new prompts and finished requests
        {"name": "assign prompt step", "op": "assign", "batch": 500, "tokens": 65000,
         "context": 4096, "page": 16, "mix": 10},
        # the new token of each request
        {"name": "append decode step", "op": "append", "dtype": "bf16", "tokens": 16, "page": 64,
         "pages": 256, "hkv": 8, "dim": 128, "mix": 11},
        # a step's prompts
        {"name": "append prompt step", "op": "append", "dtype": "fp16", "tokens": 16000,
         "page": 16, "pages": 2048, "hkv": 8, "dim": 128, "mix": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["packed", "packed", "paged", "paged", "paged", "assign", "append"])
    mix = rng.randrange(1 << 20)
    dtype = rng.choice(["bf16", "fp16"])
    dim = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    ratio = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "packed":
        hq = min(32, hkv * ratio)
        return {"op": op, "dtype": dtype, "batch": _log(rng, 1, 64), "tokens": _log(rng, 64, 12000),
                "hq": hq, "hkv": min(hkv, hq), "dim": dim, "mix": mix}
    if op == "paged":
        hq = hkv * ratio
        chunks = rng.choice([0, 0, 1, 2])
        batch = max(chunks, _log(rng, 1, 64))
        context = _log(rng, 64, 16384)
        chunk = min(context, _log(rng, 2, 1024)) if chunks else rng.choice([1, 1, 1, 2])
        # the plain form holds every request's scores padded to the largest
        while batch * hq * chunk * context > 2_500_000_000:
            batch = max(chunks, batch // 2) if batch > max(chunks, 1) else batch
            context = context if batch > max(chunks, 1) else context // 2 + 1
            chunk = min(chunk, context)
        return {"op": op, "dtype": dtype, "batch": batch, "chunks": chunks, "chunk": chunk,
                "context": context, "page": page, "hq": hq, "hkv": hkv, "dim": dim, "mix": mix}
    if op == "assign":
        batch = _log(rng, 1, 1000)
        return {"op": op, "batch": batch, "tokens": max(batch, _log(rng, 16, 65000)),
                "context": _log(rng, 64, 8192), "page": page, "mix": mix}
    tokens = _log(rng, 1, 16000)
    return {"op": op, "dtype": dtype, "tokens": tokens, "page": page,
            "pages": tokens // page + rng.randrange(2, 64), "hkv": hkv, "dim": dim, "mix": mix}


# ---- lengths: a function of the case alone ----

def _split(total, parts, rng):
    """`parts` lengths of at least one that sum to `total`, from short to long ones."""
    parts = min(parts, total)
    w = [math.exp(rng.uniform(0.0, 3.0)) for _ in range(parts)]
    free, s = total - parts, sum(w)
    n = [1 + int(free * x / s) for x in w]
    n[rng.randrange(parts)] += total - sum(n)
    return n


def _lengths(case):
    """(tokens held in all after the step, new tokens among them) of each request."""
    rng = random.Random(case["mix"])
    if case["op"] == "packed":
        n = _split(case["tokens"], case["batch"], rng)
        return n, n
    if case["op"] == "paged":
        total, new = [], []
        for b in range(case["batch"]):
            n = case["chunk"] if b < case["chunks"] or not case["chunks"] else 1
            low = max(n, case["context"] // 4)
            total.append(case["context"] if b == 0 else rng.randint(low, max(low, case["context"])))
            new.append(n)
        return total, new
    # assign: (held before, new); most requests decode, some bring a prompt, some are done
    held, new = [], []
    prompts = _split(case["tokens"] - case["batch"], max(1, case["batch"] // 4), rng) \
        if case["tokens"] > case["batch"] else []
    for b in range(case["batch"]):
        if b % 4 == 3 and prompts:
            held.append(0 if b % 8 == 3 else rng.randint(0, case["context"]))
            new.append(prompts.pop())
        elif b % 16 == 5:
            held.append(rng.randint(0, case["context"]))
            new.append(-1)
        else:
            held.append(rng.randint(1, case["context"]))
            new.append(1)
    return held, new


def _ceil(a, b):
    return -(-a // b)


# ---- inputs ----

def _normal(g, shape, dtype, scale=None):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x if scale is None else x.mul_(scale)).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + case["mix"])
    s = {"op": case["op"]}
    if case["op"] == "assign":
        held, new = _lengths(case)
        page = case["page"]
        have = [_ceil(h, page) for h in held]
        need = [max(0, _ceil(h + n, page) - p) if n > 0 else 0 for h, n, p in zip(held, new, have)]
        width = max(h + n for h, n in zip(have, need)) + 3
        pages = sum(have) + sum(need) + 17
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        has = torch.arange(width, device="cuda")[None, :] < _ints(have)[:, None]
        table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
        table[has] = order[:sum(have)]
        free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        free[:pages - sum(have)] = order[sum(have):]
        total = sum(n for n in new if n > 0)
        capacity = total + 5  # a few padded rows, as in a step of fixed size
        s.update(page=page, lengths=_ints(held), new=_ints(new), table=table, free=free,
                 num_free=_ints([pages - sum(have)]), kv=_ints(held), num_free_out=_ints([0]),
                 offsets=_ints([0] * (case["batch"] + 1)), slots=_ints([0] * capacity),
                 positions=_ints([0] * capacity), status=_ints([0]))
        return s
    dtype, dim, hkv = DTYPES[case["dtype"]], case["dim"], case["hkv"]
    # keys carry a scale per channel and head, values do not
    outlier = torch.exp(torch.randn(hkv, dim, generator=g, device="cuda"))
    if case["op"] == "append":
        t, page = case["tokens"], case["page"]
        s["k_pages"] = _normal(g, (case["pages"], hkv, page, dim), dtype)
        s["v_pages"] = _normal(g, (case["pages"], hkv, page, dim), dtype)
        s["k"] = _normal(g, (t, hkv, dim), dtype, outlier)
        s["v"] = _normal(g, (t, hkv, dim), dtype)
        s["slots"] = torch.randperm(case["pages"] * page, generator=g, device="cuda")[:t].to(torch.int32)
        return s
    total, new = _lengths(case)
    t = sum(new)
    s["q"] = _normal(g, (t, case["hq"], dim), dtype)
    ends = [0]
    for n in new:
        ends.append(ends[-1] + n)
    s["offsets"] = _ints(ends)
    s["kv_heads"] = hkv
    if case["op"] == "packed":
        s["k"] = _normal(g, (t, hkv, dim), dtype, outlier)
        s["v"] = _normal(g, (t, hkv, dim), dtype)
        return s
    page = case["page"]
    have = [_ceil(n, page) for n in total]
    pages = sum(have) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(total), max(have) + 1), dtype=torch.int32, device="cuda")
    table[torch.arange(max(have) + 1, device="cuda")[None, :] < _ints(have)[:, None]] = order[:sum(have)]
    s["k_pages"] = _normal(g, (pages, hkv, page, dim), dtype, outlier[:, None, :])
    s["v_pages"] = _normal(g, (pages, hkv, page, dim), dtype)
    s.update(table=table, kv=_ints(total), max_new=max(new))
    return s


# ---- one pass ----

def run(s):
    if own:
        return _run_own(s)
    return {"packed": _packed, "paged": _paged, "assign": _assign, "append": _append}[s["op"]](s)


def _run_own(s):
    import decode_attention_kivi_b200 as K

    if s["op"] == "assign":
        K.kivi_paged_assign(s["lengths"], s["new"], s["table"], s["free"], s["num_free"], s["page"],
                            kv_lengths=s["kv"], num_free_out=s["num_free_out"],
                            offsets=s["offsets"], slots=s["slots"], positions=s["positions"],
                            status=s["status"])
        return _assigned(s)
    if s["op"] == "append":
        K.kivi_paged_append(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"])
        return s["k_pages"], s["v_pages"]
    if "workspace" not in s:  # kept by a program for all its calls of this shape
        n = K.kivi_attention_workspace_bytes(s["kv_heads"], s["q"].shape[1], s["q"].shape[2])
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    if s["op"] == "packed":
        return K.kivi_packed_attention(s["q"], s["k"], s["v"], s["offsets"], s["workspace"])
    return K.kivi_paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv"],
                                  s["offsets"], s["workspace"], max_new=s["max_new"])


def _softmax_(x, seen):
    """Softmax weights over the last axis in place; nothing where a row sees no key."""
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = x.sum(-1, keepdim=True)
    return torch.where(total > 0, total, torch.ones_like(total))


def _packed(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    t, hq, d = q.shape
    hkv = k.shape[1]
    i = torch.arange(t, device=q.device)
    seq = torch.searchsorted(s["offsets"][1:].contiguous(), i.to(torch.int32), right=True)
    seen = (seq[:, None] == seq[None, :]) & (i[:, None] >= i[None, :])
    qg = q.view(t, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    x = torch.matmul(qg, k.permute(1, 2, 0)).mul_(1.0 / math.sqrt(d)).view(hkv, -1, t, t)
    total = _softmax_(x, seen)
    o = torch.matmul(x.view(hkv, -1, t), v.permute(1, 0, 2)).view(hkv, -1, t, d) / total
    return o.permute(2, 0, 1, 3).reshape(t, hq, d).to(s["q"].dtype)


def _paged(s):
    q, table, off = s["q"], s["table"].long(), s["offsets"].long()
    t, hq, d = q.shape
    _, hkv, page, _ = s["k_pages"].shape
    b, width = table.shape
    new = off[1:] - off[:-1]
    row = torch.arange(t, device=q.device)
    req = torch.searchsorted(off[1:].contiguous(), row, right=True)
    at = row - off[req]
    n = s["max_new"]
    padded = torch.zeros((b, n, hq, d), device=q.device)
    padded[req, at] = q.float()
    k = s["k_pages"][table].float().permute(0, 2, 4, 1, 3).reshape(b, hkv, d, width * page)
    v = s["v_pages"][table].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, width * page, d)
    key = torch.arange(width * page, device=q.device)
    kv = s["kv"].long()
    last = (kv - new)[:, None] + torch.arange(n, device=q.device)[None, :]
    seen = (key <= last[..., None]) & (key < kv[:, None, None])
    v = torch.where((key < kv[:, None])[:, None, :, None], v, torch.zeros((), device=q.device))
    g = padded.view(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    x = torch.matmul(g, k).mul_(1.0 / math.sqrt(d)).view(b, hkv, -1, n, width * page)
    total = _softmax_(x, seen[:, None, None])
    o = torch.matmul(x.view(b, hkv, -1, width * page), v).view(b, hkv, -1, n, d) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)
    return o[req, at].to(q.dtype)


def _assigned(s):
    return {k: s[k] for k in ("table", "kv", "offsets", "slots", "positions", "num_free_out",
                              "free", "status")}


def _assign(s):
    page, held, new = s["page"], s["lengths"].long(), s["new"].long()
    table, free, num_free = s["table"], s["free"], s["num_free"].long()
    b, width = table.shape
    have = (held + page - 1) // page
    done = new < 0
    add = new.clamp(min=0)
    kv = torch.where(done, torch.zeros_like(held), held + add)
    need = torch.where(done, torch.zeros_like(have), (kv + page - 1) // page - have)
    col = torch.arange(width, device=held.device)[None, :]
    back = done[:, None] & (col < have[:, None])          # pages given back, in request order
    returned = table[back]
    top = num_free + returned.numel()
    free[num_free + torch.arange(returned.numel(), device=held.device)] = returned
    take = (col >= have[:, None]) & (col < (have + need)[:, None])
    taken = torch.arange(int(need.sum()), device=held.device)
    table[take] = free[top - 1 - taken]                    # popped from the end of the stack
    off = torch.zeros_like(s["offsets"])
    off[1:] = add.cumsum(0)
    row = torch.arange(s["slots"].numel(), device=held.device)
    real = row < off[-1]
    req = torch.searchsorted(off[1:].contiguous(), row.to(torch.int32), right=True).clamp(max=b - 1)
    pos = held[req] + row - off[req]
    pos = torch.where(real, pos, torch.zeros_like(pos))
    slot = table[req, pos // page].long() * page + pos % page
    s["kv"].copy_(kv)
    s["offsets"].copy_(off)
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(real, slot, torch.full_like(slot, -1)))
    s["num_free_out"].copy_(top - need.sum())
    s["status"].zero_()
    return _assigned(s)


def _append(s):
    page = s["k_pages"].shape[2]
    slot = s["slots"].long()
    s["k_pages"][slot // page, :, slot % page] = s["k"]
    s["v_pages"][slot // page, :, slot % page] = s["v"]
    return s["k_pages"], s["v_pages"]


# ---- what a pass cannot do without ----

def work(case):
    if case["op"] == "append":
        # new rows read and written, one slot each
        return {"bytes": 8 * case["tokens"] * case["hkv"] * case["dim"] + 4 * case["tokens"],
                "flops": 0}
    held, new = _lengths(case)
    if case["op"] == "assign":
        page = case["page"]
        tokens = sum(n for n in new if n > 0)
        taken = sum(_ceil(h + n, page) - _ceil(h, page) for h, n in zip(held, new) if n > 0)
        back = sum(_ceil(h, page) for h, n in zip(held, new) if n < 0)
        # lengths in and out, offsets; slot and position per token; pages read and written
        return {"bytes": 4 * (4 * len(new) + 2 * (tokens + 5) + 2 * (taken + back)), "flops": 0}
    d, hq, hkv = case["dim"], case["hq"], case["hkv"]
    pairs = sum(n * (h - n) + n * (n + 1) // 2 for h, n in zip(held, new))
    return {"bytes": 2 * d * (2 * hkv * sum(held) + 2 * hq * sum(new)), "flops": 4 * d * hq * pairs}


# ---- the definition in 64 bits, request by request ----

def exact(case, seed):
    if case["op"] == "assign":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        page = case["page"]
        k, v = s["k_pages"].double(), s["v_pages"].double()
        flat_k, flat_v = k.transpose(1, 2).reshape(-1, case["hkv"], case["dim"]), \
            v.transpose(1, 2).reshape(-1, case["hkv"], case["dim"])
        flat_k.index_copy_(0, s["slots"].long(), s["k"].double())
        flat_v.index_copy_(0, s["slots"].long(), s["v"].double())
        back = lambda x: x.view(-1, page, case["hkv"], case["dim"]).transpose(1, 2)  # noqa: E731
        return back(flat_k), back(flat_v)
    total, new = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["dim"]
    out = torch.zeros((sum(new), hq, d), dtype=torch.float64, device="cuda")
    first = 0
    for b, (length, n) in enumerate(zip(total, new)):
        if case["op"] == "packed":
            keys, values = s["k"][first:first + n].double(), s["v"][first:first + n].double()
        else:
            ids = s["table"][b, :_ceil(length, case["page"])].long()
            keys, values = (x[ids].transpose(1, 2).reshape(-1, hkv, d)[:length].double()
                            for x in (s["k_pages"], s["v_pages"]))
        hidden = torch.ones((n, length), dtype=torch.bool, device="cuda").triu_(length - n + 1)
        for h in range(hq):
            x = (s["q"][first:first + n, h].double() / math.sqrt(d)) @ keys[:, h * hkv // hq].T
            p = torch.softmax(x.masked_fill_(hidden, -math.inf), -1)
            out[first:first + n, h] = p @ values[:, h * hkv // hq]
        first += n
    return out
