"""The serving operators' cases: what is measured of ``append_kv``, ``prompt_attention``, ``paged_attention``
and ``process_logits``, with each operator's plain form (elementary torch operations in 32 bits) and its
definition in 64 bits.

A case is a dict with an ``"op"``.  Attention cases carry heads (``hq``/``hkv``), head size ``d``, type
``dtype``, new tokens per sequence ``new`` and tokens already cached ``ctx`` (or the keys ``kv`` of each
sequence), as texts of numbers; cached cases have a ``page`` size
and the pool layout ``order`` ("hnd": page, head, row; "nhd": page, row, head).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases
def listed():
    ragged = [696, 2450, 2106, 216, 1316, 3764, 443, 949]
    spread = [128 + (i * 2477) % 3969 for i in range(32)]
    return [
        # the first short prompt of a chat on the two-layer decoder: latency
        dict(name="prompt_short", op="prompt", hq=4, hkv=2, d=64, dtype="bf16", new="17", ctx="0", page=0,
             order="hnd", causal=True),
        # eight prompts of the batch sweep's lengths, packed, with the 16-layer decoder's heads
        dict(name="prompt_packed", op="prompt", hq=32, hkv=8, d=64, dtype="bf16", new=_text(ragged), ctx=_text([0] * 8), page=0,
             order="hnd", causal=True),
        # the next chunk of three long prompts over their cached pages (chunked filling), odd lengths
        dict(name="prompt_chunk_paged", op="prompt", hq=24, hkv=8, d=128, dtype="fp16", new="511 1024 77",
             ctx="8191 0 2500", page=64, order="hnd", causal=True),
        # one long document
        dict(name="prompt_long", op="prompt", hq=32, hkv=8, d=128, dtype="bf16", new="16384", ctx="0", page=0,
             order="hnd", causal=True),
        # one sequence at the headline context, in the decoder's own slot cache (one page per slot)
        dict(name="decode_one", op="decode", hq=32, hkv=8, d=64, dtype="bf16", kv="1025", page=2048, order="hnd"),
        # a continuous batch over small pages, contexts spread over 128..4096
        dict(name="decode_batch", op="decode", hq=32, hkv=8, d=128, dtype="bf16", kv=_text(spread), page=16, order="nhd"),
        # three long sequences of very different length, few key heads
        dict(name="decode_long", op="decode", hq=28, hkv=4, d=128, dtype="fp16", kv="200001 31000 977", page=64,
             order="hnd"),
        # one new token of each sequence of a decode batch
        dict(name="append_step", op="append", hq=32, hkv=8, d=64, dtype="bf16", new=_text([1] * 64),
             ctx=_text(63 * i + 5 for i in range(64)), page=32, order="hnd", theta=10000.0),
        # a chunk of prompts going into the cache, one far into its context
        dict(name="append_prompt", op="append", hq=32, hkv=8, d=128, dtype="bf16", new="4096 1 2001 2050",
             ctx="0 300 40001 17", page=64, order="nhd", theta=500000.0),
        # one sequence's logits after a long answer: latency
        dict(name="logits_one", op="logits", rows=1, vocab=128256, dtype="fp32", hist=1500, prompt=1024, bias=0,
             mask=False),
        # a decode batch with penalties, biases and a grammar's mask
        dict(name="logits_batch", op="logits", rows=64, vocab=128256, dtype="fp32", hist=4096, prompt=700, bias=64,
             mask=True),
        # an odd vocabulary from a 16-bit product
        dict(name="logits_odd", op="logits", rows=13, vocab=32001, dtype="bf16", hist=333, prompt=40, bias=300,
             mask=True),
    ]


def _text(vals):
    return " ".join(str(v) for v in vals)


def _lens(case, key):
    return [int(v) for v in case[key].split()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hkv = rng.choice([1, 2, 4, 8])
    return hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16] if hkv < 8 else [1, 2, 3, 4]), hkv


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "append", "logits"])
    if op == "logits":
        return dict(op=op, rows=_log(rng, 1, 64), vocab=_log(rng, 1000, 128256), dtype=rng.choice(["fp32", "bf16", "fp16"]),
                    hist=_log(rng, 1, 4096), prompt=_log(rng, 1, 2048), bias=rng.choice([0, 1, _log(rng, 2, 300)]),
                    mask=rng.random() < 0.5)
    hq, hkv = _heads(rng)
    case = dict(op=op, hq=hq, hkv=hkv, d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                order=rng.choice(["hnd", "nhd"]))
    if op == "decode":
        n = _log(rng, 1, 64)
        top = min(131072, 900_000 // (n * hkv))
        case.update(kv=_text(_log(rng, 1, top) for _ in range(n)), page=rng.choice([16, 32, 64, 128, 200, 1024]))
        return case
    n = _log(rng, 1, 12)
    top = max(2, 24000 // n) if op == "append" else max(2, min(12000, 24000 // n))
    new = [_log(rng, 1, top) for _ in range(n)]
    if op == "append":
        case.update(new=_text(new), ctx=_text(rng.choice([0, _log(rng, 1, 8000)]) for _ in new),
                    page=rng.choice([16, 32, 64, 128, 200]), theta=rng.choice([10000.0, 500000.0]))
        return case
    paged = rng.random() < 0.5
    case.update(new=_text(new), ctx=_text(rng.choice([0, _log(rng, 1, 6000)]) if paged else 0 for _ in new),
                page=rng.choice([16, 32, 64, 128, 200]) if paged else 0, causal=rng.random() < 0.8)
    if not paged:
        case["order"] = "hnd"
    return case


# ------------------------------------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _pool(case, gen, lens):
    """A pool with just the pages of `lens` tokens per sequence, handed out in a shuffled order."""
    ps, hkv, d, dt = case["page"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    need = [max(1, -(-n // ps)) for n in lens]
    total = sum(need)
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    shape = (total, hkv, ps, d) if case["order"] == "hnd" else (total, ps, hkv, d)
    k, v = torch.empty(shape, dtype=dt, device=DEV), torch.empty(shape, dtype=dt, device=DEV)
    step = max(1, (1 << 26) // (hkv * ps * d))
    for i in range(0, total, step):  # in parts: the 32-bit normals of a long cache would take too much at once
        k[i:i + step] = _normal(gen, k[i:i + step].shape, dt)
        v[i:i + step] = _normal(gen, v[i:i + step].shape, dt)
    if case["order"] == "nhd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return k, v, table


def _ints(vals):
    return torch.tensor(vals, dtype=torch.int32, device=DEV)


def _cu(lens):
    return _ints([0] + list(np.cumsum(lens)))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "logits":
        R, V, H = case["rows"], case["vocab"], case["hist"]
        st["logits"] = (3.0 * torch.randn((R, V), generator=gen, device=DEV)).to(dt)
        # a text repeats itself: ids fall off as a power, so some occur many times
        u = torch.rand((R, H), generator=gen, device=DEV)
        ids = (V ** u - 1).to(torch.int32).clamp_(0, V - 1)
        st["history"] = (ids * 7919 + seed % 1000) % V
        lens = torch.randint((H + 1) // 2, H + 1, (R,), generator=gen, device=DEV, dtype=torch.int32)
        st["history_lens"] = lens
        st["prompt_lens"] = torch.minimum(lens, torch.full_like(lens, case["prompt"]))
        st["repetition"] = 1.0 + 0.3 * torch.rand(R, generator=gen, device=DEV)
        st["frequency"] = 0.2 * torch.rand(R, generator=gen, device=DEV)
        st["presence"] = 0.5 * torch.rand(R, generator=gen, device=DEV)
        st["bias"] = None
        if case["bias"]:
            n = case["bias"]
            st["bias"] = (_ints([n * r for r in range(R + 1)]),
                          torch.randint(0, V, (R * n,), generator=gen, device=DEV, dtype=torch.int32),
                          2.0 * torch.randn(R * n, generator=gen, device=DEV))
        st["mask"] = None
        if case["mask"]:  # a grammar allows about one id in four here
            words = (V + 31) // 32
            a = torch.randint(-2**31, 2**31, (2, R, words), generator=gen, device=DEV, dtype=torch.int64)
            st["mask"] = (a[0] & a[1]).to(torch.int32)
        st["out"] = torch.empty((R, V), dtype=torch.float32, device=DEV)
        return st
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "decode":
        st["q"] = _normal(gen, (len(_lens(case, "kv")), hq, d), dt)
        st["k"], st["v"], st["table"] = _pool(case, gen, _lens(case, "kv"))
        st["kv_lens"] = _ints(_lens(case, "kv"))
        if own:
            import event_tensor_task_b200 as mk
            n = mk.mk_paged_attention_workspace_bytes(len(_lens(case, "kv")), hq, hkv, d)
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        return st
    T = sum(_lens(case, "new"))
    st["cu"] = _cu(_lens(case, "new"))
    if case["op"] == "prompt":
        st["q"] = _normal(gen, (T, hq, d), dt)
        if case["page"]:
            st["k"], st["v"], st["table"] = _pool(case, gen, [a + c for a, c in zip(_lens(case, "new"), _lens(case, "ctx"))])
            st["kv_lens"] = _ints([a + c for a, c in zip(_lens(case, "new"), _lens(case, "ctx"))])
        else:
            st["k"], st["v"] = _normal(gen, (T, hkv, d), dt), _normal(gen, (T, hkv, d), dt)
        return st
    # append: q, k and v are the columns of one projection's output
    st["qkv"] = _normal(gen, (T, hq + 2 * hkv, d), dt)
    st["k"], st["v"], st["table"] = _pool(case, gen, [a + c for a, c in zip(_lens(case, "new"), _lens(case, "ctx"))])
    st["ctx"] = _ints(_lens(case, "ctx"))
    return st


# ------------------------------------------------------------------------------------------------ plain forms
def _attend(q, k, v, scale, limit, wide):
    """q [n][Hq][D], k/v [m][Hkv][D], query i sees the keys j < limit[i]; in the type `wide`."""
    n, hq, d = q.shape
    m, hkv = k.shape[0], k.shape[1]
    if m == 0:
        return torch.zeros((n, hq, d), dtype=wide, device=q.device)
    qs = q.to(wide).reshape(n, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    s = torch.matmul(qs, k.to(wide).permute(1, 2, 0)) * scale  # [Hkv][G*n][m]
    s = s.reshape(hkv, hq // hkv, n, m)
    dead = torch.arange(m, device=q.device)[None, :] >= limit[:, None]
    s = s.masked_fill(dead, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p.reshape(hkv, -1, m), v.to(wide).permute(1, 0, 2))
    return o.reshape(hkv, hq // hkv, n, d).permute(2, 0, 1, 3).reshape(n, hq, d)


def _rows(pool, table, b, n, ps):
    """The first n cached rows of sequence b, [n][Hkv][D]."""
    pages = pool[table[b, :max(1, -(-n // ps))].long()]  # [p][Hkv][ps][D]
    return pages.transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])[:n]


def _prompt(st, wide):
    case, q = st["case"], st["q"]
    out = torch.empty(q.shape, dtype=q.dtype if wide is torch.float32 else wide, device=q.device)
    scale, at = 1.0 / math.sqrt(case["d"]), 0
    for b, (n, c) in enumerate(zip(_lens(case, "new"), _lens(case, "ctx"))):
        m = n + c
        k = _rows(st["k"], st["table"], b, m, case["page"]) if case["page"] else st["k"][at:at + n]
        v = _rows(st["v"], st["table"], b, m, case["page"]) if case["page"] else st["v"][at:at + n]
        step = max(1, min(n, (1 << 28) // (case["hq"] * m)))
        for i in range(0, n, step):
            e = min(n, i + step)
            seen = c + e if case["causal"] else m  # keys after the part's last query are not looked at
            limit = torch.arange(c + i + 1, c + e + 1, device=DEV) if case["causal"] else torch.full((e - i,), m, device=DEV)
            out[at + i:at + e] = _attend(q[at + i:at + e], k[:seen], v[:seen], scale, limit, wide).to(out.dtype)
        at += n
    return out


def _decode(st, wide):
    case, q = st["case"], st["q"]
    out = torch.empty(q.shape, dtype=q.dtype if wide is torch.float32 else wide, device=q.device)
    for b, m in enumerate(_lens(case, "kv")):
        k, v = _rows(st["k"], st["table"], b, m, case["page"]), _rows(st["v"], st["table"], b, m, case["page"])
        out[b:b + 1] = _attend(q[b:b + 1], k, v, 1.0 / math.sqrt(case["d"]), torch.full((1,), m, device=DEV), wide).to(out.dtype)
    return out


def _positions(case):
    seq = np.repeat(np.arange(len(_lens(case, "new"))), _lens(case, "new"))
    at = np.concatenate([[0], np.cumsum(_lens(case, "new"))])[:-1]
    pos = np.arange(len(seq)) - at[seq] + np.asarray(_lens(case, "ctx"), dtype=np.int64)[seq]
    return torch.from_numpy(seq).to(DEV), torch.from_numpy(pos).to(DEV)


def _append(st):
    case = st["case"]
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["page"]
    qkv = st["qkv"]
    seq = torch.repeat_interleave(torch.arange(len(_lens(case, "new")), device=DEV), st["cu"].diff().long(), output_size=qkv.shape[0])
    pos = torch.arange(qkv.shape[0], device=DEV) - st["cu"].long()[seq] + st["ctx"].long()[seq]
    freq = torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device=DEV),
                     torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / -d)
    angle = pos.double()[:, None, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    x = qkv[:, :hq + hkv].float()
    lo, hi = x[..., :d // 2], x[..., d // 2:]
    turned = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1).to(qkv.dtype)
    page, row = st["table"][seq, pos // ps].long(), pos % ps
    st["k"][page, :, row] = turned[:, hq:]
    st["v"][page, :, row] = qkv[:, hq + hkv:]
    return turned[:, :hq].contiguous(), st["k"], st["v"]


def _counts(ids, lens, first, V):
    """How often each id stands at the positions first <= i < lens of each row's history."""
    at = torch.arange(ids.shape[1], device=ids.device)[None, :]
    live = ((at >= first[:, None]) & (at < lens[:, None])).to(torch.int32)
    n = torch.zeros((ids.shape[0], V), dtype=torch.int32, device=ids.device)
    return n.scatter_add_(1, ids.long(), live)


def _logits(st, wide):
    case = st["case"]
    R, V = case["rows"], case["vocab"]
    x = st["logits"].to(wide)
    every = _counts(st["history"], st["history_lens"], torch.zeros_like(st["prompt_lens"]), V)
    said = _counts(st["history"], st["history_lens"], st["prompt_lens"], V)
    rep, freq, pres = (st[n].to(wide)[:, None] for n in ("repetition", "frequency", "presence"))
    x = torch.where(every > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * said.to(wide) - pres * (said > 0).to(wide)
    if st["bias"] is not None:
        indptr, ids, vals = st["bias"]
        row = torch.repeat_interleave(torch.arange(R, device=DEV), indptr.diff().long(), output_size=ids.shape[0])
        x = x + torch.zeros_like(x).index_put_((row, ids.long()), vals.to(wide), accumulate=True)
    if st["mask"] is not None:
        at = torch.arange(V, device=DEV)
        x = x.masked_fill((st["mask"][:, at // 32] >> (at % 32)) & 1 == 0, -math.inf)
    best = torch.where(torch.isinf(x.amax(-1)), torch.full((R,), -1, device=DEV), x.argmax(-1)).to(torch.int32)
    return x, best


# ------------------------------------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        if op == "prompt":
            return _prompt(st, torch.float32)
        if op == "decode":
            return _decode(st, torch.float32)
        return _append(st) if op == "append" else _logits(st, torch.float32)
    import event_tensor_task_b200 as mk
    if op == "prompt":
        if case["page"]:
            return mk.prompt_attention(st["q"], st["k"], st["v"], st["cu"], page_table=st["table"],
                                       kv_lens=st["kv_lens"], causal=case["causal"])
        return mk.prompt_attention(st["q"], st["k"], st["v"], st["cu"], causal=case["causal"])
    if op == "decode":
        return mk.paged_attention(st["q"], st["k"], st["v"], st["table"], st["kv_lens"], workspace=st["workspace"])
    if op == "append":
        hq, hkv = case["hq"], case["hkv"]
        q, k, v = st["qkv"][:, :hq], st["qkv"][:, hq:hq + hkv], st["qkv"][:, hq + hkv:]
        return mk.append_kv(q, k, v, st["k"], st["v"], st["table"], st["ctx"], st["cu"],
                            rope_theta=case["theta"]), st["k"], st["v"]
    return mk.process_logits(st["logits"], history=st["history"], history_lens=st["history_lens"],
                             prompt_lens=st["prompt_lens"], repetition=st["repetition"], frequency=st["frequency"],
                             presence=st["presence"], bias=st["bias"], mask=st["mask"], out=st["out"])


def work(case):
    op = case["op"]
    if op == "logits":
        R, V, s = case["rows"], case["vocab"], 4 if case["dtype"] == "fp32" else 2
        cells = R * V
        return {"bytes": cells * (s + 4) + 4 * R * (3 * case["hist"] // 4) + 8 * R * case["bias"] +
                (cells // 8 if case["mask"] else 0), "flops": 4 * cells}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "decode":
        n = sum(_lens(case, "kv"))
        return {"bytes": 2 * d * (2 * hkv * n + 2 * hq * len(_lens(case, "kv"))), "flops": 4 * d * hq * n}
    T = sum(_lens(case, "new"))
    if op == "append":
        return {"bytes": 2 * 2 * T * (hq + 2 * hkv) * d, "flops": 3 * T * (hq + hkv) * d}
    pairs = sum(n * c + (n * (n + 1) // 2 if case["causal"] else n * n) for n, c in zip(_lens(case, "new"), _lens(case, "ctx")))
    return {"bytes": 2 * d * (2 * T * hq + 2 * hkv * sum(n + c for n, c in zip(_lens(case, "new"), _lens(case, "ctx")))),
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_rows(pool, table, n, ps):
    j = torch.arange(n, device=DEV)
    return pool[table[j // ps].long(), :, j % ps].double()  # [n][Hkv][D]


def _exact_attention(q, k, v, first_limit, causal):
    """Head by head: softmax(q k^T / sqrt(D)) v with query i seeing first_limit + i keys (all, when not causal)."""
    n, hq, d = q.shape
    m, hkv = k.shape[:2]
    out = torch.empty((n, hq, d), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 27) // m)
    for h in range(hq):
        kh, vh = k[:, h * hkv // hq], v[:, h * hkv // hq]
        for i in range(0, n, step):
            e = min(n, i + step)
            seen = min(m, first_limit + e - 1) if causal else m
            s = q[i:e, h].double() @ kh[:seen].T / d ** 0.5
            if causal:
                j = torch.arange(seen, device=DEV)
                s[j[None, :] - torch.arange(i, e, device=DEV)[:, None] >= first_limit] = -math.inf
            out[i:e, h] = torch.softmax(s, -1) @ vh[:seen]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "decode":
        return torch.cat([_exact_attention(st["q"][b:b + 1], _exact_rows(st["k"], st["table"][b], m, case["page"]),
                                           _exact_rows(st["v"], st["table"][b], m, case["page"]), m, False)
                          for b, m in enumerate(_lens(case, "kv"))])
    if op == "prompt":
        parts, at = [], 0
        for b, (n, c) in enumerate(zip(_lens(case, "new"), _lens(case, "ctx"))):
            if case["page"]:
                k, v = (_exact_rows(st[x], st["table"][b], n + c, case["page"]) for x in ("k", "v"))
            else:
                k, v = st["k"][at:at + n].double(), st["v"][at:at + n].double()
            parts.append(_exact_attention(st["q"][at:at + n], k, v, c + 1, case["causal"]))
            at += n
        return torch.cat(parts)
    if op == "append":
        hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["page"]
        seq, pos = _positions(case)
        x = torch.view_as_complex(st["qkv"][:, :hq + hkv].double().reshape(-1, hq + hkv, 2, d // 2).transpose(2, 3).contiguous())
        p = torch.arange(d // 2, dtype=torch.float64, device=DEV)
        angle = pos.double()[:, None] * torch.exp(-2.0 * p / d * math.log(case["theta"]))
        y = torch.view_as_real(x * torch.polar(torch.ones_like(angle), angle)[:, None]).transpose(2, 3).reshape(-1, hq + hkv, d)
        k, v = st["k"].double(), st["v"].double()
        page, row = st["table"][seq, pos // ps].long(), pos % ps
        k[page, :, row] = y[:, hq:]
        v[page, :, row] = st["qkv"][:, hq + hkv:].double()
        return y[:, :hq], k, v
    # logits: row by row on the host, from the definition; the chosen id is a whole number that a value next to
    # another's decides, so it is given only where the two best are further apart than 32 bits resolve
    R, V = case["rows"], case["vocab"]
    x = st["logits"].double().cpu().numpy()
    hist, lens, first = (st[n].cpu().numpy() for n in ("history", "history_lens", "prompt_lens"))
    rep, freq, pres = (st[n].double().cpu().numpy() for n in ("repetition", "frequency", "presence"))
    clear = True
    best = np.empty(R, dtype=np.int32)
    for r in range(R):
        every = np.bincount(hist[r, :lens[r]], minlength=V)
        said = np.bincount(hist[r, first[r]:lens[r]], minlength=V)
        x[r] = np.where(every > 0, np.where(x[r] > 0, x[r] / rep[r], x[r] * rep[r]), x[r])
        x[r] -= freq[r] * said + pres[r] * (said > 0)
        if st["bias"] is not None:
            lo, hi = (int(i) for i in st["bias"][0][r:r + 2])
            np.add.at(x[r], st["bias"][1][lo:hi].cpu().numpy(), st["bias"][2][lo:hi].double().cpu().numpy())
        if st["mask"] is not None:
            bits = np.unpackbits(st["mask"][r].cpu().numpy().view(np.uint8), bitorder="little")[:V]
            x[r][bits == 0] = -np.inf
        best[r] = int(np.argmax(x[r])) if np.isfinite(x[r].max()) else -1
        two = np.partition(x[r], -2)[-2:]
        clear = clear and not (0 < two[1] - two[0] < 1e-5 * abs(two[1]))
    return torch.from_numpy(x), torch.from_numpy(best) if clear else None
