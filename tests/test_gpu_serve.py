"""The serving operators on the GPU against their definition in 64 bits.

Tolerances, elementwise, with u = half a step of the 16-bit type:
 - a stored value is rounded once: u |x|;
 - attention: a score is a D-term fp32 sum, off by at most D 2^-24 times the sum of |q_i k_i|, which makes each
   probability off by that fraction (twice: numerator and sum); the exponential adds 2^-21, twice as well; an
   n-key sum n 2^-24; a probability rounded to the type for its product is off by u (prompt attention), as value and
   remainder by u^2 (single tokens).  Each is a fraction of the mean of |v| under the probabilities.  In fp16
   a probability below 2^-14 of the running maximum has a step of 2^-24: n 2^-25 max |v| more;
 - rotation: the reduced angle in [-pi, pi] is rounded to fp32 (2^-22.3) and sine and cosine are within two of
   their last places (2^-22): 2^-21 (|x| + |y|) for a pair (x, y);
 - logits: five fp32 steps and the bias sum, 2^-22 of the magnitudes that meet.
"""
import math

import pytest
import torch

import event_tensor_task_b200 as mk
from oracle import serve as oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def cu(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)


def i32(vals):
    return torch.tensor(vals, dtype=torch.int32)


def pool(g, lens, page, hkv, d, dtype, order="hnd", spare=2, poison=float("nan")):
    """CPU pool [n_pages][Hkv][page][D] (a view in `order`), every row that no sequence owns holding `poison`, and
    the page table (-1 where there is no page)."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    shape = (total, hkv, page, d) if order == "hnd" else (total, page, hkv, d)
    k, v = torch.full(shape, poison).to(dtype), torch.full(shape, poison).to(dtype)
    if order == "nhd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    at = 0
    for b, n in enumerate(lens):
        for i in range(need[b]):
            p = int(perm[at])
            at += 1
            table[b, i] = p
            live = min(page, n - i * page)
            k[p, :, :live] = torch.randn((hkv, live, d), generator=g).to(dtype)
            v[p, :, :live] = torch.randn((hkv, live, d), generator=g).to(dtype)
    return k, v, table


def dev(t):
    """On the device with the same strides."""
    out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=DEV)
    return out.copy_(t)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def check_attention(got, ref, dtype, n_keys, vmax, single):
    out, mag, big = ref
    d = out.shape[-1]
    u = half_step(dtype)
    frac = 2 * (d * 2.0**-24 * big + 2.0**-21) + n_keys * 2.0**-24 + (u * u if single else u)
    tol = u * out.abs() + frac * mag * (1 + u)
    if dtype == HF:
        tol = tol + n_keys * 2.0**-25 * vmax * (0.002 if single else 1.0)
    err = (got.double().cpu() - out).abs()
    assert torch.isfinite(got).all()
    worst = float((err - tol).max())
    assert worst <= 0, f"off by {float(err.max()):.3e} where {float(tol.flatten()[err.argmax()]):.3e} is allowed"


# ------------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("hq,hkv,d,dtype,order,page,theta,new,ctx", [
    (4, 2, 64, BF, "hnd", 16, 10000.0, [1], [0]),
    (4, 2, 64, BF, "hnd", 16, 10000.0, [3, 0, 17, 1], [15, 4, 0, 33]),
    (8, 8, 128, HF, "nhd", 32, 500000.0, [5, 40], [100000, 31]),
    (7, 1, 128, BF, "nhd", 200, 10000.0, [1] * 9, [0, 1, 199, 200, 201, 399, 400, 7, 8]),
    (32, 8, 64, HF, "hnd", 1024, 0.0, [33], [1000]),
    (0, 2, 64, BF, "hnd", 16, 10000.0, [20], [5]),
    (3, 3, 64, BF, "hnd", 1, 10000.0, [6], [2]),
])
def test_append(hq, hkv, d, dtype, order, page, theta, new, ctx):
    g = gen(hq * 1000 + page)
    T, tail = sum(new), 3
    # far positions need no rows below them: only the last pages exist
    lens = [a + c for a, c in zip(new, ctx)]
    k, v, table = pool(g, [min(n, 4000) for n in lens], page, hkv, d, dtype, order, poison=7.0)
    width = max(-(-n // page) for n in lens)
    full = torch.full((len(new), width), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        have = table[b][table[b] >= 0]
        last = -(-n // page)
        first = max(0, last - len(have))
        full[b, first:last] = have[:last - first]
    qkv = torch.randn((T + tail, hq + 2 * hkv, d), generator=g).to(dtype)
    kd, vd, x = dev(k), dev(v), dev(qkv)
    q = x[:, :hq] if hq else None
    q_out = torch.full((T + tail, max(hq, 1), d), 5.0, dtype=dtype, device=DEV)[:, :hq] if hq else None
    st = status_word()
    got = mk.append_kv(q, x[:, hq:hq + hkv], x[:, hq + hkv:], kd, vd, full.to(DEV), i32(ctx).to(DEV), cu(new).to(DEV),
                       rope_theta=theta, q_out=q_out, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and got is q_out
    want_k, want_v = k.double(), v.double()
    tol_k = torch.zeros_like(want_k)
    u, at = half_step(dtype), 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        for i in range(n):
            row, pos = qkv[at:at + 1], c + i
            p, r = int(full[b, pos // page]), pos % page
            turned = oracle.rotate(row[:, :hq + hkv], [pos], theta)
            mixed = row[:, :hq + hkv].double().abs()
            mixed = mixed + mixed.roll(d // 2, -1)
            tol = u * turned.abs() + 2.0**-21 * mixed
            if hq:
                assert ((q_out[at].double().cpu() - turned[0, :hq]).abs() <= tol[0, :hq]).all()
            want_k[p, :, r], tol_k[p, :, r] = turned[0, hq:], tol[0, hq:]
            want_v[p, :, r] = row[0, hq + hkv:].double()
            at += 1
    assert ((kd.double().cpu() - want_k).abs() <= tol_k).all()  # (untouched rows: equal)
    assert torch.equal(vd.double().cpu(), want_v)
    if hq:
        assert (q_out[T:] == 5.0).all()


def test_append_in_place_and_unturned_copy():
    g = gen(1)
    k, v, table = pool(g, [40], 16, 2, 64, BF)
    q = torch.randn((10, 4, 64), generator=g).to(BF)
    kv = torch.randn((2, 10, 2, 64), generator=g).to(BF)
    args = (dev(kv[0]), dev(kv[1]))
    tail = (table.to(DEV), i32([30]).to(DEV), cu([10]).to(DEV))
    a, kd, vd = dev(q), dev(k), dev(v)
    out = mk.append_kv(a, *args, kd, vd, *tail)
    same = dev(q)
    got = mk.append_kv(same, *args, kd, vd, *tail, q_out=same)
    assert got is same and torch.equal(out, same)
    plain = mk.append_kv(a, *args, kd, vd, *tail, rope_theta=0)
    assert torch.equal(plain.cpu(), q)
    assert torch.equal(kd[table[0, 2].item(), :, :8].cpu(), kv[0][2:].transpose(0, 1))


@pytest.mark.parametrize("what", ["page", "high_page", "width", "ctx", "cu"])
def test_append_refuses_on_the_device(what):
    """Bad ids and lengths: nothing is stored for the row concerned, the rest is, the status word tells."""
    g = gen(3)
    k, v, table = pool(g, [20, 20], 16, 2, 64, BF, poison=7.0)
    k.fill_(7.0), v.fill_(7.0)
    ctx, bounds = [17, 18], [0, 2, 4]
    x = torch.randn((4, 2, 64), generator=g).to(BF)
    if what == "page":
        table[0, 1] = -1
    elif what == "high_page":
        table[0, 1] = k.shape[0]
    elif what == "width":
        ctx[0] = 31  # its second token falls behind the table
    elif what == "ctx":
        ctx[0] = -1
    else:
        bounds = [-3, 2, 4]
    kd, vd, st = dev(k), dev(v), status_word()
    q = torch.full((4, 2, 64), 3.0, dtype=BF, device=DEV)
    q_out = torch.full((4, 2, 64), 9.0, dtype=BF, device=DEV)
    mk.append_kv(q, dev(x), dev(x), kd, vd, table.to(DEV), i32(ctx).to(DEV), i32(bounds).to(DEV), rope_theta=0,
                 q_out=q_out, status=st)
    assert int(st) == mk.MK_ERR_DEVICE_BOUNDS
    stored = 3 if what == "width" else 2
    assert int((vd.cpu() != 7.0).any(-1).sum()) == stored * 2
    assert int((q_out == 3.0).all(-1).sum()) == stored * 2 and int((q_out == 9.0).all(-1).sum()) == (4 - stored) * 2
    p = int(table[1, 1])
    assert torch.equal(vd[p, :, 2:4].cpu(), x[2:].transpose(0, 1))


# ------------------------------------------------------------------------------------------------ prompts
def prompt_reference(q, ks, vs, new, causal, scale):
    parts, at = [], 0
    for n, k, v in zip(new, ks, vs):
        m = k.shape[0]
        limit = [i + 1 + m - n if causal else m for i in range(n)]
        parts.append(oracle.attend(q[at:at + n], k, v, limit, scale))
        at += n
    return tuple(torch.cat([p[i] for p in parts]) for i in range(3))


@pytest.mark.parametrize("hq,hkv,d,dtype,causal,new,keys", [
    (1, 1, 64, BF, True, [1], None),
    (4, 2, 64, BF, True, [17], None),
    (4, 2, 64, BF, True, [128, 1, 0, 129, 127], None),
    (2, 2, 128, HF, True, [300, 5], None),
    (8, 1, 128, BF, True, [33, 200], None),
    (6, 2, 64, HF, False, [70, 130], None),
    (7, 1, 128, BF, False, [19], [257]),
    (5, 1, 64, BF, True, [10, 3], [140, 3]),          # a chunk after earlier keys
    (4, 4, 64, BF, True, [9, 6], [4, 0]),             # more queries than keys: the first rows see none
    (2, 1, 128, HF, False, [3, 2], [0, 400]),
    (128, 1, 64, BF, True, [3], [60]),
    (48, 1, 128, BF, True, [21], None),
    (2, 1, 64, BF, True, [1], [900]),
])
def test_prompt_packed(hq, hkv, d, dtype, causal, new, keys):
    g = gen(hq * 100 + d + sum(new))
    m = keys if keys is not None else new
    T, tail = sum(new), 2
    q = torch.randn((T + tail, hq, d), generator=g).to(dtype)
    kv = torch.randn((sum(m) + tail, 2 * hkv, d), generator=g).to(dtype)
    kv[sum(m):] = float("nan")  # rows behind the last sequence may hold anything
    st = status_word()
    out = torch.full((T + tail, hq, d), 5.0, dtype=dtype, device=DEV)
    x = dev(kv)
    mk.prompt_attention(dev(q), x[:, :hkv], x[:, hkv:], cu(new).to(DEV), cu_k=None if keys is None else cu(keys).to(DEV),
                        causal=causal, out=out, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and (out[T:] == 5.0).all()
    ks, vs, at = [], [], 0
    for n in m:
        ks.append(kv[at:at + n, :hkv])
        vs.append(kv[at:at + n, hkv:])
        at += n
    ref = prompt_reference(q[:T], ks, vs, new, causal, d ** -0.5)
    check_attention(out[:T], ref, dtype, max(m + [1]), 6.0, False)


@pytest.mark.parametrize("hq,hkv,d,dtype,order,page,new,ctx,scale", [
    (4, 2, 64, BF, "hnd", 16, [1, 30, 0], [0, 50, 9], None),
    (4, 1, 128, BF, "nhd", 64, [100, 7], [29, 500], None),
    (3, 3, 64, HF, "hnd", 32, [129], [0], 0.3),
    (2, 2, 128, HF, "nhd", 200, [60, 150], [170, 333], None),
    (4, 2, 64, BF, "hnd", 1024, [257, 3], [0, 700], None),   # the decoder's slot cache
    (2, 1, 64, BF, "hnd", 128, [130], [130], 0.02),
])
def test_prompt_paged(hq, hkv, d, dtype, order, page, new, ctx, scale):
    g = gen(hq * 100 + page)
    lens = [a + c for a, c in zip(new, ctx)]
    k, v, table = pool(g, lens, page, hkv, d, dtype, order)
    q = torch.randn((sum(new), hq, d), generator=g).to(dtype)
    st = status_word()
    out = mk.prompt_attention(dev(q), dev(k), dev(v), cu(new).to(DEV), page_table=table.to(DEV),
                              kv_lens=i32(lens).to(DEV), scale=scale, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    ks = [oracle.rows(k, table[b], n, page) for b, n in enumerate(lens)]
    vs = [oracle.rows(v, table[b], n, page) for b, n in enumerate(lens)]
    ref = prompt_reference(q, ks, vs, new, True, scale or d ** -0.5)
    check_attention(out, ref, dtype, max(lens), 6.0, False)


@pytest.mark.parametrize("hq,hkv,d,dtype,causal,new,keys", [
    (8, 2, 64, BF, True, [40, 3], [3000, 2900]),
    (4, 4, 128, HF, True, [150], [4100]),
    (3, 1, 128, BF, False, [70, 1, 130], [2500, 0, 1700]),
    (2, 1, 64, HF, True, [300], [1600]),              # causal edge inside the last pieces
    (2, 1, 64, BF, True, [1700], [1600]),             # rows without keys in a sequence that is cut
])
def test_prompt_cut_along_the_keys(hq, hkv, d, dtype, causal, new, keys):
    """Few rows and many keys: pieces of the keys on many SMs, joined.  The workspace's contents do not matter, and
    without one the same comes out within the tolerance."""
    g = gen(hq * 100 + d)
    n = mk.mk_prompt_attention_workspace_bytes(len(new), sum(new), hq, hkv, d, sum(keys))
    assert n > 0
    q = torch.randn((sum(new), hq, d), generator=g).to(dtype)
    kv = torch.randn((sum(keys) + 1, 2 * hkv, d), generator=g).to(dtype)
    kv[sum(keys):] = float("nan")
    x, args = dev(kv), (cu(new).to(DEV), cu(keys).to(DEV))
    ks = [kv[a:b, :hkv] for a, b in zip(cu(keys)[:-1], cu(keys)[1:])]
    vs = [kv[a:b, hkv:] for a, b in zip(cu(keys)[:-1], cu(keys)[1:])]
    ref = prompt_reference(q, ks, vs, new, causal, d ** -0.5)
    outs = []
    for ws in (None, torch.full((n,), 255, dtype=torch.uint8, device=DEV), torch.empty(256, dtype=torch.uint8, device=DEV)):
        st = status_word()
        out = mk.prompt_attention(dev(q), x[:, :hkv], x[:, hkv:], args[0], cu_k=args[1], causal=causal, workspace=ws,
                                  status=st)
        assert int(st) == 0
        check_attention(out, ref, dtype, max(keys), 6.0, False)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])


def test_prompt_cut_along_paged_keys():
    g = gen(31)
    new, ctx = [30, 5, 1], [2500, 40, 1999]
    lens = [a + c for a, c in zip(new, ctx)]
    for page, order in ((16, "hnd"), (200, "nhd")):
        k, v, table = pool(g, lens, page, 2, 64, BF, order)
        q = torch.randn((sum(new), 4, 64), generator=g).to(BF)
        out = mk.prompt_attention(dev(q), dev(k), dev(v), cu(new).to(DEV), page_table=table.to(DEV), kv_lens=i32(lens).to(DEV))
        ks = [oracle.rows(k, table[b], n, page) for b, n in enumerate(lens)]
        vs = [oracle.rows(v, table[b], n, page) for b, n in enumerate(lens)]
        check_attention(out, prompt_reference(q, ks, vs, new, True, 0.125), BF, max(lens), 6.0, False)


@pytest.mark.parametrize("hkv,d,dtype", [(8, 64, BF), (4, 128, HF)])
def test_prompt_more_work_than_blocks(hkv, d, dtype):
    """Many sequences (more than a warp counts at a time) and more row blocks than the device holds: every block runs
    several of them, with and without keys."""
    g = gen(hkv)
    new = [int(n) for n in torch.randint(0, 60, (90,), generator=g)]
    keys = [n + int(e) if n % 7 else 0 for n, e in zip(new, torch.randint(0, 50, (90,), generator=g))]
    q = torch.randn((sum(new), hkv, d), generator=g).to(dtype)
    kv = torch.randn((sum(keys), 2 * hkv, d), generator=g).to(dtype)
    x = dev(kv)
    out = mk.prompt_attention(dev(q), x[:, :hkv], x[:, hkv:], cu(new).to(DEV), cu_k=cu(keys).to(DEV))
    ks = [kv[a:b, :hkv] for a, b in zip(cu(keys)[:-1], cu(keys)[1:])]
    vs = [kv[a:b, hkv:] for a, b in zip(cu(keys)[:-1], cu(keys)[1:])]
    check_attention(out, prompt_reference(q, ks, vs, new, True, d ** -0.5), dtype, max(keys), 6.0, False)


def test_prompt_strided_rows():
    """Queries as every second head of a wider tensor, outputs into a wider one."""
    g = gen(5)
    qw = torch.randn((50, 8, 2, 64), generator=g).to(BF)
    k, v = torch.randn((2, 50, 2, 64), generator=g).to(BF)
    wide = torch.full((50, 4, 3, 64), 5.0, dtype=BF, device=DEV)
    out = wide[:, :, 1]
    mk.prompt_attention(dev(qw)[:, ::2, 1], dev(k), dev(v), cu([20, 30]).to(DEV), out=out)
    ref = prompt_reference(qw[:, ::2, 1], [k[:20], k[20:]], [v[:20], v[20:]], [20, 30], True, 0.125)
    check_attention(out, ref, BF, 30, 6.0, False)
    assert (wide[:, :, 0] == 5.0).all() and (wide[:, :, 2] == 5.0).all()
    wide = torch.full((50, 4, 72), 5.0, dtype=BF, device=DEV)  # rows on 16 bytes, not on 32
    again = mk.prompt_attention(dev(qw)[:, ::2, 1], dev(k), dev(v), cu([20, 30]).to(DEV), out=wide[:, :, :64])
    assert torch.equal(again, out) and (wide[:, :, 64:] == 5.0).all()


def test_prompt_large_scores():
    """Scores far apart and far from zero: the running maximum carries them."""
    g = gen(6)
    q = (30 * torch.randn((200, 2, 64), generator=g)).to(BF)
    k = (30 * torch.randn((200, 1, 64), generator=g)).to(BF)
    v = torch.randn((200, 1, 64), generator=g).to(BF)
    k[150] = 100.0
    out = mk.prompt_attention(dev(q), dev(k), dev(v), cu([200]).to(DEV))
    ref = prompt_reference(q, [k], [v], [200], True, 0.125)
    check_attention(out, ref, BF, 200, 6.0, False)


@pytest.mark.parametrize("what", ["page", "high_page", "kv_len", "negative", "cu_q", "cu_k"])
def test_prompt_refuses_on_the_device(what):
    g = gen(7)
    k, v, table = pool(g, [40, 40], 16, 1, 64, BF, poison=0.0)
    q = torch.randn((8, 2, 64), generator=g).to(BF)
    lens, cq, ck, packed = [40, 40], [0, 4, 8], [0, 20, 40], what.startswith("cu_k")
    if what == "page":
        table[0, 0] = -5
    elif what == "high_page":
        table[0, 1] = k.shape[0]
    elif what == "kv_len":
        lens[0] = 49
    elif what == "negative":
        lens[0] = -1
    elif what == "cu_q":
        cq = [0, 4, 9]
    else:
        ck = [0, 20, 41]
    st = status_word()
    if packed:
        x = torch.randn((40, 1, 64), generator=g).to(BF)
        out = mk.prompt_attention(dev(q), dev(x), dev(x), i32(cq).to(DEV), cu_k=i32(ck).to(DEV), status=st)
    else:
        out = mk.prompt_attention(dev(q), dev(k), dev(v), i32(cq).to(DEV), page_table=table.to(DEV),
                                  kv_lens=i32(lens).to(DEV), status=st)
    torch.cuda.synchronize()
    assert int(st) == mk.MK_ERR_DEVICE_BOUNDS
    assert torch.isfinite(out).all()
    if what not in ("cu_q", "cu_k"):  # the other sequence has its values
        ref = prompt_reference(q[4:], [oracle.rows(k, table[1], 40, 16)], [oracle.rows(v, table[1], 40, 16)], [4], True, 0.125)
        check_attention(out[4:], ref, BF, 40, 6.0, False)
    if what == "negative":
        assert (out[:4] == 0).all()


# ------------------------------------------------------------------------------------------------ single tokens
@pytest.mark.parametrize("hq,hkv,d,dtype,order,page,lens", [
    (1, 1, 64, BF, "hnd", 16, [1]),
    (4, 2, 64, BF, "hnd", 1088, [1025]),
    (4, 2, 64, BF, "nhd", 16, [0, 1, 15, 16, 17, 63, 64, 65, 300]),
    (16, 2, 128, BF, "hnd", 64, [500, 3, 129]),
    (16, 1, 128, HF, "nhd", 32, [257]),
    (7, 1, 64, HF, "hnd", 200, [199, 200, 201, 401]),
    (40, 2, 64, BF, "hnd", 16, [77, 150]),                # 20 heads a kv head: two tiles
    (9, 1, 128, BF, "hnd", 128, [128, 640]),
    (5, 5, 128, HF, "nhd", 1, [40, 2]),
    (2, 1, 64, BF, "hnd", 64, [6000, 10]),
])
def test_paged(hq, hkv, d, dtype, order, page, lens):
    g = gen(hq * 100 + page + d)
    k, v, table = pool(g, lens, page, hkv, d, dtype, order)
    q = torch.randn((len(lens), hq, d), generator=g).to(dtype)
    st = status_word()
    args = (dev(q), dev(k), dev(v), table.to(DEV), i32(lens).to(DEV))
    out = mk.paged_attention(*args, status=st)
    again = mk.paged_attention(*args, workspace=torch.full(
        (mk.mk_paged_attention_workspace_bytes(len(lens), hq, hkv, d),), 255, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(out, again)
    parts = [oracle.attend(q[b:b + 1], oracle.rows(k, table[b], n, page), oracle.rows(v, table[b], n, page), [n],
                           d ** -0.5) for b, n in enumerate(lens)]
    check_attention(out, tuple(torch.cat([p[i] for p in parts]) for i in range(3)), dtype, max(lens), 6.0, True)


@pytest.mark.parametrize("n,hq,hkv,d,dtype", [
    (300, 4, 2, 64, BF),
    (300, 16, 2, 64, BF),     # more rows than the join takes one by one: it goes by the cuts
    (60, 48, 2, 128, HF),     # and two tiles of heads a kv head
])
def test_paged_many_short_sequences(n, hq, hkv, d, dtype):
    """More pairs than blocks: a block's share holds many of them, whole and cut, and some sequences have no keys."""
    g = gen(11)
    lens = [int(m) for m in torch.randint(0, 200, (n,), generator=g)]
    lens[3] = lens[n - 1] = 0
    k, v, table = pool(g, lens, 16, hkv, d, dtype)
    q = torch.randn((n, hq, d), generator=g).to(dtype)
    out = mk.paged_attention(dev(q), dev(k), dev(v), table.to(DEV), i32(lens).to(DEV), scale=0.1,
                             out=torch.full((n, hq, d), float("nan"), dtype=dtype, device=DEV))
    parts = [oracle.attend(q[b:b + 1], oracle.rows(k, table[b], m, 16), oracle.rows(v, table[b], m, 16), [m], 0.1)
             for b, m in enumerate(lens)]
    check_attention(out, tuple(torch.cat([p[i] for p in parts]) for i in range(3)), dtype, 200, 6.0, True)


def test_paged_long_cache_offsets_past_32_bits():
    """Rows whose element offset does not fit 32 bits: pages far apart in one large pool."""
    n_pages, page, d = 40000, 1024, 64
    k = torch.empty((n_pages, 1, page, d), dtype=BF, device=DEV)  # 5.2 GB each
    v = torch.empty_like(k)
    ids = [39999, 3, 33000, 20000]
    table = i32([ids]).to(DEV)
    g = gen(12)
    x = torch.randn((2, 4, 1, page, d), generator=g).to(BF)
    for i, p in enumerate(ids):
        k[p].copy_(x[0, i])
        v[p].copy_(x[1, i])
    n = 3 * page + 77
    q = torch.randn((1, 2, d), generator=g).to(BF)
    lens = i32([n]).to(DEV)
    out = mk.paged_attention(dev(q), k, v, table, lens)
    rows = [t.transpose(1, 2).reshape(-1, 1, d)[:n] for t in x]
    check_attention(out, oracle.attend(q, rows[0], rows[1], [n], 0.125), BF, n, 6.0, True)
    got = mk.prompt_attention(dev(q), k, v, cu([1]).to(DEV), page_table=table, kv_lens=lens)
    check_attention(got, oracle.attend(q, rows[0], rows[1], [n], 0.125), BF, n, 6.0, False)
    new = torch.randn((1, 1, d), generator=g).to(BF)
    mk.append_kv(None, dev(new), dev(new), k, v, table, lens, cu([1]).to(DEV), rope_theta=0)
    assert torch.equal(k[ids[3], 0, 77].cpu(), new[0, 0])


@pytest.mark.parametrize("what", ["page", "high_page", "long", "negative"])
def test_paged_refuses_on_the_device(what):
    g = gen(13)
    k, v, table = pool(g, [100, 100], 16, 1, 64, BF, poison=0.0)
    q = torch.randn((2, 2, 64), generator=g).to(BF)
    lens = [100, 100]
    if what == "page":
        table[0, 3] = -1
    elif what == "high_page":
        table[0, 3] = k.shape[0]
    elif what == "long":
        lens[0] = 113
    else:
        lens[0] = -7
    st = status_word()
    out = mk.paged_attention(dev(q), dev(k), dev(v), table.to(DEV), i32(lens).to(DEV), status=st)
    assert int(st) == mk.MK_ERR_DEVICE_BOUNDS and torch.isfinite(out).all()
    ref = oracle.attend(q[1:], oracle.rows(k, table[1], 100, 16), oracle.rows(v, table[1], 100, 16), [100], 0.125)
    check_attention(out[1:], ref, BF, 100, 6.0, True)
    if what == "negative":
        assert (out[0] == 0).all()


# ------------------------------------------------------------------------------------------------ logits
def logits_case(R, V, dtype, H=0, bias=0, mask=False, seed=0):
    g = gen(seed + V)
    kw = {}
    if H:
        ids = (torch.rand((R, H), generator=g) ** 3 * V).to(torch.int32)
        ids[:, ::7] = torch.randint(-2, V + 2, (R, len(range(0, H, 7))), generator=g, dtype=torch.int32)
        lens = torch.randint(0, H + 1, (R,), generator=g, dtype=torch.int32)
        lens[0] = H
        kw.update(history=ids, history_lens=lens, prompt_lens=(lens // 3).to(torch.int32),
                  repetition=1 + torch.rand(R, generator=g), frequency=torch.rand(R, generator=g),
                  presence=torch.rand(R, generator=g) - 0.5)
    if bias:
        per = [bias if r % 3 else bias // 2 for r in range(R)]
        ids = torch.randint(-1, min(V, 4 * bias) + 1, (sum(per),), generator=g, dtype=torch.int32)
        kw["bias"] = (cu(per), ids, torch.randn(sum(per), generator=g))
    if mask:
        kw["mask"] = torch.randint(-2**31, 2**31, (R, (V + 31) // 32), generator=g, dtype=torch.int64).to(torch.int32)
    return (4 * torch.randn((R, V), generator=g)).to(dtype), kw


def to_dev(kw):
    return {n: tuple(x.to(DEV) for x in t) if isinstance(t, tuple) else t.to(DEV) for n, t in kw.items()}


def check_logits(got, best, logits, kw):
    x, want = oracle.process(logits, **kw)
    got = got.cpu().double()
    mags = logits.double().abs() * (2 if "repetition" in kw else 1) + 8.0
    if "frequency" in kw:
        mags = mags + kw["history"].shape[1]
    if "bias" in kw:
        mags = mags + 4.0 * kw["bias"][1].numel() ** 0.5
    assert torch.equal(torch.isinf(got), torch.isinf(x))
    live = torch.isfinite(x)
    assert ((got - x).abs()[live] <= 2.0**-22 * mags[live]).all()
    for r in range(x.shape[0]):  # the choice is the largest of the values that came out, ties to the lowest id
        row = got[r].clone()
        row[torch.isnan(row)] = -math.inf
        assert int(best[r]) == (int(row.argmax()) if float(row.max()) > -math.inf else -1)
        if want[r] >= 0 and int(best[r]) != int(want[r]):
            assert float(x[r, int(want[r])] - x[r, int(best[r])]) <= 2.0**-21 * float(mags[r].max())


@pytest.mark.parametrize("R,V,dtype,H,bias,mask", [
    (1, 1, torch.float32, 0, 0, False),
    (3, 33, torch.float32, 5, 3, True),
    (2, 1000, BF, 64, 40, True),
    (1, 8192, HF, 300, 0, False),
    (5, 8193, torch.float32, 0, 100, False),
    (2, 20011, torch.float32, 1000, 70, True),
    (1, 40000, BF, 33, 33, False),
    (70, 2051, HF, 17, 5, True),
    (2, 3000, torch.float32, 9000, 50, True),       # a history too long for the short marks
    (80, 70001, BF, 40, 40, True),                  # a row in one block, in two parts
    (80, 70004, torch.float32, 40, 40, False),
    (1, 90000, torch.float32, 12000, 3000, True),   # the long marks, in parts; a list with many ids twice
])
def test_logits(R, V, dtype, H, bias, mask):
    logits, kw = logits_case(R, V, dtype, H, bias, mask)
    out, best = mk.process_logits(dev(logits), **to_dev(kw))
    check_logits(out, best, logits, kw)


def test_logits_in_place_strided_and_aligned_alike():
    """Rows that start off a 16-byte boundary, a padded row stride, and the logits' own buffer as the output."""
    logits, kw = logits_case(3, 5000, torch.float32, 50, 20, True, seed=1)
    want, best = mk.process_logits(dev(logits), **to_dev(kw))
    wide = torch.full((3, 5007), 9.0, device=DEV)
    view = wide[:, 3:5003]
    view.copy_(logits)
    out, best2 = mk.process_logits(view, **to_dev(kw), out=view)
    assert out is view and torch.equal(out, want) and torch.equal(best, best2)
    assert (wide[:, :3] == 9.0).all() and (wide[:, 5003:] == 9.0).all()
    only = torch.empty(3, dtype=torch.int32, device=DEV)
    a = mk.mk_logits_args(rows=3, vocab=5000, dtype=mk.MK_DTYPE_FP32, logits=want.data_ptr(), logits_stride=5000,
                          next_tokens=only.data_ptr())
    mk.mk_process_logits(a, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(only, best)


def test_logits_ties_infinities_nan_and_empty_rows():
    inf, nan, low = math.inf, math.nan, torch.finfo(torch.float32).min
    x = torch.tensor([[1.0, 3.0, 3.0, 2.0],        # a tie: the lower id
                      [-0.0, 0.0, -1.0, -0.0],     # zeros tie whatever their sign
                      [nan, -5.0, nan, -inf],      # NaN is not chosen
                      [-inf, -inf, -inf, -inf],    # nothing is left
                      [1.0, inf, nan, inf],        # masked below: id 1
                      [low, low, low, low],
                      [5.0, 6.0, 7.0, nan]])       # masked below: all
    mask = torch.full((7, 1), -1, dtype=torch.int32)
    mask[4, 0], mask[6, 0] = ~0b0010, 0
    out, best = mk.process_logits(x.to(DEV), mask=mask.to(DEV))
    assert best.tolist() == [1, 0, 1, -1, 3, 0, -1]
    assert float(out[4, 1]) == -inf and (out[6] == -inf).all() and math.isnan(float(out[2, 0]))
    one = torch.tensor([[0b0101]], dtype=torch.int32, device=DEV)  # one mask for all rows
    out, best = mk.process_logits(x.to(DEV), mask=one)
    assert best.tolist() == [2, 0, -1, -1, 0, 0, 2]


def test_logits_repeats_of_one_id_in_list_order():
    """The same id a thousand times in the history, and biases whose sum depends on the order."""
    V = 300
    x = torch.zeros((2, V))
    x[0, 7], x[1, 7] = 2.0, -2.0
    hist = torch.full((2, 1000), 7, dtype=torch.int32)
    vals = torch.tensor([1e8, 1.0, -1e8, 1.0] * 12)
    ids = torch.tensor([9, 9, 9, 9] * 12, dtype=torch.int32)
    kw = dict(history=hist, prompt_lens=i32([0, 1000]), repetition=torch.full((2,), 1.25),
              frequency=torch.full((2,), 0.5), presence=torch.full((2,), 0.25), bias=(i32([0, 48, 48]), ids, vals))
    out, best = mk.process_logits(x.to(DEV), **to_dev(kw))
    want = torch.tensor(0.0)
    for v in vals:
        want = want + v  # fp32, in list order
    assert float(out[0, 9]) == float(want)
    # 2 / 1.25 is rounded to fp32 (2^-24 of it); the two differences lie in [256, 512), where half a step is 2^-16
    assert abs(float(out[0, 7]) - (2.0 / 1.25 - 500.0 - 0.25)) <= 2 * 2.0**-16 + 2.0**-23 and float(out[1, 7]) == -2.5


@pytest.mark.parametrize("what", ["history", "negative", "bias_end", "bias_order"])
def test_logits_refuses_on_the_device(what):
    x = torch.ones((1, 50))
    hist = torch.full((1, 8), 3, dtype=torch.int32)
    lens, indptr = [8], [0, 2]
    if what == "history":
        lens = [9]
    elif what == "negative":
        lens = [-1]
    elif what == "bias_end":
        indptr = [0, 3]
    else:
        indptr = [2, 0]
    st = status_word()
    out, best = mk.process_logits(x.to(DEV), history=hist.to(DEV), history_lens=i32(lens).to(DEV),
                                  repetition=torch.full((1,), 2.0, device=DEV),
                                  bias=(i32(indptr).to(DEV), i32([1, 2]).to(DEV), torch.ones(2, device=DEV)), status=st)
    assert int(st) == mk.MK_ERR_DEVICE_BOUNDS
    assert float(out[0, 3]) == (1.0 if what == "negative" else 0.5)
    assert float(out[0, 1]) == (1.0 if what.startswith("bias") else 2.0)


# ------------------------------------------------------------------------------------------------ calls as programs make them
def test_calls_with_nothing_to_do():
    k, v, table = pool(gen(20), [10], 16, 1, 64, BF)
    k, v, table = dev(k), dev(v), table.to(DEV)
    none = torch.empty((0, 2, 64), dtype=BF, device=DEV)
    assert mk.append_kv(none, none[:, :1], none[:, :1], k, v, table, i32([3]).to(DEV), i32([0, 0]).to(DEV)).shape == (0, 2, 64)
    assert mk.prompt_attention(none, k, v, i32([0, 0]).to(DEV), page_table=table, kv_lens=i32([3]).to(DEV)).shape == (0, 2, 64)
    assert mk.paged_attention(none, k, v, table[:0], i32([]).to(DEV)).shape == (0, 2, 64)
    out, best = mk.process_logits(torch.empty((0, 5), device=DEV))
    assert out.shape == (0, 5) and best.shape == (0,)
    # no keys at all: zero rows
    q = torch.ones((3, 2, 64), dtype=BF, device=DEV)
    got = mk.prompt_attention(q, none[:, :1], none[:, :1], i32([0, 3]).to(DEV), cu_k=i32([0, 0]).to(DEV))
    assert (got == 0).all()
    got = mk.paged_attention(q[:1], k, v, table[:, :0], i32([0]).to(DEV))
    assert (got == 0).all()


def test_captured_and_replayed_on_another_stream():
    """One graph of all four on new contents of the same buffers, next to the same calls on a second stream."""
    g = gen(21)
    k, v, table = pool(g, [90, 40], 16, 2, 64, BF, poison=0.0)
    table, ctx = table.to(DEV), i32([80, 37]).to(DEV)
    lens, bounds = i32([90, 40]).to(DEV), cu([10, 3]).to(DEV)
    qkv = [dev(torch.randn((13, 8, 64), generator=g).to(BF)) for _ in range(3)]
    logits = [dev(torch.randn((2, 3000), generator=g)) for _ in range(3)]
    hist = i32([[5, 6, 7], [8, 8, 8]]).to(DEV)
    pen = torch.full((2,), 1.5, device=DEV)

    def calls(x, lg, kc, vc):
        q = mk.append_kv(x[:, :4], x[:, 4:6], x[:, 6:], kc, vc, table, ctx, bounds)
        a = mk.prompt_attention(q, kc, vc, bounds, page_table=table, kv_lens=lens)
        b = mk.paged_attention(q[9:13:3], kc, vc, table, lens)
        return (q, a, b) + mk.process_logits(lg, history=hist, repetition=pen)

    want = []
    for x, lg in zip(qkv, logits):
        want.append([t.clone() for t in calls(x, lg, dev(k), dev(v))])
    x, lg, kc, vc = qkv[0].clone(), logits[0].clone(), dev(k), dev(v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls(x, lg, kc, vc)
    other = torch.cuda.Stream()
    for i in (1, 2, 0, 1):
        x.copy_(qkv[i])
        lg.copy_(logits[i])
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            side = calls(qkv[2], logits[2], dev(k), dev(v))
        torch.cuda.synchronize()
        for a, b in zip(outs, want[i]):
            assert torch.equal(a, b)
        for a, b in zip(side, want[2]):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mk.process_logits(logits[1], history=hist, repetition=pen, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[1][3])


def test_cut_prompts_captured_and_on_two_streams():
    """Calls that join pieces: captured, replayed on new contents, and two at a time on two streams."""
    g = gen(41)
    x = [dev(torch.randn((2600, 4, 64), generator=g).to(BF)) for _ in range(3)]
    q = [dev(torch.randn((30, 4, 64), generator=g).to(BF)) for _ in range(3)]
    bounds, keys = cu([30]).to(DEV), cu([2600]).to(DEV)

    def call(i, **kw):
        return mk.prompt_attention(q[i], x[i][:, :2], x[i][:, 2:], bounds, cu_k=keys, **kw)

    want = [call(i).clone() for i in range(3)]
    qs, xs = q[0].clone(), x[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mk.prompt_attention(qs, xs[:, :2], xs[:, 2:], bounds, cu_k=keys)
        out2 = mk.prompt_attention(qs, xs[:, :2], xs[:, 2:], bounds, cu_k=keys)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in (1, 2, 0):
        qs.copy_(q[i])
        xs.copy_(x[i])
        torch.cuda.synchronize()
        graph.replay()
        side = [call(j, stream=s) for j, s in ((1, streams[0]), (2, streams[1]), (0, streams[0]), (1, streams[1]))]
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(out2, want[i])
        for got, j in zip(side, (1, 2, 0, 1)):
            assert torch.equal(got, want[j])


@pytest.mark.parametrize("captured", [False, True])
def test_calls_that_feed_one_another_without_a_pause(captured):
    """Small calls begin while the one before them still runs: forty steps in which every call reads what the one
    before it wrote (rows, cache, lengths, tokens) come out as with a pause after each call."""
    g = gen(43)
    B, steps = 3, 40
    x0 = torch.randn((B, 8, 64), generator=g).to(BF)
    lens0 = i32([5, 200, 63])
    pool0 = [torch.randn((60, 2, 16, 64), generator=g).to(BF) for _ in range(2)]
    table = torch.randperm(60, generator=g)[:51].view(3, 17).to(torch.int32).to(DEV)
    W = dev((torch.randn((256, 512), generator=g) / 16).to(BF))
    bounds, pen = cu([1] * B).to(DEV), torch.full((B,), 1.3, device=DEV)

    def walk(x, lens, k, v, hist, pause):
        """The steps' results, from x on (x, lens, k, v, hist are written)."""
        toks = []
        for i in range(steps):
            q = mk.append_kv(x[:, :4], x[:, 4:6], x[:, 6:], k, v, table, lens, bounds)
            pause()
            lens += 1
            a = mk.prompt_attention(q, k, v, bounds, page_table=table, kv_lens=lens)
            pause()
            b = mk.paged_attention(a, k, v, table, lens)
            pause()
            out, best = mk.process_logits(b.reshape(B, 256), history=hist, repetition=pen)
            pause()
            hist[:, i] = best
            x.copy_((out.to(BF) @ W).view(B, 8, 64))
            toks.append(best)
        return torch.stack(toks)

    def fresh():
        return dev(x0), lens0.to(DEV), dev(pool0[0]), dev(pool0[1]), torch.full((B, steps), -1, dtype=torch.int32, device=DEV)

    slow = fresh()
    want = walk(*slow, torch.cuda.synchronize)
    fast = fresh()
    if captured:
        walk(*fresh(), lambda: None)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = walk(*fast, lambda: None)
        for t, u in zip(fast, fresh()):
            t.copy_(u)
        graph.replay()
    else:
        got = walk(*fast, lambda: None)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for t, u in zip(fast, slow):
        assert torch.equal(t, u)


def test_heads_that_share_their_rows():
    """Pools and rows with a head stride of zero (one head's rows shown as four)."""
    g = gen(42)
    k, v, table = pool(g, [70, 33], 16, 1, 64, BF)
    q = torch.randn((2, 8, 64), generator=g).to(BF)
    kd, vd = dev(k).expand(-1, 4, -1, -1), dev(v).expand(-1, 4, -1, -1)
    out = mk.paged_attention(dev(q), kd, vd, table.to(DEV), i32([70, 33]).to(DEV))
    parts = [oracle.attend(q[b:b + 1], oracle.rows(k, table[b], n, 16), oracle.rows(v, table[b], n, 16), [n], 0.125)
             for b, n in enumerate([70, 33])]
    check_attention(out, tuple(torch.cat([p[i] for p in parts]) for i in range(3)), BF, 70, 6.0, True)
    with pytest.raises(mk.MkError):  # nothing can be written there
        mk.append_kv(None, dev(q)[:, :4], dev(q)[:, :4], kd, vd, table.to(DEV), i32([0, 0]).to(DEV), cu([1, 1]).to(DEV))
    with pytest.raises(mk.MkError, match="overlap"):
        mk.paged_attention(dev(q), dev(k), dev(v), table.to(DEV), i32([70, 33]).to(DEV),
                           out=torch.empty((2, 1, 64), dtype=BF, device=DEV).expand(-1, 8, -1))


def test_prompt_then_decode_steps_then_choice():
    """The operators together with the decoder: a prompt goes into the decoder's slot cache layer by layer
    (projections by torch), the decode steps continue from it, and the processed logits choose the token.  The
    result is what feeding the prompt to the decoder token by token gives, within the decoder tests' 2e-2."""
    import workloads as wl
    from gpu_common import DenseCase, TOL, rel_err
    s = wl.TINY
    case = DenseCase(s, 2, 128, 2, [0, 0], debug=False)
    K2, V2 = torch.zeros_like(case.K), torch.zeros_like(case.V)
    prompts = [[3, 17, 900, 4, 55, 23, 8], [1000, 2, 2, 77]]
    # token by token
    last = [None, None]
    for b, p in enumerate(prompts):
        for i, t in enumerate(p):
            last[b] = case.gpu_step([t], [b], [i], counts=False)["logits"][0]
    # all at once
    w, eps = case.w, s.eps
    toks = torch.tensor(sum(prompts, []), device=DEV)
    bounds, ctx = cu([len(p) for p in prompts]).to(DEV), i32([0, 0]).to(DEV)
    lens = i32([len(p) for p in prompts]).to(DEV)
    slots = i32([[0], [1]]).to(DEV)

    def norm(x, gain):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gain.float()

    x = w["embed"][toks].float()
    for l in range(s.n_layers):
        L = f"layers.{l}."
        h = norm(x, w[L + "attn_norm"])
        q, k, v = ((h @ w[L + n].float().T).to(BF).view(len(toks), -1, 64) for n in ("wq", "wk", "wv"))
        q = mk.append_kv(q, k, v, K2[l], V2[l], slots, ctx, bounds, rope_theta=s.rope_theta)
        o = mk.prompt_attention(q, K2[l], V2[l], bounds, page_table=slots, kv_lens=lens)
        one = mk.paged_attention(q[[6, 10]], K2[l], V2[l], slots, lens)  # the last tokens, one by one
        assert rel_err(one, o[[6, 10]]) <= TOL
        x = x + o.reshape(len(toks), -1).float() @ w[L + "wo"].float().T
        h = norm(x, w[L + "ffn_norm"])
        x = x + (torch.nn.functional.silu(h @ w[L + "w_gate"].float().T) * (h @ w[L + "w_up"].float().T)) @ w[L + "w_down"].float().T
    logits = norm(x, w["final_norm"]) @ w["embed"].float().T
    for b, at in enumerate((6, 10)):
        assert rel_err(logits[at], last[b]) <= TOL
    for b, p in enumerate(prompts):  # (the layer's caches: post-RoPE keys and values)
        assert rel_err(K2[:, b, :, :len(p)], case.K[:, b, :, :len(p)]) <= TOL
        assert rel_err(V2[:, b, :, :len(p)], case.V[:, b, :, :len(p)]) <= TOL
    # the next step continues from either cache
    token = [11, 12]
    ref = case.gpu_step(token, [0, 1], [7, 4], counts=False)["logits"]
    case.K.copy_(K2)
    case.V.copy_(V2)
    got = case.gpu_step(token, [0, 1], [7, 4], counts=False)["logits"]
    assert rel_err(got, ref) <= TOL
    hist = i32([prompts[0] + [11], prompts[1] + [12] + [-1] * 3]).to(DEV)
    mask = torch.full((2, s.vocab // 32), -1, dtype=torch.int32)
    kw = dict(history=hist.cpu(), history_lens=i32([8, 5]), prompt_lens=i32([7, 4]), repetition=torch.full((2,), 1.2),
              frequency=torch.full((2,), 0.1), presence=torch.full((2,), 0.1), mask=mask)
    out, best = mk.process_logits(got.to(DEV), **to_dev(kw))
    check_logits(out, best, got, kw)
