"""The serving operators at calls that the first tests do not make: short prompts in great number, pools without pages,
calls from two threads and the like.  Tolerances as in test_gpu_serve.py."""
import math

import pytest
import torch

import event_tensor_task_b200 as mk
from oracle import serve as oracle
from test_gpu_serve import BF, DEV, HF, check_attention, cu, dev, gen, i32, prompt_reference, status_word

pytestmark = pytest.mark.gpu


def flush():
    """Nothing of what was there before stays in L2 (126 MB)."""
    torch.zeros(1 << 26, device=DEV)


@pytest.mark.parametrize("hkv,d,dtype", [(8, 64, BF), (4, 128, HF)])
def test_short_prompts_in_great_number(hkv, d, dtype):
    """Every block runs dozens of pieces of work of one or two key tiles, each ending inside its last value tile, out of
    key and value pools that are not in L2.  The rows are those of calls too small for a block to get a second piece."""
    g = gen(hkv)
    n, page = 1200, 64
    lens = [int(m) for m in torch.randint(1, 129, (n,), generator=g)]
    need = [-(-m // page) for m in lens]
    total = 4 * sum(need)
    where = torch.randperm(total, generator=g)[:sum(need)].to(torch.int32)
    table = torch.full((n, 2), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = where[at:at + m]
        at += m
    dgen = torch.Generator(device=DEV).manual_seed(d)
    k, v = (torch.randn((total, hkv, page, d), generator=dgen, device=DEV).to(dtype) for _ in range(2))
    q = torch.randn((sum(lens), hkv, d), generator=dgen, device=DEV).to(dtype)
    table, bounds = table.to(DEV), cu(lens)
    few = 120 // hkv
    want, st = torch.empty_like(q), status_word()
    for b in range(0, n, few):
        e = min(n, b + few)
        lo, hi = int(bounds[b]), int(bounds[e])
        want[lo:hi] = mk.prompt_attention(q[lo:hi], k, v, (bounds[b:e + 1] - lo).to(DEV), page_table=table[b:e],
                                          kv_lens=i32(lens[b:e]).to(DEV), status=st)
    assert int(st) == 0
    on_device = bounds.to(DEV), i32(lens).to(DEV)
    for _ in range(8):
        flush()
        out = mk.prompt_attention(q, k, v, on_device[0], page_table=table, kv_lens=on_device[1], status=st,
                                  out=torch.full_like(q, math.nan))
        torch.cuda.synchronize()
        assert int(st) == 0 and torch.equal(out, want)
    for b in range(0, n, 100):  # and the rows are right
        lo, m = int(bounds[b]), lens[b]
        rows = [torch.cat([pool[int(p)].transpose(0, 1) for p in table[b, :need[b]]])[:m].cpu() for pool in (k, v)]
        ref = prompt_reference(q[lo:lo + m].cpu(), rows[:1], rows[1:], [m], True, d ** -0.5)
        check_attention(out[lo:lo + m], ref, dtype, 128, 6.0, False)


@pytest.mark.parametrize("width,keys", [(3, 5), (200, 3000)])  # (few keys; enough to be cut into pieces)
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF)])
def test_a_pool_without_pages_holds_no_keys(d, dtype, width, keys):
    """Whatever the table and the lengths say: zero rows, nothing stored, and the status word."""
    k, v = torch.empty((2, 0, 2, 16, d), dtype=dtype, device=DEV)
    table, q = torch.zeros((2, width), dtype=torch.int32, device=DEV), torch.ones((6, 4, d), dtype=dtype, device=DEV)
    st = status_word()
    out = mk.prompt_attention(q, k, v, cu([5, 1]).to(DEV), page_table=table, kv_lens=i32([keys, 0]).to(DEV), status=st)
    torch.cuda.synchronize()
    assert int(st) == mk.MK_ERR_DEVICE_BOUNDS and (out == 0).all()
    st.zero_()
    out = mk.prompt_attention(q, k, v, cu([5, 1]).to(DEV), page_table=table, kv_lens=i32([0, 0]).to(DEV), status=st)
    assert int(st) == 0 and (out == 0).all()
    out = mk.paged_attention(q[:2], k, v, table, i32([keys, 0]).to(DEV), status=st)
    assert int(st) == mk.MK_ERR_DEVICE_BOUNDS and (out == 0).all()
    st.zero_()
    mk.append_kv(q, q[:, :2], q[:, 2:], k, v, table, i32([0, 0]).to(DEV), cu([5, 1]).to(DEV), status=st)
    assert int(st) == mk.MK_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF)])
def test_work_handed_out_by_every_lane(d, dtype):
    """Seventy sequences, so every lane of the warp that hands out the work finds and publishes some of it; a few are
    cut into pieces, of which the blocks that see few keys leave all but the first idle."""
    g = gen(d)
    new = [int(n) for n in torch.randint(1, 30, (70,), generator=g)]
    keys = [n + int(e) for n, e in zip(new, torch.randint(0, 100, (70,), generator=g))]
    for b in (2, 33, 69):
        new[b], keys[b] = 140, 2600
    keys[33] = 1700
    new[2] = 1500  # its first rows see about a thousand keys, its last 2,600
    q = torch.randn((sum(new), 2, d), generator=g).to(dtype)
    kv = torch.randn((sum(keys), 2, d), generator=g).to(dtype)
    x, st = dev(kv), status_word()
    args = dev(q), x[:, :1], x[:, 1:], cu(new).to(DEV)
    assert mk.mk_prompt_attention_workspace_bytes(70, sum(new), 2, 1, d, sum(keys)) > 0
    outs = [mk.prompt_attention(*args, cu_k=cu(keys).to(DEV), status=st) for _ in range(5)]
    whole = mk.prompt_attention(*args, cu_k=cu(keys).to(DEV), status=st, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert int(st) == 0 and all(torch.equal(outs[0], o) for o in outs)
    qb, kb = cu(new), cu(keys)
    for b in range(70):
        some = torch.arange(0, new[b], 97 if new[b] > 200 else 1)
        k, v = kv[kb[b]:kb[b + 1], :1], kv[kb[b]:kb[b + 1], 1:]
        ref = oracle.attend(q[qb[b] + some], k, v, [int(i) + 1 + keys[b] - new[b] for i in some], d ** -0.5)
        for out in (outs[0], whole):
            check_attention(out[int(qb[b]) + some.to(DEV)], ref, dtype, keys[b], 6.0, False)


def test_prompt_workspace_goes_by_the_call():
    """A short prompt over the decoder's slot cache takes kilobytes, not what the whole device could leave; the most that
    any call takes is what it was."""
    small = mk.mk_prompt_attention_workspace_bytes(1, 17, 4, 2, 64, 2048)
    assert 0 < small <= 1 << 20
    k, v = torch.zeros((2, 4, 2, 2048, 64), dtype=BF, device=DEV)
    q = torch.zeros((17, 4, 64), dtype=BF, device=DEV)
    args = cu([17]).to(DEV), i32([[2]]).to(DEV), i32([17]).to(DEV)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    mk.prompt_attention(q, k, v, args[0], page_table=args[1], kv_lens=args[2])
    assert torch.cuda.max_memory_allocated() - before <= 2 << 20
    for d in (64, 128):
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        tiles = 2 * sms  # of 128 rows, that the device holds
        whole = mk.mk_prompt_attention_workspace_bytes(1, 128 * sms, 1, 1, d, 1 << 22)
        assert whole == 4 * 2 * tiles * 128 * (d + 2) * 4


@pytest.mark.parametrize("page", [16, 128, 130, 255, 1024])
@pytest.mark.parametrize("hq,hkv,d,new,lens", [
    (4, 2, 64, [17], [2300]),
    (2, 1, 128, [1, 9, 260], [1800, 40, 2100]),
    (6, 2, 64, [64, 65, 1], [1700, 900, 2550]),
])
def test_prompt_workspace_is_enough(page, hq, hkv, d, new, lens):
    """Nothing is written behind it, and what comes out is what comes out with one as large as any call's."""
    g = gen(page + d)
    k, v, table = (t.to(DEV) for t in _filled_pool(g, lens, page, hkv, d))
    q = torch.randn((sum(new), hq, d), generator=g).to(BF).to(DEV)
    tail = cu(new).to(DEV), i32(lens).to(DEV)
    n = mk.mk_prompt_attention_workspace_bytes(len(new), sum(new), hq, hkv, d, page * table.shape[1])
    assert n > 0 and n % 16 == 0
    buf = torch.full((n + 4096,), 171, dtype=torch.uint8, device=DEV)
    st = status_word()
    outs = [mk.prompt_attention(q, k, v, tail[0], page_table=table, kv_lens=tail[1], workspace=w, status=st)
            for w in (buf[:n], None, torch.empty(200 << 20, dtype=torch.uint8, device=DEV))]
    torch.cuda.synchronize()
    assert int(st) == 0 and (buf[n:] == 171).all() and not (buf[:n] == 171).all()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def _filled_pool(g, lens, page, hkv, d):
    need = [-(-n // page) for n in lens]
    perm = torch.randperm(sum(need), generator=g).to(torch.int32)
    table, at = torch.full((len(lens), max(need)), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    k, v = torch.randn((2, sum(need), hkv, page, d), generator=g).to(BF)
    return k, v, table


@pytest.mark.parametrize("bounds,fine", [
    ([0, 2, 6], True),
    ([1, 2, 4], True),          # rows before the first sequence and behind the last
    ([0, 2, 7], False),         # more rows than there are
    ([0, 5, 3, 6], False),      # a sequence of fewer than no rows
    ([0, 6, 6, 5], False),
    ([0] * 299 + [6, 2], False),
    ([-1, 2, 6], False),
    ([0, 2, 2**31 - 1], False),
])
def test_append_reports_bounds_of_sequences(bounds, fine):
    g = gen(71)
    B = len(bounds) - 1
    k, v = torch.zeros((2, B, 2, 16, 64), dtype=BF, device=DEV)
    x = torch.randn((6, 2, 64), generator=g).to(BF).to(DEV)
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
    st = status_word()
    mk.append_kv(None, x, x, k, v, table, torch.zeros(B, dtype=torch.int32, device=DEV), i32(bounds).to(DEV),
                 rope_theta=0, status=st)
    assert int(st) == (0 if fine else mk.MK_ERR_DEVICE_BOUNDS)
    if fine or bounds == [0, 2, 7]:  # rows that exist are stored
        for b in range(2):
            lo, hi = bounds[b], min(bounds[b + 1], 6)
            assert torch.equal(v[b, :, :hi - lo], x[lo:hi].transpose(0, 1)) and (v[b, :, hi - lo:] == 0).all()


def _program(seed, d=64, dtype=BF):
    """A short serving step on tensors of its own: a function that runs it and returns all that it wrote."""
    g = gen(seed)
    new, ctx = [9, 1, 40], [30, 2000, 3]
    lens = [a + c for a, c in zip(new, ctx)]
    k, v, table = (t.to(DEV) for t in _filled_pool(g, lens, 16, 2, d))
    x = torch.randn((sum(new), 8, d), generator=g).to(dtype).to(DEV)
    W = (torch.randn((4 * d, 5000), generator=g) / 16).to(dtype).to(DEV)
    ctx, lens, bounds = i32(ctx).to(DEV), i32(lens).to(DEV), cu(new).to(DEV)
    last = (bounds[1:] - 1).long()
    hist, pen = torch.randint(0, 5000, (3, 50), generator=g, dtype=torch.int32).to(DEV), torch.full((3,), 1.3, device=DEV)

    def run(split=None):
        kc, vc = k.clone(), v.clone()
        q = mk.append_kv(x[:, :4], x[:, 4:6], x[:, 6:], kc, vc, table, ctx, bounds)
        if split is None:
            a = mk.prompt_attention(q, kc, vc, bounds, page_table=table, kv_lens=lens)
            b = mk.paged_attention(q[last], kc, vc, table, lens)
        else:  # the two attentions side by side
            here = torch.cuda.current_stream()
            split.wait_stream(here)
            with torch.cuda.stream(split):
                b = mk.paged_attention(q[last], kc, vc, table, lens)
            a = mk.prompt_attention(q, kc, vc, bounds, page_table=table, kv_lens=lens)
            here.wait_stream(split)
        joined = (a[last] + b).reshape(3, -1)
        out, best = mk.process_logits(joined @ W, history=hist, repetition=pen)
        return [kc, vc, q, a, b, out, best]

    return run


def test_two_host_threads_at_once():
    """Each on a stream of its own, and then both on one; a refusal in one thread does not show in the other."""
    import threading
    runs = [_program(s) for s in (80, 81)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    shared = torch.cuda.Stream()
    bad = torch.zeros((3, 1), dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    for own in (True, False):
        got, wrong = [[], []], []

        def work(i, stream):
            try:
                with torch.cuda.stream(stream):
                    for n in range(20):
                        got[i].append(runs[i]())
                        if i == 1:
                            with pytest.raises(mk.MkError, match="above 0"):
                                mk.paged_attention(want[1][2][:3], want[1][0], want[1][1], *bad, scale=-1.0)
            except BaseException as e:  # noqa: B902 (told by the test's thread)
                wrong.append(e)

        streams = [torch.cuda.Stream() if own else shared for _ in range(2)]
        threads = [threading.Thread(target=work, args=(i, streams[i])) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not wrong, wrong
        for i in range(2):
            assert len(got[i]) == 20
            for outs in got[i]:
                assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


@pytest.mark.parametrize("captured", [False, True])
def test_calls_of_two_streams_that_meet(captured):
    """The cache is filled on one stream, its two readers run on two, and the next call waits for both."""
    run = _program(82)
    want = run()
    torch.cuda.synchronize()
    split = torch.cuda.Stream()
    if captured:
        run(split)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run(split)
        for _ in range(10):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    else:
        for _ in range(30):
            got = run(split)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_every_call_repeats_itself():
    """The same bits from run to run, with the device empty or full of other work."""
    run = _program(83)
    want, other = run(), torch.cuda.Stream()
    a = torch.randn((4096, 4096), device=DEV, dtype=BF)
    for i in range(20):
        if i % 2:
            with torch.cuda.stream(other):
                for _ in range(4):
                    a @ a
        flush()
        got = run()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    torch.cuda.synchronize()


def test_first_calls_of_a_process_are_captured():
    """No call before the capture has loaded a kernel, asked for shared memory or made a tensor map."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = """
import sys
sys.path[:0] = [%r, %r]
import torch
import event_tensor_task_b200 as mk
from test_gpu_serve import i32, cu
d = "cuda:0"
for dim, dtype in ((64, torch.bfloat16), (128, torch.float16)):
    k, v = torch.randn((2, 200, 2, 16, dim), device=d).to(dtype)
    x = torch.randn((6, 8, dim), device=d).to(dtype)
    table = torch.arange(198, dtype=torch.int32, device=d).view(2, 99)
    ctx, lens, bounds = i32([1500, 3]).to(d), i32([1505, 4]).to(d), cu([5, 1]).to(d)
    logits = torch.randn((2, 5000), device=d).to(dtype)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = mk.append_kv(x[:, :4], x[:, 4:6], x[:, 6:], k, v, table, ctx, bounds)
        a = mk.prompt_attention(q, k, v, bounds, page_table=table, kv_lens=lens)
        b = mk.paged_attention(q[4:], k, v, table, lens)
        out = mk.process_logits(logits)
    graph.replay()
    torch.cuda.synchronize()
    want = mk.prompt_attention(q, k, v, bounds, page_table=table, kv_lens=lens), mk.paged_attention(q[4:], k, v, table, lens)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert torch.equal(out[1], logits.float().argmax(-1).int())
print("captured")
""" % (os.path.dirname(here), here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
