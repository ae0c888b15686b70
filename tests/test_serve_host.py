"""The serving operators' refusals and their oracle, without a GPU: the C ABI checks its arguments before it touches
a device, so made-up addresses do for what is refused."""
import math

import pytest
import torch

import event_tensor_task_b200 as mk
from oracle import serve as oracle

A = 1 << 20  # an aligned address that is never followed


def pages(**kw):
    p = mk.mk_kv_pages(k=A, v=A, dtype=mk.MK_DTYPE_BF16, n_kv_heads=2, head_dim=64, n_pages=4, page_size=16,
                       page_stride=2048, head_stride=1024, row_stride=64, page_table=A, table_width=3, table_stride=3)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def append_args():
    return mk.mk_append_args(pages=pages(), batch=2, n_tokens=4, n_q_heads=4, q=A, k=A, v=A, q_out=2 * A,
                             q_row_stride=256, q_head_stride=64, k_row_stride=128, k_head_stride=64, v_row_stride=128,
                             v_head_stride=64, qo_row_stride=256, qo_head_stride=64, cu_seqlens=A, ctx_lens=A,
                             rope_theta=10000.0)


def prompt_args():
    return mk.mk_prompt_args(pages=pages(), batch=2, n_tokens=4, n_q_heads=4, causal=1, q=A, out=A, q_row_stride=256,
                             q_head_stride=64, o_row_stride=256, o_head_stride=64, cu_q=A, kv_lens=A)


def paged_args():
    return mk.mk_paged_attn_args(pages=pages(), batch=2, n_q_heads=4, q=A, out=A, q_row_stride=256, q_head_stride=64,
                                 o_row_stride=256, o_head_stride=64, kv_lens=A, workspace=A,
                                 workspace_bytes=mk.mk_paged_attention_workspace_bytes(2, 4, 2, 64))


def logits_args():
    return mk.mk_logits_args(rows=2, vocab=100, dtype=mk.MK_DTYPE_FP32, logits=A, logits_stride=100, out=2 * A,
                             out_stride=100, next_tokens=A, history=A, history_width=8, history_stride=8,
                             repetition=A, bias_indptr=A, bias_ids=A, bias_values=A, bias_count=3, mask=A,
                             mask_stride=4)


INVALID, UNSUPPORTED, WORKSPACE = mk.MK_ERR_INVALID_ARG, mk.MK_ERR_UNSUPPORTED, mk.MK_ERR_WORKSPACE
POOL = [("pages.dtype", 2, INVALID), ("pages.head_dim", 96, UNSUPPORTED), ("pages.n_kv_heads", 0, INVALID),
        ("pages.n_pages", -1, INVALID), ("pages.page_size", 0, INVALID), ("pages.k", 0, INVALID),
        ("pages.v", A + 8, INVALID), ("pages.row_stride", 68, INVALID), ("pages.page_stride", 4, INVALID),
        ("pages.head_stride", -64, INVALID), ("pages.row_stride", 1 << 40, INVALID), ("pages.table_stride", 2, INVALID),
        ("pages.table_width", -1, INVALID), ("pages.table_width", 1 << 28, INVALID),
        ("pages.page_size", 0x7ffffd00 // 3, INVALID)]


def refused(call, args, path, value, status):
    obj = args
    *front, last = path.split(".")
    for f in front:
        obj = getattr(obj, f)
    setattr(obj, last, value)
    with pytest.raises(mk.MkError) as e:
        call(args)
    assert e.value.status == status and e.value.message


@pytest.mark.parametrize("path,value,status", POOL + [
    ("pages.page_table", 0, INVALID), ("batch", -1, INVALID), ("n_tokens", -1, INVALID), ("n_q_heads", 0, INVALID),
    ("q_out", 0, INVALID), ("q_out", A, None), ("k", 0, INVALID), ("v", A + 2, INVALID), ("k_row_stride", 65, INVALID),
    ("q", 0, INVALID), ("cu_seqlens", 0, INVALID), ("ctx_lens", A + 1, INVALID), ("rope_theta", 0.5, INVALID),
    ("rope_theta", math.nan, INVALID), ("status", 3, INVALID), ("pages.row_stride", 0, INVALID),
    ("pages.head_stride", 56, INVALID), ("pages.page_stride", 0, INVALID)])
def test_append_refuses(path, value, status):
    a = append_args()
    if status is None:  # on top of q with other strides
        a.qo_row_stride = 512
        status = INVALID
    refused(mk.mk_append_kv, a, path, value, status)


@pytest.mark.parametrize("path,value,status", POOL + [
    ("batch", -1, INVALID), ("n_tokens", -2, INVALID), ("n_q_heads", 3, INVALID), ("n_q_heads", 0, INVALID),
    ("n_q_heads", 2 * 129, UNSUPPORTED), ("causal", 2, INVALID), ("scale", -1.0, INVALID), ("scale", math.inf, INVALID),
    ("scale", math.nan, INVALID), ("q", 0, INVALID), ("out", A + 4, INVALID), ("q_row_stride", 7, INVALID),
    ("cu_q", 0, INVALID), ("kv_lens", 0, INVALID), ("pages.page_size", 48, UNSUPPORTED),
    ("pages.page_size", 8, UNSUPPORTED), ("pages.page_table", 0, INVALID), ("workspace", A + 64, WORKSPACE)])
def test_prompt_refuses(path, value, status):
    refused(mk.mk_prompt_attention, prompt_args(), path, value, status)


def test_prompt_refuses_packed_keys_in_two_pages():
    a = prompt_args()
    a.cu_k = A
    refused(mk.mk_prompt_attention, a, "pages.page_table", 0, INVALID)  # n_pages is 4


@pytest.mark.parametrize("path,value,status", POOL + [
    ("pages.page_table", 0, INVALID), ("batch", -1, INVALID), ("batch", mk.MK_PAGED_ATTN_MAX_BATCH + 1, UNSUPPORTED),
    ("n_q_heads", 5, INVALID), ("scale", -0.1, INVALID), ("q", A + 8, INVALID), ("out", 0, INVALID),
    ("o_head_stride", 60, INVALID), ("kv_lens", 0, INVALID), ("workspace", 0, WORKSPACE), ("workspace", A + 16, WORKSPACE),
    ("workspace_bytes", 1000, WORKSPACE)])
def test_paged_refuses(path, value, status):
    refused(mk.mk_paged_attention, paged_args(), path, value, status)


@pytest.mark.parametrize("path,value,status", [
    ("rows", -1, INVALID), ("rows", 65536, INVALID), ("vocab", 0, INVALID), ("vocab", (1 << 30) + 1, INVALID), ("dtype", 3, INVALID), ("logits", 0, INVALID),
    ("logits", A + 2, INVALID), ("logits_stride", 99, INVALID), ("out_stride", 99, INVALID), ("out", A + 2, INVALID),
    ("history_stride", 7, INVALID), ("history_width", -1, INVALID), ("history_width", 1 << 28, INVALID),
    ("history", 0, INVALID), ("bias_ids", 0, INVALID), ("bias_count", -1, INVALID), ("mask_stride", 3, INVALID),
    ("repetition", A + 1, INVALID)])
def test_logits_refuses(path, value, status):
    refused(mk.mk_process_logits, logits_args(), path, value, status)


def test_logits_refuses_no_output_and_wrong_alias():
    a = logits_args()
    a.out = 0
    refused(mk.mk_process_logits, a, "next_tokens", 0, INVALID)
    a = logits_args()
    a.dtype = mk.MK_DTYPE_BF16
    refused(mk.mk_process_logits, a, "out", A, INVALID)


def test_null_arguments_and_empty_calls():
    lib = mk.lib()
    for name in ("mk_append_kv", "mk_prompt_attention", "mk_paged_attention", "mk_process_logits"):
        assert getattr(lib, name)(None, 0) == INVALID and mk.mk_last_error()
    assert lib.mk_append_kv(mk.mk_append_args(batch=2, n_tokens=0), 0) == mk.MK_OK
    assert lib.mk_prompt_attention(mk.mk_prompt_args(), 0) == mk.MK_OK
    assert lib.mk_paged_attention(mk.mk_paged_attn_args(), 0) == mk.MK_OK
    assert lib.mk_process_logits(mk.mk_logits_args(vocab=9), 0) == mk.MK_OK


def tensors():
    z = torch.zeros
    return dict(q=z((4, 4, 64), dtype=torch.bfloat16), k=z((4, 2, 64), dtype=torch.bfloat16),
                pool=z((3, 2, 16, 64), dtype=torch.bfloat16), table=z((2, 3), dtype=torch.int32),
                lens=z(2, dtype=torch.int32), cu=z(3, dtype=torch.int32), logits=z((2, 70)),
                hist=z((2, 5), dtype=torch.int32), row=z(2), mask=z((2, 3), dtype=torch.int32))


def calls(x, **kw):
    """The four calls on CPU tensors; `kw` replaces arguments."""
    g = dict(x, **kw)
    return dict(
        append=lambda: mk.append_kv(g["q"], g["k"], g.get("v", x["k"]), g["pool"], g.get("vpool", g["pool"]), g["table"],
                                    g["lens"], g["cu"], q_out=g.get("q_out")),
        prompt=lambda: mk.prompt_attention(g["q"], g["k"], g.get("v", x["k"]), g["cu"], kv_lens=g.get("kv_lens"),
                                           cu_k=g.get("cu_k"), scale=g.get("scale"), out=g.get("q_out")),
        chunk=lambda: mk.prompt_attention(g["q"], g["pool"], g.get("vpool", g["pool"]), g["cu"], page_table=g["table"],
                                          kv_lens=g["lens"], cu_k=g.get("cu_k")),
        paged=lambda: mk.paged_attention(g["q"][:2], g["pool"], g.get("vpool", g["pool"]), g["table"], g["lens"],
                                         scale=g.get("scale"), workspace=g.get("ws")),
        logits=lambda: mk.process_logits(g["logits"], history=g["hist"], repetition=g["row"], mask=g["mask"],
                                         bias=g.get("bias"), out=g.get("out"), next_tokens=g.get("next")))


def test_tensor_calls_refuse_cpu_tensors():
    """Everything in order but the place: refused for that, before any launch."""
    for name, call in calls(tensors()).items():
        with pytest.raises(mk.MkError, match="CUDA device") as e:
            call()
        assert e.value.status == INVALID, name


@pytest.mark.parametrize("names,match,change", [
    ("append", "k must be", lambda x: dict(k=x["k"][:, :1])),
    ("append", "v must be", lambda x: dict(v=x["k"][:3])),
    ("append", "v must be", lambda x: dict(v=x["k"].half())),
    ("append prompt", "q must be", lambda x: dict(q=x["q"].float())),
    ("append prompt paged", "q must be", lambda x: dict(q=x["q"][:, 0])),
    ("append prompt paged", "q must be a tensor", lambda x: dict(q=[[1.0]] * 4)),
    ("append prompt", "dense", lambda x: dict(q=x["q"].transpose(1, 2).contiguous().transpose(1, 2))),
    ("append chunk paged", "page_table", lambda x: dict(table=x["table"].long())),
    ("append chunk", "page_table", lambda x: dict(table=x["table"][:1])),
    ("append chunk paged", "dense rows", lambda x: dict(table=x["table"].T.contiguous().T)),
    ("append chunk paged", "same strides", lambda x: dict(vpool=x["pool"].transpose(1, 2).contiguous().transpose(1, 2))),
    ("append chunk paged", "bf16 or fp16", lambda x: dict(pool=x["pool"].float())),
    ("append chunk paged", "k and v pages", lambda x: dict(pool=x["pool"][0])),
    ("append", "ctx_lens", lambda x: dict(lens=x["lens"].long())),
    ("append", "cu_seqlens", lambda x: dict(cu=x["cu"][:2])),
    ("chunk", "kv_lens must be", lambda x: dict(lens=torch.zeros((2, 2), dtype=torch.int32)[:, 0])),
    ("prompt", "not kv_lens", lambda x: dict(kv_lens=x["lens"])),
    ("prompt", "cu_k must be", lambda x: dict(cu_k=x["cu"][:2])),
    ("prompt", "same strides", lambda x: dict(v=torch.zeros((4, 3, 64), dtype=torch.bfloat16)[:, :2])),
    ("chunk", "not cu_k", lambda x: dict(cu_k=x["cu"])),
    ("chunk", "names no pages", lambda x: dict(table=x["table"][:, :0])),
    ("prompt paged", "scale", lambda x: dict(scale=0.0)),
    ("prompt paged", "scale", lambda x: dict(scale=-1.0)),
    ("paged", "workspace", lambda x: dict(ws=torch.zeros(9))),
    ("logits", "logits must be", lambda x: dict(logits=x["logits"].double())),
    ("logits", "logits must be", lambda x: dict(logits=x["logits"][0])),
    ("logits", "dense rows", lambda x: dict(logits=x["logits"].T.contiguous().T)),
    ("logits", "history must be", lambda x: dict(hist=x["hist"].long())),
    ("logits", "need a history", lambda x: dict(hist=None)),
    ("logits", "repetition", lambda x: dict(row=x["row"].double())),
    ("logits", "mask must be", lambda x: dict(mask=x["mask"][:, :2])),
    ("logits", "bias", lambda x: dict(bias=(x["cu"], x["lens"], None))),
    ("logits", "bias values", lambda x: dict(bias=(x["cu"], x["lens"], torch.zeros(3)))),
])
def test_tensor_calls_refuse_types_shapes_and_strides(names, match, change):
    x = tensors()
    for name in names.split():
        with pytest.raises(mk.MkError, match=match) as e:
            calls(x, **change(x))[name]()
        assert e.value.status == INVALID


# ------------------------------------------------------------------------------------------------ the oracle's pins
def test_oracle_rotation_is_complex_multiplication():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 2, 64), generator=g, dtype=torch.float64)
    z = torch.view_as_complex(torch.stack([x[..., :32], x[..., 32:]], -1).contiguous())
    pos = [0, 5, 131071]
    p = torch.arange(32, dtype=torch.float64)
    turn = torch.polar(torch.ones((3, 1, 32), dtype=torch.float64), torch.tensor(pos, dtype=torch.float64)[:, None, None] * 10000.0 ** (-p / 32))
    y = torch.view_as_real(z * turn)
    assert torch.allclose(oracle.rotate(x, pos, 10000.0), torch.cat([y[..., 0], y[..., 1]], -1), atol=1e-9)
    assert torch.equal(oracle.rotate(x, pos, 0.0), x)


def test_oracle_attention_matches_the_library_and_skips_unseen_keys():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((5, h, 64), generator=g, dtype=torch.float64) for h in (4, 2, 2))
    out, mag, big = oracle.attend(q, k, v, [1, 2, 3, 4, 5], 0.125)
    ref = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1)[None], k.transpose(0, 1).repeat_interleave(2, 0)[None],
                                                           v.transpose(0, 1).repeat_interleave(2, 0)[None], is_causal=True)
    assert torch.allclose(out, ref[0].transpose(0, 1), atol=1e-12)
    k[4], v[4] = math.nan, math.nan
    short = oracle.attend(q, k, v, [0, 2, 3, 4, 4], 0.125)[0]
    assert (short[0] == 0).all() and torch.equal(short[1:4], out[1:4]) and torch.isfinite(short).all()
    assert (mag >= out.abs() - 1e-12).all() and (big > 0).all()


def test_oracle_logits_by_hand():
    x = torch.tensor([[2.0, -2.0, 1.0, 0.5, 3.0]])
    out, best = oracle.process(x, history=torch.tensor([[0, 1, 1, 3, 9]]), history_lens=[4], prompt_lens=[2],
                               repetition=[2.0], frequency=[0.25], presence=[0.5],
                               bias=(torch.tensor([0, 2]), torch.tensor([2, 2]), torch.tensor([1.0, 0.5])),
                               mask=torch.tensor([[0b01111]]))
    # id 0: 2/2; id 1 (once in the answer): -2*2 - 0.25 - 0.5; id 2: +1.5; id 3: 0.5/2 - 0.75; id 4: masked
    assert out[0].tolist() == [1.0, -4.75, 2.5, -0.5, -math.inf] and best.tolist() == [2]
