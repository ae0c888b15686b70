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
        ("pages.table_width", -1, INVALID), ("pages.table_width", 1 << 28, INVALID)]


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
    ("rope_theta", math.nan, INVALID), ("status", 3, INVALID)])
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
    ("pages.page_size", 8, UNSUPPORTED), ("pages.page_table", 0, INVALID)])
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
    ("rows", -1, INVALID), ("rows", 65536, INVALID), ("vocab", 0, INVALID), ("dtype", 3, INVALID), ("logits", 0, INVALID),
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


def test_tensor_calls_refuse_what_the_struct_cannot_show():
    """Types, shapes, strides and places, before any launch (CPU tensors: refused for that at the latest)."""
    t = torch.zeros
    q, kv = t((2, 4, 64), dtype=torch.bfloat16), t((3, 2, 16, 64), dtype=torch.bfloat16)
    i = t((2, 3), dtype=torch.int32)
    for call in (lambda: mk.paged_attention(q, kv, kv, i, i[:, 0]), lambda: mk.paged_attention(q[0], kv, kv, i, i[:, 0]),
                 lambda: mk.prompt_attention(q, q, q, i[0]), lambda: mk.process_logits(t((2, 5))),
                 lambda: mk.process_logits(t((2, 5), dtype=torch.float64)), lambda: mk.process_logits(t(5)),
                 lambda: mk.append_kv(q, q, q, kv, kv, i, i[:, 0], i[0])):
        with pytest.raises(mk.MkError) as e:
            call()
        assert e.value.status == INVALID
    # the helpers behind them
    def fill(*a):
        p = mk.mk_kv_pages()
        mk._pages(p, *a)
        return p

    for bad in ((kv, kv.transpose(1, 2).contiguous().transpose(1, 2), i, 2),  # other strides
                (kv, kv, i.long(), 2), (kv.float(), kv.float(), i, 2), (kv, kv, i, 3), (kv[0], kv[0], i, 2),
                (kv, kv, i.T.contiguous().T, 2), (kv.transpose(2, 3), kv.transpose(2, 3), i, 2)):
        with pytest.raises(mk.MkError):
            fill(*bad)
    with pytest.raises(mk.MkError):
        mk._rows("q", q.transpose(1, 2), q.transpose(1, 2).shape, q.dtype)
    with pytest.raises(mk.MkError):
        mk._array("lens", i[:, 0], torch.int32, 2)  # not dense
    with pytest.raises(mk.MkError):
        mk._dense_rows("mask", i, torch.int32, 2, 4)
    with pytest.raises(mk.MkError):
        mk._scale(0.0)
    p = fill(kv, kv, i, 2)
    assert (p.n_pages, p.n_kv_heads, p.page_size, p.head_dim, p.table_width, p.table_stride) == (3, 2, 16, 64, 3, 3)
    assert (p.page_stride, p.head_stride, p.row_stride) == (2048, 1024, 64)
    p = fill(kv[:1], kv[1:2], i, 2)
    assert (p.page_stride, p.head_stride, p.row_stride) == (0, 1024, 64)  # (one page: its stride is not used)


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
