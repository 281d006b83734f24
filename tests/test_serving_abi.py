"""Refusals of the serving-step calls: host checks that come before any launch."""
import os

import pytest

import bit_vector_quantized_gb300 as vq

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(vq.LIB_PATH):
        from bit_vector_quantized_gb300 import build
        build.build()
    return vq.lib()


def refused(fn, args, cases):
    for kw, st in cases:
        with pytest.raises(vq.VQError) as e:
            fn(**dict(args, **kw))
        assert e.value.status == st, kw


def test_append_slots_refusals():
    args = dict(batch=2, seq_lens=FAKE, new_lens=FAKE, page_table=FAKE, max_pages_per_seq=4, free_pages=FAKE,
                free_capacity=8, num_free=FAKE, page_size=64, num_pages=8, max_tokens=16, seq_lens_out=FAKE,
                num_free_out=FAKE, cu_new_lens=FAKE, slot_mapping=FAKE, positions=FAKE)
    bad = vq.VQ_ERR_INVALID_ARG
    refused(vq.vq_append_slots, args, [
        (dict(batch=-1), bad), (dict(batch=16385), vq.VQ_ERR_UNSUPPORTED), (dict(page_size=0), bad),
        (dict(page_size=24), bad), (dict(num_pages=0), bad), (dict(max_pages_per_seq=0), bad),
        (dict(free_capacity=-1), bad), (dict(max_tokens=-1), bad), (dict(max_tokens=(1 << 30) + 1), bad),
        (dict(seq_lens=None), bad), (dict(new_lens=None), bad), (dict(page_table=None), bad),
        (dict(free_pages=None), bad), (dict(num_free=None), bad), (dict(seq_lens_out=None), bad),
        (dict(num_free_out=None), bad), (dict(cu_new_lens=None), bad), (dict(slot_mapping=None), bad),
        (dict(positions=None), bad), (dict(slot_mapping=FAKE + 8), bad)])


def test_rotary_refusals():
    args = dict(config=vq.make_rotary(), num_tokens=4, positions=FAKE, dtype=vq.VQ_FP16, q=1 << 24, q_stride=512,
                num_q_heads=4, q_out=1 << 25, k=1 << 26, k_stride=128, v=None, v_stride=0, num_kv_heads=1,
                k_out=1 << 27, v_out=None)
    bad = vq.VQ_ERR_INVALID_ARG
    mk = vq.make_rotary
    refused(vq.vq_rotary, args, [
        (dict(config=mk(head_dim=64)), vq.VQ_ERR_UNSUPPORTED), (dict(config=mk(rotary_dim=0)), bad),
        (dict(config=mk(rotary_dim=130)), bad), (dict(config=mk(rotary_dim=33)), bad), (dict(config=mk(base=0.5)), bad),
        (dict(config=mk(base=float("inf"))), bad), (dict(config=mk(attention_factor=0.0)), bad),
        (dict(config=mk(scaling="linear", factor=0.0)), bad),
        (dict(config=mk(scaling="parts", factor=2.0, low_turns=4.0, high_turns=4.0)), bad),
        (dict(config=mk(scaling="parts", factor=2.0, base=1.0)), bad),
        (dict(config=mk(scaling="wavelength", factor=2.0, original_len=0)), bad), (dict(dtype=2), bad),
        (dict(num_tokens=-1), bad), (dict(positions=None), bad), (dict(positions=FAKE + 4), bad),
        (dict(q_out=None), bad), (dict(v=1 << 28), bad), (dict(q=None, q_out=None, k=None, k_out=None), bad),
        (dict(q_stride=511), bad), (dict(q_stride=504), bad), (dict(num_q_heads=0), bad), (dict(k=(1 << 26) + 8), bad),
        (dict(q_out=(1 << 24) + 1024), bad), (dict(k_out=1 << 25), bad), (dict(q_out=1 << 24, q_stride=640), bad),
        (dict(q_out=1 << 24, dtype=vq.VQ_BF16), bad), (dict(k_out=FAKE), bad)])
    vq.vq_rotary(**dict(args, num_tokens=0, positions=None, q=None, q_out=None, k=None, k_out=None))  # no tokens: no-op


def test_chunk_attention_refusals():
    L = vq.make_layout()
    args = dict(layout=L, batch=2, num_tokens=4, q=1 << 24, lambda_=FAKE, codebook_k=FAKE, codebook_v=FAKE, k_pool=FAKE,
                v_pool=FAKE, num_pages=4, page_table=FAKE, max_pages_per_seq=4, seq_lens=FAKE, max_seq_len=100,
                cu_new_lens=FAKE, max_new_len=2, window=0, num_sinks=0, softmax_scale=0.0, out=1 << 26, workspace=FAKE,
                workspace_bytes=1 << 30)
    bad, unsupported = vq.VQ_ERR_INVALID_ARG, vq.VQ_ERR_UNSUPPORTED
    refused(vq.vq_chunk_attention, args, [
        (dict(batch=-1), bad), (dict(batch=1025), unsupported), (dict(num_tokens=-1), bad), (dict(max_new_len=-1), bad),
        (dict(window=-1), bad), (dict(num_sinks=-1), bad), (dict(num_sinks=4), bad), (dict(softmax_scale=float("nan")), bad),
        (dict(q=None), bad), (dict(lambda_=None), bad), (dict(codebook_k=None), bad), (dict(codebook_v=None), bad),
        (dict(k_pool=None), bad), (dict(v_pool=None), bad), (dict(page_table=None), bad), (dict(seq_lens=None), bad),
        (dict(out=None), bad), (dict(workspace=None), bad), (dict(cu_new_lens=FAKE + 4), bad), (dict(q=FAKE + 8), bad),
        (dict(num_pages=0), bad), (dict(max_pages_per_seq=0), bad), (dict(max_seq_len=-1), bad), (dict(max_seq_len=1025), bad),
        (dict(max_seq_len=(1 << 30) + 1, max_pages_per_seq=1 << 24), bad), (dict(out=(1 << 24) + 64), bad),
        (dict(cu_new_lens=None, num_tokens=1), bad), (dict(layout=vq.make_layout(v_sub=8)), unsupported),
        (dict(layout=vq.make_layout(page_size=8)), bad)])
    for kw in (dict(batch=0), dict(num_tokens=0), dict(max_new_len=0)):  # nothing to do
        vq.vq_chunk_attention(**dict(args, q=None, out=None, workspace=None, **kw))


def test_chunk_workspace_bytes():
    L = vq.make_layout()
    n = vq.vq_chunk_workspace_bytes(L, 4, 4, 1000, 1, 152)
    assert n > 0 and n % 256 == 0
    assert vq.vq_chunk_workspace_bytes(L, 4, 400, 1000, 100, 152) >= n
    for kw in ((-1, 4, 1000, 1), (4, -1, 1000, 1), (4, 4, -1, 1), (4, 4, 1000, -1)):
        assert vq.vq_chunk_workspace_bytes(L, *kw, 152) == 0
    assert vq.vq_chunk_workspace_bytes(vq.make_layout(v_sub=8), 4, 4, 1000, 1, 152) == 0


def test_row_offsets_need_their_bound():
    """Without it longer sequences would be left out of an output that nobody had written."""
    with pytest.raises(ValueError, match="max_new_len"):
        vq.chunk_attention(vq.make_layout(), None, None, None, None, None, None, None, None, 100, cu_new_lens=object())
