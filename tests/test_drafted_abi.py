"""Refusals of the calls around drafted tokens: host checks that come before any launch."""
import os

import pytest

import bit_vector_quantized_gb300 as vq
from test_serving_abi import FAKE, refused

bad, unsupported = vq.VQ_ERR_INVALID_ARG, vq.VQ_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(vq.LIB_PATH):
        from bit_vector_quantized_gb300 import build
        build.build()
    return vq.lib()


def test_tree_attention_refusals():
    args = dict(layout=vq.make_layout(), batch=2, num_tokens=4, q=1 << 24, lambda_=FAKE, codebook_k=FAKE, codebook_v=FAKE, k_pool=FAKE,
                v_pool=FAKE, num_pages=4, page_table=FAKE, max_pages_per_seq=4, seq_lens=FAKE, max_seq_len=100,
                cu_new_lens=FAKE, max_new_len=2, tree_masks=FAKE, mask_words=1, positions=None, window=0, num_sinks=0, softmax_scale=0.0,
                out=1 << 26, workspace=FAKE, workspace_bytes=1 << 30)
    refused(vq.vq_tree_attention, args, [
        (dict(batch=-1), bad), (dict(batch=1025), unsupported), (dict(num_tokens=-1), bad), (dict(max_new_len=-1), bad),
        (dict(max_new_len=257, mask_words=5), unsupported), (dict(max_new_len=65), bad), (dict(mask_words=0), bad), (dict(mask_words=65), bad),
        (dict(tree_masks=None), bad), (dict(tree_masks=FAKE + 8), bad), (dict(cu_new_lens=None), bad), (dict(window=5), bad),
        (dict(positions=FAKE + 4), bad), (dict(window=-1), bad), (dict(num_sinks=-1), bad), (dict(num_sinks=4), bad),
        (dict(softmax_scale=float("inf")), bad), (dict(q=None), bad), (dict(out=None), bad), (dict(workspace=None), bad), (dict(seq_lens=None), bad),
        (dict(page_table=None), bad), (dict(k_pool=None), bad), (dict(max_seq_len=1025), bad), (dict(num_pages=0), bad),
        (dict(out=(1 << 24) + 64), bad), (dict(layout=vq.make_layout(v_sub=8)), unsupported), (dict(layout=vq.make_layout(page_size=8)), bad)])
    for kw in (dict(batch=0), dict(num_tokens=0), dict(max_new_len=0)):  # nothing to do
        vq.vq_tree_attention(**dict(args, q=None, out=None, tree_masks=None, workspace=None, **kw))


def test_tree_workspace_bytes():
    for L in (vq.make_layout(), vq.make_layout(num_q_heads=40), vq.make_layout(num_q_heads=8), vq.make_layout(k_sub=8, k_bits=12, v_sub=8, v_bits=12)):
        sizes = [vq.vq_tree_workspace_bytes(L, 4, 4 * n, 1000, n, 152) for n in range(1, 257)]
        assert min(sizes) > 0 and all(n % 256 == 0 for n in sizes)
        assert sizes == sorted(sizes)  # a larger step's does for smaller ones
    for kw in ((-1, 4, 1000, 1), (4, -1, 1000, 1), (4, 4, -1, 1), (4, 4, 1000, -1)):
        assert vq.vq_tree_workspace_bytes(L, *kw, 152) == 0
    assert vq.vq_tree_workspace_bytes(vq.make_layout(v_sub=8), 4, 4, 1000, 1, 152) == 0


def test_append_kv_refusals():
    mk = vq.make_rotary
    args = dict(layout=vq.make_layout(num_q_heads=4, num_kv_heads=1), config=mk(), num_tokens=4, positions=FAKE, slot_mapping=FAKE + (1 << 12),
                dtype=vq.VQ_FP16, q=1 << 24, q_stride=512, k=1 << 26, k_stride=128, v=1 << 27, v_stride=256, lambda_=FAKE, codebook_k=FAKE,
                codebook_v=FAKE, q_out=1 << 25, k_pool=FAKE, v_pool=FAKE, num_pages=4)
    refused(vq.vq_append_kv, args, [
        (dict(config=mk(head_dim=64)), unsupported), (dict(config=mk(rotary_dim=33)), bad), (dict(config=mk(base=0.5)), bad),
        (dict(config=mk(attention_factor=0.0)), bad), (dict(config=mk(scaling="linear", factor=0.0)), bad), (dict(dtype=2), bad),
        (dict(layout=vq.make_layout(k_sub=1)), unsupported), (dict(layout=vq.make_layout(page_size=8)), bad), (dict(num_tokens=-1), bad),
        (dict(positions=None), bad), (dict(slot_mapping=None), bad), (dict(k=None), bad), (dict(v=None), bad), (dict(lambda_=None), bad),
        (dict(codebook_k=None), bad), (dict(codebook_v=None), bad), (dict(k_pool=None), bad), (dict(v_pool=None), bad), (dict(q=None), bad),
        (dict(q_out=None), bad), (dict(k=(1 << 26) + 8), bad), (dict(positions=FAKE + 4), bad), (dict(num_pages=0), bad),
        (dict(q_stride=511), bad), (dict(q_stride=504), bad), (dict(k_stride=120), bad), (dict(v_stride=129), bad),
        (dict(q_out=(1 << 24) + 1024), bad), (dict(q_out=1 << 26), bad), (dict(q_out=1 << 27), bad), (dict(q_out=1 << 24, q_stride=640), bad),
        (dict(q_out=1 << 24, dtype=vq.VQ_BF16), bad), (dict(q_out=FAKE), bad), (dict(q_out=FAKE + (1 << 12)), bad)])
    vq.vq_append_kv(**dict(args, num_tokens=0, positions=None, slot_mapping=None, k=None, v=None, q=None, q_out=None))  # no tokens: no-op


def test_keep_tokens_refusals():
    args = dict(layout=vq.make_layout(), batch=2, seq_lens=FAKE, cu_new_lens=FAKE, keep=FAKE, max_keep=3, keep_lens=FAKE, page_table=FAKE,
                max_pages_per_seq=4, num_pages=8, k_pools=[FAKE, FAKE], v_pools=[FAKE, FAKE], free_pages=FAKE, free_capacity=8, num_free=FAKE,
                seq_lens_out=FAKE, num_free_out=FAKE)
    refused(vq.vq_keep_tokens, args, [
        (dict(batch=-1), bad), (dict(batch=16385), unsupported), (dict(max_keep=-1), bad), (dict(max_keep=257), unsupported),
        (dict(k_pools=[], v_pools=[]), bad), (dict(k_pools=[FAKE] * 129, v_pools=[FAKE] * 129), unsupported),
        (dict(k_pools=[FAKE, None]), bad), (dict(v_pools=[FAKE + 8, FAKE]), bad), (dict(max_pages_per_seq=0), bad), (dict(num_pages=0), bad),
        (dict(free_capacity=-1), bad), (dict(seq_lens=None), bad), (dict(cu_new_lens=None), bad), (dict(keep=None), bad),
        (dict(keep_lens=None), bad), (dict(page_table=None), bad), (dict(free_pages=None), bad), (dict(num_free=None), bad),
        (dict(seq_lens_out=None), bad), (dict(num_free_out=None), bad), (dict(keep=FAKE + 4), bad), (dict(layout=vq.make_layout(page_size=8)), bad)])
    vq.vq_keep_tokens(**dict(args, batch=0, seq_lens=None, keep=None))
    with pytest.raises(ValueError, match="layers"):
        vq.vq_keep_tokens(**dict(args, k_pools=[FAKE]))


def test_a_tree_workspace_serves_every_call_within_its_bounds():
    """The tile height depends on all of batch, tokens and the longest sequence's; a workspace does not run short for smaller ones."""
    for L in (vq.make_layout(), vq.make_layout(num_q_heads=40, num_kv_heads=8), vq.make_layout(k_sub=8, k_bits=12, v_sub=8, v_bits=12)):
        for B, T, n in [(8, 300, 64), (8, 512, 64), (24, 1464, 61), (4, 1000, 250), (16, 100, 8), (1, 96, 96)]:
            most = vq.vq_tree_workspace_bytes(L, B, T, 5000, n, 152)
            for b in range(1, B + 1):
                for t in (1, T // 7, T // 3, T // 2, T):
                    for m in {min(m, n) for m in (1, 4, 8, 9, n // 3, n // 2, n - 1, n)}:
                        assert vq.vq_tree_workspace_bytes(L, b, t, 5000, m, 152) <= most, (B, T, n, b, t, m)
