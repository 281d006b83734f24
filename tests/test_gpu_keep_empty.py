"""Keeping tokens of an empty batch: the free stack's size is the one that came in."""
import pytest

torch = pytest.importorskip("torch")
import bit_vector_quantized_gb300 as vq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("stream", [False, True])
def test_an_empty_batch(given, stream):
    layout = vq.make_layout(128, 8, 2, 4, 8, 4, 8, 16)
    kp, vp = vq.alloc_pools(layout, 9)
    i32 = dict(dtype=torch.int32, device="cuda")
    e, num_free = torch.empty(0, **i32), torch.tensor([5], **i32)
    torch.full((1,), 77, **i32)  # (what a new tensor may find)
    out = torch.tensor([-3], **i32) if given else None
    s = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    r = vq.keep_tokens(layout, e, torch.zeros(1, **i32), torch.empty((0, 4), **i32), e, torch.empty((0, 3), **i32), [kp], [vp],
                       torch.arange(9, **i32), num_free, num_free_out=out, stream=s)
    torch.cuda.synchronize()
    assert r.seq_lens.shape == (0,) and int(r.num_free) == 5 and int(num_free) == 5
    assert out is None or r.num_free is out


def test_an_empty_batch_in_place():
    layout = vq.make_layout(128, 8, 2, 4, 8, 4, 8, 16)
    kp, vp = vq.alloc_pools(layout, 9)
    i32 = dict(dtype=torch.int32, device="cuda")
    e, num_free = torch.empty(0, **i32), torch.tensor([5], **i32)
    r = vq.keep_tokens(layout, e, torch.zeros(1, **i32), torch.empty((0, 4), **i32), e, torch.empty((0, 3), **i32), [kp], [vp],
                       torch.arange(9, **i32), num_free, seq_lens_out=e, num_free_out=num_free)
    torch.cuda.synchronize()
    assert r.num_free is num_free and int(num_free) == 5
