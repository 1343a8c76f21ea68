"""Descriptors of a pool and a batch follow their owner: sizes that change, tensors that are
replaced, whatever address they get. Nothing here touches a GPU."""
import pytest
import torch

import sink_window_attention_b200 as swa


def pool(dtype="fp8", n=4, page=16, H=2, D=64):
    return swa.PagedKVCache(n, page, H, D, dtype, device="cpu")


def fields(c):
    return c.n_pages, c.page_size, c.H, c.D, c.dtype, c.k, c.v, c.k_scale, c.v_scale


def test_a_pool_that_grows():
    c = pool("bf16")
    c.to_c()
    for name in ("k", "v"):
        setattr(c, name, torch.zeros(9, 2, 16, 64, dtype=torch.bfloat16))
    c.n_pages = 9
    assert fields(c.to_c()) == (9, 16, 2, 64, swa.LL_BF16, c.k.data_ptr(), c.v.data_ptr(), None, None)


def test_a_look_without_a_device_keeps_the_descriptor():
    """(as the workspace's size asks for it between two calls)"""
    c = pool()
    a = c.to_c(-1)
    assert c.to_c() is a and c.to_c(-1) is a
    with pytest.raises(ValueError, match="CUDA"):
        c.to_c(0)


def test_sizes_are_part_of_what_is_kept():
    """Sizes that change under the same tensors: another descriptor, or a refusal."""
    c = pool("bf16")
    a = c.to_c()
    c.k, c.v = c.k.view(4, 2, 16, 64), c.v.view(4, 2, 16, 64)
    assert fields(c.to_c()) == fields(a)
    c.n_pages, c.page_size = 2, 32
    with pytest.raises(ValueError, match="k must be"):
        c.to_c()
    c.k, c.v = c.k.view(2, 2, 32, 64), c.v.view(2, 2, 32, 64)
    b = c.to_c()
    assert (b.n_pages, b.page_size) == (2, 32) and (a.n_pages, a.page_size) == (4, 16)
    c.n_pages = 1000
    with pytest.raises(ValueError, match="k must be"):
        c.to_c()


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
def test_a_pool_tensor_that_does_not_fit(name):
    c = pool()
    c.to_c()
    right = getattr(c, name)
    for wrong in (right[:3].clone(), right.to(torch.float64), right[..., None], None):
        setattr(c, name, wrong)
        with pytest.raises(ValueError, match=f"^{name} must be"):
            c.to_c()
        with pytest.raises(ValueError, match=f"^{name} must be"):
            c.to_c()
    setattr(c, name, right)
    assert c.to_c().n_pages == 4


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
def test_a_smaller_tensor_at_the_same_address(name):
    """What an allocator does with a pool that is replaced by a smaller one."""
    c = pool()
    c.to_c()
    whole = getattr(c, name)
    setattr(c, name, whole[:2])
    assert getattr(c, name).data_ptr() == whole.data_ptr() and getattr(c, name).is_contiguous()
    with pytest.raises(ValueError, match=f"^{name} must be"):
        c.to_c()
    # the same number of elements of a smaller type
    setattr(c, name, whole)
    c.to_c()
    if whole.dtype == torch.float32:
        setattr(c, name, whole.view(torch.uint8).view(-1)[:whole.numel()].view(whole.shape))
        with pytest.raises(ValueError, match=f"^{name} must be"):
            c.to_c()


def test_codes_by_their_own_type():
    c = pool()
    c.k = c.k.view(torch.float8_e4m3fn)
    assert c.to_c().k == c.k.data_ptr()
    c = pool("bf16")
    c.k = c.k.view(torch.uint8)[..., :64].contiguous().view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="^k must be"):
        c.to_c()


def test_a_resized_tensor():
    c = pool("bf16")
    c.to_c()
    c.k.resize_(2, 2, 16, 64)
    with pytest.raises(ValueError, match="^k must be"):
        c.to_c()


def test_a_tensor_transposed_in_place():
    c = pool("bf16")
    c.to_c(-1)
    c.v.transpose_(2, 3)
    with pytest.raises(ValueError):
        c.to_c(-1)


def test_scales_that_are_missing_or_left_over():
    c = pool("bf16")
    c.k_scale = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="k_scale"):
        c.to_c()
    c = pool()
    c.k_scale = c.v_scale = None
    with pytest.raises(ValueError, match="k_scale"):
        c.to_c()


def batch(B=3, pages=5):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return swa.TokenBatch(i32(B + 1), i32(B), i32(B, pages), 2, 64)


@pytest.mark.parametrize("name", ["q_start", "kv_len", "page_table"])
def test_a_batch_tensor_that_does_not_fit(name):
    """(-1 is the device of a host tensor, so that the descriptor itself is reached.)"""
    t = batch()
    a = t.to_c(6, -1)
    assert t.to_c(6, -1) is a and (a.B, a.max_pages, a.total_q) == (3, 5, 6)
    right = getattr(t, name)
    for wrong in (right[:2], right.long(), right.clone()[:1].contiguous(), None):
        setattr(t, name, wrong)
        with pytest.raises(ValueError, match=f"^{name} must be"):
            t.to_c(6, -1)
    setattr(t, name, right)
    assert t.to_c(6, -1).B == 3


def test_a_batch_whose_sizes_change():
    t = batch()
    t.to_c(6, -1)
    t.B = 4
    with pytest.raises(ValueError, match="must be"):
        t.to_c(6, -1)
    t.B, t.max_pages = 3, 50
    with pytest.raises(ValueError, match="page_table must be"):
        t.to_c(6, -1)
    t.page_table = torch.zeros(3, 50, dtype=torch.int32)
    t.max_q = 7
    c = t.to_c(6, -1)
    assert (c.max_pages, c.max_q, c.page_table) == (50, 7, t.page_table.data_ptr())


def test_a_rotation_in_place_of_what_autograd_tracks():
    x = torch.zeros(2, 2, 64)
    pos = torch.zeros(2, dtype=torch.int32)
    for a, out in ((x.clone().requires_grad_(), x), (x, x.clone().requires_grad_())):
        with pytest.raises(ValueError, match="requires grad"):
            swa.token_rope_apply(a, pos, swa.TokenRope(64), out=out)
    y = x.clone().requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        swa.token_rope_apply(y, pos, swa.TokenRope(64), out=y)


def test_inputs_that_require_grad_are_refused():
    """The append and the attention have no gradients: under grad mode they say so."""
    c, t = pool("bf16"), batch()
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    y = x.clone().requires_grad_()
    for call in (lambda: swa.paged_append(c, t, y, x), lambda: swa.paged_append(c, t, x, y),
                 lambda: swa.paged_attention(y, c, t), lambda: swa.paged_attention(x, c, t, out=y)):
        with pytest.raises(ValueError, match="no_grad"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # the next check: host tensors
            call()
