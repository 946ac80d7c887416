"""Refusals of the exact-attention entry points that concern arguments beside
q, k and v (fake pointers, as no device call is made).  CPU only."""
import pytest
import torch

from structured_sub_quadratic_b200 import _build, api

P = 1 << 30  # fake pointers, 1 GiB apart


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return api.load_library()


@pytest.mark.parametrize("sizes,lens", [
    ((2, 4, 2, 16, 16, 64), 4 * P + 64),            # out
    ((2, 4, 2, 16, 16, 64), 5 * P + 4),             # lse
    ((2, 4, 2, 16, 16, 64), 5 * P + 2 * 4 * 16 * 4 - 4),  # its last element
    ((2, 4, 2, 16, 16, 64), 5 * P - 4),             # the second length in its first one
    ((1, 4, 2, 1, 4096, 64), 10 * P + 128),         # the workspace of a split call
])
def test_forward_refuses_outputs_over_the_lengths(lib, sizes, lens):
    assert lib.monarch_attn_dense_fwd(0, P, 2 * P, 3 * P, 4 * P, 5 * P, *sizes, None, 0, lens,
                                      0.125, 10 * P, 1 << 24, None) == api.MONARCH_ERR_INVALID_ARG


@pytest.mark.parametrize("lens", [7 * P + 4, 8 * P, 9 * P + 8, 10 * P + 4, 7 * P - 4])
def test_backward_refuses_outputs_over_the_lengths(lib, lens):
    ptrs = [(i + 1) * P for i in range(9)]  # ..., dq, dk, dv
    assert lib.monarch_attn_dense_bwd(0, *ptrs, 2, 4, 2, 16, 16, 64, None, 0, lens, 0.125, 10 * P,
                                      1 << 20, None) == api.MONARCH_ERR_INVALID_ARG


def test_text_of_a_bad_index_says_what_the_kernels_do(lib):
    """Keys of a page outside the cache are zeros, and stay in the softmax."""
    text = lib.monarch_attn_strerror(api.MONARCH_ERR_BAD_INDEX)
    assert b"zero" in text and b"left out" not in text


@pytest.mark.parametrize("shape,strides", [
    ((1, 1, 3, 8), (100, 100, 1, 1)),      # windows that step by one channel
    ((2, 1, 16, 8), (1, 100, 8, 1)),       # sequences that do
    ((2, 3, 16, 8), (1, 1, 8, 1)),
    ((2, 3, 16, 8), (384, 8, 24, 1)),      # token-major
    ((2, 3, 16, 8), (0, 0, 8, 1)),         # broadcast
    ((2, 3, 16, 1), (48, 16, 1, 7)),       # one channel
])
def test_results_have_contiguous_channels(shape, strides):
    """Whatever the strides of an input, what is allocated like it can be written."""
    t = torch.zeros(1000).as_strided(shape, strides)
    y = api._like(t)
    assert y.shape == t.shape and (y.stride(-1) == 1 or shape[-1] == 1)
    # distinct elements
    y.copy_(torch.arange(float(y.numel())).view(shape))
    assert torch.equal(y.flatten(), torch.arange(float(y.numel())))
