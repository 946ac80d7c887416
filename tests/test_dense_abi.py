"""Refusals of the exact-attention entry points: they answer before any device
call, so fake aligned pointers are enough.  CPU only."""
import ctypes

import pytest
import torch

from structured_sub_quadratic_b200 import _build, api

P = 1 << 30  # fake pointers, 1 GiB apart
BAD, UNSUPPORTED = api.MONARCH_ERR_INVALID_ARG, api.MONARCH_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return api.load_library()


def longs(*x):
    return (ctypes.c_longlong * len(x))(*x)


def fwd(lib, dtype=0, ptrs=None, sizes=(2, 4, 2, 16, 16, 64), strides=None, causal=0, lens=None,
        scale=0.125, ws=10 * P, ws_bytes=1 << 24):
    ptrs = [P, 2 * P, 3 * P, 4 * P, 5 * P] if ptrs is None else ptrs
    return lib.monarch_attn_dense_fwd(dtype, *ptrs, *sizes, strides, causal, lens, scale, ws,
                                      ws_bytes, None)


@pytest.mark.parametrize("change,expect", [
    (dict(dtype=2), BAD),
    (dict(sizes=(0, 4, 2, 16, 16, 64)), BAD),
    (dict(sizes=(2, 4, 3, 16, 16, 64)), BAD),       # 4 query heads over 3
    (dict(sizes=(2, 4, 2, -1, 16, 64)), BAD),
    (dict(sizes=(2, 4, 2, 16, 16, 0)), UNSUPPORTED),
    (dict(sizes=(2, 4, 2, 16, 16, 257)), UNSUPPORTED),
    (dict(sizes=(1 << 20, 1 << 9, 1, 1 << 20, 1, 64)), BAD),  # more tiles than a grid
    (dict(causal=2), BAD),
    (dict(scale=0.0), BAD),
    (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD),
    (dict(ptrs=[None, 2 * P, 3 * P, 4 * P, 5 * P]), BAD),
    (dict(ptrs=[P + 1, 2 * P, 3 * P, 4 * P, 5 * P]), BAD),    # half an element
    (dict(ptrs=[P, 2 * P, 3 * P, 4 * P, None]), BAD),         # no lse
    (dict(ptrs=[P, 2 * P, 3 * P, P + 64, 5 * P]), BAD),       # out over q
    (dict(ptrs=[P, 2 * P, 3 * P, 4 * P, 2 * P]), BAD),        # lse over k
    (dict(ptrs=[P, 2 * P, 3 * P, 4 * P, 4 * P + 256]), BAD),  # lse over out
    (dict(lens=P + 2), BAD),
    # one query over 4096 keys is split: too little workspace, none, over k
    (dict(sizes=(1, 4, 2, 1, 4096, 64), ws_bytes=64), BAD),
    (dict(sizes=(1, 4, 2, 1, 4096, 64), ws=None), BAD),
    (dict(sizes=(1, 4, 2, 1, 4096, 64), ws=2 * P), BAD),
    # out with repeated elements, and a negative stride
    (dict(strides=longs(4096, 1024, 64, 2048, 1024, 64, 2048, 1024, 64, 0, 1024, 64)), BAD),
    (dict(strides=longs(4096, 1024, 64, 2048, 1024, 64, 2048, 1024, 64, 4096, 1024, 32)), BAD),
    (dict(strides=longs(4096, -1024, 64, 2048, 1024, 64, 2048, 1024, 64, 4096, 1024, 64)), BAD),
])
def test_forward_refusals(lib, change, expect):
    assert fwd(lib, **change) == expect


def bwd(lib, ptrs=None, sizes=(2, 4, 2, 16, 16, 64), ws=10 * P, ws_bytes=1 << 20, scale=0.125):
    ptrs = [(i + 1) * P for i in range(9)] if ptrs is None else ptrs
    return lib.monarch_attn_dense_bwd(0, *ptrs, *sizes, None, 0, None, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("change", [
    dict(ws=None), dict(ws=10 * P + 8), dict(ws_bytes=2 * 4 * 16 * 4 - 1), dict(ws=P), dict(ws=7 * P),
    dict(scale=-1.0), dict(sizes=(2, 4, 0, 16, 16, 64)),
    dict(ptrs=[P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 8 * P, 8 * P + 64]),  # dk over dv
    dict(ptrs=[P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 4 * P, 8 * P, 9 * P]),       # dq over out
    dict(ptrs=[P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 5 * P, 8 * P, 9 * P]),       # dq over lse
    dict(ptrs=[P, 2 * P, 3 * P, 4 * P, None, 6 * P, 7 * P, 8 * P, 9 * P]),
])
def test_backward_refusals(lib, change):
    assert lib.monarch_attn_dense_fwd_workspace_bytes(0, 1, 4, 1, 4096, 64) > 0
    assert lib.monarch_attn_dense_fwd_workspace_bytes(0, 32, 12, 197, 197, 64) == 0
    assert lib.monarch_attn_dense_fwd_workspace_bytes(1, 1, 4, 1, 4096, 64) > 0
    assert lib.monarch_attn_dense_fwd_workspace_bytes(1, 1, 4, 1, 64, 64) == 0
    assert bwd(lib, **change) == BAD
    assert lib.monarch_attn_dense_bwd_workspace_bytes(2, 4, 16) == 2 * 4 * 16 * 4
    assert lib.monarch_attn_dense_bwd_workspace_bytes(0, 4, 16) == 0


def dec(lib, ptrs=None, sizes=(2, 4, 2, 64, 8, 16, 4), strides=None, scale=0.125, ws=10 * P,
        ws_bytes=1 << 24):
    ptrs = [(i + 1) * P for i in range(7)] if ptrs is None else ptrs
    return lib.monarch_attn_dense_decode(0, *ptrs, *sizes, strides, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("change,expect", [
    (dict(sizes=(0, 4, 2, 64, 8, 16, 4)), BAD),
    (dict(sizes=(2, 4, 3, 64, 8, 16, 4)), BAD),
    (dict(sizes=(2, 4, 2, 300, 8, 16, 4)), UNSUPPORTED),
    (dict(sizes=(2, 4, 2, 64, -1, 16, 4)), BAD),
    (dict(sizes=(2, 4, 2, 64, 8, 0, 4)), BAD),
    (dict(sizes=(2, 4, 2, 64, 8, 1 << 20, 1 << 11)), BAD),      # more than 2^30 keys
    (dict(scale=0.0), BAD),
    # 6400 keys are split: too little workspace, none, over the cache
    (dict(sizes=(2, 4, 2, 64, 800, 16, 400), ws_bytes=16), BAD),
    (dict(sizes=(2, 4, 2, 64, 800, 16, 400), ws=None), BAD),
    (dict(sizes=(2, 4, 2, 64, 800, 16, 400), ws=2 * P), BAD),
    (dict(ptrs=[P, 2 * P, 3 * P, None, 5 * P, 6 * P, 7 * P]), BAD),
    (dict(ptrs=[P, 2 * P, 3 * P, 4 * P, 5 * P + 1, 6 * P, 7 * P]), BAD),
    (dict(ptrs=[P, 2 * P, 3 * P, 4 * P, 5 * P, P, 7 * P]), BAD),  # out over q
    (dict(ptrs=[P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 5 * P]), BAD),  # lse over lens
])
def test_decode_refusals(lib, change, expect):
    assert dec(lib, **change) == expect


def rot(lib, ptrs=(P, 2 * P, 3 * P, 4 * P), sizes=(2, 4, 2, 16, 64), strides=None, axes=(64,),
        grid=None, positions=5 * P, step=0, freqs=None, magnitude=1.0, flags=(0, 0)):
    freqs = [1.0] * 32 if freqs is None else freqs
    return lib.monarch_attn_rotary(
        0, *ptrs, *sizes, strides, len(axes), (ctypes.c_int * len(axes))(*axes),
        None if grid is None else (ctypes.c_int * len(grid))(*grid), positions, step,
        (ctypes.c_double * len(freqs))(*freqs), magnitude, *flags, None)


PACKED = longs(*[16 * 768, 64, 768] * 4)  # views of a (B, N, 12, 64) projection


@pytest.mark.parametrize("change,expect", [
    (dict(sizes=(2, 0, 0, 16, 64)), BAD),
    (dict(sizes=(2, 4, 2, 16, 300)), UNSUPPORTED),
    (dict(axes=(63,)), BAD),
    (dict(axes=(64, 2)), BAD),                            # 66 of 64 channels
    (dict(axes=(2,) * 5), UNSUPPORTED),
    (dict(grid=(16,)), BAD),                              # grid and positions
    (dict(positions=None), BAD),                          # neither
    (dict(positions=None, grid=(15,)), BAD),
    (dict(positions=5 * P + 2), BAD),
    (dict(step=15), BAD),
    (dict(freqs=[float("inf")] * 32), BAD),
    (dict(magnitude=float("nan")), BAD),
    (dict(flags=(2, 0)), BAD),
    (dict(ptrs=(P, 2 * P, P + 128, 4 * P)), BAD),         # q_out shifted over q
    (dict(ptrs=(P, 2 * P, 2 * P, 4 * P)), BAD),           # q_out over k
    (dict(ptrs=(P, 2 * P, 3 * P, 3 * P)), BAD),           # both outputs in one place
    (dict(ptrs=(P, 2 * P, 5 * P, 4 * P)), BAD),           # q_out over the positions
    # in place in one projection, k's heads over q's last one
    (dict(ptrs=(P, P + 3 * 128, P, P + 3 * 128), strides=PACKED), BAD),
])
def test_rotary_refusals(lib, change, expect):
    assert rot(lib, **change) == expect


def test_empty_calls_launch_nothing(lib):
    assert rot(lib, sizes=(2, 4, 2, 0, 64), ptrs=(None,) * 4) == api.MONARCH_OK
    assert fwd(lib, sizes=(2, 4, 2, 0, 16, 64), ptrs=[None, 2 * P, 3 * P, None, None]) == \
        api.MONARCH_OK
    assert lib.monarch_attn_last_launches() == 0


def test_binding_refuses_host_tensors_and_odd_arguments():
    q = torch.zeros(1, 2, 4, 8)
    with pytest.raises(ValueError):
        api.monarch_attn_dense_fwd(q, q, q)
    with pytest.raises(ValueError):
        api.monarch_attn_dense_fwd(q, q[:, :, :, :4], q)
    with pytest.raises(ValueError):
        api.monarch_attn_dense_bwd(q, q, q, q, q[..., 0], q)
    with pytest.raises(ValueError):
        api.monarch_attn_dense_decode(q[:, :, 0], q, q, torch.zeros(1, 1, dtype=torch.int32),
                                      torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        api.monarch_attn_rotary(q, q, grid=(4,))
    with pytest.raises(ValueError):
        api.monarch_attn_rotary(q, q, grid=(4,), axis_dims=(3,))
    assert b"page" in api.load_library().monarch_attn_strerror(api.MONARCH_ERR_BAD_INDEX)
