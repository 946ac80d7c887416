"""Exact attention where values are not numbers."""
import pytest
import torch

from test_gpu_dense import BF16, F32, decode_case, dense_case

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


# --------------------------------------------------------------------------
# a NaN or an infinite score among the visible keys
# --------------------------------------------------------------------------
@pytest.mark.parametrize("fill", [NAN, INF])
@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 24), (BF16, 128), (BF16, 72), (BF16, 200),
                                     (F32, 64)])
@pytest.mark.parametrize("Nq,Nk,first", [(70, 150, 0), (70, 150, 75), (300, 700, 530),
                                         (2, 2600, 1290)])
def test_no_key_hides_a_nan(cuda_lib, Nq, Nk, first, dtype, d, fill):
    """Head h has it in key first + h alone: each of its rows is NaN, whatever
    the key's place in a tile, and the last head is as it was."""
    H = 17
    q, k, v, _, _ = dense_case(1, H, H, Nq, Nk, d, False, None, "head", dtype)
    q[..., 0] = q[..., 0].abs() + 1  # an infinite key scores +inf: exp(inf - inf)
    clean, clean_lse = cuda_lib.monarch_attn_dense_fwd(q, k, v)
    for h in range(H - 1):
        k[0, h, first + h, 0] = fill
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v)
    cuda_lib.check()
    assert torch.isnan(out[:, :-1]).all() and torch.isnan(lse[:, :-1]).all()
    assert torch.equal(out[:, -1], clean[:, -1]) and torch.equal(lse[:, -1], clean_lse[:, -1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,Hkv", [(16, 16), (40, 2)])
@pytest.mark.parametrize("keys", [150, 3000])
def test_no_cached_key_hides_a_nan(cuda_lib, keys, H, Hkv, dtype):
    q, k, v, table, lens = decode_case(1, H, Hkv, [keys], 16, 64, dtype)
    clean, _ = cuda_lib.monarch_attn_dense_decode(q, k, v, table, lens)
    for h in range(Hkv - 1):
        j = keys - 40 + h
        k[table[0, j // 16].item(), h, j % 16, 3] = NAN
    out, lse = cuda_lib.monarch_attn_dense_decode(q, k, v, table, lens)
    cuda_lib.check()
    last = H - H // Hkv
    assert torch.isnan(out[:, :last]).all() and torch.isnan(lse[:, :last]).all()
    assert torch.equal(out[:, last:], clean[:, last:])
