"""Exact attention where values are not numbers, scores are infinite, pages lie
outside the cache, sums cancel, rows overlap or offsets pass 32 bits."""
import numpy as np
import pytest
import torch

from oracle import dense_ref
from test_gpu_dense import BF16, F32, close, decode_bounds, decode_case, dense_case, f64, half_step

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


# --------------------------------------------------------------------------
# scores of -inf
# --------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 24, 128])
@pytest.mark.parametrize("Nq,Nk", [(70, 150), (200, 600), (2, 2600)])
def test_scores_of_minus_infinity(cuda_lib, Nq, Nk, d):
    """Keys that score -inf weigh nothing; a row that has no others is a row
    without keys, in one range of keys or several, and takes no part in the
    gradients."""
    q, k, v, do, _ = dense_case(1, 3, 3, Nq, Nk, d, False, None, "head", BF16)
    q[..., 0] = q[..., 0].abs() + 1
    k[0, 0, :, 0] = -INF                     # every key of head 0
    gone = torch.arange(Nk, device="cuda") % 7 < 3
    k[0, 1, gone, 0] = -INF                  # some keys of head 1
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v)
    _, dk, dv = cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do)
    cuda_lib.check()
    assert (out[0, 0] == 0).all() and torch.isneginf(lse[0, 0]).all()
    assert (dk[0, 0] == 0).all() and (dv[0, 0] == 0).all()
    for h, kept in ((1, ~gone), (2, torch.ones_like(gone))):
        x = [f64(t) for t in (q[:, h:h + 1], k[:, h:h + 1, kept], v[:, h:h + 1, kept],
                              do[:, h:h + 1])]
        refs = (*dense_ref.dense_forward(*x[:3]), *dense_ref.dense_backward(*x)[1:])
        eO, eL, _, eK, eV = dense_ref.dense_errors(*x, half_step(BF16))
        got = (out[:, h:h + 1], lse[:, h:h + 1], dk[:, h:h + 1, kept], dv[:, h:h + 1, kept])
        # (a sum of all keys for one of the kept ones: 7 / 4 of its terms)
        for name, a, ref, e in zip(("out", "lse", "dk", "dv"), got, refs, (eO, eL, eK, eV)):
            close(name, a, ref, 1.75 * e)


@pytest.mark.parametrize("Nq,Nk", [(40, 100), (2, 2000)])
def test_scores_that_overflow(cuda_lib, Nq, Nk):
    """fp32 scores of -1e40 are -inf: rows without keys, split or not."""
    q, v, do = (torch.full((1, 2, n, 32), x, device="cuda")
                for n, x in ((Nq, 1e20), (Nk, 1.0), (Nq, 1.0)))
    k = torch.full_like(v, -1e20)
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v)
    grads = cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do)
    cuda_lib.check()
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert all((g == 0).all() for g in grads)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (40, 2)])
@pytest.mark.parametrize("keys", [100, 3000])
def test_cached_scores_of_minus_infinity(cuda_lib, keys, H, Hkv, dtype):
    q, k, v, table, lens = decode_case(1, H, Hkv, [keys], 16, 64, dtype)
    q[..., 0] = q[..., 0].abs() + 1
    clean, _ = cuda_lib.monarch_attn_dense_decode(q, k, v, table, lens)
    k[:, 0, :, 0] = -INF
    out, lse = cuda_lib.monarch_attn_dense_decode(q, k, v, table, lens)
    cuda_lib.check()
    first = H // Hkv
    assert (out[:, :first] == 0).all() and torch.isneginf(lse[:, :first]).all()
    assert torch.equal(out[:, first:], clean[:, first:])


# --------------------------------------------------------------------------
# pages outside the cache
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys,page", [(100, 16), (100, 7), (2500, 64)])
def test_keys_of_bad_pages_are_zero(cuda_lib, keys, page, dtype):
    """A page outside the cache stands for zero keys and values, which score 0."""
    q, k, v, table, lens = decode_case(2, 4, 2, [keys, 20], page, 64, dtype, spare=3)
    spare = torch.ones(k.shape[0], dtype=torch.bool, device="cuda")
    spare[table.flatten().long()] = False
    zero = int(spare.nonzero()[0])
    k[zero], v[zero] = 0, 0
    bad, ref = table.clone(), table.clone()
    bad[0, 1], bad[0, 3] = -1, k.shape[0]
    ref[0, 1], ref[0, 3] = zero, zero
    out, lse = cuda_lib.monarch_attn_dense_decode(q, k, v, bad, lens)
    with pytest.raises(cuda_lib.MonarchError) as exc:
        cuda_lib.check()
    assert exc.value.status == cuda_lib.MONARCH_ERR_BAD_INDEX
    x = [f64(t) for t in (q, k, v)]
    O, L, A = dense_ref.decode(*x, ref.cpu().numpy(), lens.tolist())
    eO, eL = decode_bounds(*x, O, A, lens.tolist(), dtype)
    close("out", out, O, eO)
    close("lse", lse, L, np.full(L.shape, eL))
    assert all(torch.equal(a, b) for a, b in zip(
        (out, lse), cuda_lib.monarch_attn_dense_decode(q, k, v, ref, lens)))
    cuda_lib.check()


# --------------------------------------------------------------------------
# values with a large common part
# --------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nk,causal,lens", [(300, False, None), (600, False, [36, 600, 129]),
                                            (700, True, None), (1100, True, [1100, 512, 90])])
def test_gradients_of_rows_with_few_keys(cuda_lib, Nk, causal, lens, d):
    """Values of 256 or 258: dO V^T - delta cancels all but the 2, and a delta
    from out, rounded to a multiple of 2, would be off by as much.  Rows that
    see up to 512 keys take it from the probabilities, however long the
    tensors of their batch are."""
    B = 1 if lens is None else len(lens)
    q, k, v, do, kl = dense_case(B, 2, 1, Nk, Nk, d, causal, lens, "head", BF16)
    v = 256 + 2 * (v > 0).to(BF16)
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v, causal=causal, k_lens=kl)
    dq, dk, _ = cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do, causal=causal, k_lens=kl)
    cuda_lib.check()
    x = [f64(t) for t in (q, k, v, do)]
    # the keys that the last row of each row's tile of 128 sees
    last = np.minimum(np.arange(Nk) // 128 * 128 + 127, Nk - 1)
    sees = np.minimum(np.reshape([Nk] * B if lens is None else lens, (B, 1)),
                      last + 1 if causal else Nk)
    few = np.broadcast_to(sees <= 512, (B, Nk))[:, None]
    refs = dense_ref.dense_backward(*x, causal, lens)
    bounds = dense_ref.dense_errors(*x, half_step(BF16), causal, lens, exact_delta=few)
    close("dq", dq, refs[0], bounds[2])
    close("dk", dk, refs[1], bounds[3])


# --------------------------------------------------------------------------
# layouts
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,Nq,Nk,causal", [(12, 300, 520, True), (24, 520, 130, False)])
def test_one_key_head_for_many(cuda_lib, H, Nq, Nk, causal, dtype):
    q, k, v, do, _ = dense_case(1, H, 1, Nq, Nk, 128, causal, None, "token", dtype)
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v, causal=causal)
    grads = cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do, causal=causal)
    cuda_lib.check()
    x = [f64(t) for t in (q, k, v, do)]
    refs = (*dense_ref.dense_forward(*x[:3], causal), *dense_ref.dense_backward(*x, causal))
    bounds = dense_ref.dense_errors(*x, half_step(dtype), causal, rounded_weights=dtype is BF16)
    for name, got, ref, bound in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads), refs,
                                     bounds):
        close(name, got, ref, bound)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Nq,step", [(3, 1), (20, 8), (20, 3)])
def test_rows_that_overlap(cuda_lib, Nq, step, dtype):
    """Rows that are windows of one signal give what their copies give."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(4000, generator=g, device="cuda").to(dtype)
    q, k, v = (x[o:].as_strided((1, 2, n, 32), (700, 350, step, 1))
               for o, n in ((0, Nq), (1400, 25), (2800, 25)))
    do = torch.randn(1, 2, Nq, 32, generator=g, device="cuda").to(dtype)
    a = cuda_lib.monarch_attn_dense_fwd(q, k, v)
    grads = cuda_lib.monarch_attn_dense_bwd(q, k, v, *a, do)
    turned = cuda_lib.monarch_attn_rotary(q, grid=(Nq,))[0]
    cuda_lib.check()
    c = [t.contiguous() for t in (q, k, v)]
    x = [f64(t) for t in (*c, do)]
    refs = (*dense_ref.dense_forward(*x[:3]), *dense_ref.dense_backward(*x))
    bounds = dense_ref.dense_errors(*x, half_step(dtype), rounded_weights=dtype is BF16)
    for name, got, ref, bound in zip(("out", "lse", "dq", "dk", "dv"), (*a, *grads), refs, bounds):
        close(name, got, ref, bound)
    assert torch.equal(turned, cuda_lib.monarch_attn_rotary(c[0], grid=(Nq,))[0])


def far(t, dim):
    """t in a buffer of its own where dimension `dim` steps so far that its last
    entry starts above 2^31 elements."""
    rest = list(t.shape)
    n = rest.pop(dim)
    strides = list(torch.empty(rest, device="meta").stride())
    step = (2**31 // (n - 1) + 128) // 128 * 128
    strides.insert(dim, step)
    view = torch.empty(step * (n - 1) + t.numel(), device="cuda", dtype=t.dtype) \
        .as_strided(t.shape, strides)
    assert step * (n - 1) >= 2**31
    return view.copy_(t)


@pytest.mark.parametrize("dim", [0, 1, 2])
@pytest.mark.parametrize("dtype,d", [(BF16, 64), (F32, 64)])
def test_offsets_above_32_bits(cuda_lib, dtype, d, dim):
    q, k, v, do, _ = dense_case(2, 2, 2, 130, 140, d, True, None, "head", dtype)
    ref = cuda_lib.monarch_attn_dense_fwd(q, k, v, causal=True)
    grads = cuda_lib.monarch_attn_dense_bwd(q, k, v, *ref, do, causal=True)
    turned = cuda_lib.monarch_attn_rotary(q, grid=(130,))[0]
    fq, fk, fv, fo = (far(t, dim) for t in (q, k, v, q))
    got = cuda_lib.monarch_attn_dense_fwd(fq, fk, fv, causal=True, out=fo)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    fg = cuda_lib.monarch_attn_dense_bwd(fq, fk, fv, *got, far(do, dim), causal=True)
    assert all(torch.equal(a, b) for a, b in zip(fg, grads))
    cuda_lib.monarch_attn_rotary(fq, grid=(130,), q_out=fo)
    assert torch.equal(fo, turned)
    cuda_lib.check()


@pytest.mark.parametrize("dim", [0, 1, 2])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cache_offsets_above_32_bits(cuda_lib, dtype, dim):
    q, k, v, table, lens = decode_case(2, 4, 2, [100, 70], 16, 64, dtype, "head")
    ref = cuda_lib.monarch_attn_dense_decode(q, k, v, table, lens)
    got = cuda_lib.monarch_attn_dense_decode(q, far(k, dim), far(v, dim), table, lens)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    cuda_lib.check()
