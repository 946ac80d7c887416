"""Exact attention, paged decode and rotary positions on the GPU against their
float64 forms.

Tolerances are element by element and derived from the arithmetic
(oracle/dense_ref.py: every output rounded once to its type, weights of the
bf16 products rounded once more, everything else fp32).
"""
import numpy as np
import pytest
import torch

from oracle import dense_ref
from structured_sub_quadratic_b200.inputs import video_qkv

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(x):
    return x.detach().double().cpu().numpy()


def heads(g, B, H, N, d, dtype, order="head"):
    """(B, H, N, d) on the GPU: contiguous, token-major, or a slice of wider rows."""
    if order == "head":
        return torch.randn(B, H, N, d, generator=g, device="cuda").to(dtype)
    if order == "token":
        return torch.randn(B, N, H, d, generator=g, device="cuda").to(dtype).transpose(1, 2)
    # rows and pointers of odd alignment
    return torch.randn(B, H, N, d + 3, generator=g, device="cuda").to(dtype)[..., 1:d + 1]


def close(name, got, ref, bound):
    got = f64(got)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{name}: infinities differ"
    assert np.isfinite(got[~inf]).all(), f"{name}: not finite"
    over = (np.abs(got[~inf] - ref[~inf]) - bound[~inf]).max(initial=0.0)
    assert over <= 1e-30, f"{name}: {over:.3e} above its bound"


CASES = [
    # B, H, Hkv, Nq, Nk, d, causal, lens, order
    (1, 1, 1, 1, 1, 64, False, None, "head"),
    (1, 2, 2, 16, 16, 64, True, None, "head"),
    (2, 3, 3, 197, 197, 64, False, None, "token"),
    (1, 4, 2, 128, 128, 128, True, None, "head"),
    (2, 6, 2, 129, 257, 128, True, [257, 100], "token"),
    (3, 2, 1, 130, 130, 64, True, [0, 1, 130], "head"),     # an empty sequence, one key
    (1, 2, 2, 300, 90, 128, True, None, "head"),            # the first 210 rows see nothing
    (1, 2, 1, 90, 300, 64, False, [0], "head"),             # no key at all
    (2, 2, 2, 65, 383, 128, False, [128, 256], "head"),     # lengths at tile ends
    (1, 8, 1, 1, 500, 128, True, None, "token"),            # one query
    (1, 2, 2, 33, 70, 80, True, [69], "token"),             # d between the tile widths
    (1, 3, 1, 200, 140, 40, False, None, "head"),
    (1, 2, 2, 40, 50, 24, True, None, "head"),
    (2, 2, 1, 140, 150, 8, False, [150, 9], "token"),       # the smallest rows of 16 bytes
    (1, 1, 1, 20, 30, 7, True, None, "head"),               # d odd
    (1, 2, 1, 70, 100, 200, False, [99], "head"),           # d above the tensor-core tiles
    (1, 1, 1, 40, 33, 256, True, None, "head"),
    (1, 2, 2, 70, 100, 64, True, None, "odd"),              # unaligned rows
    (2, 2, 1, 520, 520, 64, True, [520, 391], "head"),      # several tiles of either axis
    (1, 40, 8, 40, 330, 64, True, [300], "token"),          # many short heads
    (1, 60, 60, 300, 260, 16, False, None, "head"),
    # few queries over many keys: split over the keys and joined
    (1, 1, 1, 1, 2000, 64, False, None, "head"),
    (2, 2, 1, 70, 2500, 128, True, [2500, 700], "token"),   # ranges that one batch never reaches
    (1, 4, 2, 130, 1300, 80, True, None, "head"),
    (2, 1, 1, 3, 1100, 40, False, [0, 1], "head"),
]


def dense_case(B, H, Hkv, Nq, Nk, d, causal, lens, order, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 131 * Nq + Nk + d)
    q, do = (heads(g, B, H, Nq, d, dtype, order) for _ in range(2))
    k, v = (heads(g, B, Hkv, Nk, d, dtype, order) for _ in range(2))
    kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    return q, k, v, do, kl


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:7])))
def test_dense_forward_and_gradients(cuda_lib, case, dtype):
    B, H, Hkv, Nq, Nk, d, causal, lens, order = case
    q, k, v, do, kl = dense_case(*case, dtype)
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v, causal=causal, k_lens=kl)
    assert cuda_lib.last_launches() > 0
    grads = cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do, causal=causal, k_lens=kl)
    cuda_lib.check()
    x = [f64(t) for t in (q, k, v, do)]
    refs = (*dense_ref.dense_forward(*x[:3], causal, lens),
            *dense_ref.dense_backward(*x, causal, lens))
    bounds = dense_ref.dense_errors(*x, half_step(dtype), causal, lens,
                                    rounded_weights=dtype is BF16)
    for name, got, ref, bound in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads), refs,
                                     bounds):
        close(name, got, ref, bound)
    assert out.dtype == dtype and all(a.shape == b.shape for a, b in zip(grads, (q, k, v)))


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (BF16, 200), (F32, 64)])
def test_keys_past_the_length_are_never_used(cuda_lib, dtype, d):
    """NaN and infinities past the lengths change nothing, bit for bit."""
    lens = [77, 0, 200]
    q, k, v, do, kl = dense_case(3, 4, 2, 150, 200, d, True, lens, "head", dtype)
    results = []
    for fill in (0.0, float("nan"), float("inf")):
        kk, vv = k.clone(), v.clone()
        for b, n in enumerate(lens):
            kk[b, :, n:] = fill
            vv[b, :, n:] = -fill
        out, lse = cuda_lib.monarch_attn_dense_fwd(q, kk, vv, causal=True, k_lens=kl)
        results.append((out, lse, *cuda_lib.monarch_attn_dense_bwd(q, kk, vv, out, lse, do,
                                                                   causal=True, k_lens=kl)))
    cuda_lib.check()
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
    _, _, dq, dk, dv = results[0]
    assert (dq[1] == 0).all() and (dk[1] == 0).all()
    assert (dk[0, :, 77:] == 0).all() and (dv[0, :, 77:] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores_and_scale(cuda_lib, dtype):
    """Scores of hundreds: the running maximum carries the softmax."""
    q, k, v, do, _ = dense_case(1, 2, 1, 140, 300, 64, False, None, "head", dtype)
    q = (q.float() * 12).to(dtype)
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v, scale=0.5)
    grads = cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do, scale=0.5)
    x = [f64(t) for t in (q, k, v, do)]
    refs = (*dense_ref.dense_forward(*x[:3], scale=0.5),
            *dense_ref.dense_backward(*x, scale=0.5))
    bounds = dense_ref.dense_errors(*x, half_step(dtype), scale=0.5,
                                    rounded_weights=dtype is BF16)
    for name, got, ref, bound in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads), refs,
                                     bounds):
        close(name, got, ref, bound)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (F32, 32)])
def test_gradient_against_differences_of_the_kernel(cuda_lib, dtype, d):
    """The directional derivative of the fp32-summed loss, by differences of
    the float64 form, agrees with the gradients within their bounds."""
    q, k, v, do, _ = dense_case(1, 2, 2, 60, 60, d, True, None, "head", dtype, seed=5)
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v, causal=True)
    grads = [f64(t) for t in cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do, causal=True)]
    x = [f64(t) for t in (q, k, v, do)]
    bounds = dense_ref.dense_errors(*x, half_step(dtype), True, rounded_weights=dtype is BF16)[2:]
    r = np.random.default_rng(0)
    for a in range(3):
        u = r.standard_normal(x[a].shape)
        h = 1e-5
        up, down = ([t + (h * u if i == a else 0) * s for i, t in enumerate(x[:3])]
                    for s in (1, -1))
        slope = ((dense_ref.dense_forward(*up, True)[0] -
                  dense_ref.dense_forward(*down, True)[0]) * x[3]).sum() / (2 * h)
        bound = (bounds[a] * np.abs(u)).sum() + 1e-6 * np.abs(grads[a] * u).sum()
        assert abs((grads[a] * u).sum() - slope) <= bound


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_broadcast_inputs(cuda_lib, dtype):
    """Keys and values expanded over the batch, queries over the heads."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(2, 1, 150, 64, generator=g, device="cuda").to(dtype).expand(2, 4, 150, 64)
    k, v = (torch.randn(1, 2, 170, 64, generator=g, device="cuda").to(dtype).expand(2, 2, 170, 64)
            for _ in range(2))
    do = torch.randn(2, 4, 150, 64, generator=g, device="cuda").to(dtype)
    a = cuda_lib.monarch_attn_dense_fwd(q, k, v)
    b = cuda_lib.monarch_attn_dense_fwd(*(t.contiguous() for t in (q, k, v)))
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    ga = cuda_lib.monarch_attn_dense_bwd(q, k, v, *a, do)
    gb = cuda_lib.monarch_attn_dense_bwd(*(t.contiguous() for t in (q, k, v)), *b, do)
    assert all(torch.equal(s, t) for s, t in zip(ga, gb))
    assert ga[0].shape == q.shape and ga[1].shape == k.shape


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_repeats_are_bit_identical_and_leave_neighbours_alone(cuda_lib, dtype):
    q, k, v, do, kl = dense_case(2, 4, 2, 333, 333, 64, True, [333, 200], "token", dtype)
    wide = torch.full((2, 4, 340, 72), 7.0, device="cuda", dtype=dtype)
    out = wide[:, :, 3:336, 8:]
    for _ in range(2):
        cuda_lib.monarch_attn_dense_fwd(q, k, v, causal=True, k_lens=kl, out=out)
        first = out.clone()
    ref, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v, causal=True, k_lens=kl)
    assert torch.equal(out, first) and torch.equal(out, ref)
    rest = wide.clone()
    rest[:, :, 3:336, 8:] = 7.0
    assert (rest == 7.0).all()
    a, b = (cuda_lib.monarch_attn_dense_bwd(q, k, v, ref, lse, do, causal=True, k_lens=kl)
            for _ in range(2))
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("d,H,N,causal", [(64, 40, 700, False), (128, 40, 700, True),
                                          (64, 300, 130, True), (128, 20, 1900, False)])
def test_more_ctas_than_the_device_holds(cuda_lib, d, H, N, causal):
    """Waves of CTAs beside each other on an SM, softmaxes ahead of the
    products and behind: each head as it is alone."""
    q, k, v, do, _ = dense_case(1, H, H, N, N, d, causal, None, "head", BF16, seed=3)
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v, causal=causal)
    grads = cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do, causal=causal)
    cuda_lib.check()
    for h in (0, H // 2, H - 1):
        x = [f64(t[:, h:h + 1]) for t in (q, k, v, do)]
        refs = (*dense_ref.dense_forward(*x[:3], causal), *dense_ref.dense_backward(*x, causal))
        bounds = dense_ref.dense_errors(*x, half_step(BF16), causal)
        for name, got, ref, bound in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads),
                                         refs, bounds):
            close(name, got[:, h:h + 1], ref, bound)


def test_empty_queries_and_keys(cuda_lib):
    q, k, v, do, _ = dense_case(1, 2, 2, 5, 0, 64, False, None, "head", BF16)
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v)
    dq, dk, dv = cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do)
    assert (out == 0).all() and torch.isneginf(lse).all() and (dq == 0).all()
    assert dk.numel() == dv.numel() == 0
    q, k, v, do, _ = dense_case(1, 2, 2, 0, 5, 64, False, None, "head", BF16)
    out, lse = cuda_lib.monarch_attn_dense_fwd(q, k, v)
    dq, dk, dv = cuda_lib.monarch_attn_dense_bwd(q, k, v, out, lse, do)
    assert out.numel() == dq.numel() == 0 and (dk == 0).all() and (dv == 0).all()
    cuda_lib.check()


# --------------------------------------------------------------------------
# paged decode
# --------------------------------------------------------------------------
def decode_case(B, H, Hkv, lens, page, d, dtype, major="token", seed=0, spare=2):
    g = torch.Generator(device="cuda").manual_seed(seed + page + d)
    per = max(1, -(-max(lens) // page)) + 1
    pages = B * per + spare
    shape = (pages, page, Hkv, d) if major == "token" else (pages, Hkv, page, d)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2))
    if major == "token":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = order[:B * per].view(B, per).contiguous()
    q = torch.randn(B, H, d, generator=g, device="cuda").to(dtype)
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def decode_bounds(q, k, v, O, A, lens, dtype):
    """As dense_errors, with the largest score bounded by the largest norms."""
    eps, d = 2.0 ** -23, q.shape[-1]
    s = np.abs(q).sum(-1).max() * np.abs(k).max() / np.sqrt(d)
    worst = 2 * (d + 8) * eps * s
    e = worst + 2.0 ** -21 + 2 * max(lens) * eps
    w = half_step(dtype) if dtype is BF16 else 0
    return half_step(dtype) * np.abs(O) + (w + e) * A, e + 30 * eps


DECODE = [
    # B, H, Hkv, lens, page, d, major
    (1, 1, 1, [1], 1, 64, "token"),
    (3, 4, 4, [17, 0, 33], 16, 64, "token"),
    (2, 8, 2, [1000, 129], 64, 128, "head"),
    (2, 12, 1, [300, 257], 24, 128, "token"),      # 12 shared heads, pages that cross tiles
    (1, 40, 2, [700], 128, 128, "head"),           # 20 shared heads
    (4, 2, 1, [5, 64, 65, 63], 256, 96, "token"),
    (2, 6, 3, [90, 91], 7, 80, "head"),
    (1, 2, 2, [130], 16, 7, "token"),              # d odd
    (1, 4, 2, [260], 32, 256, "token"),
    (1, 4, 1, [9000], 16, 128, "token"),           # split over the cache
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{c[1]}-{c[2]}-{max(c[3])}-{c[4]}-{c[5]}")
def test_decode(cuda_lib, case, dtype):
    B, H, Hkv, lens, page, d, major = case
    q, k, v, table, ln = decode_case(*case[:6], dtype, major)
    out, lse = cuda_lib.monarch_attn_dense_decode(q, k, v, table, ln)
    cuda_lib.check()
    x = [f64(t) for t in (q, k, v)]
    O, L, A = dense_ref.decode(*x, table.cpu().numpy(), lens)
    eO, eL = decode_bounds(x[0], x[1], x[2], O, A, lens, dtype)
    close("out", out, O, eO)
    close("lse", lse, L, np.full(L.shape, eL))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_ignores_what_lies_past_the_length(cuda_lib, dtype):
    lens = [70, 128, 0]
    q, k, v, table, ln = decode_case(3, 8, 2, lens, 32, 128, dtype)
    a = cuda_lib.monarch_attn_dense_decode(q, k, v, table, ln)
    for b, n in enumerate(lens):
        for p in range(table.shape[1]):
            rows = slice(max(0, n - 32 * p), 32)
            k[table[b, p].item(), :, rows] = float("nan")
            v[table[b, p].item(), :, rows] = float("inf")
        table[b, -(-n // 32):] = 1 << 29  # entries past the sequence's pages are not read
    c = cuda_lib.monarch_attn_dense_decode(q, k, v, table, ln)
    cuda_lib.check()
    assert all(torch.equal(s, t) for s, t in zip(a, c))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_reports_bad_pages_and_lengths(cuda_lib, dtype):
    """Both are checked before any access; the other sequences are right."""
    q, k, v, table, ln = decode_case(3, 4, 2, [100, 90, 80], 16, 64, dtype)
    good = cuda_lib.monarch_attn_dense_decode(q, k, v, table, ln)[0]
    cuda_lib.check()
    bad = table.clone()
    bad[1, 2], bad[1, 3] = k.shape[0], -1
    out = cuda_lib.monarch_attn_dense_decode(q, k, v, bad, ln)[0]
    with pytest.raises(cuda_lib.MonarchError) as exc:
        cuda_lib.check()
    assert exc.value.status == cuda_lib.MONARCH_ERR_BAD_INDEX
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    assert torch.isfinite(out).all()
    top = table.shape[1] * 16
    for n in (top + 1, -3, 2**31 - 1):
        long = ln.clone()
        long[0] = n
        out = cuda_lib.monarch_attn_dense_decode(q, k, v, table, long)[0]
        with pytest.raises(cuda_lib.MonarchError) as exc:
            cuda_lib.check()
        assert exc.value.status == cuda_lib.MONARCH_ERR_BAD_INDEX
        long[0] = max(0, min(n, top))
        assert torch.equal(out, cuda_lib.monarch_attn_dense_decode(q, k, v, table, long)[0])
    cuda_lib.check()


# --------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------
ROTARY = [
    # B, H, Hkv, N, d, axes, grid or None, scaling, order
    (1, 1, 1, 1, 64, (64,), None, None, "head"),
    (2, 3, 1, 37, 128, (128,), None, ("parts", 8.0, 4096.0, 1.0, 32.0), "token"),
    (1, 2, 2, 60, 128, (44, 42, 42), (3, 4, 5), None, "head"),
    (2, 4, 2, 60, 96, (32, 16, 16), (3, 4, 5), None, "token"),   # part of the head
    (1, 12, 12, 24, 64, (16,), None, ("ntk", 4.0), "head"),
    (1, 5, 3, 30, 80, (40,), None, ("linear", 2.5), "token"),
    (1, 2, 1, 21, 31, (10, 6), None, None, "head"),              # odd rows
    (1, 2, 1, 21, 64, (2, 2, 4, 8), None, None, "odd"),
    (1, 1, 2, 9, 256, (256,), None, None, "head"),
]


def rotary_case(case, dtype):
    B, H, Hkv, N, d, axes, grid, scaling, order = case
    g = torch.Generator(device="cuda").manual_seed(N + d)
    q, k = heads(g, B, H, N, d, dtype, order), heads(g, B, Hkv, N, d, dtype, order)
    if grid is None:
        pos = torch.randint(-1000, 1000000, (B, len(axes), N), generator=g, device="cuda",
                            dtype=torch.int32)
        where = pos.cpu().numpy()
    else:
        pos = None
        where = np.stack(np.unravel_index(np.arange(N), grid))[None]
    return q, k, pos, where


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", ROTARY, ids=lambda c: f"{c[3]}-{c[4]}-{c[5]}-{c[8]}")
def test_rotary(cuda_lib, case, interleaved, inverse, dtype):
    axes, grid, scaling = case[5:8]
    q, k, pos, where = rotary_case(case, dtype)
    got = cuda_lib.monarch_attn_rotary(q, k, pos, axis_dims=axes, grid=grid, scaling=scaling,
                                       interleaved=interleaved, inverse=inverse)
    freqs, mag = cuda_lib.rotary_frequencies(axes, scaling=scaling)
    u = half_step(dtype)
    for x, y in zip((q, k), got):
        x = f64(x)
        ref = dense_ref.rotary(x, where, axes, freqs, mag, interleaved, inverse)
        # cosine and sine off by 2^-21 (angle to 2^-23, two fp32 roundings and
        # the function's own), the two products and their sum by 2^-23 each
        size = mag * np.sqrt(2) * np.abs(x).max()
        close("rotated", y, ref, u * np.abs(ref) + 2.0 ** -20 * size)
        rot = sum(axes)
        assert np.array_equal(f64(y)[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_in_place_in_one_projection(cuda_lib, dtype, interleaved):
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(2, 33, 8, 64, generator=g, device="cuda").to(dtype)
    q, k = x[:, :, :4].transpose(1, 2), x[:, :, 4:6].transpose(1, 2)
    ref = cuda_lib.monarch_attn_rotary(q, k, grid=(33,), interleaved=interleaved)
    v = x[:, :, 6:].clone()
    a, b = cuda_lib.monarch_attn_rotary(q, k, grid=(33,), q_out=q, k_out=k,
                                        interleaved=interleaved)
    assert a is q and b is k and torch.equal(q, ref[0]) and torch.equal(k, ref[1])
    assert torch.equal(x[:, :, 6:], v)
    with pytest.raises(cuda_lib.MonarchError):
        cuda_lib.monarch_attn_rotary(q, q, grid=(33,), q_out=q, k_out=q)
    only, none = cuda_lib.monarch_attn_rotary(ref[0], grid=(33,), inverse=True,
                                              interleaved=interleaved)
    assert none is None and only.shape == q.shape


def test_video_path_rotates_by_place_in_the_latent(cuda_lib):
    f, h, w, d = 2, 6, 10, 64
    q, k, v = (x.cuda() for x in video_qkv(1, 2, (f, h, w), d, BF16, seed=1))
    q0 = q.clone()
    turn = dict(axis_dims=(24, 20, 20), interleaved=True)
    for layout in ("fh,w", "w,fh", "h,fw"):
        got = cuda_lib.monarch_attn_fwd_video(q, k, v, f, h, w, layout, 1, rotary=turn)
        qr, kr = cuda_lib.monarch_attn_rotary(q, k, grid=(f, h, w), **turn)
        assert torch.equal(got, cuda_lib.monarch_attn_fwd_video(qr, kr, v, f, h, w, layout, 1))
    assert torch.equal(q, q0)
    plain = cuda_lib.monarch_attn_fwd_video(q, k, v, f, h, w, "fh,w", 1)
    assert not torch.equal(plain, got)


# --------------------------------------------------------------------------
# together, as a model uses them
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_then_decode_step(cuda_lib, dtype):
    """Rotate, attend causally, keep k and v in pages, decode the next token:
    the row that the whole sequence's forward pass gives."""
    g = torch.Generator(device="cuda").manual_seed(9)
    B, H, Hkv, N, d, page = 2, 4, 2, 150, 64, 16
    q, k, v = (heads(g, B, n, N, d, dtype, "token") for n in (H, Hkv, Hkv))
    pos = torch.arange(N, device="cuda", dtype=torch.int32)
    qr, kr = cuda_lib.monarch_attn_rotary(q, k, pos)
    whole, lse = cuda_lib.monarch_attn_dense_fwd(qr, kr, v, causal=True)
    per = -(-N // page)
    caches = []
    for t in (kr, v):
        c = torch.zeros(B * per, page, Hkv, d, device="cuda", dtype=dtype)
        c.view(B, per * page, Hkv, d)[:, :N] = t.transpose(1, 2)
        caches.append(c.transpose(1, 2))
    table = torch.arange(B * per, device="cuda", dtype=torch.int32).view(B, per)
    lens = torch.full((B,), N, device="cuda", dtype=torch.int32)
    one, _ = cuda_lib.monarch_attn_rotary(q[:, :, -1:], positions=pos[-1:])
    out, l1 = cuda_lib.monarch_attn_dense_decode(one[:, :, 0], *caches, table, lens)
    assert torch.equal(one[:, :, 0], qr[:, :, -1])
    x = [f64(t) for t in (qr[:, :, -1:], kr, v)]
    eO, eL = dense_ref.dense_errors(*x, x[0], half_step(dtype),
                                    rounded_weights=dtype is BF16)[:2]
    # both are within their bound of the exact row
    assert (np.abs(f64(out) - f64(whole[:, :, -1])) <= 2 * eO[:, :, 0]).all()
    assert (np.abs(f64(l1) - f64(lse[:, :, -1])) <= 2 * eL[:, :, 0]).all()


def run_all(api, q, k, v, do, caches, table, lens, stream=None):
    qr, kr = api.monarch_attn_rotary(q, k, grid=(q.shape[2],), stream=stream)
    out, lse = api.monarch_attn_dense_fwd(qr, kr, v, causal=True, stream=stream)
    dq, dk, dv = api.monarch_attn_dense_bwd(qr, kr, v, out, lse, do, causal=True, stream=stream)
    dq, dk = api.monarch_attn_rotary(dq, dk, grid=(q.shape[2],), inverse=True, stream=stream)
    step, l1 = api.monarch_attn_dense_decode(q[:, :, 0], *caches, table, lens, stream=stream)
    return out, lse, dq, dk, dv, step, l1


def all_inputs(seed, dtype=BF16):
    q, k, v, do, _ = dense_case(2, 4, 2, 200, 200, 64, True, None, "head", dtype, seed)
    one, kc, vc, table, lens = decode_case(2, 4, 2, [900, 300], 16, 64, dtype, seed=seed)
    return q, k, v, do, (kc, vc), table, lens


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_graphs_are_independent(cuda_lib, dtype):
    """Two captured passes replayed in turn, and at the same time on two
    streams, give what eager calls give; lengths are read at replay."""
    sets = [all_inputs(s, dtype) for s in (1, 2)]
    eager = [[t.clone() for t in run_all(cuda_lib, *s)] for s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_all(cuda_lib, *s))
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert all(torch.equal(a, b) for a, b in zip(o, e))
    sets[0][6][0] = 500
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][5], run_all(cuda_lib, *sets[0])[5])
    cuda_lib.check()


def test_captured_split_forward(cuda_lib):
    """Few queries over many keys: the ranges' workspace belongs to the graph,
    and lengths that empty some ranges are read at replay."""
    q, k, v, _, kl = dense_case(2, 4, 2, 5, 2600, 64, False, [2600, 2600], "head", BF16)
    cuda_lib.monarch_attn_dense_fwd(q, k, v, k_lens=kl)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = cuda_lib.monarch_attn_dense_fwd(q, k, v, k_lens=kl)
    for lens in ([2600, 2600], [100, 0], [2599, 1], [1400, 2600]):
        kl.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        ref = cuda_lib.monarch_attn_dense_fwd(q, k, v, k_lens=kl)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        x = [f64(t) for t in (q, k, v)]
        O, L = dense_ref.dense_forward(*x, lens=lens)
        eO, eL = dense_ref.dense_errors(*x, x[0], half_step(BF16), lens=lens)[:2]
        close("out", got[0], O, eO)
        close("lse", got[1], L, eL)
    cuda_lib.check()


def test_calls_on_their_own_stream(cuda_lib):
    """The stream argument carries allocations and launches; several at once."""
    sets = [all_inputs(s) for s in range(4)]
    eager = [run_all(cuda_lib, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[run_all(cuda_lib, *s, stream=st) for _ in range(3)] for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for runs, e in zip(got, eager):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, e))
    cuda_lib.check()


@pytest.mark.parametrize("split", [False, True])
def test_monarch_call_right_behind_a_dense_one(cuda_lib, split):
    """The Monarch kernels, which may start while the kernel before them
    ends, read what an exact forward pass or decode has just written."""
    B, H, b1, b2, d = 1, 4, 16, 20, 64
    n = b1 * b2
    q, k, v, _, _ = dense_case(B, H, H, n, 2600 if split else n, d, False, None, "head", BF16)
    outs = []
    for wait in (True, False, False):
        o, _ = cuda_lib.monarch_attn_dense_fwd(q, k, v)
        if wait:
            torch.cuda.synchronize()
        m = cuda_lib.monarch_attn_fwd(o, o, o, b1, b2, 1)
        if wait:
            torch.cuda.synchronize()
        outs.append(cuda_lib.monarch_attn_dense_fwd(m, k, v)[0])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    cuda_lib.check()
