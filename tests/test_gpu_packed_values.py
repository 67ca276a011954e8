"""Values at the edges of the packed operators' ranges: NaN and infinities in a query, signed zeros, unusual scales and
caps, and every combination of weight type and layout."""
import math

import pytest
import torch

from tests import ragged_reference as R
from tests.test_gpu_ragged import SCALE, _cu, _dev, _prefill, _prefill_inputs, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from mla_latent_kv_fp8_gb300 import build
    build.build()
    from mla_latent_kv_fp8_gb300 import _lib
    _lib.lib()
    assert _lib.mla_device_error() == 0
    return _lib


# ---------------------------------------------------------------- codes

def _append_both(L, latent, scale):
    """The codes of latent rows [n, 576] by mla_append_rotated (no norm, angles of 0) and by mla_append_latent."""
    n = latent.shape[0]
    table = torch.zeros((n, 64), device="cuda")
    table[:, :32] = 1
    pages = -(-n // 64)
    bt, start = torch.arange(pages, dtype=torch.int32, device="cuda")[None], _dev([0])
    a = torch.full((pages, 64, 576), 0xAA, dtype=torch.uint8, device="cuda")
    b = a.clone()
    sc = _dev([scale], torch.float32)
    L.mla_append_rotated(latent, None, 0.0, table, 1, _dev([0, n]), sc, bt, start, a)
    L.mla_append_latent(latent[None], sc, bt, start, b)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    return a.view(-1, 576)[:n], b.view(-1, 576)[:n]


def test_codes_of_signed_zeros(L):
    """-0 keeps its sign, as a division does."""
    latent = torch.zeros((2, 576), dtype=torch.bfloat16, device="cuda")
    latent[1, :512] = -0.0
    a, b = _append_both(L, latent, 0.031)
    assert torch.equal(a, b)
    assert bool((a[0] == 0).all()) and bool((a[1, :512] == 0x80).all())


@pytest.mark.parametrize("scale", [
    0.031, 1.0, 1.53173798, 0.0113, 448.0, 3e-5, float.fromhex("0x1.881dfcp+0"),
    float.fromhex("0x1.00000ap+3"), float.fromhex("0x1.1fffeep-5"), float.fromhex("0x1.fffff4p-1"),  # near 2^20 multiples
    2.0 ** -90, 2.0 ** 90, float.fromhex("0x1.fffffep-91"), float.fromhex("0x1.000002p+90"),        # ends of the fast range
    1e-38, 1e-42, 3e38, 0.0, -0.02, math.inf, -math.inf, math.nan,                                  # the general division
])
def test_codes_are_those_of_a_plain_division(L, scale):
    """Byte for byte those of mla_append_latent, whatever the scale: values around every border between codes and
    random ones, zeros, infinities and NaN of both signs, the smallest and the largest numbers."""
    unit = scale if 0 < abs(scale) < math.inf else 1.0
    t = torch.arange(16, 32, dtype=torch.float64)
    border = torch.cat([t * 2.0 ** e for e in range(-14, 6)])
    x = torch.cat([border * unit * (1 + d * 2.0 ** -8) for d in range(-2, 3)]
                  + [torch.randn(20000, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * unit * g
                     for g in (0.01, 1.0, 100.0)]
                  + [torch.tensor([0.0, math.inf, math.nan, 2.0 ** -133, 3e38, 2.0 ** -126])])
    x = torch.cat([x, -x])
    rows = -(-len(x) // 512)
    latent = torch.ones((rows, 576), dtype=torch.float64)
    flat = torch.zeros(rows * 512, dtype=torch.float64)
    flat[:len(x)] = x
    latent[:, :512] = flat.view(rows, 512)
    a, b = _append_both(L, latent.to(torch.bfloat16).cuda(), scale)
    assert torch.equal(a, b)


# ---------------------------------------------------------------- NaN and infinities in a query

@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("n_splits", [1, 4])
@pytest.mark.parametrize("lq,lk", [([1], [40]), ([100], [900]), ([3, 260], [700, 2100]), ([40] * 40, [50] * 40)])
def test_nan_queries_give_nan_and_nothing_else_changes(L, lq, lk, n_splits, cap):
    """A NaN in one dim, in the rotated dims, and in all of a query row: NaN in out and lse of that row and head, not
    the answer of a row without a key and not an ordinary number; every other row is the same bit for bit."""
    H, n = 2, sum(lq)
    q, kn, kp, v = _prefill_inputs(lq, lk, H, 500 + n, pad=2)
    want, want_lse = _prefill(L, (q, kn, kp, v), lq, lk, n_splits, cap)
    rows = sorted({0, n // 2, n - 1})
    bad = torch.zeros((n + 2, H), dtype=torch.bool, device="cuda")
    q = q.clone()
    for at, (row, dims) in enumerate(zip(rows, (slice(5, 6), slice(150, 151), slice(0, 192)))):
        q[row, at % H, dims] = math.nan
        bad[row, at % H] = True
    out, lse = _prefill(L, (q, kn, kp, v), lq, lk, n_splits, cap)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])


@pytest.mark.parametrize("n_splits", [1, 3])
@pytest.mark.parametrize("n", [1, 300])
def test_infinite_queries(L, n, n_splits):
    """One infinity in a query: its scores are infinities of both signs.  Without a cap the softmax is not a number;
    with one they are +-cap.  Two infinities of opposite signs: not a number either way."""
    H, cap, keys = 1, 20.0, 800
    q, kn, kp, v = _prefill_inputs([n], [keys], H, 600 + n)
    kn = kn.clone()
    kn[:, 0, 3] = torch.where(kn[:, 0, 3] == 0, 1.0, kn[:, 0, 3])
    q[n // 2, 0, 3] = math.inf
    for c, nan in ((0.0, True), (cap, False)):
        out, lse = _prefill(L, (q, kn, kp, v), [n], [keys], n_splits, c, causal=0)
        torch.cuda.synchronize()
        row, z = out[n // 2, 0].double(), lse[n // 2, 0].double()
        if nan:
            assert bool(row.isnan().all()) and bool(z.isnan())
            continue
        s = cap * torch.sign(kn[:, 0, 3].double())
        p = torch.softmax(s, 0)
        ref, ref_z = p @ v[:, 0].double(), torch.logsumexp(s, 0)
        # the scores are off by at most cap * 2^-20, probabilities are rounded to bf16 and so is the output
        e = cap * 2.0 ** -20
        assert bool(((row - ref).abs() <= (p @ v[:, 0].double().abs()) * (R.BF16_HALF + 2 * e + 2.0 ** -12)
                     + R.BF16_HALF * 1.01 * ref.abs()).all())
        assert abs(float(z - ref_z)) <= 2 * e + 2.0 ** -21 * float(ref_z) + 2.0 ** -18
    q[n // 2, 0, 4] = -math.inf
    same = kn[:, 0, 3] * kn[:, 0, 4] > 0             # inf - inf in these keys' scores
    assert bool(same.any())
    out, lse = _prefill(L, (q, kn, kp, v), [n], [keys], n_splits, cap, causal=0)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    assert bool(out[n // 2].isnan().all()) and bool(lse[n // 2].isnan().all())
    rest = torch.arange(n, device="cuda") != n // 2
    assert not bool(out[rest].isnan().any()) and not bool(lse[rest].isnan().any())


@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_nan_scores_of_hidden_keys_only(L, cap):
    """Scores that are not numbers, but only at keys that the row does not see (past its place under the causal mask, and
    past the sequence's end): the row's answer is an ordinary one."""
    H, n, pad = 1, 200, 100
    q, kn, kp, v = _prefill_inputs([n], [n], H, 71, pad=pad)     # rows past the sequence are NaN and infinities
    kn = kn.clone()
    q[50, 0, :2] = torch.tensor([math.inf, -math.inf])           # inf - inf where k[0] k[1] > 0
    kn[:n, 0, 0] = 1.0
    kn[:n, 0, 1] = torch.where(torch.arange(n, device="cuda") <= 50, -1.0, 1.0)   # visible: +inf, hidden: NaN
    out, lse = _prefill(L, (q, kn, kp, v), [n], [n], 1, cap)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    if cap:                                                       # all 51 visible scores are the cap
        ref = v[:51, 0].double().mean(0)
        bound = v[:51, 0].double().abs().mean(0) * (2 * R.BF16_HALF + 2.0 ** -12) + R.BF16_HALF * ref.abs()
        assert bool(((out[50, 0].double() - ref).abs() <= bound).all())
        assert abs(float(lse[50, 0]) - (cap + math.log(51))) <= cap * 2.0 ** -19 + 2.0 ** -18
    else:
        assert bool(out[50].isnan().all()) and bool(lse[50].isnan().all())
    assert not bool(out[51:n].isnan().any()) and not bool(out[:50].isnan().any())
    assert bool((out[n:] == 7).all())


# ---------------------------------------------------------------- caps

@pytest.mark.parametrize("cap", [2.0 ** -10, 0.05, 1.0, 64.0, 64.5, 300.0, 4096.0])
@pytest.mark.parametrize("n_splits,most", [(1, 2), (3, 2), (1, 24)])
def test_caps_over_their_range(L, cap, n_splits, most):
    """Scores small and large against the cap, from whole numbers, so that the products and their sums are exact in fp32
    and what is left is the cap: out and lse are as close as its stated accuracy lets them be."""
    lq, lk, H, scale = [300, 5], [900, 130], 2, 1 / 16
    q, kn, kp, v = _prefill_inputs(lq, lk, H, 41)
    g = torch.Generator().manual_seed(most)
    whole = lambda shape, m: torch.randint(-m, m + 1, shape, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, kn, kp = whole(q.shape, most), whole(kn.shape, 2), whole(kp.shape, 2)
    cu_q, cu_k = _cu(lq), _cu(lk)
    out = torch.empty((sum(lq), H, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((sum(lq), H), device="cuda")
    L.mla_prefill_ragged(q, kn, kp, v, _dev(cu_q), _dev(cu_k), max(lq), max(lk), n_splits, scale, cap, 0, 0, None, out, lse)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    ref, z, _, _ = R.prefill(q, kn, kp, v, cu_q, cu_k, scale, cap, False)
    for b in range(2):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in range(H):
            k = torch.cat([kn[keys, h].double(), kp[keys].double()], 1)
            s = cap * torch.tanh(q[rows, h].double() @ k.T * scale / cap)
            # a score: its cap as documented, and a few roundings of its multiples and of the reference it is held
            # against, relative to it (to the cap, where it is held as a difference to the cap)
            e = (2.0 ** -20 + 8 * R.F32_HALF) * (cap if cap <= 64 else s.abs().amax(1)) + 2.0 ** -20
            e = torch.as_tensor(e, device="cuda").expand(s.shape[0])
            p = torch.softmax(s, 1)
            bound = (p @ v[keys, h].double().abs()) * (R.BF16_HALF + 2 * e[:, None] + 2.0 ** -12) \
                + R.BF16_HALF * 1.01 * ref[rows, h].abs() + 1e-30
            assert bool(((out[rows, h].double() - ref[rows, h]).abs() <= bound).all())
            lse_bound = 2 * e + 2.0 ** -21 * z[rows, h].abs() + 2.0 ** -18
            assert bool(((lse[rows, h].double() - z[rows, h]).abs() <= lse_bound).all())


@pytest.mark.parametrize("cap", [0.0, 2.0 ** -10])
def test_smallest_and_largest_scales(L, cap):
    """A scale so small that every score is 0: the mean of the values; the largest one: the value of the best key (with
    a cap, where every score is +-cap: finite)."""
    n, keys, H = 130, 300, 2
    q, kn, kp, v = _prefill_inputs([n], [keys], H, 81)
    outs = []
    for scale in (2.0 ** -100, 2.0 ** 20):
        out = torch.empty((n, H, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((n, H), device="cuda")
        L.mla_prefill_ragged(q, kn, kp, v, _dev([0, n]), _dev([0, keys]), n, keys, 1, scale, cap, 0, 0, None, out, lse)
        torch.cuda.synchronize()
        assert L.mla_device_error() == 0
        outs.append((out.double(), lse.double()))
    mean = v.double().mean(0)
    # probabilities of 2^0, exact in bf16; sums of 300 fp32 terms; the output's rounding
    bound = R.BF16_HALF * 1.01 * mean.abs() + 300 * R.F32_HALF * v.double().abs().mean(0) + 2.0 ** -20 * cap
    assert bool(((outs[0][0] - mean).abs() <= bound).all())
    assert bool(((outs[0][1] - math.log(keys)).abs() <= 2.0 ** -18).all())
    out, lse = outs[1]
    assert not bool(out.isnan().any()) and bool(lse.isfinite().all())
    if cap == 0:
        k = torch.cat([kn.double(), kp.double()[:, None].expand(-1, H, -1)], -1)
        s = torch.einsum("nhd,mhd->nhm", q.double(), k)
        size = torch.einsum("nhd,mhd->nhm", q.double().abs(), k.abs()).amax(2)
        two = s.topk(2, 2).values
        sure = two[..., 0] - two[..., 1] > 2 * 200 * R.F32_HALF * size      # more than the products' sums may be off
        best = v.double().permute(1, 0, 2)[torch.arange(H, device="cuda")[None], s.argmax(2)]
        # The best key's probability is 2^d before the division by the sum, d the rounding of the reference (scores of
        # 2^26 have a step of 4): out is v * bf16(2^d) / 2^d, off by up to half a bf16 step, and rounded once more.
        near = (out - best).abs() <= (2 * R.BF16_HALF + R.BF16_HALF ** 2) * best.abs()
        assert bool(sure.float().mean() > 0.9) and bool(near[sure].all())


# ---------------------------------------------------------------- every weight type and layout

WEIGHTS = [None, torch.bfloat16, torch.float32]


def _weight(dims, dtype, seed):
    if dtype is None:
        return None
    return (1 + 0.2 * torch.randn(dims, generator=torch.Generator().manual_seed(seed))).to(dtype)


@pytest.mark.parametrize("dtype", WEIGHTS)
@pytest.mark.parametrize("interleaved", [0, 1])
@pytest.mark.parametrize("n", [1, 70, 2500])
def test_append_forms(L, dtype, interleaved, n):
    latent, weight, scale = _randn((n, 576), 3 * n), _weight(512, dtype, n), 0.0123
    table, past = R.cos_sin(n + 30), 30
    pages = -(-(n + past) // 64)
    cache = torch.zeros((pages, 64, 576), dtype=torch.uint8, device="cuda")
    kept = torch.zeros((n, 576), dtype=torch.bfloat16, device="cuda")
    L.mla_append_rotated(latent.cuda(), weight.cuda() if weight is not None else None, 1e-6, table.cuda(), interleaved,
                         _dev([0, n]), _dev([scale], torch.float32),
                         torch.arange(pages, dtype=torch.int32, device="cuda")[None], _dev([past]), cache, kept)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    ref, size = R.new_latents(latent, weight, 1e-6, table, interleaved, torch.arange(n) + past)
    sc = float(torch.tensor(scale))
    R.assert_bf16(kept.cpu(), ref, size, "kept")
    R.assert_codes(cache.cpu().view(-1, 576)[past:past + n], ref / sc, size / sc, "codes")


@pytest.mark.parametrize("dtype", WEIGHTS)
@pytest.mark.parametrize("interleaved", [0, 1])
@pytest.mark.parametrize("n,H", [(1, 1), (33, 12), (700, 5)])
def test_rotate_forms(L, dtype, interleaved, n, H):
    q, weight, table = _randn((n, H, 192), 7 * n + H), _weight(192, dtype, n), R.cos_sin(n + 9)
    nope = torch.zeros((n, H, 128), dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros((n, H, 64), dtype=torch.bfloat16, device="cuda")
    L.mla_rotate_query(q.cuda(), weight.cuda() if weight is not None else None, 1e-6, table.cuda(), interleaved,
                       _dev([0, n]), _dev([9]), nope, pe)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    x = q.double() if weight is None else R.norm(q.double(), weight, 1e-6)
    ref, size = R.rotate(x[..., 128:], table[torch.arange(n) + 9][:, None], interleaved)
    R.assert_bf16(pe.cpu(), ref, size, "rotated")
    R.assert_bf16(nope.cpu(), x[..., :128], x[..., :128].abs(), "other dims")
