"""The largest and smallest calls that the packed operators take: 65,535 sequences, 65,535 heads, tensors without rows,
pages, positions or columns, outputs with the heads outermost."""
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


def _many():
    """Lengths of 65,535 sequences, most of them empty: the first, the last, neighbours and lone ones have rows."""
    lens = [0] * 65535
    g = torch.Generator().manual_seed(4)
    for b in torch.randperm(65535, generator=g)[:1500].tolist() + [0, 1, 2, 40000, 40001, 65533, 65534]:
        lens[b] = 1 + b % 3
    return lens


def test_most_sequences_append_rotate_gather(L):
    lens = _many()
    n, B = sum(lens), len(lens)
    used = [b for b in range(B) if lens[b]]
    start = torch.zeros(B, dtype=torch.int32)
    bt = torch.full((B, 2), -5, dtype=torch.int32)
    for i, b in enumerate(used):
        start[b] = 60 + b % 9
        bt[b, 0], bt[b, 1] = 2 * i, 2 * i + 1
    seq = torch.tensor([b for b in used for _ in range(lens[b])])
    pos = torch.tensor([int(start[b]) + i for b in used for i in range(lens[b])])
    table = R.cos_sin(80)
    latent, q = _randn((n + 2, 576), 1), _randn((n + 2, 3, 192), 2)
    cache = torch.zeros((2 * len(used), 64, 576), dtype=torch.uint8, device="cuda")
    kept = torch.full((n + 2, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    cu, gs, gbt, scale = _dev(_cu(lens)), start.cuda(), bt.cuda(), _dev([0.02], torch.float32)
    gq = q.cuda()
    L.mla_append_rotated(latent.cuda(), None, 0.0, table.cuda(), 1, cu, scale, gbt, gs, cache, kept)
    L.mla_rotate_query(gq, None, 0.0, table.cuda(), 0, cu, gs, None, gq[..., 128:])
    hist = torch.full((n + 2, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    L.mla_gather_latent(cache, scale, gbt, cu, gs, hist[:, :512], hist[:, 512:])
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    ref, size = R.new_latents(latent[:n], None, 0.0, table, 1, pos)
    R.assert_bf16(kept.cpu()[:n], ref, size, "kept")
    codes = cache.cpu()[bt[seq, pos // 64].long(), pos % 64]
    sc = float(torch.tensor(0.02))
    R.assert_codes(codes, ref / sc, size / sc, "codes")
    assert torch.equal(hist[:n].cpu(), (codes.view(torch.float8_e4m3fn).float() * torch.tensor(0.02)).to(torch.bfloat16))
    ref, size = R.rotate(q[:n, :, 128:].double(), table[pos][:, None], 0)
    R.assert_bf16(gq.cpu()[:n, :, 128:], ref, size, "rotated")
    assert bool((kept[n:] == 7).all()) and bool((hist[n:] == 7).all()) and torch.equal(gq[n:].cpu(), q[n:])


@pytest.mark.parametrize("n_splits", [1, 3])
def test_most_sequences_prefill(L, n_splits):
    lq = _many()
    lk = [150 + b % 200 if n else b % 2 for b, n in enumerate(lq)]      # keys of sequences without a query too
    x = _prefill_inputs(lq, lk, 1, 9, pad=1)
    out, lse = _prefill(L, x, lq, lk, n_splits)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    n = sum(lq)
    R.assert_prefill(out, lse, R.prefill(*x, _cu(lq), _cu(lk), SCALE), slice(0, n))
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())


def test_most_heads_prefill(L):
    H, nq, nk = 65535, 2, 5
    q, kn, kp, v = _prefill_inputs([nq], [nk], H, 3)
    out, lse = _prefill(L, (q, kn, kp, v), [nq], [nk])
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    k = torch.cat([kn, kp[:, None].expand(-1, H, -1)], -1).double()
    s = torch.einsum("nhd,mhd->hnm", q.double(), k) * SCALE
    size = torch.einsum("nhd,mhd->hnm", q.double().abs(), k.abs()) * SCALE
    see = torch.arange(nk, device="cuda")[None] <= torch.arange(nq, device="cuda")[:, None] + nk - nq
    s, size = s.masked_fill(~see, -math.inf), size.masked_fill(~see, 0.0)
    z, p = torch.logsumexp(s, 2), torch.softmax(s, 2)
    e = 200 * R.F32_HALF * size.amax(2) + 8 * R.F32_HALF * s.masked_fill(~see, 0.0).abs().amax(2) + 2.0 ** -20
    ref = torch.einsum("hnm,mhd->nhd", p, v.double())
    bound = torch.einsum("hnm,mhd->nhd", p, v.double().abs()) * (R.BF16_HALF + 2 * e.t()[..., None] + 2.0 ** -12) \
        + R.BF16_HALF * 1.01 * ref.abs() + 1e-30
    assert bool(((out.double() - ref).abs() <= bound).all())
    assert bool(((lse.double() - z.t()).abs() <= (2 * e + 2.0 ** -21 * z.abs() + 2.0 ** -18).t()).all())


def test_many_heads_rotate(L):
    H, n = 70001, 3
    q, table = _randn((n, H, 192), 5), R.cos_sin(9)
    g = q.cuda()
    L.mla_rotate_query(g, None, 0.0, table.cuda(), 1, _dev([0, n]), _dev([4]), None, g[..., 128:])
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    ref, size = R.rotate(q[..., 128:].double(), table[4:4 + n][:, None], 1)
    R.assert_bf16(g.cpu()[..., 128:], ref, size, "rotated")
    assert torch.equal(g.cpu()[..., :128], q[..., :128])


def test_calls_without_rows_do_nothing(L):
    e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    cu, cu0, start, start0 = _dev([0, 0, 0]), _dev([0]), _dev([0, 0]), e(0, dtype=torch.int32)
    table, scale = R.cos_sin(4).cuda(), _dev([0.1], torch.float32)
    cache, bt = torch.full((2, 64, 576), 3, dtype=torch.uint8, device="cuda"), _dev([[0], [1]])
    for c, s, b in ((cu, start, bt), (cu0, start0, e(0, 1, dtype=torch.int32))):
        for n in (0, 5):                            # no rows at all, and rows of no sequence
            kept, hist = torch.full((n, 576), 7.0, dtype=torch.bfloat16, device="cuda"), _randn((n, 576), 1).cuda()
            before, q = hist.clone(), _randn((n, 2, 192), 2).cuda()
            q0 = q.clone()
            L.mla_append_rotated(_randn((n, 576), 3).cuda(), None, 0.0, table, 1, c, scale, b, s, cache, kept)
            L.mla_rotate_query(q, None, 0.0, table, 1, c, s, None, q[..., 128:])
            L.mla_gather_latent(cache, scale, b, c, s, hist[:, :512], hist[:, 512:])
            out, lse = torch.full((n, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((n, 2), 7.0, device="cuda")
            for keys in (0, 3):
                L.mla_prefill_ragged(q, _randn((keys, 2, 128), 4).cuda(), _randn((keys, 64), 5).cuda(),
                                     _randn((keys, 2, 128), 6).cuda(), c, c, 0, 0, 0, SCALE, 0.0, 1, 0, None, out, lse)
            torch.cuda.synchronize()
            assert L.mla_device_error() == 0
            assert bool((kept == 7).all()) and torch.equal(hist, before) and torch.equal(q, q0)
            assert bool((out == 7).all()) and bool((lse == 7).all())
    assert bool((cache == 3).all())
    # no heads
    L.mla_rotate_query(e(3, 0, 192), None, 0.0, table, 1, _dev([0, 3]), _dev([0]), None, e(3, 0, 64))
    L.mla_prefill_ragged(e(3, 0, 192), e(3, 0, 128), e(3, 64), e(3, 0, 128), _dev([0, 3]), _dev([0, 3]), 3, 3, 0, SCALE, 0.0,
                         1, 0, None, e(3, 0, 128), e(3, 0, dtype=torch.float32))
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0


def test_caches_without_pages_columns_or_positions(L):
    """Every row is out of range: reported, nothing written (the gather writes zeros)."""
    latent, table, scale = _randn((2, 576), 1).cuda(), R.cos_sin(4).cuda(), _dev([0.1], torch.float32)
    cu, start = _dev([0, 2]), _dev([0])
    pages, none = (torch.full((k, 64, 576), 3, dtype=torch.uint8, device="cuda") for k in (2, 0))
    columns, empty = _dev([[0]]), torch.empty((1, 0), dtype=torch.int32, device="cuda")
    for cache, bt, t, code in ((none, columns, table, 2), (pages, empty, table, 3),
                               (pages, columns, torch.empty((0, 64), device="cuda"), 3)):
        kept = torch.full((2, 576), 7.0, dtype=torch.bfloat16, device="cuda")
        L.mla_append_rotated(latent, None, 0.0, t, 1, cu, scale, bt, start, cache, kept)
        torch.cuda.synchronize()
        assert L.mla_device_error() == code
        assert bool((kept == 7).all()) and bool((cache == 3).all())
        if t is table:
            L.mla_gather_latent(cache, scale, bt, cu, start, kept[:, :512], kept[:, 512:])
            torch.cuda.synchronize()
            assert L.mla_device_error() == code and bool((kept == 0).all())


@pytest.mark.parametrize("n_splits", [1, 3])
def test_prefill_output_with_the_heads_outermost(L, n_splits):
    lq, lk, H = [130, 300], [200, 700], 3
    q, kn, kp, v = _prefill_inputs(lq, lk, H, 12)
    box = torch.full((H, 430, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = box.transpose(0, 1)[..., :128], torch.empty((430, H), device="cuda")
    L.mla_prefill_ragged(q, kn, kp, v, _dev(_cu(lq)), _dev(_cu(lk)), 300, 700, n_splits, SCALE, 0.0, 1, 0, None, out, lse)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    R.assert_prefill(out, lse, R.prefill(q, kn, kp, v, _cu(lq), _cu(lk), SCALE))
    assert bool((box[..., 128:] == 7).all())
