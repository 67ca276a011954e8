"""Kernels of one stream in a row, without a synchronisation between them: each one reads what the ones before it
have written.  The packed operators and the decode are programmatic dependents, resident while their predecessors run,
so every call here changes what the next one reads at the same addresses."""
import math

import pytest
import torch

from mla_latent_kv_fp8_gb300 import synth
from tests.test_gpu_ragged import SCALE, _cu, _dev, _prefill_inputs, _randn

pytestmark = pytest.mark.gpu

ROUNDS = 12


@pytest.fixture(scope="module")
def L():
    from mla_latent_kv_fp8_gb300 import build
    build.build()
    from mla_latent_kv_fp8_gb300 import _lib
    _lib.lib()
    assert _lib.mla_device_error() == 0
    return _lib


@pytest.mark.parametrize("n", [3, 200, 6000])
def test_append_then_gather_of_changing_rows(L, n):
    """The same cache slots written anew and read back, round after round: exact values."""
    pages = -(-n // 64) + 1
    table = torch.zeros((n, 64), device="cuda")
    table[:, :32] = 1                              # no turn: the codes are those of a plain division
    cache = torch.zeros((pages, 64, 576), dtype=torch.uint8, device="cuda")
    bt = torch.randperm(pages, generator=torch.Generator().manual_seed(n))[None].to(torch.int32).cuda()
    cu, start, scale = _dev([0, n]), _dev([0]), _dev([0.02], torch.float32)
    rows = [_randn((n, 576), 10 * n + r).cuda() for r in range(ROUNDS)]
    got = [torch.empty((n, 576), dtype=torch.bfloat16, device="cuda") for _ in rows]
    torch.cuda.synchronize()
    for x, y in zip(rows, got):
        L.mla_append_rotated(x, None, 0.0, table, 0, cu, scale, bt, start, cache)
        L.mla_gather_latent(cache, scale, bt, cu, start, y[:, :512], y[:, 512:])
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    for r, (x, y) in enumerate(zip(rows, got)):
        codes = (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(y, (codes.float() * scale).to(torch.bfloat16)), f"round {r}"


@pytest.mark.parametrize("lq,lk,H,n_splits", [([1], [9000], 2, 16), ([40, 7], [3000, 800], 3, 5), ([300], [4000], 2, 4)])
def test_split_prefills_of_changing_inputs(L, lq, lk, H, n_splits):
    """Calls that share the stream's split scratch, each with its own queries, keys and values, equal the same calls
    made one at a time: a partial answer left from the call before would differ."""
    xs = [_prefill_inputs(lq, lk, H, 1000 + 7 * r) for r in range(ROUNDS)]
    cu_q, cu_k = _dev(_cu(lq)), _dev(_cu(lk))

    def call(x, out, lse):
        L.mla_prefill_ragged(*x, cu_q, cu_k, max(lq), max(lk), n_splits, SCALE, 0.0, 1, 0, None, out, lse)

    def empty():
        return (torch.full((sum(lq), H, 128), math.nan, dtype=torch.bfloat16, device="cuda"),
                torch.full((sum(lq), H), math.nan, device="cuda"))

    alone, together = [empty() for _ in xs], [empty() for _ in xs]
    for x, o in zip(xs, alone):
        torch.cuda.synchronize()
        call(x, *o)
    torch.cuda.synchronize()
    for x, o in zip(xs, together):
        call(x, *o)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    for r, (a, b) in enumerate(zip(alone, together)):
        assert not bool(a[0].isnan().any())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), f"round {r}"


@pytest.mark.parametrize("H,lens,n_splits", [(12, [900, 130], 4), (96, [700], 2), (12, [40], 1), (12, [3000] * 40, 8)])
def test_rotation_then_decode_of_changing_queries(L, H, lens, n_splits):
    """Each round rotates new queries into the same absorbed query and decodes it: the split and unsplit 12-head kernel,
    the wide one and the longest-first launch read the rows that the rotation has just written."""
    case = synth.make_decode_case(5, lens, H, 1).to("cuda")
    B = len(lens)
    table = torch.zeros((max(lens), 64), device="cuda")
    table[:, :32] = 1
    cu, start = _dev(list(range(B + 1))), _dev([n - 1 for n in lens])
    qs = [_randn((B, H, 192), 300 + r, 3.0).cuda() for r in range(ROUNDS)]
    absorbed = case.q.clone()

    def call(q, out, lse):
        L.mla_rotate_query(q, None, 0.0, table, 0, cu, start, None, absorbed.view(B, H, 576)[..., 512:])
        L.mla_decode_paged(absorbed, case.kv_cache, case.kv_scale, case.block_table, case.seq_lens, n_splits,
                           case.sm_scale, out, lse)

    def empty():
        return (torch.full((B, 1, H, 512), math.nan, dtype=torch.bfloat16, device="cuda"),
                torch.full((B, 1, H), math.nan, device="cuda"))

    alone, together = [empty() for _ in qs], [empty() for _ in qs]
    for q, o in zip(qs, alone):
        torch.cuda.synchronize()
        call(q, *o)
    torch.cuda.synchronize()
    for q, o in zip(qs, together):
        call(q, *o)
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    for r, (a, b) in enumerate(zip(alone, together)):
        assert not bool(a[0].isnan().any())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), f"round {r}"
    assert not torch.equal(alone[0][0], alone[1][0])


def test_replayed_chain_of_changing_inputs(L):
    """The chain append, rotate, gather, split prefill captured once and replayed back to back on the same buffers, with
    copies of new inputs between the replays, answers as the calls do one at a time."""
    n, past, H = 50, 2000, 2
    total = n + past
    pages = -(-total // 64)
    bt = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[None].to(torch.int32).cuda()
    cache = torch.randint(0, 120, (pages, 64, 576), dtype=torch.uint8, generator=torch.Generator().manual_seed(2)).cuda()
    angle = torch.arange(total, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    table = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    weight = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    cu, cu_k, start, scale = _dev([0, n]), _dev([0, total]), _dev([past]), _dev([0.01], torch.float32)
    kn, v = _randn((total, H, 128), 3).cuda(), _randn((total, H, 128), 4).cuda()
    ins = [(_randn((n, 576), 20 + r).cuda(), _randn((n, H, 192), 40 + r).cuda()) for r in range(ROUNDS)]
    latent, q = (torch.empty_like(t) for t in ins[0])
    hist = torch.empty((total, 576), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((n, H, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((n, H), device="cuda")

    def chain():
        L.mla_append_rotated(latent, weight, 1e-6, table, 1, cu, scale, bt, start, cache)
        L.mla_rotate_query(q, None, 0.0, table, 1, cu, start, None, q[..., 128:])
        L.mla_gather_latent(cache, scale, bt, cu_k, None, hist[:, :512], hist[:, 512:])
        L.mla_prefill_ragged(q, kn, hist[:, 512:], v, cu, cu_k, n, total, 4, SCALE, 0.0, 1, 0, None, out, lse)

    def feed(r):
        latent.copy_(ins[r][0])
        q.copy_(ins[r][1])

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        alone = []
        for r in range(ROUNDS):
            feed(r)
            torch.cuda.synchronize()
            chain()
            torch.cuda.synchronize()
            alone.append((hist.clone(), out.clone(), lse.clone()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        chain()
    torch.cuda.synchronize()
    replayed = []
    with torch.cuda.stream(s):
        for r in range(ROUNDS):
            feed(r)
            g.replay()
            replayed.append((hist.clone(), out.clone(), lse.clone()))
    torch.cuda.synchronize()
    assert L.mla_device_error() == 0
    for r, (a, b) in enumerate(zip(alone, replayed)):
        assert all(torch.equal(x, y) for x, y in zip(a, b)), f"round {r}"
