"""Shared-prefix decode on the GPU (sha_decode_prefix) against its definition in 64 bits."""
import math

import pytest
import torch

from prefix_plan import SEVERAL_ROW_TILES
from prefix_reference import Case

pytestmark = pytest.mark.gpu

FILL = -77.0


@pytest.fixture(scope="module")
def sha():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import head_sparse_decode_b200 as h
    return h


def _run(sha, c, scale=None, **kw):
    q, kp, vp, idx, lens, table, pt = c.on()
    out = torch.full_like(q, FILL)
    got = sha.sha_decode_prefix(q, kp, vp, idx, lens, table, c.prefix, pt,
                                c.scale if scale is None else scale, out, **kw)
    assert got is out
    torch.cuda.synchronize()
    return out


def _check(sha, c, scale=None, status=0, rows=None, **kw):
    out = _run(sha, c, scale, **kw)
    assert sha.sha_get_device_status() == status
    want, bound = c.reference(scale, rows)
    if rows is not None:
        out = out[rows]
        want, bound = want[rows], bound[rows]
    c.check(out, want, bound, FILL)
    return out


# page sizes, prefixes around page and tile ends, suffixes from none on
@pytest.mark.parametrize("prefix,suffix,page_size", [
    (1, 1, 8), (1, 0, 256), (7, 3, 8), (8, 0, 8), (16, 16, 16), (127, 2, 16), (128, 128, 16),
    (129, 5, 64), (100, 300, 128), (255, 7, 256), (256, 130, 128), (300, 1, 256), (500, 129, 8),
    (513, 40, 32)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix_and_page_ends(sha, prefix, suffix, page_size, d):
    _check(sha, Case(3, 8, 2, d, 1, prefix, suffix, page_size, "fp16", seed=prefix + d))


@pytest.mark.parametrize("H_q,H_kv,top_k", [(6, 6, 3), (8, 4, 2), (9, 3, 2), (32, 4, 4), (16, 1, 1),
                                            (14, 2, 1), (72, 72, 22), (32, 2, 2), (20, 4, 1)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_groups_and_types(sha, H_q, H_kv, top_k, dtype):
    for d in (64, 128):
        _check(sha, Case(5, H_q, H_kv, d, top_k, 200, 90, 16, dtype, seed=H_q + d))


@pytest.mark.parametrize("B,H_q,H_kv,top_k", [
    (1, 4, 4, 1), (1, 16, 1, 1), (150, 2, 2, 2), (40, 16, 2, 2), (33, 8, 1, 1), (130, 1, 1, 1),
    (70, 3, 1, 1), (17, 16, 1, 1)])
def test_batches_across_row_tiles(sha, B, H_q, H_kv, top_k):
    """Heads selected by one row and by more rows than one tile of queries holds."""
    _check(sha, Case(B, H_q, H_kv, 128, top_k, 140, 20, 8, "bf16", seed=B))


def test_uneven_selection(sha):
    """One head taken by every row, some by one row, some by none."""
    B, H = 140, 24
    idx = torch.zeros((B, 2), dtype=torch.int32)
    idx[:, 1] = 5
    idx[0, 1], idx[77, 1], idx[139, 1] = 23, 9, 1
    _check(sha, Case(B, H, H, 64, 2, 260, 30, 16, "fp16", seed=4, idx=idx))


@pytest.mark.parametrize("prefix", [2000, 4099])
def test_long_prefix_split_over_many_blocks(sha, prefix):
    _check(sha, Case(2, 8, 1, 128, 1, prefix, 64, 64, "bf16", seed=prefix))
    _check(sha, Case(3, 2, 2, 64, 1, prefix, 0, 128, "fp16", seed=prefix + 1))


@pytest.mark.parametrize("B,H_q,H_kv,d,top_k,prefix,page_size,dtype", [
    (8, 72, 72, 128, 18, 1930, 16, "fp16"), (8, 80, 80, 64, 20, 1345, 64, "bf16"),
    (6, 160, 40, 128, 20, 1984, 32, "bf16"), (5, 90, 90, 64, 36, 2049, 8, "fp16")])
def test_long_runs_that_end_in_a_short_tile(sha, B, H_q, H_kv, d, top_k, prefix, page_size, dtype):
    """Many heads of few rows each: runs of many key tiles, the last with up to 64 keys, in which
    the second stream has no step."""
    c = Case(B, H_q, H_kv, d, top_k, prefix, 9, page_size, dtype, seed=prefix)
    first = _check(sha, c)
    for _ in range(5):
        assert torch.equal(_run(sha, c), first)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H_q,H_kv,d,prefix,suffix,sink", [
    (4, 4, 128, 9000, 40, 17), (16, 1, 64, 9000, 40, 8999), (2, 2, 64, 40, 6000, 40),
    (8, 1, 128, 3000, 3000, 0), (32, 2, 128, 200, 7000, 7199)])
def test_many_small_weights_beside_a_large_one(sha, H_q, H_kv, d, prefix, suffix, sink, dtype):
    """One key takes nearly all the weight and has the value 0; the others, each below 2^-25 of
    it, together make the output."""
    c = Case(2, H_q, H_kv, d, H_kv, prefix, suffix, 64, dtype, seed=45)
    n = prefix + suffix
    u = torch.randn(d, generator=torch.Generator().manual_seed(6)).sign()
    c.q[:] = u.to(c.dtype)
    for pool in (c.k_pages, c.v_pages):
        pool[~torch.isnan(pool)] = 0.0 if pool is c.k_pages else 1.0
    page = c.prefix_table[sink // 64] if sink < prefix else c.table[1, sink // 64]
    c.k_pages[int(page), :, sink % 64] = u.to(c.dtype)
    c.v_pages[int(page), :, sink % 64] = 0.0
    c.idx, c.lens[0] = c.idx.sort(dim=1).values, prefix
    scale = 18.0 / d                                      # the sink's score; the others' is 0
    out = _run(sha, c, scale)[1].cpu().double()
    assert sha.sha_get_device_status() == sha.SHA_OK
    w = math.exp(-18.0)                                   # 2^-25.97
    want = (n - 1) * w / (1.0 + (n - 1) * w)
    # the output's rounding (the least fp16 here is normal) and the weights', half a step each,
    # fp16 weights by up to 2^-36 of the largest where they are subnormal; exp2 2^-21, twice; the
    # score in log2 units, 26, off by two roundings of the scale; sums of n terms, 2^-23 a step
    u = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    bound = want * (2 * u + 2.0 ** -20 + 40 * 2.0 ** -24 + n * 2.0 ** -23)
    if dtype == "fp16":
        bound += n * 2.0 ** -36
    assert ((out - want).abs() <= bound).all()


@pytest.mark.parametrize("args", SEVERAL_ROW_TILES, ids=str)
def test_blocks_of_several_row_tiles(sha, args):
    """One block takes row tile after row tile: other queries, other heads, wide and narrow ones,
    pieces of split ones."""
    c = Case(*args, seed=args[5])
    first = _run(sha, c)
    _check(sha, c, rows=sorted({c.B - 1, c.B // 4} if c.B > 3 else {c.B - 1}))
    for _ in range(5):
        assert torch.equal(_run(sha, c), first)


def test_suffixes_longer_than_the_prefix(sha):
    """Own keys split over blocks and joined with the shared part."""
    _check(sha, Case(2, 8, 1, 128, 1, 9, 3000, 16, "bf16", seed=12))
    _check(sha, Case(3, 3, 3, 64, 1, 130, 2500, 64, "fp16", seed=13))
    _check(sha, Case(2, 16, 1, 128, 1, 40, 1500, 16, "fp16", seed=14))


def test_rows_that_end_with_the_prefix(sha):
    c = Case(4, 8, 2, 128, 2, 137, 60, 16, "fp16", seed=21, lens=[137, 197, 137, 138])
    _check(sha, c)
    c = Case(4, 8, 2, 128, 2, 144, 0, 16, "fp16", seed=22, lens=[144] * 4)
    _check(sha, c)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0, 30.0, 1e-6])
def test_scales(sha, scale):
    """Flat, reversed and one-hot weights."""
    for dtype in ("fp16", "bf16"):
        _check(sha, Case(3, 8, 2, 64, 1, 300, 70, 16, dtype, seed=31), scale=scale)


def test_scores_that_rise_along_the_prefix(sha):
    """The running maximum moves at every key: later keys are ever nearer to the query."""
    c = Case(2, 4, 1, 128, 1, 700, 50, 16, "fp16", seed=41)
    n = int(c.lens[1])
    u = torch.randn(128, generator=torch.Generator().manual_seed(5)).sign()
    c.q[:] = u.to(c.dtype)
    for i in range(n):
        for b in range(c.B):
            page = c.prefix_table[i // 16] if i < c.prefix else c.table[b, i // 16]
            if i < int(c.lens[b]):
                c.k_pages[int(page), 0, i % 16] = (u * (i / n * 8)).to(c.dtype)
    _check(sha, c)


def test_equals_the_paged_decode(sha):
    """On one batch, the result of sha_decode_paged up to both sides' rounding."""
    c = Case(6, 16, 4, 128, 2, 160, 100, 16, "bf16", seed=51)
    c.table[:, :10] = c.prefix_table[None, :10]
    out = _run(sha, c)
    q, kp, vp, idx, lens, table, _ = c.on()
    paged = torch.full_like(q, FILL)
    sha.sha_decode_paged(q, kp, vp, idx, lens, table, c.scale, paged)
    want, bound = c.reference()
    c.check(paged, want, bound, FILL)
    c.check(out, want, bound, FILL)


def test_bad_ids_and_lengths(sha):
    """Bad heads and lengths: those units are left alone and flagged, the others are right."""
    c = Case(6, 8, 4, 64, 2, 150, 40, 16, "fp16", seed=61)
    c.idx[1, 0], c.idx[2, 1] = 4, -1
    good = c.lens.clone()
    c.lens[3], c.lens[4], c.lens[5] = 149, 16 * c.table.shape[1] + 1, -5
    out = _run(sha, c)
    assert sha.sha_get_device_status() == sha.SHA_ERR_BAD_INDEX
    assert sha.sha_get_device_status() == sha.SHA_OK
    assert (out[3:] == FILL).all()
    c.lens = good
    want, bound = c.reference(rows=[0, 1, 2])
    c.check(out, want, bound, FILL)


@pytest.mark.parametrize("where", ["prefix", "row"])
def test_bad_pages_are_flagged(sha, where):
    c = Case(3, 4, 4, 64, 2, 40, 40, 8, "fp16", seed=62, lens=[80, 80, 80])
    for bad in (-1, c.k_pages.shape[0], 2 ** 31 - 1):
        if where == "prefix":
            c.prefix_table[2] = bad
        else:
            c.table[1, 7] = bad
        out = _run(sha, c)
        assert sha.sha_get_device_status() == sha.SHA_ERR_BAD_INDEX
    if where == "row":
        want, bound = c.reference(rows=[0, 2])
        c.check(out[[0, 2]], want[[0, 2]], bound[[0, 2]], FILL)


def test_all_heads_bad(sha):
    c = Case(3, 4, 4, 64, 2, 40, 10, 8, "fp16", seed=63)
    c.idx[:] = 9
    out = _run(sha, c)
    assert (out == FILL).all()
    assert sha.sha_get_device_status() == sha.SHA_ERR_BAD_INDEX


def test_repeated_calls_are_bit_identical(sha):
    c = Case(40, 32, 4, 128, 2, 1500, 300, 16, "bf16", seed=71)
    first = _run(sha, c)
    for _ in range(5):
        assert torch.equal(_run(sha, c), first)


def test_one_workspace_for_calls_of_all_sizes(sha):
    """Whatever an earlier call left in it, and whatever it holds at first."""
    cases = [Case(20, 8, 8, 128, 3, 300, 200, 16, "fp16", seed=81),
             Case(2, 8, 1, 64, 1, 33, 900, 32, "bf16", seed=82),
             Case(90, 16, 2, 128, 2, 129, 5, 8, "bf16", seed=83)]
    need = max(sha.sha_decode_prefix_workspace_size(c.B, c.H_q, c.H_kv, c.d, c.idx.shape[1])
               for c in cases)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    for c in cases + cases[::-1]:
        _check(sha, c, workspace=ws)
    small = torch.empty(need // 2 // 256 * 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(sha.ShaError) as e:
        _run(sha, cases[2], workspace=small[:256])
    assert e.value.status == sha.SHA_ERR_WORKSPACE


def test_workspace_stays_within_its_bytes(sha):
    c = Case(90, 16, 2, 128, 2, 129, 300, 8, "bf16", seed=84)
    need = sha.sha_decode_prefix_workspace_size(c.B, c.H_q, c.H_kv, c.d, 2)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    _check(sha, c, workspace=ws[:need])
    assert (ws[need:] == 0xA5).all()


def test_streams_and_graphs(sha):
    """Another stream, and two captured graphs replayed in turn with changed inputs."""
    c1 = Case(6, 16, 4, 128, 2, 300, 50, 16, "bf16", seed=91)
    c2 = Case(9, 4, 4, 64, 3, 77, 200, 8, "fp16", seed=92)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    _check(sha, c1, stream=s)
    graphs = []
    for c in (c1, c2):
        args = c.on()
        out = torch.full_like(args[0], FILL)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sha.sha_decode_prefix(*args[:6], c.prefix, args[6], c.scale, out)
        graphs.append((c, args, out, g))
    for seed in (1, 2):
        for c, args, out, g in graphs:
            c.q = torch.randn(c.q.shape, generator=torch.Generator().manual_seed(seed)).to(c.dtype)
            args[0].copy_(c.q)
            out.fill_(FILL)
            g.replay()
    torch.cuda.synchronize()
    assert sha.sha_get_device_status() == sha.SHA_OK
    for c, args, out, g in graphs:
        c.check(out, *c.reference(), FILL)


def test_two_calls_at_once(sha):
    """Calls on two streams, each with its own workspace."""
    cases = [Case(30, 32, 4, 128, 2, 1000, 100, 16, "bf16", seed=95),
             Case(30, 8, 8, 64, 4, 700, 60, 16, "fp16", seed=96)]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [c.on() for c in cases]
    outs = [torch.full_like(a[0], FILL) for a in args]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, a, o, s in zip(cases, args, outs, streams):
            sha.sha_decode_prefix(*a[:6], c.prefix, a[6], c.scale, o, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o, *c.reference(), FILL)


def test_behind_other_kernels_of_the_stream(sha):
    """The pages are written by the append just before, and the queries by its rotation."""
    c = Case(8, 16, 4, 128, 2, 64, 40, 16, "bf16", seed=97, lens=[104] * 8)
    q, kp, vp, idx, lens, table, pt = c.on()
    out = torch.full_like(q, FILL)
    g = torch.Generator().manual_seed(3)
    k_new = torch.randn((8, 4, 128), generator=g).to(torch.bfloat16)
    v_new = torch.randn((8, 4, 128), generator=g).to(torch.bfloat16)
    pos = torch.full((8,), 103, dtype=torch.int32, device="cuda")
    freq = torch.zeros(64, dtype=torch.float64, device="cuda")       # turns nothing
    kg, vg = k_new.cuda(), v_new.cuda()
    torch.cuda.synchronize()
    rot = sha.sha_append_paged(kg, vg, kp, vp, table, pos, inv_freq=freq, q=q)
    sha.sha_decode_prefix(rot, kp, vp, idx, lens, table, c.prefix, pt, c.scale, out)
    for b in range(8):
        c.k_pages[int(c.table[b, 6]), :, 7] = k_new[b]
        c.v_pages[int(c.table[b, 6]), :, 7] = v_new[b]
    c.check(out, *c.reference(), FILL)


def test_python_refusals_on_the_gpu(sha):
    c = Case(3, 8, 2, 64, 1, 40, 10, 8, "fp16", seed=98)
    q, kp, vp, idx, lens, table, pt = c.on()
    out = torch.empty_like(q)

    def call(q=q, kp=kp, vp=vp, idx=idx, lens=lens, table=table, prefix=40, pt=pt, out=out, **kw):
        sha.sha_decode_prefix(q, kp, vp, idx, lens, table, prefix, pt, 0.1, out, **kw)

    for kw in (dict(q=q[:2]), dict(vp=vp[:1]), dict(idx=idx.long()), dict(idx=idx[:2]),
               dict(lens=lens[:2]), dict(lens=lens.long()), dict(table=table[:, ::2]),
               dict(table=table[:2]), dict(prefix=0), dict(prefix=41), dict(pt=pt[:4]),
               dict(pt=pt.long()), dict(out=out[:2]), dict(out=out.float()),
               dict(q=q.float()), dict(q=q.cpu()), dict(workspace=torch.empty(1 << 24, 1)),
               dict(q=q[:, :, None].expand(3, 8, 2, 64))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(sha.ShaError) as e:
        call(kp=kp.reshape(-1, 2, 4, 64), vp=vp.reshape(-1, 2, 4, 64), prefix=20)
    assert e.value.status == sha.SHA_ERR_UNSUPPORTED
    call(q=q[:, :, None])
    assert sha.sha_get_device_status() == sha.SHA_OK


def test_many_calls_back_to_back(sha):
    """Calls that follow one another without a pause, each beginning while the last one ends: none
    waits for anything that has gone by (a bounded wait would cost it seconds)."""
    cases = [Case(32, 64, 8, 128, 5, 384, 60, 16, "bf16", seed=101),
             Case(24, 12, 12, 128, 4, 640, 33, 8, "fp16", seed=102),
             Case(16, 8, 8, 64, 4, 900, 70, 32, "bf16", seed=103)]
    args = [c.on() for c in cases]
    outs = [torch.full_like(a[0], FILL) for a in args]

    def calls():
        for _ in range(4):
            for c, a, o in zip(cases, args, outs):
                sha.sha_decode_prefix(*a[:6], c.prefix, a[6], c.scale, o)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(10):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert begin.elapsed_time(end) < 1000.0
    assert sha.sha_get_device_status() == sha.SHA_OK
    for c, o in zip(cases, outs):
        c.check(o, *c.reference(), FILL)
