"""Rotary positions and paged appending on the GPU against their definitions in 64 bits."""
import pytest
import torch

import rope_reference as ref

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sha():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import head_sparse_decode_b200 as h
    return h


def _randn(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


def _positions(T, most, seed):
    return torch.randint(0, most, (T,), generator=torch.Generator().manual_seed(seed + 1),
                         dtype=torch.int32)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,d,rotary", [
    (1, 1, 64, 64), (1, 32, 128, 128), (7, 5, 128, 64), (33, 9, 64, 24), (5, 3, 64, 2),
    (6, 2, 72, 50), (4, 72, 128, 128), (130, 3, 8, 4), (3, 2, 512, 512), (3, 2, 512, 510),
    (257, 1, 64, 36), (64, 40, 128, 16)])
def test_rotation(sha, T, H, d, rotary, interleaved):
    for dtype in DT:
        x = _randn((T, H, d), T + d, dtype)
        pos = _positions(T, 1 << 17, T)
        freq = ref.frequencies(rotary)
        got = sha.sha_rope(x.cuda(), pos.cuda(), freq.cuda(), interleaved=interleaved, mscale=1.25)
        ref.assert_rotated(got, x, pos, freq, interleaved, 1.25)
        assert sha.sha_get_device_status() == sha.SHA_OK


def test_far_positions_keep_their_angles(sha):
    """Positions up to 2^31 - 1 and negative ones: an fp32 angle would be 128 rad off."""
    pos = torch.tensor([2 ** 31 - 1, 2 ** 30 + 1, -(2 ** 31), -17, 0, 2 ** 24 + 1],
                       dtype=torch.int32)
    x = _randn((6, 2, 128), 3, "fp16")
    freq = ref.frequencies(128)
    got = sha.sha_rope(x.cuda(), pos.cuda(), freq.cuda())
    # the angle's product rounds at 2^-53 of 2^31 rad, 2.4e-7: within the bound's slack
    want = ref.rotate(x, pos, freq)
    slack = 1e-6 * (x.double()[..., :64].abs() + x.double()[..., 64:].abs()).repeat(1, 1, 2)
    assert ((got.cpu().double() - want).abs()
            <= ref.bound(x, want, freq, False, 1.0) + slack).all()


def test_position_zero_is_the_identity_and_the_tail_is_copied(sha):
    x = _randn((4, 3, 64), 5, "bf16").cuda()
    got = sha.sha_rope(x, torch.zeros(4, dtype=torch.int32, device="cuda"),
                       ref.frequencies(32).cuda())
    assert torch.equal(got, x)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_strided_views(sha, interleaved):
    """A slice of a fused projection's rows, rotated in place and into a head-major tensor."""
    T, d = 19, 128
    fused = _randn((T, 12, d), 6, "fp16")
    pos, freq = _positions(T, 5000, 6).cuda(), ref.frequencies(96).cuda()
    g = fused.cuda()
    q = g[:, 3:10]
    head_major = torch.full((7, T, d), 7.0, dtype=torch.float16, device="cuda").transpose(0, 1)
    sha.sha_rope(q, pos, freq, out=head_major, interleaved=interleaved)
    ref.assert_rotated(head_major, fused[:, 3:10], pos, freq, interleaved)
    assert torch.equal(g.cpu(), fused)                    # the input as it was
    same = sha.sha_rope(q, pos, freq, out=q, interleaved=interleaved)
    assert same is q and torch.equal(q, head_major)
    assert torch.equal(g[:, :3].cpu(), fused[:, :3]) and torch.equal(g[:, 10:].cpu(), fused[:, 10:])


def test_broadcast_input_and_single_rows_of_odd_strides(sha):
    pos, freq = _positions(6, 100, 8), ref.frequencies(64)
    one = _randn((1, 1, 64), 8, "bf16")
    x = one.expand(6, 4, 64)                              # strides 0
    got = sha.sha_rope(one.cuda().expand(6, 4, 64), pos.cuda(), freq.cuda())
    ref.assert_rotated(got, x, pos, freq)
    odd = torch.as_strided(one.cuda(), (1, 1, 64), (3, 5, 1))  # strides of size-1 dimensions
    ref.assert_rotated(sha.sha_rope(odd, pos[:1].cuda(), freq.cuda()), one, pos[:1], freq)


def test_gradient_is_the_rotation_backwards(sha):
    """d<w, rope(x)>/dx = mscale * R(-p) w, against central differences of the 64-bit formula."""
    T, H, d, m = 3, 2, 16, 1.5
    pos, freq = torch.tensor([0, 5, 1000], dtype=torch.int32), ref.frequencies(8)
    w = _randn((T, H, d), 9, "fp16")
    got = sha.sha_rope(w.cuda(), -pos.cuda(), freq.cuda(), mscale=m).cpu().double()
    # a copied element's gradient is w itself
    x = torch.randn((T, H, d), generator=torch.Generator().manual_seed(10), dtype=torch.float64)
    diff = torch.empty_like(x)
    for i in range(x.numel()):
        step = torch.zeros(x.numel(), dtype=torch.float64)
        step[i] = 0.5
        step = step.reshape(x.shape)
        up = ref.rotate(x + step, pos, freq, mscale=m) - ref.rotate(x - step, pos, freq, mscale=m)
        diff.view(-1)[i] = (up * w.double()).sum()
    # linear in x: the differences are exact but for 64-bit rounding
    assert ((got - diff).abs() <= ref.bound(w, diff, freq, False, m) + 1e-9).all()


def test_empty_calls(sha):
    freq = ref.frequencies(64).cuda()
    x = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    assert sha.sha_rope(x, torch.empty(0, dtype=torch.int32, device="cuda"), freq).shape == x.shape


def test_other_stream_and_graph_replay(sha):
    x, pos = _randn((40, 8, 128), 11, "bf16"), _positions(40, 9999, 11)
    freq = ref.frequencies(128)
    xg, pg, fg = x.cuda(), pos.cuda(), freq.cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty_like(xg)
    sha.sha_rope(xg, pg, fg, out=out, stream=s)
    s.synchronize()
    ref.assert_rotated(out, x, pos, freq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = sha.sha_rope(xg, pg, fg)
    pg.add_(3)
    graph.replay()
    torch.cuda.synchronize()
    ref.assert_rotated(captured, x, pos + 3, freq)


def test_python_refusals_on_the_gpu(sha):
    x = torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda")
    pos, freq = torch.zeros(4, dtype=torch.int32, device="cuda"), ref.frequencies(64).cuda()
    for bad in (lambda: sha.sha_rope(x, pos.long(), freq), lambda: sha.sha_rope(x, pos[:3], freq),
                lambda: sha.sha_rope(x, pos, freq.float()), lambda: sha.sha_rope(x, pos.cpu(), freq),
                lambda: sha.sha_rope(x[..., ::2], pos, freq), lambda: sha.sha_rope(x[0], pos, freq),
                lambda: sha.sha_rope(x, pos, freq, out=x[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        sha.sha_rope(x.float(), pos, freq)
    with pytest.raises(TypeError):
        sha.sha_rope(x, pos, freq, out=x.bfloat16())
    with pytest.raises(sha.ShaError) as e:                # not 16-byte aligned
        sha.sha_rope(x.flatten()[1:449].reshape(-1, 1, 64), pos[:1].expand(7).contiguous(), freq)
    assert e.value.status == sha.SHA_ERR_MISALIGNED


# ---------------------------------------------------------------- appending

def _cache(B, pages, ps, H_kv, d, dtype, seed, spare=3):
    g = torch.Generator().manual_seed(seed)
    n = B * pages + spare
    kp = torch.randn((n, H_kv, ps, d), generator=g).to(DT[dtype])
    vp = torch.randn((n, H_kv, ps, d), generator=g).to(DT[dtype])
    table = torch.randperm(n, generator=g)[:B * pages].reshape(B, pages).to(torch.int32)
    return kp, vp, table


def _check_append(sha, k, v, kp, vp, table, pos, rows=None, freq=None, q=None, interleaved=False,
                  mscale=1.0, skipped=()):
    """Runs the call and compares pools and queries; tokens in `skipped` must leave no trace."""
    T, H_kv, d = k.shape
    ps = kp.shape[2]
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    kg, vg = kp.cuda(), vp.cuda()
    q_out = None if q is None else torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    got = sha.sha_append_paged(cu(k), cu(v), kg, vg, cu(table), cu(pos), rows=cu(rows),
                               inv_freq=cu(freq), interleaved=interleaved, mscale=mscale, q=cu(q),
                               q_out=q_out)
    torch.cuda.synchronize()
    live = [t for t in range(T) if t not in skipped]
    row = rows if rows is not None else torch.arange(T)
    touched = torch.zeros(kp.shape[0], ps, dtype=torch.bool)
    kc, vc = kg.cpu(), vg.cpu()
    new_k = torch.empty_like(k)
    for t in live:
        page, off = int(table[int(row[t]), int(pos[t]) // ps]), int(pos[t]) % ps
        assert not touched[page, off]
        touched[page, off] = True
        new_k[t] = kc[page, :, off]
        assert torch.equal(vc[page, :, off], v[t])
    if freq is None:
        assert all(torch.equal(new_k[t], k[t]) for t in live)
    elif live:
        ref.assert_rotated(new_k[live], k[live], pos[live], freq, interleaved, mscale)
    for before, after in ((kp, kc), (vp, vc)):            # every other slot as it was
        keep = ~touched[:, None, :, None].expand(before.shape)
        assert torch.equal(before[keep], after[keep])
    if q is not None:
        assert got is q_out
        if live:
            ref.assert_rotated(got[live], q[live], pos[live], freq, interleaved, mscale)
        for t in skipped:
            assert (got[t] == 3.0).all()
    return sha.sha_get_device_status()


@pytest.mark.parametrize("page_size", [1, 5, 16, 128])
@pytest.mark.parametrize("B,H_q,H_kv,d,rotary,interleaved", [
    (1, 32, 32, 128, 128, False), (9, 8, 1, 64, 64, False), (37, 64, 8, 128, 64, True),
    (4, 6, 2, 72, 36, False), (3, 0, 72, 64, 22, True)])
def test_append_decode_step(sha, B, H_q, H_kv, d, rotary, interleaved, page_size):
    """One token for each row, at each row's own length."""
    for dtype in DT:
        pages = -(-40 // page_size)
        kp, vp, table = _cache(B, pages, page_size, H_kv, d, dtype, B + page_size)
        qkv = _randn((B, H_q + 2 * H_kv, d), B, dtype)
        q, k, v = qkv.split([H_q, H_kv, H_kv], dim=1)
        pos = _positions(B, pages * page_size, B)
        assert _check_append(sha, k, v, kp, vp, table, pos, freq=ref.frequencies(rotary),
                             q=q if H_q else None, interleaved=interleaved,
                             mscale=0.75) == sha.SHA_OK


def test_append_ragged_prompts(sha):
    """Chunks of several sequences behind what they hold, one of them empty."""
    H_kv, d, ps = 4, 128, 16
    share, past = [33, 0, 1, 130], [7, 0, 15, 20]
    kp, vp, table = _cache(4, 10, ps, H_kv, d, "bf16", 21)
    rows = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(share)])
    pos = torch.cat([torch.arange(p, p + n, dtype=torch.int32) for p, n in zip(past, share)])
    T = int(pos.numel())
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(2))
    rows, pos = rows[perm], pos[perm]                     # in any order
    qkv = _randn((T, 8 + 2 * H_kv, d), 22, "bf16")
    q, k, v = qkv.split([8, H_kv, H_kv], dim=1)
    assert _check_append(sha, k, v, kp, vp, table, pos, rows=rows, freq=ref.frequencies(d),
                         q=q) == sha.SHA_OK


def test_append_without_rotation(sha):
    kp, vp, table = _cache(3, 2, 16, 2, 64, "fp16", 31)
    k, v = _randn((3, 2, 64), 32, "fp16"), _randn((3, 2, 64), 33, "fp16")
    assert _check_append(sha, k, v, kp, vp, table, _positions(3, 32, 31)) == sha.SHA_OK


def test_append_padded_batch(sha):
    """Position -1 marks no token: nothing of it is read into the cache, and nothing is flagged."""
    kp, vp, table = _cache(4, 2, 16, 2, 64, "fp16", 41)
    qkv = _randn((4, 8, 64), 42, "fp16")
    qkv[1] = float("nan")
    q, k, v = qkv.split([4, 2, 2], dim=1)
    pos = torch.tensor([3, -1, 31, -1], dtype=torch.int32)
    table[1] = 10 ** 6                                    # a padding row's table is not read
    assert _check_append(sha, k, v, kp, vp, table, pos, freq=ref.frequencies(64), q=q,
                         skipped=(1, 3)) == sha.SHA_OK
    none = torch.full((4,), -1, dtype=torch.int32)
    assert _check_append(sha, k, v, kp, vp, table, none, freq=ref.frequencies(64), q=q,
                         skipped=(0, 1, 2, 3)) == sha.SHA_OK


@pytest.mark.parametrize("what", ["position", "negative", "row", "row_negative", "page",
                                  "page_negative"])
def test_append_bad_slots_are_flagged_and_left_alone(sha, what):
    kp, vp, table = _cache(4, 2, 16, 2, 64, "bf16", 51)
    qkv = _randn((4, 8, 64), 52, "bf16")
    q, k, v = qkv.split([4, 2, 2], dim=1)
    pos, rows = torch.tensor([3, 9, 31, 0], dtype=torch.int32), torch.arange(4, dtype=torch.int32)
    if what == "position":
        pos[1] = 32
    elif what == "negative":
        pos[1] = -2
    elif what == "row":
        rows[1] = 4
    elif what == "row_negative":
        rows[1] = -1
    elif what == "page":
        table[1, 0] = kp.shape[0]
    else:
        table[1, 0] = -1
    assert _check_append(sha, k, v, kp, vp, table, pos, rows=rows, freq=ref.frequencies(64), q=q,
                         skipped=(1,)) == sha.SHA_ERR_BAD_INDEX
    assert sha.sha_get_device_status() == sha.SHA_OK


def test_append_queries_in_place(sha):
    kp, vp, table = _cache(5, 1, 16, 2, 128, "bf16", 61)
    qkv = _randn((5, 10, 128), 62, "bf16")
    pos, freq = _positions(5, 16, 61), ref.frequencies(128)
    g = qkv.cuda()
    q, k, v = g.split([6, 2, 2], dim=1)
    got = sha.sha_append_paged(k, v, kp.cuda(), vp.cuda(), table.cuda(), pos.cuda(),
                               inv_freq=freq.cuda(), q=q, q_out=q)
    assert got is q
    ref.assert_rotated(q, qkv[:, :6], pos, freq)
    assert torch.equal(g[:, 6:].cpu(), qkv[:, 6:])


def test_append_beyond_32_bits(sha):
    """A slot whose element offset in the pool is past 2^32 (a 9 GiB pool a side)."""
    H_kv, ps, d = 8, 64, 128
    n = (1 << 32) // (H_kv * ps * d) + 64
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GiB of free device memory")
    kp = torch.zeros((n, H_kv, ps, d), dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    k, v = _randn((1, H_kv, d), 71, "fp16"), _randn((1, H_kv, d), 72, "fp16")
    table = torch.tensor([[n - 1]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([63], dtype=torch.int32)
    freq = ref.frequencies(128)
    sha.sha_append_paged(k.cuda(), v.cuda(), kp, vp, table, pos.cuda(), inv_freq=freq.cuda())
    ref.assert_rotated(kp[n - 1, :, 63][None], k, pos, freq)
    assert torch.equal(vp[n - 1, :, 63].cpu(), v[0])
    assert int((vp != 0).sum()) == int((v != 0).sum())


def test_append_then_decode_reads_what_was_written(sha):
    """A step over a cache grown token by token equals the decode of the same keys rotated at once."""
    B, H_q, H_kv, d, ps, n = 2, 8, 2, 64, 8, 21
    kp, vp, table = _cache(B, 3, ps, H_kv, d, "bf16", 81)
    kp, vp, table = kp.cuda(), vp.cuda(), table.cuda()
    qkv = _randn((n, B, H_q + 2 * H_kv, d), 82, "bf16")
    freq = ref.frequencies(d)
    idx = torch.arange(H_kv, dtype=torch.int32, device="cuda").expand(B, H_kv).contiguous()
    for t in range(n):
        q, k, v = qkv[t].cuda().split([H_q, H_kv, H_kv], dim=1)
        pos = torch.full((B,), t, dtype=torch.int32, device="cuda")
        rot = sha.sha_append_paged(k, v, kp, vp, table, pos, inv_freq=freq.cuda(), q=q)
    out = torch.zeros((B, H_q, d), dtype=torch.bfloat16, device="cuda")
    sha.sha_decode_paged(rot, kp, vp, idx, pos + 1, table, d ** -0.5, out)
    assert sha.sha_get_device_status() == sha.SHA_OK
    q, k, v = qkv.double().split([H_q, H_kv, H_kv], dim=2)
    at = torch.arange(n)
    for b in range(B):
        kr = ref.rotate(k[:, b], at, freq).to(torch.bfloat16).double()
        qr = ref.rotate(q[n - 1, b][None], at[-1:], freq)[0].to(torch.bfloat16).double()
        for h in range(H_q):
            w = torch.softmax(kr[:, h // 4] @ qr[h] * d ** -0.5, dim=0)
            want = (w[:, None] * v[:, b, h // 4]).sum(0)
            # the decode's own bound at these inputs (parity.TOLERANCE of bf16)
            assert (out[b, h].cpu().double() - want).abs().max() <= 1.5e-2
