"""The serving operators as they are used together: decode steps that append, rotate and attend
over a paged cache (append_decode_paged), with and without a shared prefix, against the same
steps in 64 bits; and their pipeline waits giving up."""
import math
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import rope_reference as rope
from prefix_reference import HALF_STEP

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sha():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import head_sparse_decode_b200 as h
    return h


class Steps:
    """B rows behind a prompt of `prefix` keys in shared pages, `steps` tokens decoded for each."""

    def __init__(self, B, H_q, H_kv, d, top_k, prefix, steps, page_size, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        self.B, self.H_q, self.H_kv, self.d, self.G = B, H_q, H_kv, d, H_q // H_kv
        self.prefix, self.steps, self.page_size, self.dtype = prefix, steps, page_size, dtype
        # quarter turns: a rotation that swaps and negates, so that rounding it changes nothing
        # and the decode's own bound holds for the whole step
        self.freq = (torch.arange(d // 2) % 4).double() * (math.pi / 2)
        self.prompt = [torch.randn((prefix, H_kv, d), generator=g).to(dtype) for _ in range(2)]
        self.fused = torch.randn((steps, B, H_q + 2 * H_kv, d), generator=g).to(dtype)
        first, shared = prefix // page_size, -(-prefix // page_size)
        pages = -(-(prefix + steps) // page_size)
        n = shared + B * (pages - first) + 2
        perm = torch.randperm(n, generator=g).to(torch.int32)
        self.prefix_table = perm[:shared].contiguous()
        self.table = torch.cat([self.prefix_table[:first].expand(B, first),
                                perm[shared:shared + B * (pages - first)].reshape(B, -1)], dim=1)
        self.table = self.table.contiguous()
        self.k_pages = torch.full((n, H_kv, page_size, d), float("nan"), dtype=dtype)
        self.v_pages = self.k_pages.clone()
        self.idx = [torch.rand((B, H_kv), generator=g).argsort(dim=1)[:, :top_k]
                    .to(torch.int32).contiguous() for _ in range(steps)]

    def split(self, t):
        return self.fused[t].split([self.H_q, self.H_kv, self.H_kv], dim=1)

    def run(self, sha, shared, stream=None):
        """Prefill, then the steps; the outputs of every step (rows not selected are 9)."""
        dev = "cuda"
        kp, vp = self.k_pages.to(dev), self.v_pages.to(dev)
        table, pt, freq = self.table.to(dev), self.prefix_table.to(dev), self.freq.to(dev)
        pos = torch.arange(self.prefix, dtype=torch.int32, device=dev)
        row = torch.zeros(self.prefix, dtype=torch.int32, device=dev)
        k, v = (x.to(dev) for x in self.prompt)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        sha.sha_append_paged(k, v, kp, vp, pt[None].contiguous(), pos, rows=row, inv_freq=freq,
                             stream=stream)
        if not shared or self.prefix % self.page_size:
            # without sharing every row's first pages hold the prompt; with it only the last
            # shared page's keys have a copy in each row's own page, and it is not read
            for b in range(self.B if not shared else 0):
                sha.sha_append_paged(k, v, kp, vp, table, pos, rows=row + b, inv_freq=freq)
        outs = []
        for t in range(self.steps):
            q, k, v = (x.to(dev) for x in self.split(t))
            at = torch.full((self.B,), self.prefix + t, dtype=torch.int32, device=dev)
            out = torch.full((self.B, self.H_q, self.d), 9.0, dtype=self.dtype, device=dev)
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            got = sha.append_decode_paged(q, k, v, kp, vp, self.idx[t].to(dev), at, at + 1, table,
                                          inv_freq=freq, prefix_len=self.prefix if shared else 0,
                                          prefix_table=pt if shared else None,
                                          scale=self.d ** -0.5, out=out, stream=stream)
            assert got is out
            if stream is not None:
                stream.synchronize()
            outs.append(out.cpu())
        assert sha.sha_get_device_status() == sha.SHA_OK
        return outs

    def check(self, outs):
        """The bound is that of the decode (prefix_reference)."""
        u = HALF_STEP[self.dtype]
        at = torch.arange(self.prefix + self.steps)
        keys = torch.cat([self.prompt[0][:, None].expand(-1, self.B, -1, -1),
                          torch.stack([self.split(t)[1] for t in range(self.steps)])])
        vals = torch.cat([self.prompt[1][:, None].expand(-1, self.B, -1, -1),
                          torch.stack([self.split(t)[2] for t in range(self.steps)])])
        for t, out in enumerate(outs):
            n = self.prefix + t + 1
            q = self.split(t)[0]
            want = torch.full(out.shape, 9.0, dtype=torch.float64)
            bound = torch.zeros_like(want)
            for b in range(self.B):
                k = rope.rotate(keys[:n, b], at[:n], self.freq).to(self.dtype).double()
                v = vals[:n, b].double()
                qr = rope.rotate(q[b][None], at[n - 1:n], self.freq)[0].to(self.dtype).double()
                for h in self.idx[t][b].tolist():
                    qh = qr[h * self.G:(h + 1) * self.G]
                    w = torch.softmax(qh @ k[:, h].T * self.d ** -0.5, dim=1)
                    o, A = w @ v[:, h], w @ v[:, h].abs()
                    S = self.d ** -0.5 * (qh.abs() @ k[:, h].abs().T).max()
                    want[b, h * self.G:(h + 1) * self.G] = o
                    bound[b, h * self.G:(h + 1) * self.G] = \
                        u * (o.abs() + A) + n * 2.0 ** -25 * v[:, h].abs().max() \
                        + A * (2 * (self.d + 2) * 2.0 ** -23 * S + 2.0 ** -20 + n * 2.0 ** -23)
            excess = (out.double() - want).abs() - bound
            assert excess.max() <= 0, f"step {t}: {float(excess.max())} over the bound"


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,H_q,H_kv,d,top_k,prefix,page_size,dtype", [
    (3, 8, 2, 64, 1, 37, 8, torch.bfloat16), (5, 6, 6, 128, 4, 64, 16, torch.float16),
    (2, 32, 2, 128, 2, 130, 64, torch.bfloat16)])
def test_decode_steps(sha, B, H_q, H_kv, d, top_k, prefix, page_size, dtype, shared):
    s = Steps(B, H_q, H_kv, d, top_k, prefix, 11, page_size, dtype, seed=B + prefix)
    s.check(s.run(sha, shared))


def test_decode_steps_on_another_stream(sha):
    s = Steps(4, 8, 4, 64, 2, 50, 6, 16, torch.float16, seed=7)
    first = s.run(sha, True)
    other = s.run(sha, True, stream=torch.cuda.Stream())
    assert all(torch.equal(a, b) for a, b in zip(first, other))


def test_new_tensors_belong_to_the_stream_that_uses_them(sha):
    """Memory just freed on the current stream, whose work on it may be pending, is not handed to
    a call on another stream."""
    other = torch.cuda.Stream()
    x = torch.zeros((512, 16, 128), dtype=torch.float16, device="cuda")
    pos = torch.zeros(512, dtype=torch.int32, device="cuda")
    freq = torch.zeros(64, dtype=torch.float64, device="cuda")
    torch.cuda.synchronize()
    for stream in (other, other.cuda_stream):
        freed = torch.empty_like(x)
        at = freed.data_ptr()
        del freed
        out = sha.sha_rope(x, pos, freq, stream=stream)
        assert out.data_ptr() != at
        other.synchronize()
        del out
        again = torch.empty_like(x)                       # it is still the current stream's
        assert again.data_ptr() == at
        del again


def test_captured_step(sha):
    """A step captured once and replayed for each token: positions and lengths move on the device."""
    s = Steps(3, 8, 2, 128, 1, 40, 9, 8, torch.bfloat16, seed=8)
    want = s.run(sha, True)
    dev = "cuda"
    kp, vp = s.k_pages.to(dev), s.v_pages.to(dev)
    table, pt, freq = s.table.to(dev), s.prefix_table.to(dev), s.freq.to(dev)
    sha.sha_append_paged(s.prompt[0].to(dev), s.prompt[1].to(dev), kp, vp, pt[None].contiguous(),
                         torch.arange(40, dtype=torch.int32, device=dev),
                         rows=torch.zeros(40, dtype=torch.int32, device=dev), inv_freq=freq)
    fused = torch.zeros_like(s.fused[0], device=dev)
    q, k, v = fused.split([8, 2, 2], dim=1)
    idx = torch.zeros((3, 1), dtype=torch.int32, device=dev)
    at = torch.full((3,), -1, dtype=torch.int32, device=dev)
    lens = torch.full((3,), 40, dtype=torch.int32, device=dev)
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device=dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sha.append_decode_paged(q, k, v, kp, vp, idx, at, lens, table, inv_freq=freq, prefix_len=40,
                                prefix_table=pt, scale=128 ** -0.5, out=out)
    for t in range(9):
        fused.copy_(s.fused[t])
        idx.copy_(s.idx[t])
        at.fill_(40 + t)
        lens.fill_(41 + t)
        out.fill_(9.0)
        graph.replay()
        assert torch.equal(out.cpu(), want[t])
    assert sha.sha_get_device_status() == sha.SHA_OK


def test_refusals(sha):
    s = Steps(2, 4, 2, 64, 1, 16, 2, 8, torch.float16, seed=9)
    q, k, v = (x.cuda() for x in s.split(0))
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    args = (s.k_pages.cuda(), s.v_pages.cuda(), s.idx[0].cuda(), i, i + 1, s.table.cuda())
    with pytest.raises(ValueError):
        sha.append_decode_paged(q[:1], k, v, *args)
    with pytest.raises(ValueError):
        sha.append_decode_paged(q[0], k, v, *args)
    with pytest.raises(ValueError):                       # not contiguous, and nothing turns it
        sha.append_decode_paged(s.fused[0].cuda()[:, :4], k, v, *args)


@pytest.mark.parametrize("prefix_len", [0, 16])
def test_a_refused_step_has_written_nothing(sha, prefix_len):
    """Whatever is wrong with a step's arguments, and however late it is found: the cache, the
    queries and the output stay as they were."""
    s = Steps(2, 4, 2, 64, 1, 16, 2, 8, torch.float16, seed=9)
    fused = s.fused[0].cuda()
    q, k, v = fused.split([4, 2, 2], dim=1)
    at = torch.full((2,), 16, dtype=torch.int32, device="cuda")
    kp, vp = (torch.full_like(p, 5.0, device="cuda") for p in (s.k_pages, s.v_pages))
    pt, freq = s.prefix_table.cuda(), s.freq.cuda()
    out = torch.full((2, 4, 64), 9.0, dtype=torch.float16, device="cuda")
    good = dict(q=q, k=k, v=v, k_pages=kp, v_pages=vp, batch_head_index=s.idx[0].cuda(),
                positions=at, seqlens=at + 1, block_table=s.table.cuda(), inv_freq=freq,
                prefix_len=prefix_len, prefix_table=pt, scale=0.125, out=out)
    odd = torch.full((kp.shape[0], 2, 12, 64), 5.0, dtype=torch.float16, device="cuda")
    refused = [
        (ValueError, dict(batch_head_index=s.idx[0].cuda().long())),
        (ValueError, dict(batch_head_index=s.idx[0].cuda()[:1])),
        (ValueError, dict(seqlens=at[:1])), (ValueError, dict(seqlens=at.long())),
        (ValueError, dict(block_table=s.table.cuda()[:1])), (ValueError, dict(positions=at.cpu())),
        (ValueError, dict(out=out[:1])), (ValueError, dict(out=out.float())),
        (ValueError, dict(out=out.cpu())), (ValueError, dict(inv_freq=freq.float())),
        (ValueError, dict(inv_freq=None)), (ValueError, dict(prefix_len=-1)),
        (ValueError, dict(workspace=torch.empty(1 << 24))), (ValueError, dict(v_pages=vp[1:])),
        (ValueError, dict(prefix_len=17)), (ValueError, dict(prefix_len=16, prefix_table=None)),
        (ValueError, dict(prefix_len=16, prefix_table=pt.long())),
        (sha.ShaError, dict(scale=float("inf"))), (sha.ShaError, dict(mscale=float("nan"))),
        (sha.ShaError, dict(k_pages=odd, v_pages=odd)),
        (sha.ShaError, dict(batch_head_index=torch.zeros((2, 3), dtype=torch.int32,
                                                         device="cuda"))),
        (sha.ShaError, dict(prefix_len=80, prefix_table=torch.zeros(10, dtype=torch.int32,
                                                                    device="cuda"))),
        (sha.ShaError, dict(prefix_len=16, workspace=torch.empty(512, dtype=torch.uint8,
                                                                 device="cuda"))),
    ]
    before = fused.clone()
    for error, bad in refused:
        with pytest.raises(error):
            sha.append_decode_paged(**{**good, **bad})
    torch.cuda.synchronize()
    assert (kp == 5.0).all() and (vp == 5.0).all() and (odd == 5.0).all() and (out == 9.0).all()
    assert torch.equal(fused, before)
    assert sha.sha_get_device_status() == sha.SHA_OK
    sha.append_decode_paged(**good)                       # and as it stands it is taken
    assert sha.sha_get_device_status() == sha.SHA_OK
    assert (kp != 5.0).any() and (out != 9.0).any()


def test_steps_without_a_rotation(sha):
    """Nothing turned: the queries are read where they are, and the keys appended as they are."""
    B, H_q, H_kv, d, n = 3, 8, 2, 64, 20
    g = torch.Generator().manual_seed(17)
    kp, vp = (torch.full((2 * B, H_kv, 16, d), float("nan"), dtype=torch.float16, device="cuda")
              for _ in range(2))
    table = torch.randperm(2 * B, generator=g).reshape(B, 2).to(torch.int32).cuda()
    idx = torch.tensor([[0, 1], [1, 0], [0, 1]], dtype=torch.int32, device="cuda")
    qkv = torch.randn((n, B, H_q + 2 * H_kv, d), generator=g).half()
    for t in range(n):
        q, k, v = qkv[t].cuda().split([H_q, H_kv, H_kv], dim=1)
        at = torch.full((B,), t, dtype=torch.int32, device="cuda")
        out = sha.append_decode_paged(q.contiguous(), k, v, kp, vp, idx, at, at + 1, table)
        assert out.shape == (B, H_q, d)
    assert sha.sha_get_device_status() == sha.SHA_OK
    q, k, v = qkv.double().split([H_q, H_kv, H_kv], dim=2)
    for b in range(B):
        for h in range(H_q):
            w = torch.softmax(k[:, b, h // 4] @ q[-1, b, h] * d ** -0.5, dim=0)
            want, A = w @ v[:, b, h // 4], w @ v[:, b, h // 4].abs()
            S = d ** -0.5 * (q[-1, b, h].abs() @ k[:, b, h // 4].abs().T).max()
            # the decode's bound (prefix_reference)
            bound = 2.0 ** -11 * (want.abs() + A) + n * 2.0 ** -25 * v.abs().max() \
                + A * (2 * (d + 2) * 2.0 ** -23 * S + 2.0 ** -20 + n * 2.0 ** -23)
            assert ((out[b, h].cpu().double() - want).abs() <= bound).all()


class Split:
    """A step whose units are split over blocks and merged through the workspace: few rows, long
    ones.  The keys lie in the cache already, as the step would write them."""

    def __init__(self, B, H_q, H_kv, d, keys, seed):
        g = torch.Generator().manual_seed(seed)
        ps = 64
        pages = -(-keys // ps)
        mk = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        self.kp, self.vp = mk(B * pages, H_kv, ps, d), mk(B * pages, H_kv, ps, d)
        self.table = torch.randperm(B * pages, generator=g).reshape(B, pages).to(torch.int32).cuda()
        self.q = mk(B, H_q, d)
        at = torch.tensor([keys - 1 - 7 * b for b in range(B)])
        rows = torch.arange(B, device="cuda")
        page = self.table[rows, (at // ps).cuda()].long()
        self.k, self.v = (p[page, :, (at % ps).cuda()].clone() for p in (self.kp, self.vp))
        self.at = at.to(torch.int32).cuda()
        self.idx = torch.arange(H_kv, dtype=torch.int32, device="cuda").expand(B, H_kv).contiguous()
        self.lens = self.at + 1
        self.sizes = (B, H_q, H_kv, d, H_kv, pages * ps)
        self.out = torch.empty((B, H_q, d), dtype=torch.bfloat16, device="cuda")

    def step(self, sha, **kw):
        return sha.append_decode_paged(self.q, self.k, self.v, self.kp, self.vp, self.idx, self.at,
                                       self.lens, self.table, out=self.out, **kw)

    def want(self, sha):
        """The same decode by itself."""
        return sha.sha_decode_paged(self.q, self.kp, self.vp, self.idx, self.lens, self.table, None,
                                    torch.empty_like(self.out))


@pytest.mark.parametrize("H_q,H_kv", [(4, 4), (16, 2)])
def test_a_step_without_a_prefix_takes_the_workspace_it_is_given(sha, H_q, H_kv):
    """Whatever the workspace holds, within its bytes, and none that is too small."""
    s = Split(2, H_q, H_kv, 128, 6000, seed=21)
    want = s.want(sha)
    need = sha.append_decode_workspace_size(*s.sizes)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        s.out.zero_()
        s.step(sha, workspace=ws[:need])
        assert torch.equal(s.out, want)
        ws[:need].fill_(0xFF)
    assert (ws[need:] == 0xA5).all()
    with pytest.raises(sha.ShaError) as e:
        s.step(sha, workspace=ws[:256])
    assert e.value.status == sha.SHA_ERR_WORKSPACE
    assert sha.sha_get_device_status() == sha.SHA_OK


def test_steps_without_a_prefix_at_once(sha):
    """Steps on two streams, each with a workspace of its own (given, or new), then captured in
    two graphs that are replayed at once."""
    steps = [Split(2, 16, 2, 128, 9000, seed=31), Split(3, 4, 4, 64, 7000, seed=32)]
    wants = [s.want(sha).clone() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    spaces = [torch.empty(sha.append_decode_workspace_size(*s.sizes), dtype=torch.uint8,
                          device="cuda") for s in steps]
    torch.cuda.synchronize()
    for given in (True, False):
        for _ in range(20):
            for s, stream, ws in zip(steps, streams, spaces):
                s.step(sha, workspace=ws if given else None, stream=stream)
        torch.cuda.synchronize()
        for s, want in zip(steps, wants):
            assert torch.equal(s.out, want)
            s.out.zero_()
    graphs = []
    for s in steps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.step(sha)
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for s, want in zip(steps, wants):
        assert torch.equal(s.out, want)
    assert sha.sha_get_device_status() == sha.SHA_OK


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("H_q,H_kv,d", [(8, 2, 128), (4, 4, 64)])
def test_captured_step_with_padded_rows(sha, H_q, H_kv, d, shared):
    """A step captured for six rows and replayed for fewer: rows without a token leave cache and
    output as they were, raise no flag, and change nothing for the others."""
    s = Steps(6, H_q, H_kv, d, 2, 40, 9, 8, torch.bfloat16, seed=18)
    want = s.run(sha, shared)
    dev = "cuda"
    kp, vp = s.k_pages.to(dev), s.v_pages.to(dev)
    table, pt, freq = s.table.to(dev), s.prefix_table.to(dev), s.freq.to(dev)
    tables = [pt[None].contiguous()] if shared else [table[b:b + 1].contiguous() for b in range(6)]
    for t in tables:
        sha.sha_append_paged(s.prompt[0].to(dev), s.prompt[1].to(dev), kp, vp, t,
                             torch.arange(40, dtype=torch.int32, device=dev),
                             rows=torch.zeros(40, dtype=torch.int32, device=dev), inv_freq=freq)
    fused = torch.zeros_like(s.fused[0], device=dev)
    q, k, v = fused.split([H_q, H_kv, H_kv], dim=1)
    idx = torch.zeros((6, 2), dtype=torch.int32, device=dev)
    at = torch.full((6,), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(6, dtype=torch.int32, device=dev)
    rows_table = table.clone()
    out = torch.empty((6, H_q, d), dtype=torch.bfloat16, device=dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sha.append_decode_paged(q, k, v, kp, vp, idx, at, lens, rows_table, inv_freq=freq,
                                prefix_len=40 if shared else 0, prefix_table=pt if shared else None,
                                scale=d ** -0.5, out=out)
    done = [0] * 6                                        # tokens that each row has
    for rows in ([0, 1, 2, 3, 4, 5], [0, 2], [5], [], [1, 3, 4], [0, 1, 2, 3, 4, 5]):
        fused.fill_(float("nan"))
        # a padded row's token, head ids and pages do not matter
        idx.fill_(-3 if len(rows) % 2 else 1)
        rows_table.fill_(10 ** 6)
        at.fill_(-1)
        lens.zero_()
        for b in rows:
            fused[b].copy_(s.fused[done[b]][b])
            idx[b].copy_(s.idx[done[b]][b])
            rows_table[b].copy_(table[b])
            at[b] = 40 + done[b]
            lens[b] = 41 + done[b]
        out.fill_(9.0)
        graph.replay()
        got = out.cpu()
        assert sha.sha_get_device_status() == sha.SHA_OK
        for b in range(6):
            if b not in rows:
                assert (got[b] == 9.0).all()
                continue
            # cut otherwise than in the full batch: equal up to the order of fp32 sums, and one
            # rounding of the weights and of the output a side (the bound of `check`, twice)
            w, t = want[done[b]][b].double(), done[b]
            vals = torch.cat([s.prompt[1], torch.stack([s.split(i)[2][b] for i in range(t + 1)])])
            assert ((got[b].double() - w).abs()
                    <= 2 * 2.0 ** -8 * (w.abs() + vals.double().abs().max()) + 1e-4)[w != 9.0].all()
            assert (got[b][want[t][b] == 9.0] == 9.0).all()
            done[b] += 1
    # by themselves the decodes take such a row for bad input
    q = torch.zeros((6, H_q, d), dtype=torch.bfloat16, device=dev)
    sha.sha_decode_paged(q, kp, vp, idx, lens * 0, table, 1.0, out)
    assert sha.sha_get_device_status() == sha.SHA_ERR_BAD_INDEX
    sha.sha_decode_prefix(q, kp, vp, idx, lens * 0, table, 40, pt, 1.0, out)
    assert sha.sha_get_device_status() == sha.SHA_ERR_BAD_INDEX


def test_waits_that_give_up(sha):
    """With the test build's wait limit at 1 ns the shared-prefix call's waits run out: it returns,
    reports the timeout, and the next call with the limit restored is right.  In a process of its
    own, since the test build is another library."""
    from head_sparse_decode_b200 import build
    script = textwrap.dedent("""
        import ctypes, torch
        import head_sparse_decode_b200 as sha
        from prefix_reference import Case
        sha._lib.sha_test_set_wait_limit.argtypes = [ctypes.c_ulonglong]
        for c in (Case(40, 16, 2, 128, 2, 700, 300, 16, "bf16", seed=3),
                  Case(5, 4, 4, 64, 2, 300, 40, 8, "fp16", seed=4),
                  Case(3, 32, 2, 128, 1, 200, 100, 64, "fp16", seed=5)):
            q, kp, vp, idx, lens, table, pt = c.on()
            out = torch.zeros_like(q)
            call = lambda: sha.sha_decode_prefix(q, kp, vp, idx, lens, table, c.prefix, pt, c.scale, out)
            assert sha._lib.sha_test_set_wait_limit(1) == 0
            call()
            assert sha.sha_get_device_status() == sha.SHA_ERR_TIMEOUT
            assert sha._lib.sha_test_set_wait_limit(4000000000) == 0
            out.fill_(-77.0)
            call()
            assert sha.sha_get_device_status() == sha.SHA_OK
            c.check(out, *c.reference(), -77.0)
        print("waits gave up and recovered")
    """)
    env = dict(os.environ, SHA_DECODE_LIBRARY=build.build_test_hooks(),
               PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", script], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "waits gave up and recovered" in r.stdout
