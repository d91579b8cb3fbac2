"""What a decode step (sha_append_decode_paged) refuses before any launch (CPU)."""
import ctypes

import pytest
import torch

P = 0x1000
S2 = ctypes.c_int64 * 2


@pytest.fixture(scope="module")
def sha():
    import head_sparse_decode_b200 as h
    return h


def _step(sha, q=P, qs=(512, 64), k=P, ks=(128, 64), v=P, vs=(128, 64), kp=P, vp=P, bt=P, idx=P,
          pos=P, lens=P, freq=P, rotary=64, inter=0, mscale=1.0, turned=P, pt=P, prefix_len=0, B=2,
          H_q=8, H_kv=2, num_pages=9, page_size=16, max_pages=4, d=64, top_k=1, scale=0.125, out=P,
          dtype=0, ws=0x1000, ws_bytes=0):
    return sha._lib.sha_append_decode_paged(
        q, S2(*qs), k, S2(*ks), v, S2(*vs), kp, vp, bt, idx, pos, lens, freq, rotary, inter, mscale,
        turned, pt, prefix_len, B, H_q, H_kv, num_pages, page_size, max_pages, d, top_k, scale, out,
        dtype, ws, ctypes.c_size_t(ws_bytes), None)


@pytest.mark.parametrize("prefix_len", [0, 20])
@pytest.mark.parametrize("kw,code", [
    # the append's
    (dict(dtype=3), 2), (dict(rotary=63), 1), (dict(rotary=66), 1), (dict(inter=2), 1),
    (dict(mscale=float("nan")), 1), (dict(B=-1), 1), (dict(H_kv=0), 1), (dict(num_pages=0), 1),
    (dict(max_pages=1 << 27), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1),
    (dict(turned=None), 1), (dict(freq=None), 1), (dict(pos=None), 1), (dict(k=P + 8), 3),
    (dict(q=P + 8), 3), (dict(turned=P + 8), 3), (dict(freq=P + 4), 3), (dict(pos=P + 2), 3),
    (dict(qs=(516, 64)), 3), (dict(ks=(-128, 64)), 1),
    # the decode's
    (dict(d=72), 2), (dict(H_q=9), 1), (dict(H_q=0), 1), (dict(H_q=34), 2), (dict(page_size=12), 2),
    (dict(top_k=3), 1), (dict(top_k=-1), 1), (dict(scale=float("nan")), 1), (dict(idx=None), 1),
    (dict(lens=None), 1), (dict(bt=None), 1), (dict(out=None), 1), (dict(idx=P + 2), 3),
    (dict(lens=P + 2), 3), (dict(out=P + 8), 3),
    # without a rotation
    (dict(rotary=0, q=None), 1), (dict(rotary=0, q=P + 8), 3),
])
def test_host_checks(sha, kw, code, prefix_len):
    assert _step(sha, prefix_len=prefix_len, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(prefix_len=-1), 1), (dict(prefix_len=65), 1), (dict(prefix_len=20, pt=None), 1),
    (dict(prefix_len=20, pt=P + 2), 3), (dict(prefix_len=20, ws=P + 16), 3),
    (dict(prefix_len=20, H_q=2000, H_kv=2000, ks=(128000, 64), vs=(128000, 64),
          qs=(128000, 64)), 2),
    (dict(B=0), 0), (dict(B=0, q=None, k=None, v=None, out=None, ws=None), 0),
])
def test_host_checks_of_the_prefix_and_empty_steps(sha, kw, code):
    assert _step(sha, **kw) == code


def test_workspace_sizes_of_sizes_it_would_reject(sha):
    size = sha._lib.sha_append_decode_workspace_size
    assert size(2, 8, 2, 64, 1, 0, 0) == 0                # no keys
    assert size(2, 8, 2, 72, 1, 64, 0) == size(2, 9, 2, 64, 1, 64, 0) == 0
    assert size(0, 8, 2, 64, 1, 64, 0) == size(2, 8, 2, 64, 0, 64, 0) == 0
    assert size(2, 8, 2, 64, 1, 64, -1) == 0


def test_python_refusals(sha):
    t = torch.zeros(2, 2, 64, dtype=torch.float16)
    i = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError):                       # not on a GPU
        sha.append_decode_paged(t, t, t, t[None], t[None], i, i[:, 0], i[:, 0], i)
