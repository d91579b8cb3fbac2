"""What sha_decode_prefix refuses before any launch (CPU)."""
import ctypes

import pytest
import torch

P = 0x1000


@pytest.fixture(scope="module")
def sha():
    import head_sparse_decode_b200 as h
    return h


def _call(sha, q=P, k=P, v=P, idx=P, lens=P, bt=P, pt=P, prefix_len=20, B=2, H_q=8, H_kv=2,
          num_pages=9, page_size=16, max_pages=4, d=64, top_k=1, scale=0.125, out=P, dtype=0,
          ws=0x1000, ws_bytes=0):
    return sha._lib.sha_decode_prefix(q, k, v, idx, lens, bt, pt, prefix_len, B, H_q, H_kv,
                                      num_pages, page_size, max_pages, d, top_k, scale, out, dtype,
                                      ws, ctypes.c_size_t(ws_bytes), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 2), (dict(d=96), 2), (dict(H_q=34, H_kv=2), 2), (dict(page_size=12), 2),
    (dict(page_size=4, prefix_len=3), 2), (dict(page_size=1, prefix_len=3), 2), (dict(H_q=2000, H_kv=2000), 2),
    (dict(num_pages=1 << 30, H_kv=8), 2), (dict(B=1 << 24, top_k=2), 2),
    (dict(prefix_len=0), 1), (dict(prefix_len=-3), 1), (dict(prefix_len=65), 1),
    (dict(num_pages=0), 1), (dict(page_size=0), 1), (dict(max_pages=0), 1),
    (dict(max_pages=1 << 27), 1), (dict(B=-1), 1), (dict(H_q=9), 1), (dict(H_kv=0), 1),
    (dict(top_k=3), 1), (dict(top_k=-1), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(idx=None), 1),
    (dict(lens=None), 1), (dict(bt=None), 1), (dict(pt=None), 1), (dict(out=None), 1),
    (dict(q=P + 8), 3), (dict(k=P + 8), 3), (dict(v=P + 8), 3), (dict(out=P + 8), 3),
    (dict(idx=P + 2), 3), (dict(lens=P + 2), 3), (dict(bt=P + 2), 3), (dict(pt=P + 2), 3),
    (dict(ws=P + 16), 3),
    (dict(B=0), 0), (dict(top_k=0), 0), (dict(B=0, q=None, ws=None), 0),
])
def test_host_checks(sha, kw, code):
    assert _call(sha, **kw) == code


def test_python_refusals(sha):
    t = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):                       # not on a GPU
        sha.sha_decode_prefix(t[:, :, 0], t, t, t, t, t, 1, t, 0.1, t)
