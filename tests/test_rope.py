"""Rotary tables, and what sha_rope and sha_append_paged refuse before any launch (CPU)."""
import ctypes
import math
import random

import pytest
import torch

import rope_reference as ref


@pytest.fixture(scope="module")
def sha():
    import head_sparse_decode_b200 as h
    return h


P = 0x1000
S2 = ctypes.c_int64 * 2


def _rope(sha, x=P, pos=P, freq=P, T=3, H=2, d=64, rotary=64, inter=0, mscale=1.0, xs=(128, 64),
          out=P, os=(128, 64), dtype=0):
    return sha._lib.sha_rope(x, pos, freq, T, H, d, rotary, inter, mscale, S2(*xs), out, S2(*os),
                             dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(d=520), 2), (dict(d=60, rotary=32), 2),
    (dict(T=-1), 1), (dict(H=-1), 1), (dict(rotary=0), 1), (dict(rotary=63), 1),
    (dict(rotary=66), 1), (dict(rotary=-2), 1), (dict(inter=2), 1),
    (dict(mscale=float("nan")), 1), (dict(mscale=float("inf")), 1),
    (dict(x=None), 1), (dict(out=None), 1), (dict(pos=None), 1), (dict(freq=None), 1),
    (dict(x=P + 8), 3), (dict(out=P + 2), 3), (dict(pos=P + 2), 3), (dict(freq=P + 4), 3),
    (dict(xs=(132, 64)), 3), (dict(xs=(128, 60)), 3), (dict(os=(132, 64)), 3),
    (dict(xs=(-128, 64)), 1), (dict(os=(0, 64)), 1), (dict(os=(128, 0)), 1),
    (dict(os=(128, 56)), 1),
    (dict(T=0), 0), (dict(H=0), 0), (dict(T=0, x=None, out=None, pos=None, freq=None), 0),
])
def test_rope_host_checks(sha, kw, code):
    assert _rope(sha, **kw) == code


def _append(sha, k=P, v=P, ks=(128, 64), vs=(128, 64), T=3, H_kv=2, d=64, kp=P, vp=P, bt=P,
            rows=P, pos=P, B=2, num_pages=4, page_size=16, max_pages=2, freq=P, rotary=64, inter=0,
            mscale=1.0, q=P, qs=(256, 64), H_q=4, qo=P, qos=(256, 64), dtype=1):
    return sha._lib.sha_append_paged(k, v, S2(*ks), S2(*vs), T, H_kv, d, kp, vp, bt, rows, pos, B,
                                     num_pages, page_size, max_pages, freq, rotary, inter, mscale,
                                     q, S2(*qs), H_q, qo, S2(*qos), dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), 2), (dict(d=12, rotary=12), 2), (dict(T=-1), 1), (dict(H_kv=0), 1),
    (dict(H_q=-1), 1), (dict(B=-1), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1),
    (dict(max_pages=0), 1), (dict(page_size=1 << 20, max_pages=1 << 12), 1),
    (dict(rows=None, T=3, B=2), 1),                       # token t is row t's: T <= B
    (dict(rotary=0), 1),                                  # queries, but nothing to do to them
    (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1), (dict(vp=None), 1),
    (dict(bt=None), 1), (dict(pos=None), 1), (dict(freq=None), 1), (dict(q=None), 1),
    (dict(qo=None), 1),
    (dict(k=P + 4), 3), (dict(v=P + 8), 3), (dict(kp=P + 8), 3), (dict(vp=P + 8), 3),
    (dict(bt=P + 1), 3), (dict(rows=P + 2), 3), (dict(pos=P + 2), 3), (dict(q=P + 2), 3),
    (dict(qo=P + 2), 3), (dict(freq=P + 4), 3), (dict(ks=(130, 64)), 3), (dict(vs=(128, 65)), 3),
    (dict(qs=(257, 64)), 3), (dict(qos=(0, 64)), 1), (dict(qos=(256, 8)), 1),
    (dict(T=0), 0), (dict(T=0, k=None, v=None, q=None, qo=None), 0),
])
def test_append_host_checks(sha, kw, code):
    assert _append(sha, **kw) == code


@pytest.mark.parametrize("T,H,s0,s1", [
    (2, 2, 64, 64), (3, 2, 64, 72), (4, 3, 128, 192), (2, 4, 136, 192), (64, 40, 64, 64)])
def test_outputs_whose_rows_overlap_are_refused(sha, T, H, s0, s1):
    """Two rows that share elements have no one result."""
    assert _rope(sha, T=T, H=H, xs=(0, 0), os=(s0, s1)) == 1
    assert _append(sha, T=T, B=T, H_q=H, qs=(0, 0), qos=(s0, s1)) == 1


def test_overlap_check_is_exact(sha):
    """Against the rows' addresses, sorted; nested views and interleaved ones."""
    from head_sparse_decode_b200 import build
    lib = ctypes.CDLL(build.build_test_hooks())
    lib.sha_test_rows_lie_apart.argtypes = [ctypes.c_int64] * 5
    rng, seen = random.Random(3), []
    for _ in range(20000):
        T, H, d = rng.randint(2, 9), rng.randint(2, 9), rng.choice([8, 64])
        s0, s1 = (8 * rng.randint(d // 8, 90) for _ in range(2))
        rows = sorted(t * s0 + h * s1 for t in range(T) for h in range(H))
        apart = all(y - x >= d for x, y in zip(rows, rows[1:]))
        assert bool(lib.sha_test_rows_lie_apart(s0, T, s1, H, d)) == apart
        nested = s0 >= s1 * (H - 1) + d or s1 >= s0 * (T - 1) + d
        seen.append((apart, nested))
    assert {(True, True), (True, False), (False, False)} == set(seen)
    far = (1 << 62) // 8 * 8
    assert lib.sha_test_rows_lie_apart(far, 3, far - 8, 3, 8)
    assert not lib.sha_test_rows_lie_apart(far, 3, far - 8, 3, 16)


def test_python_refusals(sha):
    x = torch.zeros(2, 3, 64, dtype=torch.float16)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):                       # not on a GPU
        sha.sha_rope(x, pos, ref.frequencies(64))
    with pytest.raises(ValueError):
        sha.sha_append_paged(x, x, x, x, pos, pos)


def test_frequencies_plain(sha):
    freq, m = sha.rope_frequencies(128, 500000.0)
    assert freq.dtype == torch.float64 and m == 1.0
    want = torch.tensor([500000.0 ** (-2.0 * i / 128) for i in range(64)], dtype=torch.float64)
    assert torch.allclose(freq, want, rtol=1e-14, atol=0)


def test_frequencies_scaled(sha):
    r, n, f = 64, 4096, 4.0
    plain, _ = sha.rope_frequencies(r)
    linear, m = sha.rope_frequencies(r, scaling={"kind": "linear", "factor": f})
    assert m == 1.0 and torch.allclose(linear * f, plain, rtol=1e-14, atol=0)
    # ntk: the first pair as it was, the last one divided by f
    ntk, m = sha.rope_frequencies(r, scaling={"kind": "ntk", "factor": f})
    assert m == 1.0 and float(ntk[0]) == 1.0
    assert math.isclose(float(ntk[-1] * f), float(plain[-1]), rel_tol=1e-12)
    # bands: fast pairs kept, slow ones divided, the rest between, in order
    bands, m = sha.rope_frequencies(r, scaling={"kind": "bands", "factor": f, "original_length": n})
    turns = ref.turns_of_table(plain, n)
    assert m == 1.0 and (bands[turns >= 4] == plain[turns >= 4]).all()
    assert torch.allclose(bands[turns <= 1] * f, plain[turns <= 1], rtol=1e-14, atol=0)
    between = (turns > 1) & (turns < 4)
    assert between.any() and (bands[between] < plain[between]).all()
    assert (bands[between] * f > plain[between]).all()
    # yarn: the same at both ends, and a factor on the result
    yarn, m = sha.rope_frequencies(r, scaling={"kind": "yarn", "factor": f, "original_length": n})
    assert math.isclose(m, 0.1 * math.log(f) + 1.0)
    assert (yarn[turns >= 40] == plain[turns >= 40]).all()
    assert torch.allclose(yarn[turns <= 0.5] * f, plain[turns <= 0.5], rtol=1e-14, atol=0)
    assert (yarn <= plain).all() and (yarn * f >= plain * (1 - 1e-14)).all()
    _, m = sha.rope_frequencies(r, scaling={"kind": "yarn", "factor": f, "original_length": n,
                                            "mscale": 1.0})
    assert m == 1.0


@pytest.mark.parametrize("args,kw", [
    ((3,), {}), ((0,), {}), ((64, 1.0), {}), ((64, float("nan")), {}),
    ((64,), {"scaling": {"kind": "other"}}), ((64,), {"scaling": {"kind": "linear"}}),
    ((64,), {"scaling": {"kind": "linear", "factor": 0.0}}),
    ((64,), {"scaling": {"kind": "linear", "factor": 2.0, "low": 1.0}}),
    ((64,), {"scaling": {"kind": "bands", "factor": 2.0}}),
    ((64,), {"scaling": {"kind": "bands", "factor": 2.0, "original_length": 64, "low": 4.0}}),
    ((2,), {"scaling": {"kind": "ntk", "factor": 2.0}}),
])
def test_frequencies_refusals(sha, args, kw):
    with pytest.raises(ValueError):
        sha.rope_frequencies(*args, **kw)
