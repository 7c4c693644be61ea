"""The 4-bit KV cache calls refuse bad arguments on the host, before any launch (no GPU needed), and the
oracle's format agrees with its definition."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_long_context_pq_b200 as P
from oracle import kv4_oracle as O4
from sparse_long_context_pq_b200 import build as B

FAKE = 1 << 20   # 256-byte aligned, never touched


@pytest.fixture(scope="module")
def lib():
    B.build()
    if torch.cuda.is_available():
        pytest.skip("host-validation tests with fake device pointers: CPU-only")
    return P.load_library()


def _kv(B_=2, Hq=8, Hkv=2, D=128, page_size=16, max_pages=8, num_pages=16, seq=100, cache=FAKE, table=FAKE, lens=FAKE):
    host = np.full(B_, seq, dtype=np.int32)
    return P._KV4(cache, table, lens, host.ctypes.data, B_, Hq, Hkv, D, page_size, max_pages, num_pages), host


def _cu(*steps):
    return np.cumsum((0,) + steps).astype(np.int32)


def _rows(data=FAKE, token=256, head=128):
    return P._KV4Rows(data, token, head)


def _ws(lib):
    kv, host = _kv()
    return lib.hsa_kv4_workspace_bytes(ctypes.byref(kv))


def _decode(lib, kv, q=FAKE, out=FAKE, lse=None, dtype=1, scale=0.1, window=0, ws=FAKE, n=None):
    return lib.dense_decode_kv4(ctypes.byref(kv), q, out, lse, dtype, scale, window, ws, _ws(lib) if n is None else n, None)


def _prefill(lib, kv, cu, q=FAKE, stride=1024, dtype=1, scale=0.1, causal=1, window=0, cu_dev=FAKE, out=FAKE):
    return lib.dense_prefill_kv4(ctypes.byref(kv), q, stride, out, None, dtype, cu_dev, cu.ctypes.data, scale, causal,
                                 window, FAKE, _ws(lib), None)


def _write(lib, kv, cu, k=None, v=None, dtype=1, cu_dev=FAKE, n=None):
    k, v = k or _rows(), v or _rows()
    return lib.hsa_kv4_write(ctypes.byref(kv), ctypes.byref(k), ctypes.byref(v), dtype, cu_dev, cu.ctypes.data, FAKE,
                             _ws(lib) if n is None else n, None)


def _read(lib, kv, start, cu, k=None, v=None, dtype=1, start_dev=FAKE):
    k, v = k or _rows(), v or _rows()
    return lib.hsa_kv4_read(ctypes.byref(kv), ctypes.byref(k), ctypes.byref(v), dtype, start_dev, start.ctypes.data, FAKE,
                            cu.ctypes.data, FAKE, _ws(lib), None)


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=6, Hkv=4), 1), (dict(B_=0), 1), (dict(Hkv=0), 1), (dict(max_pages=0), 1), (dict(cache=None), 1),
    (dict(table=None), 1), (dict(lens=None), 1),
    (dict(Hq=129, Hkv=1), 2), (dict(D=64), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=256), 2),
    (dict(max_pages=1 << 28), 2),
    (dict(seq=129), 3), (dict(seq=-1), 3),
    (dict(cache=FAKE + 128), 4), (dict(table=FAKE + 2), 4), (dict(lens=FAKE + 2), 4),
])
def test_every_call_refuses_a_bad_cache(lib, kw, status):
    kv, host = _kv(**kw)
    cu = _cu(*[1] * max(1, kw.get("B_", 2)))
    start = np.zeros(2, dtype=np.int32)
    assert lib.hsa_kv4_workspace_bytes(ctypes.byref(kv)) == 0
    assert _decode(lib, kv) == status
    assert _prefill(lib, kv, cu) == status
    assert _write(lib, kv, cu) == status
    assert _read(lib, kv, start, cu) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(window=-1), 1), (dict(q=FAKE + 8), 4), (dict(out=FAKE + 8), 4),
    (dict(lse=FAKE + 2), 4), (dict(ws=None), 5), (dict(ws=FAKE + 64), 5), (dict(n=256), 5),
])
def test_decode_refuses(lib, kw, status):
    kv, host = _kv()
    assert _decode(lib, kv, **kw) == status


@pytest.mark.parametrize("steps,kw,status", [
    ((1, 2), dict(causal=2), 1), ((1, 2), dict(causal=0, window=4), 1), ((1, 2), dict(cu_dev=None), 1),
    ((1, -1), {}, 1), ((1, 2), dict(stride=1028), 4), ((1, 2), dict(cu_dev=FAKE + 2), 4), ((1, 2), dict(q=FAKE + 2), 4),
])
def test_prefill_refuses(lib, steps, kw, status):
    kv, host = _kv()
    assert _prefill(lib, kv, _cu(*steps), **kw) == status


def test_prefill_without_rows_is_fine(lib):
    kv, host = _kv()
    assert _prefill(lib, kv, _cu(0, 0)) == 0
    shifted = _cu(1, 1)
    shifted += 1
    assert _prefill(lib, kv, shifted) == 1   # offsets start at 0


@pytest.mark.parametrize("steps,kw,status", [
    ((1, 101), {}, 3), ((2, -1), {}, 1), ((1, 1), dict(dtype=7), 1), ((1, 1), dict(cu_dev=None), 1),
    ((1, 1), dict(k=_rows(None)), 1), ((1, 1), dict(k=_rows(FAKE + 8)), 4), ((1, 1), dict(v=_rows(token=100)), 4),
    ((1, 1), dict(v=_rows(head=4)), 4), ((1, 1), dict(n=16), 5), ((0, 0), {}, 0),
])
def test_write_refuses(lib, steps, kw, status):
    kv, host = _kv()
    assert _write(lib, kv, _cu(*steps), **kw) == status


@pytest.mark.parametrize("start,steps,status", [
    ((0, 90), (1, 11), 3), ((-1, 0), (1, 1), 1), ((0, 0), (101, 0), 3), ((100, 100), (0, 0), 0),
])
def test_read_refuses(lib, start, steps, status):
    kv, host = _kv()
    assert _read(lib, kv, np.array(start, dtype=np.int32), _cu(*steps)) == status


@pytest.mark.parametrize("Hkv,steps,k,ok", [
    (2, (1, 2), (256, 128), True), (2, (1, 2), (128, 384), True), (2, (1, 2), (1024, 512), True), (1, (1, 2), (128, 0), True),
    (2, (1, 0), (0, 128), True), (1, (1, 0), (0, 0), True),
    (2, (1, 2), (0, 128), False), (2, (1, 2), (256, 0), False), (2, (1, 2), (128, 128), False), (2, (1, 2), (128, 256), False),
    (2, (1, 2), (192, 128), False), (1, (1, 2), (64, 0), False), (2, (1, 0), (0, 64), False), (2, (1, 2), (-256, 128), True),
    (2, (1, 2), (-128, 128), False),
])
def test_read_refuses_outputs_that_share_elements(lib, Hkv, steps, k, ok):
    kv, host = _kv(Hkv=Hkv)
    start, cu, far = np.zeros(2, dtype=np.int32), _cu(*steps), _rows(2 * FAKE, 4096, 2048)
    want = 6 if ok else 1                                              # 6: no device here
    assert _read(lib, kv, start, cu, k=_rows(FAKE, *k), v=far) == want
    assert _read(lib, kv, start, cu, k=far, v=_rows(FAKE, *k)) == want
    assert _read(lib, kv, start, cu, k=far, v=far) == 1


def test_read_refuses_null_start(lib):
    kv, host = _kv()
    assert _read(lib, kv, np.zeros(2, dtype=np.int32), _cu(1, 1), start_dev=None) == 1


def test_binding_refuses_host_tensors_and_wrong_shapes():
    i32 = torch.int32
    cache = P.KV4Cache.empty(4, 2, 32, "cpu")
    assert cache.shape == (4, 2, 2, P.KV4_TILE_BYTES)
    table, lens = torch.zeros(1, 4, dtype=i32), torch.zeros(1, dtype=i32)
    with pytest.raises(ValueError):
        P.KV4Cache(cache, table, lens, lens, 4)                       # host memory
    with pytest.raises(ValueError):
        P.KV4Cache(cache[..., :100], table, lens, lens, 4)
    with pytest.raises(ValueError):
        P.KV4Cache(cache, table.long(), lens, lens, 4)
    with pytest.raises(ValueError):
        P.KV4Cache(cache, table, torch.zeros(2, dtype=i32), lens, 4)
    with pytest.raises(ValueError):
        P.KV4Cache.empty(4, 2, 24, "cpu")


def test_limits(lib):
    kv, host = _kv(B_=1, max_pages=(1 << 30) // 16)                    # positions up to 2^30
    assert lib.hsa_kv4_workspace_bytes(ctypes.byref(kv)) == 0
    kv, host = _kv(Hkv=8, num_pages=1 << 28)                           # 2^31 tiles
    assert _decode(lib, kv, n=1 << 30) == 2
    kv, host = _kv(B_=65536)
    assert _decode(lib, kv, n=1 << 30) == 2
    kv, host = _kv(Hq=256, Hkv=2)
    assert _prefill(lib, kv, _cu(1 << 18, 0), out=2 * FAKE) == 2       # 2^25 query rows a head


@pytest.mark.parametrize("steps,kw", [
    ((1 << 20, 0), dict(causal=0)),                                    # 2^15 row tiles x 2^13 steps x 8 heads
    ((1 << 20, 1 << 20), {}),                                          # causal: half of that, twice
    ((1 << 20, 0), dict(causal=0, dtype=0)),                           # the kernel of few rows
])
def test_attention_refuses_more_steps_than_it_counts(lib, steps, kw):
    kv, host = _kv(Hq=64, Hkv=8, max_pages=1 << 16, seq=1 << 20)
    assert _prefill(lib, kv, _cu(*steps), stride=64 * 128, out=2 * FAKE, **kw) == 2


def test_a_window_keeps_long_chunks_within_the_limit(lib):
    """2^20 tokens of 64 query heads under a window of 1000: their number times the tokens is too large, their steps are not."""
    kv, host = _kv(Hq=64, Hkv=8, max_pages=1 << 16, seq=1 << 20)
    assert _prefill(lib, kv, _cu(1 << 20, 0), stride=64 * 128, out=2 * FAKE, window=1000) == 6   # no device here


def test_attention_refuses_to_write_over_its_queries(lib):
    kv, host = _kv()
    assert _decode(lib, kv) == 1
    assert _prefill(lib, kv, _cu(1, 1)) == 1


# ---- the oracle's format, from its definition ----

def test_scales_are_shifted_halves():
    half = (np.arange(248, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(half, O4.SCALES[:248])
    assert O4.SCALES[O4.MAX_SCALE_BYTE] == 10240 and np.isnan(O4.SCALES[255])


def test_quantise_by_exhaustive_search():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 128)) * np.exp(rng.uniform(-14, 9, (40, 1)))
    x[0] = 0
    x[1, :16] = 70000.0
    x[2, :16] = np.arange(16) * 0.25           # ties of every kind: scale 0.625 -> nearest of 3.75 / 6
    code, byte = O4.quantise(x)
    v = O4.values(code, byte)
    for n in range(40):
        for blk in range(8):
            xs = x[n, 16 * blk:16 * blk + 16]
            top = np.abs(xs).max()
            d = np.abs(O4.SCALES[:227] - top / 6)
            assert d[byte[n, blk]] <= d.min() * (1 + 1e-12)
            s = O4.SCALES[byte[n, blk]]
            grid = np.concatenate([O4.MAGNITUDES, -O4.MAGNITUDES]) * s
            best = np.abs(grid[None] - xs[:, None]).min(1)
            assert np.allclose(np.abs(v[n, 16 * blk:16 * blk + 16] - xs), best, rtol=1e-12, atol=0)
    assert v[0].max() == 0 and v[1, 0] == 61440


def test_put_and_get_are_inverse_and_touch_one_token():
    rng = np.random.default_rng(6)
    cache = rng.integers(0, 256, (3, 2, 2, O4.TILE_BYTES), dtype=np.uint8)
    table = np.array([2, 0, 1])
    k, v = rng.standard_normal((2, 96, 128))
    before = cache.copy()
    O4.put(cache, table, 1, 37, 32, k[0], v[0])
    same = cache == before
    assert (~same).sum() <= 64 + 128 + 16 and same[:, 0].all()
    for pos in range(96):
        O4.put(cache, table, 1, pos, 32, k[pos], v[pos])
    kk, vv = O4.get(cache, table, 1, range(96), 32)
    assert np.array_equal(kk, O4.values(*O4.quantise(k))) and np.array_equal(vv, O4.values(*O4.quantise(v)))
    assert np.array_equal(cache[:, 0], before[:, 0])
