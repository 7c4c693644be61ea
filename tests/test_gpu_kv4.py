"""The 4-bit KV cache on the GPU against the float64 oracle: bytes written, values read back, attention of one and of
several query tokens, at the sizes and masks where they can go wrong."""
import math

import numpy as np
import pytest
import torch

import sparse_long_context_pq_b200 as P
from oracle import kv4_oracle as O4

pytestmark = pytest.mark.gpu

D = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32)


class Case:
    """Pages in a shuffled order, with random codes and scales in the range of real keys and values."""

    def __init__(self, lens, Hkv, G, page, seed=0, spare=2, scales=(104, 120), filler=None):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.Hkv, self.G, self.page = rng, list(lens), Hkv, G, page
        need = [-(-t // page) for t in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.bytes = rng.integers(0, 256, (pages, Hkv, page // 16, O4.TILE_BYTES), dtype=np.uint8)
        self.bytes[..., 2048:] = rng.integers(*scales, self.bytes[..., 2048:].shape, dtype=np.uint8)
        if filler is not None:   # bytes of tokens past the end, and of pages that nobody uses
            keep = np.zeros(self.bytes.shape, dtype=bool)
            d = np.arange(D)
            for b, t in enumerate(lens):
                for pos in range(t):
                    for h in range(Hkv):
                        tile = O4.tile_of(keep, self.table[b], h, pos, page)
                        for value in (False, True):
                            a, _, s = O4._address(pos % 16, d, value)
                            tile[a] = True
                            tile[s] = True
            self.bytes = np.where(keep, self.bytes, filler).astype(np.uint8)

    def device(self):
        dev = torch.device("cuda:0")
        self.kv = P.KV4Cache(torch.from_numpy(self.bytes.copy()).to(dev), torch.from_numpy(self.table).to(dev),
                             i32(self.lens).to(dev), i32(self.lens), self.Hkv * self.G)
        self.ws = P.workspace(P.hsa_kv4_workspace_bytes(self.kv), dev)
        return self.kv

    def held(self, b, h, lo=0, hi=None):
        return O4.get(self.bytes, self.table[b], h, range(lo, self.lens[b] if hi is None else hi), self.page)

    def error(self):
        return P.hsa_read_error(self.ws)


def rows(rng, shape, kind):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(TYPES[kind])


def cu_of(news):
    return i32(np.cumsum([0] + list(news)))


def check(got, lse, q, case, news, scale, kind, causal=True, window=0, units=None):
    """Compare with the oracle. How far a row may be off, relative to the largest |value| in its reach:
    - a logit: q in 22 bits (11 in one fp16 number of a 16-bit q, which holds it to 2^-25 of its largest element:
      2^-22 covers both) and at most 16 fp32 sums of 2^-23, of scale * sum |q||k|; the power of two adds 2^-21;
      weights and their sum each take that error;
    - a weight in 16-bit calls is rounded to fp16, 2^-11; the rounding of the result is eps / 2;
    - sums over tokens: one fp32 addition of 2^-23 for each 16-token step, in warps of at most T / 16 steps."""
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    qn = q.double().cpu().numpy()
    cu = np.cumsum([0] + list(news))
    G = case.G
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[kind]
    for b, n in enumerate(news):
        T = case.lens[b]
        for h in range(case.Hkv):
            if n == 0 or (units is not None and (b, h) not in units):
                continue
            k, v = case.held(b, h)
            pos = T - n + np.arange(n)
            j = np.arange(T)
            seen = np.ones((n, T), dtype=bool)
            if causal:
                seen = j[None] <= pos[:, None]
                if window:
                    seen &= j[None] > pos[:, None] - window
            finite_k, finite_v = np.nan_to_num(np.abs(k)), np.nan_to_num(np.abs(v))
            for g in range(G):
                r = qn[cu[b]:cu[b + 1], h * G + g]
                ref, ref_lse = O4.attend(r, k, v, scale, seen)
                mine, mine_lse = got[cu[b]:cu[b + 1], h * G + g], lse[cu[b]:cu[b + 1], h * G + g]
                logit = abs(scale) * (np.abs(r) @ finite_k.T).max(1, initial=0.0) if T else np.zeros(n)
                rel = 2 * (logit * (2.0 ** -22 + 16 * 2.0 ** -23) + 2.0 ** -21 + (T / 16 + 16) * 2.0 ** -23)
                if kind != "f32":
                    rel = rel + 2.0 ** -11
                tol = rel * finite_v.max(initial=0.0) + np.abs(np.nan_to_num(ref)).max(1) * half
                nan = np.isnan(ref)
                assert np.array_equal(np.isnan(mine), nan), (b, h, g)
                off = np.abs(np.where(nan, 0, mine - np.where(nan, 0, ref))).max(1)
                assert (off <= tol).all(), (b, h, g, float((off / np.maximum(tol, 1e-300)).max()))
                empty = np.isneginf(ref_lse)
                assert np.array_equal(np.isneginf(mine_lse), empty), (b, h, g)
                known = ~empty & ~np.isnan(ref_lse)
                assert np.array_equal(np.isnan(mine_lse[~empty]), np.isnan(ref_lse[~empty])), (b, h, g)
                lse_tol = rel + 2.0 ** -22 * np.abs(np.nan_to_num(ref_lse, neginf=0.0))
                assert (np.abs(mine_lse - ref_lse)[known] <= lse_tol[known]).all(), (b, h, g)


# ---- write -----------------------------------------------------------------------------------------------------


def written(case, k, v, news):
    """The oracle's bytes after the write."""
    want = case.bytes.copy()
    at = 0
    for b, n in enumerate(news):
        for i in range(n):
            for h in range(case.Hkv):
                O4.put(want, case.table[b], h, case.lens[b] - n + i, case.page, k[at, h].double().numpy(),
                       v[at, h].double().numpy())
            at += 1
    return want


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,news,Hkv,page", [
    ([1], [1], 1, 16), ([16, 17, 15], [16, 1, 2], 2, 16), ([33, 40, 7, 64], [20, 0, 7, 1], 3, 32), ([130, 100], [129, 37], 2, 64),
    ([200], [131], 1, 128),
])
def test_write_gives_the_oracles_bytes(cuda_device, kind, lens, news, Hkv, page):
    case = Case(lens, Hkv, 1, page, seed=len(lens))
    kv = case.device()
    k, v = rows(case.rng, (sum(news), Hkv, D), kind), rows(case.rng, (sum(news), Hkv, D), kind) * 3
    cu = cu_of(news)
    P.hsa_kv4_write(kv, k.to(cuda_device), v.to(cuda_device), cu.to(cuda_device), cu, workspace_buf=case.ws)
    assert np.array_equal(kv.cache.cpu().numpy(), written(case, k, v, news))
    assert case.error() == 0


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_write_at_the_edges_of_the_format(cuda_device, kind):
    """Zeros, the smallest and largest scales, saturation, blocks with NaN and infinities, exact ties."""
    n = 24
    case = Case([n], 1, 1, 16, seed=3)
    kv = case.device()
    x = torch.from_numpy(case.rng.standard_normal((n, 1, D)).astype(np.float32))
    x *= torch.exp2(torch.linspace(-40, 30, n))[:, None, None]
    x[0] = 0
    x[1, 0, 16:32] = -0.0
    x[2, 0, 3] = float("nan")
    x[2, 0, 40] = float("inf")
    x[2, 0, 70] = -float("inf")
    x[3, 0, :16] = torch.arange(16) * 0.25               # ties of the codes (scale 0.625)
    x[4, 0] = 0
    x[4, 0, 0::16] = 6.0 * torch.tensor([(8 + i + 0.5) / 8 for i in range(8)])   # ties of the scales
    x[5, 0] = 6.0 * 2.0 ** -18                           # below half of the smallest scale step: a tie, to zero
    x[6, 0] = 6.1 * 2.0 ** -18
    x[7, 0] = 61440.0
    x[8, 0] = 65000.0
    if kind == "f32":
        x[9, 0] = 3.0e38
        x[10, 0] = 1e-44
    x = x.to(TYPES[kind])
    y = x.flip(0)
    cu = cu_of([n])
    P.hsa_kv4_write(kv, x.to(cuda_device), y.to(cuda_device), cu.to(cuda_device), cu, workspace_buf=case.ws)
    assert np.array_equal(kv.cache.cpu().numpy(), written(case, x, y, [n]))


def test_write_of_single_steps_equals_one_write(cuda_device):
    """21 tokens one by one, and at once; keys and values as views of a fused projection."""
    n, Hkv = 21, 2
    one, many = Case([5 + n, 3 + n], Hkv, 2, 16, seed=9), Case([5 + n, 3 + n], Hkv, 2, 16, seed=9)
    kv1, kv2 = one.device(), many.device()
    fused = rows(one.rng, (2 * n, 8, D), "bf16").to(cuda_device)
    k, v = fused[:, 4:6], fused[:, 6:8]
    cu = cu_of([n, n])
    P.hsa_kv4_write(kv1, k, v, cu.to(cuda_device), cu)
    step = cu_of([1, 1])
    for i in range(n):
        lens = i32([5 + i + 1, 3 + i + 1])
        kv2.seq_lens.copy_(lens)
        kv2.seq_lens_host.copy_(lens)
        sel = torch.tensor([i, n + i], device=cuda_device)
        P.hsa_kv4_write(kv2, k[sel], v[sel], step.to(cuda_device), step)
    assert torch.equal(kv1.cache, kv2.cache)


# ---- read ------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,start,news,page", [
    ([1], [0], [1], 16), ([40, 33, 90], [3, 33, 0], [30, 0, 90], 16), ([300], [131], [100], 128), ([77, 64], [15, 16], [2, 48], 32),
])
def test_read_is_exact(cuda_device, kind, lens, start, news, page):
    Hkv = 2
    case = Case(lens, Hkv, 1, page, seed=sum(lens), scales=(0, 227))
    kv = case.device()
    cu, st = cu_of(news), i32(start)
    n = sum(news)
    room = torch.full((2, n + 1, Hkv + 1, D + 8), 7.0, dtype=TYPES[kind], device=cuda_device)
    ko, vo = room[0, :n, :Hkv, :D], room[1, :n, :Hkv, :D]
    P.hsa_kv4_read(kv, st.to(cuda_device), st, cu.to(cuda_device), cu, k_out=ko, v_out=vo, workspace_buf=case.ws)
    at = 0
    for b, m in enumerate(news):
        for h in range(Hkv):
            k, v = case.held(b, h, start[b], start[b] + m)
            assert np.array_equal(ko[at:at + m, h].double().cpu().numpy(), k)
            assert np.array_equal(vo[at:at + m, h].double().cpu().numpy(), v)
        at += m
    assert (room[:, n:] == 7).all() and (room[:, :, Hkv:] == 7).all() and (room[..., D:] == 7).all()
    k2, v2 = P.hsa_kv4_read(kv, st.to(cuda_device), st, cu.to(cuda_device), cu, dtype=TYPES[kind])
    assert torch.equal(k2, ko) and torch.equal(v2, vo)
    assert case.error() == 0


# ---- decode ----------------------------------------------------------------------------------------------------


def decode(case, q, scale, window=0, stream=None):
    lse = torch.full(q.shape[:2], float("nan"), device="cuda:0")
    out = P.dense_decode_kv4(case.kv, q.to("cuda:0"), scale=scale, window=window, lse=lse, workspace_buf=case.ws,
                             stream=stream)
    return out, lse


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,Hkv,G,page,window", [
    ([1], 1, 1, 16, 0),
    ([0, 5, 0], 2, 4, 16, 0),
    ([15, 16, 17, 31, 33], 2, 2, 16, 0),
    ([1000], 2, 4, 16, 0),
    ([700, 3, 129], 1, 8, 64, 0),
    ([257, 640], 2, 5, 32, 0),
    ([300, 31], 1, 16, 128, 0),
    ([513], 1, 20, 16, 0),
    ([190], 1, 40, 32, 0),
    ([1000, 64, 2], 2, 4, 16, 33),
    ([129, 500], 1, 3, 32, 1),
])
def test_decode(cuda_device, kind, lens, Hkv, G, page, window):
    case = Case(lens, Hkv, G, page, seed=7 * len(lens) + G, filler=255)
    case.device()
    q = rows(case.rng, (len(lens), Hkv * G, D), kind)
    scale = D ** -0.5
    out, lse = decode(case, q, scale, window)
    check(out, lse, q, case, [1] * len(lens), scale, kind, window=window)
    assert case.error() == 0


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_decode_long_units_over_many_blocks(cuda_device, kind):
    """Long enough that every unit is shared by several blocks, beside short ones; sampled units."""
    lens = [30011, 40, 16000, 0, 1]
    case = Case(lens, 4, 4, 16, seed=21)
    case.device()
    q = rows(case.rng, (len(lens), 16, D), kind)
    out, lse = decode(case, q, 0.1)
    check(out, lse, q, case, [1] * 5, 0.1, kind, units={(0, 1), (1, 3), (2, 0), (4, 2)})
    assert torch.equal(out[3], torch.zeros_like(out[3])) and torch.isneginf(lse[3]).all()
    again, _ = decode(case, q, 0.1)
    assert torch.equal(out, again)   # no atomics: the same bits every time


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_decode_large_logits_and_growing_maximum(cuda_device, kind):
    """Logits of several hundred whose maximum grows from tile to tile; zero, tiny and huge queries."""
    case = Case([600], 1, 4, 16, seed=5)
    kv = case.device()
    k = torch.zeros(600, 1, D)
    k[:, 0, 0] = torch.linspace(0.1, 30.0, 600)
    k[:, 0, 17] = 1.0
    cu = cu_of([600])
    P.hsa_kv4_write(kv, k.to(cuda_device), torch.randn(600, 1, D).to(cuda_device), cu.to(cuda_device), cu)
    case.bytes = kv.cache.cpu().numpy()
    q = rows(case.rng, (1, 4, D), kind)
    q[0, 0, 0] = 20.0
    q[0, 1] = 0
    q[0, 2] *= 1e-4 if kind == "f16" else 1e-30
    q[0, 3] = 0
    q[0, 3, 0] = 60000.0 if kind == "f16" else 1e20
    out, lse = decode(case, q, 0.5 if kind == "f16" else 1.0)
    check(out[:, :3], lse[:, :3], q[:, :3], _with_groups(case, 3), [1], 0.5 if kind == "f16" else 1.0, kind)
    best = case.held(0, 0)[1][-8:]   # the largest keys tie or lead: all the weight is on the last ones
    assert np.isfinite(out.double().cpu().numpy()).all()
    assert (np.abs(out[0, 3].double().cpu().numpy()) <= np.abs(best).max(0) * 1.01 + 1e-6).all()


def _with_groups(case, G):
    other = Case.__new__(Case)
    other.__dict__.update(case.__dict__)
    other.G = G
    return other


def test_a_negative_and_a_zero_scale(cuda_device):
    case = Case([100], 1, 2, 16, seed=4)
    case.device()
    q = rows(case.rng, (1, 2, D), "f32")
    for scale in (-0.2, 0.0):
        out, lse = decode(case, q, scale)
        check(out, lse, q, case, [1], scale, "f32")


def test_masked_nan_does_not_spread(cuda_device):
    """A token whose key or value blocks are NaN: only rows that see it are NaN (a value block in its own dims)."""
    lens, n = [50], 9
    case = Case(lens, 1, 2, 16, seed=8)
    kv = case.device()
    k, v = torch.randn(n, 1, D), torch.randn(n, 1, D)
    v[4, 0, 37] = float("nan")        # dims 32..47 of position 45
    k[7, 0, 5] = float("inf")         # position 48
    v[8, 0, 100] = float("inf")       # position 49
    cu = cu_of([n])
    P.hsa_kv4_write(kv, k.to(cuda_device), v.to(cuda_device), cu.to(cuda_device), cu)
    case.bytes = kv.cache.cpu().numpy()
    for kind in ("f32", "bf16"):
        q = rows(case.rng, (n, 2, D), kind)
        for window in (0, 3):
            out, lse = prefill(case, q, [n], 0.1, window=window)
            bad = torch.isnan(out).cpu()
            assert not bad[:4].any() and bad[4, :, 32:48].all() and not bad[4, :, :32].any()
            assert bad[7].all() and bad[8].all()
            if window == 3:
                assert not bad[6, :, :32].any() and bad[6, :, 32:48].all()
            check(out, lse, q, case, [n], 0.1, kind, window=window)


# ---- prefill ---------------------------------------------------------------------------------------------------


def prefill(case, q, news, scale, causal=True, window=0, pad=0):
    cu = cu_of(news)
    lse = torch.full((q.shape[0], q.shape[1]), float("nan"), device="cuda:0")
    qd = q.to("cuda:0")
    if pad:   # a view with a longer token stride
        wide = torch.full((q.shape[0], q.shape[1] + pad, D), float("nan"), dtype=q.dtype, device="cuda:0")
        wide[:, :q.shape[1]] = qd
        qd = wide[:, :q.shape[1]]
    out = P.dense_prefill_kv4(case.kv, qd, cu.to("cuda:0"), cu, scale=scale, causal=causal, window=window, lse=lse,
                              workspace_buf=case.ws)
    return out, lse


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,news,Hkv,G,page,causal,window", [
    ([1], [1], 1, 1, 16, True, 0),
    ([20, 5], [5, 5], 2, 4, 16, True, 0),
    ([100, 64, 33], [5, 0, 33], 1, 8, 32, True, 0),
    ([3, 40], [9, 2], 1, 4, 16, True, 0),                 # more query tokens than tokens: rows without a mask
    ([0, 17], [3, 3], 2, 2, 16, True, 0),
    ([130], [130], 2, 1, 64, True, 0),
    ([257, 300], [257, 129], 1, 4, 128, True, 0),
    ([257, 300], [70, 129], 1, 4, 16, True, 40),
    ([150, 90], [60, 90], 2, 2, 16, False, 0),
    ([400], [100], 1, 7, 32, True, 0),
    ([90, 200], [33, 3], 1, 24, 16, True, 17),
    ([600], [1], 1, 64, 64, True, 0),
    ([513, 12, 300], [513, 12, 260], 1, 2, 16, True, 0),
    ([700], [300], 2, 4, 32, True, 1),
])
def test_prefill(cuda_device, kind, lens, news, Hkv, G, page, causal, window):
    case = Case(lens, Hkv, G, page, seed=sum(lens) + G, filler=255)
    case.device()
    q = rows(case.rng, (sum(news), Hkv * G, D), kind)
    out, lse = prefill(case, q, news, 0.09, causal, window, pad=3 if G == 4 else 0)
    check(out, lse, q, case, news, 0.09, kind, causal, window)
    assert case.error() == 0


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lens,news,Hkv,G,units", [
    ([9000], [30], 1, 4, None),                           # 120 rows, one unit over many blocks, steps on both halves
    ([5000, 130], [70, 130], 2, 4, {(0, 1), (1, 0)}),     # 280 rows: a full unit and a rest of 24
    ([128], [100], 1, 1, None),                           # a single step
    ([257], [65], 1, 1, None),                            # three steps on two halves
    ([40, 300], [90, 80], 1, 2, None),                    # rows before the first token, in units and beside them
    ([12, 33], [200, 260], 1, 1, None),                   # units whose rows all see nothing
])
def test_prefill_units_of_many_rows(cuda_device, kind, lens, news, Hkv, G, units):
    case = Case(lens, Hkv, G, 32, seed=sum(lens) + 1, filler=None if max(lens) > 2000 else 255)
    case.device()
    q = rows(case.rng, (sum(news), Hkv * G, D), kind)
    out, lse = prefill(case, q, news, 0.11)
    check(out, lse, q, case, news, 0.11, kind, units=units)
    again, _ = prefill(case, q, news, 0.11)
    assert torch.equal(out, again)
    assert case.error() == 0


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_prefill_large_logits_and_growing_maximum(cuda_device, kind):
    """Logits of several hundred that grow from step to step and within a step, rows of zeros, negative scales."""
    T, n = 420, 70
    case = Case([T], 1, 2, 16, seed=6)
    kv = case.device()
    k = torch.randn(T, 1, D) * 0.3
    k[:, 0, 0] = torch.linspace(0.1, 30.0, T)
    cu = cu_of([T])
    P.hsa_kv4_write(kv, k.to(cuda_device), torch.randn(T, 1, D).to(cuda_device), cu.to(cuda_device), cu)
    case.bytes = kv.cache.cpu().numpy()
    q = rows(case.rng, (n, 2, D), kind)
    q[:, 0, 0] = 25.0
    q[3] = 0
    q[5] *= 2.0 ** -12
    for scale in (0.5, -0.5, 0.0):
        out, lse = prefill(case, q, [n], scale)
        check(out, lse, q, case, [n], scale, kind)


@pytest.mark.parametrize("n", [9, 100])
@pytest.mark.parametrize("kind,factor", [(k, f) for k in ("f32", "bf16", "f16") for f in (1e5, 1e6, 3e6, 1e7, 3e7, 1e9)
                                         if (k, f) != ("f16", 1e9)])      # q of that size is not finite in fp16
def test_huge_logits_stay_finite(cuda_device, kind, factor, n):
    """Logits up to 10^10: nearly all weight is on the largest, and nothing overflows."""
    if kind == "f16":
        factor /= 65536.0
    T = 300
    case = Case([T], 1, 1, 16, seed=16)
    case.device()
    q = rows(case.rng, (n, 1, D), kind) * factor
    scale = 65536.0 if kind == "f16" else 1.0
    out, lse = prefill(case, q, [n], scale)
    k, v = case.held(0, 0)
    best = (q[:, 0].double().numpy() @ k.T) * scale
    best[np.arange(T)[None] > (T - n + np.arange(n))[:, None]] = -np.inf
    at = best.argmax(1)
    got = out[:, 0].double().cpu().numpy()
    assert np.isfinite(got).all() and torch.isfinite(lse).all()
    gap = np.sort(best, 1)[:, -1] - np.sort(best, 1)[:, -2]
    clear = gap > 1e-5 * np.abs(best.max(1)) + 100       # far more than the rounding of a logit
    assert clear.any()
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[kind]
    ref = v[at]
    assert (np.abs(got - ref)[clear] <= (2 * half + 2.0 ** -11) * np.abs(ref)[clear] + 1e-30).all()


@pytest.mark.parametrize("n", [1, 2, 4, 12])
def test_sums_of_32_bit_calls_have_no_bias(cuda_device, n):
    """Equal values come back as themselves on the mean. The tensor cores cut sums off: at most two cuts of less than
    2^-23 to a tile of 16 tokens (one hi and one lo product), or to a sum over tiles where there is no lo product of its
    own (n = 1: four rows); all else rounds to nearest. A bias that adds up over the tiles of a segment is far larger."""
    B, T = 148, 600
    cache = P.KV4Cache.empty(B * 5, 1, 128, cuda_device)
    table = torch.arange(B * 5, dtype=torch.int32).view(B, 5)
    kv = P.KV4Cache(cache, table.to(cuda_device), i32([T] * B).to(cuda_device), i32([T] * B), 4)
    gen = torch.Generator(device=cuda_device).manual_seed(5)
    cu = cu_of([T] * B)
    k = torch.randn(B * T, 1, D, generator=gen, device=cuda_device)
    P.hsa_kv4_write(kv, k, torch.full_like(k, 6.0), cu.to(cuda_device), cu)
    cu = cu_of([n] * B)
    q = torch.randn(B * n, 4, D, generator=gen, device=cuda_device)
    out = P.dense_prefill_kv4(kv, q, cu.to(cuda_device), cu, scale=0.1)
    assert abs((out.double() / 6 - 1).mean().item()) <= 2 * 2.0 ** -23 + 2.0 ** -24


@pytest.mark.parametrize("rows_of", ["few", "many"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_many_sequences(cuda_device, kind, rows_of):
    """More sequences than lanes of a warp, many of them empty or without queries."""
    rng = np.random.default_rng(40)
    B = 70
    lens = [int(x) for x in rng.integers(0, 90, B)]
    lens[0], lens[50] = 700, 1500
    news = [int(rng.integers(0, 4)) for _ in range(B)]
    if rows_of == "many":
        news[0], news[50] = 90, 33
    case = Case(lens, 1, 4, 16, seed=41)
    case.device()
    q = rows(case.rng, (sum(news), 4, D), kind)
    out, lse = prefill(case, q, news, 0.1)
    check(out, lse, q, case, news, 0.1, kind)
    q1 = rows(case.rng, (B, 4, D), kind)
    out, lse = decode(case, q1, 0.1)
    check(out, lse, q1, case, [1] * B, 0.1, kind)
    assert case.error() == 0


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_units_of_all_row_counts(cuda_device, kind):
    """1 to 130 query rows a KV head: every row tile of the streaming kernel, the border to the other, its two shapes."""
    case = Case([333], 1, 1, 16, seed=50)
    case.device()
    for n in (1, 4, 5, 8, 9, 16, 17, 24, 25, 32, 33, 40, 63, 64, 65, 127, 128, 129, 130):
        q = rows(case.rng, (n, 1, D), kind)
        out, lse = prefill(case, q, [n], 0.1)
        check(out, lse, q, case, [n], 0.1, kind)


# ---- what the calls promise ------------------------------------------------------------------------------------


@pytest.mark.parametrize("n", [60, 200])
def test_masked_nan_does_not_spread_in_long_chunks(cuda_device, n):
    """The same in units of 128 and of 256 rows, bad tokens in several steps."""
    T = 400
    case = Case([T], 1, 2, 16, seed=18)
    kv = case.device()
    k, v = torch.randn(T, 1, D), torch.randn(T, 1, D)
    v[T - 40, 0, 37] = float("nan")
    v[T - 3, 0, 100] = float("inf")
    k[T - 20, 0, 5] = float("nan")
    cu = cu_of([T])
    P.hsa_kv4_write(kv, k.to(cuda_device), v.to(cuda_device), cu.to(cuda_device), cu)
    case.bytes = kv.cache.cpu().numpy()
    q = rows(case.rng, (n, 2, D), "bf16")
    for window in (0, 10):
        out, lse = prefill(case, q, [n], 0.1, window=window)
        bad = torch.isnan(out).cpu()
        assert not bad[:n - 40].any() and bad[n - 40, :, 32:48].all() and not bad[n - 40, :, :32].any()
        assert bad[n - 20].all()
        check(out, lse, q, case, [n], 0.1, "bf16", window=window)


def test_bad_pages_in_long_chunks(cuda_device):
    """Tokens of a page that the block table does not name take no part, and are flagged."""
    T, n = 500, 90
    case = Case([T], 1, 2, 32, seed=19)
    kv = case.device()
    kv.block_table[0, 3] = -1
    kv.block_table[0, 9] = 1 << 20
    q = rows(case.rng, (n, 2, D), "bf16")
    out, lse = prefill(case, q, [n], 0.1)
    assert case.error() == P.HSA_DEVERR_PAGE
    k, v = case.held(0, 0)
    j = np.arange(T)
    seen = j[None] <= (T - n + np.arange(n))[:, None]
    seen &= ~((j // 32 == 3) | (j // 32 == 9))[None]
    for g in range(2):
        ref, ref_lse = O4.attend(q[:, g].double().numpy(), k, v, 0.1, seen)
        assert np.abs(out[:, g].double().cpu().numpy() - ref).max() <= (2.0 ** -8 + 2.0 ** -10) * np.abs(v).max()
        assert np.abs(lse[:, g].double().cpu().numpy() - ref_lse).max() <= 1e-4


def test_prefill_captured_and_replayed(cuda_device):
    """A captured chunk (write, attend) replayed with other data and lengths."""
    case = Case([900, 500], 2, 4, 16, seed=60)
    kv = case.device()
    n = [70, 40]
    cu = cu_of(n)
    cud = cu.to(cuda_device)
    k, v = torch.randn(110, 2, D, device=cuda_device).half(), torch.randn(110, 2, D, device=cuda_device).half()
    q = torch.randn(110, 8, D, device=cuda_device).half()
    out = torch.empty_like(q)

    def step(w):
        P.hsa_kv4_write(kv, k, v, cud, cu, workspace_buf=w)
        P.dense_prefill_kv4(kv, q, cud, cu, out, scale=0.1, workspace_buf=w)

    step(case.ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(case.ws)
    for lens in ([900, 500], [330, 41], [70, 300]):
        kv.seq_lens.copy_(i32(lens))
        for x in (k, v, q):
            x.normal_()
        graph.replay()
        got = out.clone()
        kv.seq_lens_host.copy_(i32(lens))
        step(P.workspace(P.hsa_kv4_workspace_bytes(kv), cuda_device))
        assert torch.equal(got, out)
    assert case.error() == 0


def test_bad_pages_are_flagged_and_skipped(cuda_device):
    lens = [70, 50]
    case = Case(lens, 2, 4, 16, seed=2)
    kv = case.device()
    kv.block_table[0, 2] = 1000
    kv.block_table[1, 1] = -7
    q = rows(case.rng, (2, 8, D), "f32")
    out, lse = decode(case, q, 0.1)
    assert case.error() == P.HSA_DEVERR_PAGE and case.error() == 0
    k0 = [p for p in range(70) if not 32 <= p < 48]     # the tokens that are left
    for h in range(2):
        k, v = case.held(0, h)
        ref, _ = O4.attend(q[0, h * 4:h * 4 + 4].double().numpy(), k[k0], v[k0], 0.1, np.ones((4, len(k0)), dtype=bool))
        assert np.abs(out[0, h * 4:h * 4 + 4].double().cpu().numpy() - ref).max() <= 1e-5 * np.abs(v).max()
    before = kv.cache.clone()
    cu = cu_of([70, 0])
    k = torch.randn(70, 2, D, device=cuda_device)
    P.hsa_kv4_write(kv, k, k, cu.to(cuda_device), cu, workspace_buf=case.ws)
    assert case.error() == P.HSA_DEVERR_PAGE
    touched = (kv.cache != before).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert set(touched) <= set(case.table[0, [0, 1, 3, 4]].tolist())
    st = i32([0, 0])
    ko, vo = P.hsa_kv4_read(kv, st.to(cuda_device), st, cu.to(cuda_device), cu, dtype=torch.float32, workspace_buf=case.ws)
    assert case.error() == P.HSA_DEVERR_PAGE
    assert (ko[32:48] == 0).all() and (vo[32:48] == 0).all() and (ko[:32] != 0).any()


def test_capture_and_replay_with_other_lengths(cuda_device):
    """One captured step (write a token, attend) replayed while the sequences grow, against eager calls."""
    lens = [40, 700]
    case = Case([t + 40 for t in lens], 2, 4, 16, seed=12)
    kv = case.device()
    k, v = torch.randn(2, 2, D, device=cuda_device), torch.randn(2, 2, D, device=cuda_device)
    q = torch.randn(2, 8, D, device=cuda_device)
    out = torch.empty_like(q)
    cu = cu_of([1, 1])
    cud = cu.to(cuda_device)
    ws2 = P.workspace(P.hsa_kv4_workspace_bytes(kv), cuda_device)

    def step(w):
        P.hsa_kv4_write(kv, k, v, cud, cu, workspace_buf=w)
        P.dense_decode_kv4(kv, q, out, scale=0.1, workspace_buf=w)

    kv.seq_lens.copy_(i32(lens))
    kv.seq_lens_host.copy_(i32(lens))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(case.ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(case.ws)
    for i in range(1, 40, 3):
        now = i32([t + i for t in lens])
        kv.seq_lens.copy_(now)
        for x in (k, v, q):
            x.normal_()
        graph.replay()
        got = out.clone()
        kv.seq_lens_host.copy_(now)
        step(ws2)
        # other block shares (planned from the host lengths): the same sums in another order
        assert (got - out).abs().max() <= 1e-5 * 8
    assert case.error() == 0


def test_other_streams_with_their_own_workspaces(cuda_device):
    case = Case([3000, 200], 2, 4, 16, seed=30)
    kv = case.device()
    q = rows(case.rng, (2, 8, D), "bf16").to(cuda_device)
    want = P.dense_decode_kv4(kv, q, scale=0.1)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [P.dense_decode_kv4(kv, q, scale=0.1, stream=s) for s in streams for _ in range(3)]
    outs.append(P.dense_decode_kv4(kv, q, scale=0.1, stream=streams[0].cuda_stream))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_offsets_past_32_bits(cuda_device):
    """A cache of more than 4 GiB whose sequence lives in its last pages."""
    Hkv, page, T = 8, 128, 300
    pages = (5 << 30) // (Hkv * page // 16 * O4.TILE_BYTES)
    cache = P.KV4Cache.empty(pages, Hkv, page, cuda_device)
    table = i32([[pages - 1, 0, pages - 2]])
    kv = P.KV4Cache(cache, table.to(cuda_device), i32([T]).to(cuda_device), i32([T]), Hkv)
    k, v = torch.randn(T, Hkv, D), torch.randn(T, Hkv, D)
    cu, st = cu_of([T]), i32([0])
    P.hsa_kv4_write(kv, k.to(cuda_device), v.to(cuda_device), cu.to(cuda_device), cu)
    ko, vo = P.hsa_kv4_read(kv, st.to(cuda_device), st, cu.to(cuda_device), cu, dtype=torch.float32)
    for got, x in ((ko, k), (vo, v)):
        want = O4.values(*O4.quantise(x.double().numpy()))
        assert np.array_equal(got.double().cpu().numpy(), want)
    q = torch.randn(1, Hkv, D)
    out = P.dense_decode_kv4(kv, q.to(cuda_device), scale=0.1)
    ref, _ = O4.attend(q[0, 5:6].double().numpy(), ko[:, 5].double().cpu().numpy(), vo[:, 5].double().cpu().numpy(), 0.1,
                       np.ones((1, T), dtype=bool))
    assert np.abs(out[0, 5].double().cpu().numpy() - ref[0]).max() <= 1e-5 * 8


def test_refusals_with_device_tensors(cuda_device):
    case = Case([40], 2, 2, 16)
    kv = case.device()
    q = torch.zeros(1, 4, D, device=cuda_device)
    cu = cu_of([2])
    cud = cu.to(cuda_device)
    for bad in (q[:, :3], q.double(), q[..., :64], torch.zeros(1, 4, 2 * D, device=cuda_device)[..., ::2]):
        with pytest.raises(ValueError):
            P.dense_decode_kv4(kv, bad, scale=0.1)
    with pytest.raises(ValueError):
        P.dense_decode_kv4(kv, q, torch.empty(1, 4, D, dtype=torch.bfloat16, device=cuda_device), scale=0.1)
    with pytest.raises(ValueError):
        P.dense_decode_kv4(kv, q, scale=0.1, lse=torch.empty(4, device=cuda_device))
    with pytest.raises(ValueError):
        P.dense_decode_kv4(kv, q.cpu(), scale=0.1)
    with pytest.raises(P.HSAError):
        P.dense_decode_kv4(kv, q, scale=0.1, window=-1)
    with pytest.raises(P.HSAError):
        P.dense_decode_kv4(kv, q, scale=0.1, workspace_buf=torch.zeros(256, dtype=torch.uint8, device=cuda_device))
    k = torch.zeros(2, 2, D, device=cuda_device)
    with pytest.raises(ValueError):
        P.hsa_kv4_write(kv, k, k.half(), cud, cu)
    with pytest.raises(ValueError):
        P.hsa_kv4_write(kv, k[:1], k, cud, cu)
    with pytest.raises(ValueError):
        P.hsa_kv4_write(kv, k, k, cud, cu.long())
    with pytest.raises(ValueError):
        P.hsa_kv4_write(kv, k.transpose(1, 2).contiguous().transpose(1, 2), k, cud, cu)
    many = cu_of([41])
    k41 = torch.zeros(41, 2, D, device=cuda_device)
    with pytest.raises(P.HSAError):
        P.hsa_kv4_write(kv, k41, k41, many.to(cuda_device), many)
    with pytest.raises(ValueError):
        P.dense_prefill_kv4(kv, torch.zeros(2, 4, 2 * D, device=cuda_device)[..., :D].transpose(0, 1), cud, cu, scale=0.1)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_windows_larger_than_any_sequence(cuda_device, kind):
    """A window that leaves nothing out, up to the largest int and past it, with rows before the first token."""
    case = Case([50, 3], 1, 2, 16, seed=80)
    case.device()
    for news in ([10, 20], [90, 1]):
        q = rows(case.rng, (sum(news), 2, D), kind)
        want, want_lse = prefill(case, q, news, 0.1)
        for window in (64, (1 << 31) - 1, (1 << 32) + 5):
            out, lse = prefill(case, q, news, 0.1, window=window)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_sequences_that_share_pages(cuda_device, kind):
    """The same pages at the front of every sequence, and twice in one."""
    case = Case([64, 80, 100], 2, 2, 16, seed=81)
    case.table[1, :3] = case.table[0, :3]
    case.table[2, :3] = case.table[0, :3]
    case.table[2, 4] = case.table[0, 1]
    case.device()
    for news in ([1, 1, 1], [40, 50, 60]):
        q = rows(case.rng, (sum(news), 4, D), kind)
        out, lse = prefill(case, q, news, 0.1)
        check(out, lse, q, case, news, 0.1, kind)


@pytest.mark.parametrize("n", [3, 40])
def test_rows_apart_and_behind_stay(cuda_device, n):
    """q as a view of a fused projection; a tensor behind out and lse keeps its bytes; a single row of any stride."""
    case = Case([200], 2, 4, 16, seed=82)
    kv = case.device()
    fused = torch.randn(n, 8 + 2 + 2, D, device=cuda_device).bfloat16()
    big = torch.full((n + 4, 8, D), 7.0, device=cuda_device, dtype=torch.bfloat16)
    lse = torch.full((n + 4, 8), 7.0, device=cuda_device)
    cu = cu_of([n])
    q = fused[:, :8]
    P.dense_prefill_kv4(kv, q, cu.to(cuda_device), cu, big[:n], scale=0.1, lse=lse[:n])
    check(big[:n], lse[:n], q.cpu(), case, [n], 0.1, "bf16")
    assert (big[n:] == 7).all() and (lse[n:] == 7).all()
    one = torch.randn(8, D, device=cuda_device).bfloat16().as_strided((1, 8, D), (3, D, 1))
    cu = cu_of([1])
    out = P.dense_prefill_kv4(kv, one, cu.to(cuda_device), cu, scale=0.1)
    assert torch.equal(out, P.dense_decode_kv4(kv, one.contiguous().view(1, 8, D), scale=0.1))


def test_chunks_on_two_streams(cuda_device):
    """Writes and chunks of two caches on two streams at once, each with its workspace, against one after the other."""
    cases = [Case([3000], 2, 4, 16, seed=90 + i) for i in range(2)]
    work = []
    for c in cases:
        kv = c.device()
        n = 150
        cu = cu_of([n])
        k, v = (torch.randn(n, 2, D, device=cuda_device).half() for _ in range(2))
        q = torch.randn(n, 8, D, device=cuda_device).half()
        work.append((kv, k, v, q, cu.to(cuda_device), cu, P.workspace(P.hsa_kv4_workspace_bytes(kv), cuda_device)))

    def run(w, stream=None):
        kv, k, v, q, cud, cu, ws = w
        outs = []
        for _ in range(4):
            P.hsa_kv4_write(kv, k, v, cud, cu, workspace_buf=ws, stream=stream)
            outs.append(P.dense_prefill_kv4(kv, q, cud, cu, scale=0.1, workspace_buf=ws, stream=stream))
        return outs

    want = [run(w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [run(w, s) for w, s in zip(work, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert all(P.hsa_read_error(w[-1]) == 0 for w in work)


# ---- together --------------------------------------------------------------------------------------------------


def test_a_sequence_from_prompt_to_decoded_tokens(cuda_device):
    """Prompts written and attended in chunks, tokens appended and decoded one by one, the cache read back into bf16
    pages: dense_decode over those gives what dense_decode_kv4 gives, and an index is trained on the keys."""
    B, Hkv, G, page, total = 2, 2, 4, 16, 600
    Hq, scale = Hkv * G, D ** -0.5
    lens = [0, 0]
    target = [total, 480]
    case = Case(target, Hkv, G, page, seed=77)
    kv = case.device()
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    k = [torch.randn(t, Hkv, D, generator=gen, device=cuda_device).bfloat16() for t in target]
    v = [torch.randn(t, Hkv, D, generator=gen, device=cuda_device).bfloat16() for t in target]
    held = [[torch.from_numpy(O4.values(*O4.quantise(x.double().cpu().numpy()))) for x in side] for side in (k, v)]

    def advance(news):
        cu = cu_of(news)
        for b in range(B):
            lens[b] += news[b]
        kv.seq_lens.copy_(i32(lens))
        kv.seq_lens_host.copy_(i32(lens))
        pick = lambda x: torch.cat([x[b][lens[b] - news[b]:lens[b]] for b in range(B)])  # noqa: E731
        P.hsa_kv4_write(kv, pick(k), pick(v), cu.to(cuda_device), cu, workspace_buf=case.ws)
        q = torch.randn(sum(news), Hq, D, generator=gen, device=cuda_device)
        if max(news) == 1 and min(news) == 1:
            out = P.dense_decode_kv4(kv, q, scale=scale, workspace_buf=case.ws)
        else:
            out = P.dense_prefill_kv4(kv, q, cu.to(cuda_device), cu, scale=scale, workspace_buf=case.ws)
        got, at = out.double().cpu().numpy(), 0
        for b in range(B):
            T, n = lens[b], news[b]
            pos = T - n + np.arange(n)
            seen = np.arange(T)[None] <= pos[:, None]
            for hq in range(0, Hq, 3):
                h = hq // G
                ref, _ = O4.attend(q[at:at + n, hq].double().cpu().numpy(), held[0][b][:T, h].numpy(),
                                   held[1][b][:T, h].numpy(), scale, seen)
                if n:
                    assert np.abs(got[at:at + n, hq] - ref).max() <= 2e-5 * 5
            at += n
        return out, q

    advance([300, 0])
    advance([250, 470])
    advance([5, 5])
    for _ in range(5):
        out, q = advance([1, 1])
    while lens[0] < total:
        out, q = advance([min(20, total - lens[0]), 0])
    q = torch.randn(B, Hq, D, generator=gen, device=cuda_device)
    out = P.dense_decode_kv4(kv, q, scale=scale, workspace_buf=case.ws)
    # back into bf16 pages of the same block table
    cu, st = cu_of(target), i32([0, 0])
    kb, vb = P.hsa_kv4_read(kv, st.to(cuda_device), st, cu.to(cuda_device), cu, workspace_buf=case.ws)
    pages = kv.cache.shape[0]
    kc = torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=cuda_device)
    vc = torch.zeros_like(kc)
    for b in range(B):
        pos = torch.arange(target[b], device=cuda_device)
        page_of = kv.block_table[b][pos // page].long()
        kc[page_of, :, pos % page] = kb[cu[b]:cu[b + 1]]
        vc[page_of, :, pos % page] = vb[cu[b]:cu[b + 1]]
    bf = P.PagedKV(kc, vc, kv.block_table.clamp(min=0), kv.seq_lens, kv.seq_lens_host, Hq)
    dense = P.dense_decode(bf, q, scale=scale)
    # dense_decode splits q and P into two bf16 parts (2^-16 each) of logits up to about 10
    assert (dense - out).abs().max() <= 5 * 4 * 2.0 ** -15 * 10
    ix = P.PQIndex.allocate(B, Hkv, 4, 600, 4, cuda_device)
    slots = torch.randint(0, 400, (B, Hkv, 4 + 16 * 256), dtype=torch.int32, device=cuda_device)
    P.hsa_train_index(bf, ix, 400, slots, coarse_iters=1, pq_iters=1)
    P.hsa_append_encode(bf, ix, 400)
    sparse = P.hsa_decode(bf, ix, q, scale=scale, budget=1.0)    # every token selected: dense attention
    assert (sparse - out).abs().max() <= 5 * 4 * 2.0 ** -15 * 10
    assert case.error() == 0


# ---- sums, ranges and limits -----------------------------------------------------------------------------------


@pytest.mark.parametrize("stairs", ["inside", "everywhere"])
@pytest.mark.parametrize("n", [60, 200])
def test_maximum_that_jumps_inside_a_step(cuda_device, n, stairs):
    """The maximum of a third of the rows grows by more than the weights' head room (15 in log2 units) between the two
    halves of a 128-token step, so that weights already stored are scaled: from the first half to the second only, or
    from every half to the next. Other rows keep theirs or have it at the front."""
    T = 640
    case = Case([T], 1, 2, 16, seed=61)
    kv = case.device()
    gen = torch.Generator().manual_seed(62)
    k = torch.randn(T, 1, D, generator=gen) * 0.05
    half = torch.arange(T) // 64
    k[:, 0, 0] = ((half + 1) // 2 if stairs == "inside" else half).float()
    cu = cu_of([T])
    P.hsa_kv4_write(kv, k.to(cuda_device), torch.randn(T, 1, D, generator=gen).to(cuda_device), cu.to(cuda_device), cu)
    case.bytes = kv.cache.cpu().numpy()
    for kind in ("bf16", "f16"):
        q = rows(case.rng, (n, 2, D), kind)
        q[0::3, :, 0], q[1::3, :, 0], q[2::3, :, 0] = 48.0, 0.125, -48.0      # 24 natural units a stair, 34 in log2
        out, lse = prefill(case, q, [n], 0.5)
        check(out, lse, q, case, [n], 0.5, kind)


@pytest.mark.parametrize("kind,n", [("f32", 16), ("bf16", 1056)])
def test_device_lengths_past_the_limits_are_flagged(cuda_device, kind, n):
    """A replay's lengths (here: the device's alone) that make more steps than a call may have: 2^31 of 32 tokens with
    8 tiles of 16 rows, 33 x 2^26 of 128 tokens with 8448 rows. Nothing is written, no step is taken."""
    Hkv, G, T = 8, 8, (1 << 30) - 128
    cache = P.KV4Cache.empty(1, Hkv, 128, cuda_device)
    table = torch.zeros(1, T // 128, dtype=torch.int32, device=cuda_device)
    kv = P.KV4Cache(cache, table, i32([T]).to(cuda_device), i32([n]), Hkv * G)
    ws = P.workspace(P.hsa_kv4_workspace_bytes(kv), cuda_device)
    q = torch.zeros(n, Hkv * G, D, dtype=TYPES[kind], device=cuda_device)
    out = torch.full_like(q, 7.0)
    cu = cu_of([n])
    P.dense_prefill_kv4(kv, q, cu.to(cuda_device), cu, out, scale=0.1, causal=False, workspace_buf=ws)
    assert P.hsa_read_error(ws) == P.HSA_DEVERR_LIMIT
    assert (out == 7).all()


@pytest.mark.parametrize("n", [1, 2, 4, 12])
def test_sums_of_32_bit_calls_have_no_bias_over_long_segments(cuda_device, n):
    """Equal values come back as themselves on the mean, however long the segments: 148 sequences of 32768 tokens, one a
    block, are 128 tiles and more a warp (n = 1, 2: 16 warps; n = 4, 12: 8). A step's products are cut off at most once for
    each of its at most four matrix instructions, less than 2^-23 of the step's own sum, half of that on the mean, and the
    partial sums that they cut are half of that sum on the mean: 2^-23 together. The rest rounds to nearest."""
    B, T = 148, 32768
    pages = T // 128
    cache = P.KV4Cache.empty(B * pages, 1, 128, cuda_device)
    table = torch.arange(B * pages, dtype=torch.int32).view(B, pages)
    kv = P.KV4Cache(cache, table.to(cuda_device), i32([T] * B).to(cuda_device), i32([T] * B), 4)
    gen = torch.Generator(device=cuda_device).manual_seed(5)
    cu = cu_of([T] * B)
    k = torch.randn(B * T, 1, D, generator=gen, device=cuda_device, dtype=torch.bfloat16)
    P.hsa_kv4_write(kv, k, torch.full_like(k, 6.0), cu.to(cuda_device), cu)
    cu = cu_of([n] * B)
    q = torch.randn(B * n, 4, D, generator=gen, device=cuda_device)
    out = P.dense_prefill_kv4(kv, q, cu.to(cuda_device), cu, scale=0.1)
    assert abs((out.double() / 6 - 1).mean().item()) <= 2.0 ** -23 + 2.0 ** -24


def long_bias(n, kind, device, Hkv=2, G=4, T=1 << 20, B=148):
    """Mean relative error of values of one sign over a million tokens, B sequences of the same pages so that a unit's
    tokens are shared by few warps or blocks; the last rows of one sequence against 64 bits."""
    gen = torch.Generator(device=device).manual_seed(9)
    cache = P.KV4Cache.empty(T // 128, Hkv, 128, device)
    table = torch.arange(T // 128, dtype=torch.int32, device=device).view(1, -1)
    one = P.KV4Cache(cache, table, i32([T]).to(device), i32([T]), Hkv * G)
    k = torch.randn(T, Hkv, D, generator=gen, device=device, dtype=torch.bfloat16)
    v = torch.rand(T, Hkv, D, generator=gen, device=device, dtype=torch.bfloat16) + 0.5
    cu, st = cu_of([T]), i32([0])
    P.hsa_kv4_write(one, k, v, cu.to(device), cu)
    k, v = P.hsa_kv4_read(one, st.to(device), st, cu.to(device), cu)
    kv = P.KV4Cache(cache, table.expand(B, -1).contiguous(), i32([T] * B).to(device), i32([T] * B), Hkv * G)
    q = torch.randn(n, Hkv * G, D, generator=gen, device=device).to(TYPES[kind])
    cu = cu_of([n] * B)
    out = P.dense_prefill_kv4(kv, q.repeat(B, 1, 1), cu.to(device), cu, scale=0.1).view(B, n, Hkv, G, D)
    m = min(n, 4)
    errors = []
    for h in range(Hkv):
        x = 0.1 * (q.view(n, Hkv, G, D)[n - m:, h].reshape(-1, D).double() @ k[:, h].double().T)
        seen = torch.arange(T, device=device)[None] <= torch.arange(T - m, T, device=device).repeat_interleave(G)[:, None]
        ref = torch.softmax(x.masked_fill_(~seen, -math.inf), -1) @ v[:, h].double()
        errors.append((out[B // 2, n - m:, h].reshape(-1, D).double() / ref - 1).mean().item())
    return float(np.mean(errors))


@pytest.mark.parametrize("n", [2, 4, 8])
def test_sums_of_16_bit_calls_over_long_segments(cuda_device, n):
    """65536 to 131072 tokens a warp. Sums of at most 512 tiles are cut off by less than 2^-23 each; the results of 256
    dims round apart from one another by at most 2^-11 of a value, evenly spread (of all rows alike, as rows see nearly
    the same mean): four standard deviations of their mean."""
    assert abs(long_bias(n, "f16", cuda_device)) <= 512 * 2.0 ** -23 + 4 * 2.0 ** -11 / math.sqrt(3 * 256)


@pytest.mark.parametrize("n", [30, 64])
def test_sums_of_long_chunks_over_long_segments(cuda_device, n):
    """Units of 120 and of 256 rows, a million tokens a block. As above, with 128 steps of 8 matrix instructions a sum."""
    assert abs(long_bias(n, "f16", cuda_device)) <= 1024 * 2.0 ** -23 + 4 * 2.0 ** -11 / math.sqrt(3 * 256)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n", [20, 64, 90])
def test_chunks_whose_sums_are_put_by(cuda_device, kind, n):
    """Units of up to 400 steps, on one half or two (a half's sums are put by after 128), beside short ones, some whole and
    some shared by two blocks of about 490 steps (128 heads; 980 with units of two row tiles), maxima that grow on the way;
    against 64 bits."""
    lens = [51200, 700, 20011]
    Hkv, G, B = 128, 4, len(lens)
    pages = [-(-t // 128) for t in lens]
    cache = P.KV4Cache.empty(sum(pages), Hkv, 128, cuda_device)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = torch.arange(at, at + pages[b])
        at += pages[b]
    kv = P.KV4Cache(cache, table.to(cuda_device), i32(lens).to(cuda_device), i32(lens), Hkv * G)
    gen = torch.Generator(device=cuda_device).manual_seed(n)
    total = sum(lens)
    k = torch.randn(total, Hkv, D, generator=gen, device=cuda_device, dtype=torch.bfloat16)
    pos = torch.cat([torch.arange(t) for t in lens]).to(cuda_device)
    k[:, :, 3] = (pos // 6000)[:, None].to(k.dtype)          # grows by a stair every 6000 tokens
    v = torch.randn(total, Hkv, D, generator=gen, device=cuda_device, dtype=torch.bfloat16)
    cu, st = cu_of(lens), i32([0] * B)
    P.hsa_kv4_write(kv, k, v, cu.to(cuda_device), cu)
    k, v = P.hsa_kv4_read(kv, st.to(cuda_device), st, cu.to(cuda_device), cu)
    news = [n, n, n]
    q = torch.randn(3 * n, Hkv * G, D, generator=gen, device=cuda_device).to(TYPES[kind])
    q[::2, :, 3] = 6.0
    cn = cu_of(news)
    ws = P.workspace(P.hsa_kv4_workspace_bytes(kv), cuda_device)
    lse = torch.empty(3 * n, Hkv * G, device=cuda_device)
    scale = 0.1
    out = P.dense_prefill_kv4(kv, q, cn.to(cuda_device), cn, scale=scale, lse=lse, workspace_buf=ws).view(3 * n, Hkv, G, D)
    again = P.dense_prefill_kv4(kv, q, cn.to(cuda_device), cn, scale=scale, workspace_buf=ws).view(3 * n, Hkv, G, D)
    assert torch.equal(out, again)
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[kind]
    for b in range(B):
        for h in range(b, Hkv, 13):
            kk, vv = (x[cu[b]:cu[b + 1], h].double() for x in (k, v))
            rows_of = q.view(3 * n, Hkv, G, D)[b * n:(b + 1) * n, h].reshape(-1, D).double()
            x = scale * (rows_of @ kk.T)
            t = torch.arange(lens[b], device=cuda_device)
            x.masked_fill_(t[None] > (lens[b] - n + torch.arange(n, device=cuda_device)).repeat_interleave(G)[:, None], -math.inf)
            ref = torch.softmax(x, -1) @ vv
            got = out[b * n:(b + 1) * n, h].reshape(-1, D).double()
            # check()'s bound: logits, weights, sums (cut off 1024 times at most, less than 2^-23 each), the result
            logit = scale * (rows_of.abs() @ kk.abs().T).max(1).values
            rel = 2 * (logit * 18 * 2.0 ** -23 + 2.0 ** -21 + 1024 * 2.0 ** -23) + 2.0 ** -11
            tol = rel * vv.abs().max() + ref.abs().max(1).values * half
            assert ((got - ref).abs().max(1).values <= tol).all(), (b, h)
            off = (lse.view(3 * n, Hkv, G)[b * n:(b + 1) * n, h].reshape(-1).double() - torch.logsumexp(x, -1)).abs()
            assert (off <= rel + 2.0 ** -22 * torch.logsumexp(x, -1).abs()).all(), (b, h)


@pytest.mark.parametrize("kind,factor", [("f32", 1e4), ("f32", 1e5), ("bf16", 1e4), ("bf16", 1e6), ("f16", 1e5)])
@pytest.mark.parametrize("n", [1, 5, 12, 40, 200])
def test_large_elements_of_q_leave_the_others_their_bits(cuda_device, n, kind, factor):
    """One element of q is `factor` times the others, where the keys are zero: the logits are the others' alone. check()
    holds them to 2^-22 of scale sum |q||k|, to which that element adds nothing. (fp32: q is held to 2^-38 of its largest
    element, 2^-21 of a unit with 10^5, a third of that on the mean; its 128 errors are independent.)"""
    T = 300
    case = Case([T], 1, 4, 16, seed=63)
    kv = case.device()
    gen = torch.Generator().manual_seed(64)
    k = torch.randn(T, 1, D, generator=gen)
    k[:, 0, 21] = 0
    cu = cu_of([T])
    P.hsa_kv4_write(kv, k.to(cuda_device), torch.randn(T, 1, D, generator=gen).to(cuda_device), cu.to(cuda_device), cu)
    case.bytes = kv.cache.cpu().numpy()
    q = rows(case.rng, (n, 4, D), "f32")
    small = 1.0 if kind != "f16" else 0.25        # 25000: finite in fp16
    q[..., 21] = factor
    q = (q * small).to(TYPES[kind])
    assert torch.isfinite(q).all()
    scale = 0.1 / small
    out, lse = prefill(case, q, [n], scale)
    check(out, lse, q, case, [n], scale, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 12, 40, 200])
def test_queries_up_to_the_largest_number(cuda_device, n, kind):
    """Rows of q whose largest element is 2^125 to just below 2^128, and rows of the smallest numbers, with a scale that
    makes ordinary logits of the large ones."""
    case = Case([200], 1, 4, 16, seed=65)
    case.device()
    q = rows(case.rng, (n, 4, D), kind)
    q = q / q.abs().amax(-1, keepdim=True)
    top = torch.tensor([2.0 ** 125, 2.0 ** 126, 2.0 ** 127, 3.3895e38])
    q = (q.float() * top[None, :, None]).to(TYPES[kind])
    if n > 2:
        q[2] = 2.0 ** -126 * torch.sign(q[2].float())
    assert torch.isfinite(q).all()
    scale = 2.0 ** -126
    out, lse = prefill(case, q, [n], scale)
    check(out, lse, q, case, [n], scale, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [1, 5, 12, 40, 200])
def test_logits_far_below_zero(cuda_device, n, kind):
    """All logits of a row between -3e30 and -1e38: the nearest to zero has all the weight."""
    T = 260
    case = Case([T], 1, 1, 16, seed=66)
    kv = case.device()
    gen = torch.Generator().manual_seed(67)
    k = torch.zeros(T, 1, D)
    k[:, 0, 40] = torch.tensor([1.5, 2.0, 3.0, 4.0, 6.0])[torch.randint(0, 5, (T,), generator=gen)]
    k[:, 0, 41] = 6.0                    # the block's scale is 1, its codes are the values
    k[T - n - 7, 0, 40] = 1.0            # every row sees this one
    cu = cu_of([T])
    v = torch.randn(T, 1, D, generator=gen)
    P.hsa_kv4_write(kv, k.to(cuda_device), v.to(cuda_device), cu.to(cuda_device), cu)
    case.bytes = kv.cache.cpu().numpy()
    q = torch.zeros(n, 1, D)
    for top in (3e30, 1e37):
        q[:, 0, 40] = -32768.0
        scale = float(np.float32(top / 32768.0))
        out, lse = prefill(case, q.to(TYPES[kind]), [n], scale)
        want = case.held(0, 0)[1][T - n - 7]
        got = out[:, 0].double().cpu().numpy()
        half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[kind]
        assert (np.abs(got - want) <= (half + 2.0 ** -20) * np.abs(want)).all()
        assert (torch.abs(lse.double().cpu() / -top - 1) <= 2.0 ** -20).all()


@pytest.mark.parametrize("n", [1, 20])
def test_strides_of_dims_of_one_are_not_looked_at(cuda_device, n):
    """One KV head, or one row, whose stride says nothing (torch leaves any number there)."""
    case = Case([60], 1, 1, 16, seed=83)
    kv = case.device()
    cu, st = cu_of([n]), i32([60 - n])
    cud, std = cu.to(cuda_device), st.to(cuda_device)
    k, v, q = (torch.randn(n, 1, D, device=cuda_device).half() for _ in range(3))
    odd = lambda x: x.as_strided((n, 1, D), (D if n > 1 else 3, 5, 1))  # noqa: E731
    P.hsa_kv4_write(kv, k, v, cud, cu)
    want = kv.cache.clone()
    kv.cache[:] = torch.from_numpy(case.bytes).to(cuda_device)
    P.hsa_kv4_write(kv, odd(k), odd(v), cud, cu)
    assert torch.equal(kv.cache, want)
    ko, vo = P.hsa_kv4_read(kv, std, st, cud, cu, dtype=torch.float16)
    k2, v2 = odd(torch.empty_like(ko)), odd(torch.empty_like(vo))
    P.hsa_kv4_read(kv, std, st, cud, cu, k_out=k2, v_out=v2)
    assert torch.equal(k2, ko) and torch.equal(v2, vo)
    out = P.dense_prefill_kv4(kv, odd(q), cud, cu, scale=0.1)
    assert torch.equal(out, P.dense_prefill_kv4(kv, q, cud, cu, scale=0.1))


def test_workspaces_that_are_not_whole_are_refused(cuda_device):
    """An expanded byte has the workspace's size and none of its memory."""
    case = Case([40], 2, 2, 16)
    kv = case.device()
    ws = torch.zeros(1, dtype=torch.uint8, device=cuda_device).expand(P.hsa_kv4_workspace_bytes(kv))
    with pytest.raises(ValueError):
        P.dense_decode_kv4(kv, torch.zeros(1, 4, D, device=cuda_device), scale=0.1, workspace_buf=ws)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [1, 5, 12, 40, 200])
def test_rows_of_q_that_are_not_finite(cuda_device, n, kind):
    """An infinite or NaN element makes its row NaN, also where every logit comes out as -inf; other rows keep theirs."""
    T = 230
    case = Case([T], 1, 4, 16, seed=68)
    kv = case.device()
    gen = torch.Generator().manual_seed(69)
    k = torch.randn(T, 1, D, generator=gen)
    k[:, 0, 7] = -k[:, 0, 7].abs() - 1.0
    cu = cu_of([T])
    P.hsa_kv4_write(kv, k.to(cuda_device), torch.randn(T, 1, D, generator=gen).to(cuda_device), cu.to(cuda_device), cu)
    case.bytes = kv.cache.cpu().numpy()
    q = rows(case.rng, (n, 4, D), kind)
    q[0, 1, 7], q[n // 2, 3, 7], q[n - 1, 0, 7] = math.inf, -math.inf, math.nan
    out, lse = prefill(case, q, [n], 0.1)
    bad = torch.isnan(out).cpu()
    assert bad[0, 1].all() and bad[n // 2, 3].all() and bad[n - 1, 0].all() and bad.sum() == 3 * D
    assert torch.isnan(lse).sum() == 3 and torch.isnan(lse[0, 1])
    q[0, 1, 7], q[n // 2, 3, 7], q[n - 1, 0, 7] = 0.0, 0.0, 0.0
    fine, _ = prefill(case, q, [n], 0.1)
    assert torch.equal(out.cpu()[~bad], fine.cpu()[~bad])
