"""Rotary positions and the 4-bit KV cache on the GPU against plain 64-bit forms.

Tolerances.
  Rotation: the bf16 result is off by half a step, 2^-8 |y|; before that, fp32 products and an fp32 sum (three
  roundings, 2^-24 each of at most m (|x0| + |x1|)) and cos/sin from an fp32 argument: half turns r, |r| <= 1, off by
  2^-25, so an angle off by pi 2^-25 < 2^-23, plus the functions' own 2^-23.  Together below 2^-21 m (|x0| + |x1|).
  Codes and scales: equal, bit for bit (the definition's fp32 steps; K is rotated in fp64 and rounded once, and an
  fp64 angle's 2^-40 moves no code of these inputs).
  Read: code * scale is exact, the factor one fp32 rounding, bf16 half a step: (2^-8 + 2^-23) |v|.
  Attention: with e = max_j sum_d |q_d k_jd| sm_scale, a score is an fp32 sum of D products, off by at most
  (D + 4) 2^-24 e; the exponent's argument is off by as much again (its difference to the maximum, in fp32, and a
  power-of-two conversion), so a weight by a factor exp(+-d), d = 2 (D + 4) 2^-24 e, its own evaluation (2^-21) and its
  rounding to f16 (2^-11, or 2^-24 of the largest weight where subnormal).  The sum over n keys in fp32 adds at most
  n 2^-24.  Numerator and denominator each: |o' - o| <= 2 (d + 2^-20 + 2^-11 + n 2^-24) a + n 2^-24 max|v| + 2^-8 |o|,
  a = sum of w |v|.  lse: d + 2^-11 (where the sum is of rounded weights) + n 2^-24, and 2^-23 |lse|.
"""
import ctypes
import threading

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_amax_b200 as fq
from tests import _kv4 as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
LLAMA3 = {"type": "llama3", "factor": 8.0, "low": 1.0, "high": 4.0, "original_max_position": 8192.0}
ERR_BAD_SLOT, ERR_BAD_PAGE, ERR_BAD_LENGTH = 0x201, 0x202, 0x203


@pytest.fixture(scope="module", autouse=True)
def _built():
    from fp8_w8a8_quantized_amax_b200 import build
    build.build()
    fq.device_error(clear=True)
    yield
    assert fq.device_error(clear=True) == 0


def heads(T, H, D, seed, wide=0, at=0, head_major=False, offset=0):
    """bf16 [T, H, D]: contiguous, part of wider rows, head-major or `offset` elements off an allocation's start."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, max(wide, H + at), D), generator=g).to(torch.bfloat16)
    if head_major:
        return x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)[:, at:at + H]
    if offset:
        flat = torch.zeros(x.numel() + offset, dtype=torch.bfloat16, device=DEV)
        flat[offset:] = x.reshape(-1).to(DEV)
        return flat[offset:].view(x.shape)[:, at:at + H]
    return x.to(DEV)[:, at:at + H]


# ------------------------------------------------------------------- rope ---

def check_rope(y, x, positions, freq, **kw):
    ref = O.rotate(O.f64(x), positions.cpu().numpy(), freq.cpu().numpy(), **kw)
    size = np.abs(O.rotate(np.abs(O.f64(x)), np.zeros(len(positions)), freq.cpu().numpy()))
    n = freq.numel()
    i = np.arange(n)
    d0, d1 = (2 * i, 2 * i + 1) if kw.get("interleaved") else (i, i + n)
    both = size[..., d0] + size[..., d1]
    size = np.zeros_like(size)
    size[..., d0] = size[..., d1] = both
    err = np.abs(O.f64(y) - ref)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * kw.get("mscale", 1.0) * size
    assert np.all(err <= tol), f"worst excess {np.max(err - tol):.3g} of {np.abs(ref).max():.3g}"


@pytest.mark.parametrize("T,H,D,R,kw", [
    (1, 1, 128, 128, {}),
    (7, 72, 128, 128, dict(wide=80)),
    (33, 5, 64, 64, dict(wide=9, at=2)),
    (301, 8, 128, 64, {}),                       # part of the head
    (19, 3, 64, 32, dict(head_major=True)),
    (40, 3, 80, 32, {}),                         # another head size
    (11, 4, 96, 6, {}),                          # pairs that no vector holds
    (23, 2, 128, 128, dict(offset=1)),           # rows that are not 16-byte aligned
    (17, 3, 50, 50, {}),                         # rows of an odd number of 16-byte parts
    (5, 2, 2, 2, {}),
    (700, 40, 128, 128, dict(wide=48)),
    (5, 3, 128, 16, {}), (5, 3, 128, 24, {}), (9, 130, 64, 64, {}),
])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(T, H, D, R, kw, interleaved):
    x = heads(T, H, D, T + H + D, **kw)
    g = torch.Generator().manual_seed(T)
    positions = torch.randint(0, 131072, (T,), generator=g).to(DEV)
    freq = fq.fp8q_rope_frequencies(R, scaling=LLAMA3)
    keep = x.clone()
    y = fq.fp8q_rope(x, positions, freq, interleaved=interleaved)
    assert torch.equal(x, keep)
    check_rope(y, x, positions, freq, interleaved=interleaved)
    assert torch.equal(y[..., R:], x[..., R:])
    # in place, and into a strided output, give the same
    z = torch.empty((T, H + 1, D + 8), dtype=torch.bfloat16, device=DEV)[:, 1:, :D]
    assert torch.equal(fq.fp8q_rope(x, positions, freq, interleaved=interleaved, out=z), y)
    fq.fp8q_rope(x, positions, freq, interleaved=interleaved, out=x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inverse_is_the_gradient_and_undoes_it(interleaved):
    T, H, D, R = 37, 3, 128, 96
    x, g = heads(T, H, D, 1), heads(T, H, D, 2)
    positions = torch.arange(1000, 1000 + T, device=DEV)
    freq = fq.fp8q_rope_frequencies(R)
    gx = fq.fp8q_rope(g, positions, freq, interleaved=interleaved, inverse=True)
    check_rope(gx, g, positions, freq, interleaved=interleaved, inverse=True)
    # the gradient of sum(g * rope(x)) by differences of the (linear) 64-bit form: one element at a time
    p, f = positions.cpu().numpy(), freq.cpu().numpy()
    G, X = O.f64(g), O.f64(x)
    rng = np.random.default_rng(0)
    for _ in range(20):
        t, h, d = rng.integers(T), rng.integers(H), rng.integers(D)
        up, down = X.copy(), X.copy()
        up[t, h, d] += 0.5
        down[t, h, d] -= 0.5
        diff = (G * O.rotate(up, p, f, interleaved=interleaved)).sum() - \
            (G * O.rotate(down, p, f, interleaved=interleaved)).sum()
        # 64-bit sums of 14,000 terms of size up to 16; bf16's half step; the 2^-21 of the rotation
        assert abs(float(gx[t, h, d]) - diff) <= 2.0 ** -8 * abs(diff) + 2.0 ** -18 + 1e-9
    back = fq.fp8q_rope(fq.fp8q_rope(x, positions, freq, interleaved=interleaved), positions, freq,
                        interleaved=interleaved, inverse=True)
    i = np.arange(R // 2)
    size = np.zeros_like(X)
    d0, d1 = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    size[..., d0] = size[..., d1] = np.hypot(X[..., d0], X[..., d1])
    size[..., R:] = np.abs(X[..., R:])
    # a pair keeps its length r: the forward rounding moves it by at most 2^-8 r in each element (sqrt 2 after turning
    # back), the second by 2^-8 of a result that is at most r (1 + 2^-7)
    assert np.all(np.abs(O.f64(back) - X) <= 2.0 ** -8 * 2.45 * size)


def test_rope_far_negative_and_repeated_positions_and_mscale():
    T, H, D = 9, 2, 128
    x = heads(T, H, D, 4)
    positions = torch.tensor([0, 0, 1, -5, 131071, 1 << 20, (1 << 20) + 1, -(1 << 20), 12345], device=DEV)
    freq = fq.fp8q_rope_frequencies(D, 10000.0, {"type": "yarn", "factor": 16.0, "original_max_position": 4096.0})
    for m in (1.0, 1.2772588722239781, 0.5):
        check_rope(fq.fp8q_rope(x, positions, freq, mscale=m), x, positions, freq, mscale=m)
    assert torch.equal(fq.fp8q_rope(x[:2], positions[:2], freq), x[:2])     # position 0 turns nothing


def test_rope_no_tokens():
    freq = fq.fp8q_rope_frequencies(64)
    x = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    assert fq.fp8q_rope(x, torch.empty(0, dtype=torch.int64, device=DEV), freq).shape == x.shape


# ----------------------------------------------------------------- append ---

def new_cache(pages, H, page, D, kg=0.004, vg=2.0 ** -7, seed=0):
    """A cache full of random bytes."""
    g = torch.Generator().manual_seed(seed + 99)
    k, v = (torch.randint(0, 256, (pages, H, page * D * 9 // 16), generator=g, dtype=torch.uint8).to(DEV)
            for _ in range(2))
    return fq.KV4Cache(k, v, page, D, kg, vg)


def check_append(cache, before, k, v, slots, positions=None, freq=None, interleaved=False, mscale=1.0):
    kr = O.f64(k)
    if positions is not None:
        kr = O.rotate(kr, positions.cpu().numpy(), freq.cpu().numpy(), interleaved=interleaved,
                      mscale=float(np.float32(mscale)))
    s = slots.cpu().numpy()
    keep = (s >= 0) & (s < cache.num_pages * cache.page_size)
    p, r = torch.from_numpy(s[keep] // cache.page_size).to(DEV), torch.from_numpy(s[keep] % cache.page_size).to(DEV)
    for pages, old, x, g, what in ((cache.k_pages, before[0], kr, cache.k_scale, "k"),
                                   (cache.v_pages, before[1], O.f64(v), cache.v_scale, "v")):
        codes, scales = O.quantize(x, g)
        want = old.clone()
        wc, ws = O.views(want, cache.page_size, cache.head_dim)
        wc[p, :, r] = torch.from_numpy(codes[keep]).to(DEV)
        ws[p, :, r] = torch.from_numpy(scales[keep]).to(DEV)
        bad = (pages != want).sum().item()
        assert bad == 0, f"{what}: {bad} bytes differ"


APPENDS = [  # T, H, D, page, rot, layout
    (1, 8, 128, 16, 128, {}),
    (64, 8, 128, 64, 128, dict(wide=48, at=3)),
    (37, 3, 64, 32, 64, {}),
    (101, 5, 64, 16, 32, dict(head_major=True)),
    (50, 1, 128, 256, 64, {}),
    (13, 2, 128, 128, 8, {}),
    (13, 2, 128, 128, 24, {}),
    (13, 7, 64, 16, 40, {}),
    (29, 4, 128, 32, 0, {}),
    (1000, 8, 128, 64, 128, dict(wide=48)),
]


@pytest.mark.parametrize("T,H,D,page,rot,kw", APPENDS)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(T, H, D, page, rot, kw, interleaved):
    pages = T // page + 5
    cache = new_cache(pages, H, page, D, seed=T)
    before = cache.k_pages.clone(), cache.v_pages.clone()
    k, v = heads(T, H, D, T, **kw), heads(T, H, D, T + 1, **kw)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.1] = -1
    slots = slots.to(DEV)
    positions = torch.randint(0, 131072, (T,), generator=g).to(DEV) if rot else None
    freq = fq.fp8q_rope_frequencies(rot, scaling=LLAMA3) if rot else None
    fq.fp8q_kv4_append(cache, k, v, slots, positions, freq, interleaved=interleaved, mscale=1.0)
    check_append(cache, before, k, v, slots, positions, freq, interleaved)
    check_read(cache, slots)


def check_read(cache, slots):
    """Read back equals the values of the cache's own bytes."""
    kb, vb = fq.fp8q_kv4_read(cache, slots)
    s = slots.cpu().numpy()
    keep = s >= 0
    at = np.where(keep, s, 0)
    for y, pages, g in ((kb, cache.k_pages, cache.k_scale), (vb, cache.v_pages, cache.v_scale)):
        codes, scales = O.views(pages, cache.page_size, cache.head_dim)
        p, r = torch.from_numpy(at // cache.page_size).to(DEV), torch.from_numpy(at % cache.page_size).to(DEV)
        ref = O.values(codes[p, :, r].cpu().numpy(), scales[p, :, r].cpu().numpy(), g) * keep[:, None, None]
        assert np.all(np.abs(O.f64(y) - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref))


def test_append_special_values():
    """Zeros, -0, blocks whose scale rounds to zero or saturates, values on the codes' borders, tiny and huge ones."""
    D, H, page = 128, 1, 16
    rows = []
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    for s in (1.0, 0.0078125, 0.25, 448.0, 3.75):
        rows.append(torch.cat([grid * s, -grid * s] * 4))
    rows.append(torch.zeros(D))
    rows.append(-torch.zeros(D))
    rows.append(torch.full((D,), 1e-30))
    rows.append(torch.full((D,), 2e5))
    rows.append(torch.linspace(-3e38, 3e38, D))
    rows.append(torch.tensor([2.0 ** -133 * i for i in range(D)]))
    rows.append(torch.tensor([(-2.0) ** (i % 16 - 14) for i in range(D)]))
    x = torch.stack(rows).to(torch.bfloat16).view(-1, H, D).to(DEV)
    T = x.shape[0]
    slots = torch.arange(T, device=DEV)
    for g in (1.0, 2.0 ** -7, 0.011, 3.0):
        cache = new_cache(2, H, page, D, kg=g, vg=g)
        before = cache.k_pages.clone(), cache.v_pages.clone()
        fq.fp8q_kv4_append(cache, x, x, slots)
        check_append(cache, before, x, x, slots)


def test_append_every_bf16_magnitude_against_its_blocks_scale():
    """All finite positive bf16 values, each in a block whose first element sets the scale."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).float()
    x = x[(x > 2e-3) & (x < 7.0)]
    n = x.numel() // 120 * 120
    x = x[:n].view(-1, 8, 15)
    for top in (6.0, 5.5, 7.25):
        b = torch.cat([torch.full((x.shape[0], 8, 1), top), x], -1).reshape(-1, 1, 128).to(torch.bfloat16).to(DEV)
        cache = new_cache(b.shape[0] // 16 + 1, 1, 16, 128, kg=1.0, vg=0.37)
        before = cache.k_pages.clone(), cache.v_pages.clone()
        slots = torch.arange(b.shape[0], device=DEV)
        fq.fp8q_kv4_append(cache, b, b, slots)
        check_append(cache, before, b, b, slots)


def test_append_slots_past_the_cache_are_skipped_and_reported():
    T, H, D, page = 6, 2, 128, 16
    cache = new_cache(3, H, page, D)
    before = cache.k_pages.clone(), cache.v_pages.clone()
    k, v = heads(T, H, D, 1), heads(T, H, D, 2)
    slots = torch.tensor([5, 48, 47, -1, 1 << 40, 0], device=DEV)
    fq.fp8q_kv4_append(cache, k, v, slots)
    assert fq.device_error(clear=True) == ERR_BAD_SLOT
    check_append(cache, before, k, v, slots)
    kb, _ = fq.fp8q_kv4_read(cache, slots)
    assert fq.device_error(clear=True) == ERR_BAD_SLOT
    assert (kb[torch.tensor([1, 3, 4])] == 0).all() and (kb[0] != 0).any()


# -------------------------------------------------------------- attention ---

class Batch:
    """Sequences in a paged cache, filled through fp8q_kv4_append (or with random bytes)."""

    def __init__(self, lens, rows, Hq, H, D, page, seed=0, pad=0, kg=0.0041, vg=2.0 ** -8, spare=3, q_kw=None,
                 spread=1.0):
        g = torch.Generator().manual_seed(seed + 7)
        self.lens, self.rows, self.D, self.page, self.H = lens, rows, D, page, H
        most = max(1, max((n + page - 1) // page for n in lens))
        need = sum((n + page - 1) // page for n in lens)
        ids = torch.randperm(need + spare, generator=g)
        # entries that no token needs point nowhere
        self.table = torch.full((len(lens), most), -7, dtype=torch.int32)
        at = 0
        slots = []
        for b, n in enumerate(lens):
            m = (n + page - 1) // page
            self.table[b, :m] = ids[at:at + m]
            at += m
            j = torch.arange(n)
            slots.append(self.table[b].long()[j // page] * page + j % page)
        k_pages, v_pages = (torch.full((need + spare, H, page * D * 9 // 16), 0x7F, dtype=torch.uint8, device=DEV)
                            for _ in range(2))           # scales of 0x7F are NaN: nothing may read them
        self.cache = fq.KV4Cache(k_pages, v_pages, page, D, kg, vg)
        slots = torch.cat(slots).to(DEV)
        k = (torch.randn((slots.numel(), H, D), generator=g) * spread).to(torch.bfloat16).to(DEV)
        v = torch.randn((slots.numel(), H, D), generator=g).to(torch.bfloat16).to(DEV)
        if slots.numel():
            fq.fp8q_kv4_append(self.cache, k, v, slots)
        T = sum(rows) + pad
        self.q = heads(T, Hq, D, seed + 3, **(q_kw or {}))
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV)
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.table_dev = self.table.to(DEV)

    def call(self, out=None, lse=None, **kw):
        T, Hq, D = self.q.shape
        out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
        lse = torch.full((T, Hq), 7.0, dtype=torch.float32, device=DEV) if lse is None else lse
        kw.setdefault("max_q_len", max(max(self.rows), 1))
        kw.setdefault("q_start", self.q_start)
        fq.fp8q_kv4_attention(self.q, self.cache, self.table_dev, self.kv_len, out=out, lse=lse, **kw)
        return out, lse

    def check(self, out, lse, sm_scale=None, causal=True, window=0, only=None):
        D = self.D
        sm = float(np.float32(D ** -0.5 if sm_scale is None else sm_scale))
        q = O.f64(self.q)
        r0 = 0
        for b, (n, m) in enumerate(zip(self.lens, self.rows)):
            if (only is None or b in only) and m:
                row = self.table[b].tolist()
                k = O.cached(self.cache.k_pages, self.page, D, self.cache.k_scale, row, n)
                v = O.cached(self.cache.v_pages, self.page, D, self.cache.v_scale, row, n)
                o, l, a, e = O.attention(q[r0:r0 + m], k, v, sm, causal, window)
                d = 2 * (D + 4) * 2.0 ** -24 * e
                big = np.abs(v).max() if n else 0.0
                tol = 2 * (d[..., None] + 2.0 ** -20 + 2.0 ** -11 + n * 2.0 ** -24) * a + n * 2.0 ** -24 * big + \
                    2.0 ** -8 * np.abs(o)
                err = np.abs(O.f64(out[r0:r0 + m]) - o)
                assert np.all(err <= tol), f"sequence {b}: worst excess {np.nanmax(err - tol):.3g}, nan {np.isnan(err).sum()}"
                got = lse[r0:r0 + m].cpu().numpy().astype(np.float64)
                dead = np.isinf(l)
                assert np.array_equal(got[dead], l[dead])
                tol = d + 2.0 ** -11 + n * 2.0 ** -24 + 2.0 ** -23 * np.abs(l, where=~dead, out=np.zeros_like(l))
                assert np.all(np.abs(got - l)[~dead] <= tol[~dead])
            r0 += m
        assert (out[r0:] == 7.0).all() and (lse[r0:] == 7.0).all()      # rows of no sequence


ATTENTIONS = [  # lens, rows, Hq, H, D, page, options
    ([1], [1], 1, 1, 128, 16, {}),
    ([500], [1], 32, 8, 128, 16, {}),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300], [1] * 13, 8, 2, 128, 16, dict(pad=2)),
    ([1000, 3, 700], [1, 1, 1], 24, 8, 128, 64, {}),                    # three query heads to a key head
    ([333, 222], [1, 1], 10, 2, 64, 32, {}),
    ([400], [1], 64, 8, 128, 256, {}),
    ([90, 900], [1, 1], 33, 3, 128, 128, {}),                           # eleven
    ([200, 100], [1, 1], 40, 1, 64, 16, {}),                            # forty
    ([100, 260, 31], [4, 5, 3], 16, 2, 128, 32, dict(pad=3)),           # drafted tokens
    ([100, 260, 31, 2, 0], [7, 0, 31, 5, 2], 6, 2, 128, 32, dict(pad=1)),   # rows that see nothing, none at all
    ([300], [300], 4, 1, 128, 64, {}),                                  # a whole prompt
    ([300, 77, 129], [130, 77, 128], 6, 2, 64, 16, dict(pad=5)),
    ([513], [129], 8, 8, 128, 64, {}),
    ([700], [64], 12, 4, 64, 128, dict(q_kw=dict(wide=20, at=1))),      # queries inside fused rows
    ([180], [90], 5, 5, 128, 16, dict(q_kw=dict(head_major=True))),
    ([300, 90], [3, 2], 16, 2, 128, 16, {}),                            # 24 rows, 25, 80 and 81: where the tiles change
    ([300, 90], [5, 2], 25, 5, 64, 32, {}),
    ([300, 90], [10, 3], 16, 2, 128, 64, dict(pad=1)),
    ([300, 290], [27, 3], 6, 2, 64, 16, {}),
]


@pytest.mark.parametrize("lens,rows,Hq,H,D,page,kw", ATTENTIONS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50), (False, 9), (True, 1)])
def test_attention(lens, rows, Hq, H, D, page, kw, causal, window):
    b = Batch(lens, rows, Hq, H, D, page, seed=len(lens) + Hq, **kw)
    out, lse = b.call(causal=causal, window=window)
    b.check(out, lse, causal=causal, window=window)


@pytest.mark.parametrize("spread,sm_scale", [(30.0, None), (0.01, 3.0), (1.0, 1e-6), (30.0, 1.0)])
def test_attention_peaked_and_flat(spread, sm_scale):
    b = Batch([257, 900], [1, 40], 8, 2, 128, 64, seed=5, spread=spread, kg=0.0041 * spread)
    out, lse = b.call(sm_scale=sm_scale)
    b.check(out, lse, sm_scale=sm_scale)


def test_attention_queries_of_very_different_sizes():
    """Rows of large and tiny queries, and elements 2^40 apart within a row."""
    b = Batch([300, 130], [1, 70], 8, 2, 128, 32, seed=6)
    for i, f in enumerate((1.0, 50.0, 1e-4, 1e-20, 0.0, 1e-38)):
        b.q[i::6] *= f
    b.q[:, 1, ::7] *= 2.0 ** -40
    b.q[:, 2, 5] *= 2.0 ** 20
    out, lse = b.call()
    b.check(out, lse)


def test_attention_without_q_start_and_without_lse():
    b = Batch([40, 0, 900], [1, 1, 1], 16, 4, 128, 32, seed=1, pad=2)
    out, lse = b.call(q_start=None)
    b.check(out, lse)
    again = torch.full_like(out, 7.0)
    fq.fp8q_kv4_attention(b.q, b.cache, b.table_dev, b.kv_len, out=again)
    assert torch.equal(out, again)


def test_attention_into_strided_and_head_major_outputs():
    b = Batch([70, 410], [3, 66], 8, 2, 128, 16, seed=2)
    want, lse = b.call()
    T = b.q.shape[0]
    for out in (torch.full((T, 11, 136), 5.0, dtype=torch.bfloat16, device=DEV)[:, 2:10, :128],
                torch.full((8, T, 128), 5.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)):
        b.call(out=out)
        assert torch.equal(out, want)
    assert (torch.full((T, 11, 136), 5.0)[:, :2] == 5.0).all()


@pytest.mark.parametrize("rows,Hq", [([1] * 6, 32), ([3] * 6, 16), ([70] * 6, 8)])
def test_attention_is_deterministic_and_leaves_its_workspace_zero(rows, Hq):
    b = Batch([2000, 3100, 77, 500, 1900, 1024], rows, Hq, 8, 128, 64, seed=3)
    need = fq.fp8q_kv4_attention_workspace_size(b.cache, 6, b.q.shape[0], Hq, max(rows))
    ws = torch.zeros(need + 64, dtype=torch.uint8, device=DEV)
    first = b.call(workspace=ws)
    for _ in range(5):
        again = b.call(workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert int(ws[:8192].count_nonzero()) == 0
    b.check(*first, only=[2, 3])


@pytest.mark.parametrize("rows", [1, 8])
def test_attention_one_long_item_over_all_ctas_and_another_behind_it(rows):
    """Hundreds of parts joined while the CTA that joins them has the next item's keys on their way."""
    b = Batch([130_000, 260, 200], [rows] * 3, 4, 1, 64, 64, seed=12)
    first = b.call()
    b.check(*first)
    for _ in range(20):
        again = b.call()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("rows", [1, 8, 70])
def test_attention_a_window_longer_than_any_context_is_none(rows):
    b = Batch([500, 130], [rows, rows], 8, 2, 128, 32, seed=5)
    want, lse = b.call()
    for window in (500, 2 ** 31, 2 ** 62, 2 ** 63 - 1):
        got = b.call(window=window)
        assert torch.equal(got[0], want) and torch.equal(got[1], lse), window


def test_attention_bad_lengths_and_pages_are_reported():
    """A bad index on the device leads nowhere: the error word names it, the other sequences are right."""
    b = Batch([100, 200, 300], [1, 1, 1], 8, 2, 128, 32, seed=4)
    good = b.table_dev.clone()
    for bad in (-1, b.cache.num_pages, 1 << 30):
        b.table_dev[1, 2] = bad
        out, lse = b.call()
        assert fq.device_error(clear=True) == ERR_BAD_PAGE
        b.check(out, lse, only=[0, 2])
    b.table_dev = good
    for bad in (-1, b.table.shape[1] * 32 + 1):
        b.kv_len[1] = bad
        out, lse = b.call()
        assert fq.device_error(clear=True) == ERR_BAD_LENGTH
        b.check(out, lse, only=[0, 2])
    b.kv_len[1] = 200
    for starts in ([0, 1, 2, 4], [0, 1, 0, 3], [-2, 1, 2, 3], [0, 1, 2, 1 << 30]):
        b.q_start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        b.call()
        assert fq.device_error(clear=True) == ERR_BAD_LENGTH
    b.q_start = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    out, lse = b.call()
    b.check(out, lse)


@pytest.mark.parametrize("rows", [1, 6, 80])
def test_attention_captured_and_replayed_with_other_lengths(rows):
    """One graph of append and attention, replayed as the sequences grow; two graphs share a workspace."""
    H, Hq, D, page, B = 2, 8, 128, 32, 3
    lens = [150, 90, 333]
    b = Batch([400] * B, [rows] * B, Hq, H, D, page, seed=8)
    ws = torch.zeros(max(16, fq.fp8q_kv4_attention_workspace_size(b.cache, B, B * rows, Hq, rows)), dtype=torch.uint8,
                     device=DEV)
    out = torch.zeros_like(b.q)
    lse = torch.zeros((B * rows, Hq), device=DEV)
    b.kv_len.copy_(torch.tensor(lens))
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        b.call(out=out, lse=lse, workspace=ws)
        for window in (0, 70):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                b.call(out=out, lse=lse, workspace=ws, window=window)
            graphs.append((g, window))
    torch.cuda.synchronize()
    for step in (0, 17, 50):
        now = [n + step for n in lens]
        b.kv_len.copy_(torch.tensor(now))
        b.lens = now
        for g, window in graphs:
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            b.check(out, lse, window=window)


def test_attention_on_another_stream():
    b = Batch([800, 300], [1, 1], 8, 2, 128, 64, seed=9)
    want, _ = b.call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got, _ = b.call()
    s.synchronize()
    assert torch.equal(want, got)


def test_calls_at_once_from_two_threads_on_two_streams():
    """Each with a workspace of its own: appends into one cache's different pages, attention of one token and of many."""
    kinds = [Batch([1500, 700], [1, 1], 8, 2, 128, 64, seed=10), Batch([900, 333], [130, 70], 8, 2, 128, 64, seed=11)]
    want = [b.call() for b in kinds]
    shared = fq.KV4Cache.empty(20, 2, 64, 128, 0.004, 0.004)
    k, v = heads(640, 2, 128, 1), heads(640, 2, 128, 2)
    slots = torch.arange(1280, device=DEV).view(2, 640)
    freq, positions = fq.fp8q_rope_frequencies(128), torch.arange(640, device=DEV)
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        b, T = kinds[i], kinds[i].q.shape[0]
        with torch.cuda.stream(torch.cuda.Stream()):
            ws = torch.zeros(fq.fp8q_kv4_attention_workspace_size(b.cache, 2, T, 8, max(b.rows)), dtype=torch.uint8,
                             device=DEV)
            for _ in range(30):
                fq.fp8q_kv4_append(shared, k, v, slots[i], positions, freq)
                out, lse = b.call(workspace=ws)
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    got = fq.fp8q_kv4_read(shared, slots.view(-1))
    alone = fq.KV4Cache.empty(20, 2, 64, 128, 0.004, 0.004)
    for i in range(2):
        fq.fp8q_kv4_append(alone, k, v, slots[i], positions, freq)
    assert all(torch.equal(a, b) for a, b in zip(got, fq.fp8q_kv4_read(alone, slots.view(-1))))


def test_attention_over_a_cache_past_four_gigabytes():
    """Pages whose byte offsets pass 32 bits."""
    H, D, page = 8, 128, 256
    pages = (1 << 32) // (page * 72 * H) + 40
    one = torch.zeros(pages, H, page * 72, dtype=torch.uint8, device=DEV)
    two = torch.zeros_like(one)
    cache = fq.KV4Cache(one, two, page, D, 0.004, 0.004)
    n = 700
    ids = torch.tensor([[pages - 1, pages - 30, pages - 7]], dtype=torch.int32)
    j = torch.arange(n)
    slots = (ids[0].long()[j // page] * page + j % page).to(DEV)
    k, v = heads(n, H, D, 1), heads(n, H, D, 2)
    fq.fp8q_kv4_append(cache, k, v, slots)
    kb, vb = fq.fp8q_kv4_read(cache, slots)
    small = new_cache(3, H, page, D, 0.004, 0.004)
    fq.fp8q_kv4_append(small, k, v, j.to(DEV))
    ks, vs = fq.fp8q_kv4_read(small, j.to(DEV))
    assert torch.equal(kb, ks) and torch.equal(vb, vs)
    for rows in (1, 3, 90):
        q = heads(rows, 32, D, 3)
        start = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        length = torch.tensor([n], dtype=torch.int32, device=DEV)
        a = fq.fp8q_kv4_attention(q, cache, ids.to(DEV), length, start, rows)
        c = fq.fp8q_kv4_attention(q, small, torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV), length, start,
                                  rows)
        assert torch.equal(a, c)


def test_nothing_to_do():
    cache = new_cache(2, 2, 16, 128)
    before = cache.k_pages.clone()
    none = torch.empty((0, 2, 128), dtype=torch.bfloat16, device=DEV)
    slots = torch.empty(0, dtype=torch.int64, device=DEV)
    fq.fp8q_kv4_append(cache, none, none, slots)
    assert fq.fp8q_kv4_read(cache, slots)[0].shape == (0, 2, 128)
    q = torch.empty((0, 4, 128), dtype=torch.bfloat16, device=DEV)
    out = fq.fp8q_kv4_attention(q, cache, torch.zeros((0, 3), dtype=torch.int32, device=DEV),
                                torch.zeros(0, dtype=torch.int32, device=DEV))
    assert out.shape == q.shape and torch.equal(before, cache.k_pages)


# ------------------------------------------------------- the run of them ---

@pytest.mark.parametrize("H,Hq,D,page,interleaved", [(2, 8, 128, 16, False), (3, 3, 64, 32, True)])
def test_prompt_then_tokens(H, Hq, D, page, interleaved):
    """A prompt in two parts, then single tokens, as a model's layer runs them: rotate the queries, append, attend.
    Every step is compared with the 64-bit forms of the whole chain: keys rotated from the same bf16 rows, quantized
    by the definition, and attention over those values with the rotated bf16 queries."""
    B, cap = 2, 400
    freq = fq.fp8q_rope_frequencies(D, scaling=LLAMA3)
    cache = fq.KV4Cache.empty(B * cap // page + 2, H, page, D, 0.004, 0.004)
    perm = torch.randperm(B * cap // page + 2, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = perm[:B * (cap // page)].view(B, -1).to(DEV)
    k_all = [np.zeros((H, 0, D)) for _ in range(B)]
    v_all = [np.zeros((H, 0, D)) for _ in range(B)]
    lens = [0, 0]
    steps = [[100, 37], [71, 140]] + [[1, 1]] * 4 + [[3, 2]]
    for step, rows in enumerate(steps):
        T = sum(rows)
        qkv = heads(T, Hq + 2 * H, D, 50 + step)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        positions = torch.cat([torch.arange(n, n + m) for n, m in zip(lens, rows)]).to(DEV)
        owner = torch.cat([torch.full((m,), b) for b, m in enumerate(rows)]).to(DEV)
        slots = table[owner, positions // page].long() * page + positions % page
        lens = [n + m for n, m in zip(lens, rows)]
        start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV)
        length = torch.tensor(lens, dtype=torch.int32, device=DEV)
        raw_k, raw_v = O.f64(k), O.f64(v)
        fq.fp8q_rope(q, positions, freq, interleaved=interleaved, out=q)
        fq.fp8q_kv4_append(cache, k, v, slots, positions, freq, interleaved=interleaved)
        lse = torch.empty((T, Hq), device=DEV)
        out = fq.fp8q_kv4_attention(q, cache, table, length, start, max(rows), lse=lse)
        p = positions.cpu().numpy()
        kr = O.values(*O.quantize(O.rotate(raw_k, p, freq.cpu().numpy(), interleaved=interleaved), 0.004), 0.004)
        vr = O.values(*O.quantize(raw_v, 0.004), 0.004)
        r = 0
        for b, m in enumerate(rows):
            k_all[b] = np.concatenate([k_all[b], kr[r:r + m].transpose(1, 0, 2)], 1)
            v_all[b] = np.concatenate([v_all[b], vr[r:r + m].transpose(1, 0, 2)], 1)
            o, l, a, e = O.attention(O.f64(q[r:r + m]), k_all[b], v_all[b], float(np.float32(D ** -0.5)))
            d = 2 * (D + 4) * 2.0 ** -24 * e
            n = lens[b]
            tol = 2 * (d[..., None] + 2.0 ** -20 + 2.0 ** -11 + n * 2.0 ** -24) * a + \
                n * 2.0 ** -24 * np.abs(v_all[b]).max() + 2.0 ** -8 * np.abs(o)
            assert np.all(np.abs(O.f64(out[r:r + m]) - o) <= tol)
            r += m


# ------------------------------------------------------------- the binding ---

def test_cpp_and_python_calls_agree(monkeypatch):
    """The operands' way through the C++ binding and through ctypes: the same results, the same refusals."""
    b = Batch([200, 70], [2, 1], 8, 2, 128, 32, seed=11)
    freq, pos = fq.fp8q_rope_frequencies(128), torch.tensor([5, 6, 9], device=DEV)
    k, v = heads(3, 2, 128, 1, wide=6, at=2), heads(3, 2, 128, 2)
    slots = torch.tensor([3, -1, 40], device=DEV)
    ws = torch.zeros(fq.fp8q_kv4_attention_workspace_size(b.cache, 2, 3, 8, 2), dtype=torch.uint8, device=DEV)

    def everything():
        cache = new_cache(4, 2, 32, 128, seed=5)
        fq.fp8q_kv4_append(cache, k, v, slots, pos, freq, interleaved=True, mscale=1.25)
        out, lse = b.call(workspace=ws, window=33)
        return [fq.fp8q_rope(b.q, pos, freq, inverse=True), cache.k_pages, cache.v_pages,
                *fq.fp8q_kv4_read(cache, slots), out, lse]

    def refusals():
        for call in (lambda: fq.fp8q_rope(b.q.float(), pos, freq), lambda: fq.fp8q_rope(b.q, pos[:2], freq),
                     lambda: fq.fp8q_rope(b.q, pos, freq.float()), lambda: fq.fp8q_rope(b.q.cpu(), pos, freq),
                     lambda: fq.fp8q_kv4_append(b.cache, k[:2], v, slots), lambda: fq.fp8q_kv4_append(b.cache, k, v, slots, pos),
                     lambda: fq.fp8q_kv4_read(b.cache, slots.int()), lambda: b.call(workspace=ws.float()),
                     lambda: b.call(workspace=ws, q_start=b.q_start[:2]), lambda: b.call(workspace=ws, lse=torch.zeros(3, 8))):
            with pytest.raises(ValueError):
                call()
        for call in (lambda: fq.fp8q_rope(b.q, pos, freq, mscale=0.0), lambda: b.call(workspace=ws, window=-1),
                     lambda: b.call(workspace=ws[:100]), lambda: b.call(workspace=ws, max_q_len=0),
                     lambda: fq.fp8q_kv4_append(b.cache, k, v, slots, pos, freq, mscale=float("nan"))):
            with pytest.raises(fq.FP8QError) as e:
                call()
            assert e.value.status == fq.ERR_INVALID_ARG

    fast = everything()
    refusals()

    class Never:
        def __getattr__(self, name):
            return lambda *a: None

    monkeypatch.setattr(fq, "_binding", Never())
    slow = everything()
    refusals()
    for x, y in zip(fast, slow):
        assert torch.equal(x, y)
