"""The 4-bit KV cache's operators where parts of long contexts meet, where weights and scores are very small or large,
and beside strided outputs: against 64-bit sums on the device."""
import math

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_amax_b200 as fq
from tests import _kv4 as O
from tests.test_gpu_kv4 import DEV, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from fp8_w8a8_quantized_amax_b200 import build
    build.build()
    fq.device_error(clear=True)
    yield
    assert fq.device_error(clear=True) == 0


def cached(pages, page, g, row, n, h):
    """float64 [n, D] on the device: head h of the first n tokens of the pages in `row`."""
    D = pages.shape[2] * 16 // 9 // page
    codes, scales = O.views(pages[row.long()[:(n + page - 1) // page], h:h + 1], page, D)
    codes, scales = codes.reshape(-1, D // 2)[:n].long(), scales.reshape(-1, D // 16)[:n].long()
    e2m1 = torch.tensor(np.concatenate([O.E2M1, -O.E2M1]), device=DEV)
    e4m3 = torch.tensor(np.concatenate([O.E4M3, [math.nan]]), device=DEV)
    v = torch.stack([e2m1[codes & 15], e2m1[codes >> 4]], -1).reshape(n, D // 16, 16) * e4m3[scales][..., None]
    return v.reshape(n, D) * float(np.float32(g))


def attention(b, i, sm=None):
    """What tests._kv4.attention gives for sequence i of a causal batch, as float64 tensors on the device; and max |v|."""
    n, m, D, H = b.lens[i], b.rows[i], b.D, b.H
    r0 = sum(b.rows[:i])
    q = b.q[r0:r0 + m].double()
    G = q.shape[1] // H
    sm = float(np.float32(D ** -0.5 if sm is None else sm))
    hide = torch.arange(n, device=DEV)[None] > torch.arange(n - m, n, device=DEV)[:, None]
    o, a, big = torch.empty_like(q), torch.empty_like(q), 0.0
    lse, e = (torch.empty(q.shape[:2], dtype=torch.float64, device=DEV) for _ in range(2))
    for h in range(H):
        k = cached(b.cache.k_pages, b.page, b.cache.k_scale, b.table_dev[i], n, h)
        v = cached(b.cache.v_pages, b.page, b.cache.v_scale, b.table_dev[i], n, h)
        big = max(big, float(v.abs().max()))
        for x in range(h * G, (h + 1) * G):
            s = (q[:, x] @ k.T * sm).masked_fill_(hide, -math.inf)
            lse[:, x] = torch.logsumexp(s, -1)
            w = torch.exp(s - lse[:, x, None])
            o[:, x], a[:, x] = w @ v, w @ v.abs()
            e[:, x] = (q[:, x].abs() @ k.abs().T * sm).masked_fill_(hide, 0.0).amax(-1)
    return o, lse, a, e, big


def check(b, i, out, lse, sm=None):
    """Sequence i's rows of a call within the bounds that tests/test_gpu_kv4.py derives, but for what small weights lose
    in f16 (n 2^-32 of max|v|, see below)."""
    n, r0 = b.lens[i], sum(b.rows[:i])
    o, l, a, e, big = attention(b, i, sm)
    out, lse = (x[r0:r0 + b.rows[i]].double() for x in (out, lse))
    d = 2 * (b.D + 4) * 2.0 ** -24 * e
    tol = 2 * (d[..., None] + 2.0 ** -20 + 2.0 ** -11 + n * 2.0 ** -24) * a + n * 2.0 ** -32 * big + 2.0 ** -8 * o.abs()
    err = (out - o).abs()
    assert bool((err <= tol).all()), f"sequence {i}: worst excess {float((err - tol).max()):.3g}"
    assert bool(((lse - l).abs() <= d + 2.0 ** -11 + n * 2.0 ** -24 + 2.0 ** -23 * l.abs()).all()), f"sequence {i}: lse"


@pytest.mark.parametrize("lens,H,Hq,D", [
    ([91885, 182], 8, 8, 128), ([32000, 1000, 16384, 100000], 8, 32, 128), ([65536, 1000, 16000, 65536], 8, 32, 128),
    ([16384] * 4, 8, 8, 128), ([131072] * 5, 7, 7, 128), ([700, 33000, 12000, 2500, 21000, 500, 30000, 9000], 8, 16, 64)])
def test_items_whose_parts_leave_one_over_beside_other_items(lens, H, Hq, D):
    """Items of 17, 33, ... parts, the last of them in a CTA that begins with the next item: every row is written, the
    same in every call on one workspace, whose header is left zero."""
    b = Batch(lens, [1] * len(lens), Hq, H, D, 64, seed=21)
    need = fq.fp8q_kv4_attention_workspace_size(b.cache, len(lens), len(lens), Hq)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    first = b.call(workspace=ws)
    assert int(ws[:8192].count_nonzero()) == 0
    for _ in range(30):
        again = b.call(workspace=ws)
        assert int(ws[:8192].count_nonzero()) == 0
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    for i in range(len(lens)):
        check(b, i, *first)


@pytest.mark.parametrize("rows,Hq,H,D", [(1, 8, 2, 128), (1, 6, 2, 64), (8, 4, 1, 128), (8, 4, 1, 64), (90, 2, 2, 128), (70, 4, 1, 64)])
@pytest.mark.parametrize("gap", [9.0, 14.0, 16.5, 17.0, 17.4, 18.5])
def test_many_small_weights_beside_dominant_ones(rows, Hq, H, D, gap):
    """One key in 32 dominates and has values of zero; what comes out is the others', e^-gap and less each.

    A weight is rounded to f16, 2^-11 of itself or, where that has no more bits, 2^-25 of the unit, which is at most 2^-7 of
    the row's largest weight (2^0 by 2^7 at the least).  So n keys lose at most n 2^-32 of the largest weight times max|v|,
    and the sum they are divided by is S = sum exp(s - max s) times that weight.  The other terms are those of
    tests/test_gpu_kv4.py, whose n 2^-24 max|v| this one replaces."""
    n = 700
    b = Batch([n], [rows], Hq, H, D, 64, seed=31, kg=2.0 ** -8, vg=2.0 ** -8)
    j = torch.arange(n)
    slots = (b.table[0].long()[j // 64] * 64 + j % 64).to(DEV)
    g = torch.Generator().manual_seed(5)
    sink = (j % 32 == 3).view(-1, 1, 1)
    # 0.75 = 6 * 32 * 2^-8 is a value of the cache; v has one sign, so that nothing cancels
    k = torch.where(sink, 0.75, 0.0).expand(n, H, D).to(torch.bfloat16).contiguous().to(DEV)
    v = torch.where(sink, 0.0, torch.randn((n, H, D), generator=g).abs()).to(torch.bfloat16).to(DEV)
    fq.fp8q_kv4_append(b.cache, k, v, slots)
    # rows of smaller and smaller gaps: 1 - r / 256 is a bf16
    b.q.copy_((1.0 - torch.arange(rows, device=DEV) / 256.0).view(-1, 1, 1).expand_as(b.q))
    sm = float(np.float32(gap / (0.75 * D)))
    out, lse = b.call(sm_scale=sm)
    o, l, a, e, big = attention(b, 0, sm)
    d = 2 * (D + 4) * 2.0 ** -24 * e
    S = torch.exp(l - e)                             # (a row's largest score is e: the products have one sign)
    tol = 2 * (d[..., None] + 2.0 ** -20 + 2.0 ** -11 + n * 2.0 ** -24) * a + n * 2.0 ** -32 * big / S[..., None] + 2.0 ** -8 * o
    err = (out.double() - o).abs()
    assert bool((err <= tol).all()), f"off by {float((err / o).max()):.3g} of itself, allowed {float((tol / o).max()):.3g}"
    assert bool(((lse.double() - l).abs() <= d + 2.0 ** -11 + n * 2.0 ** -24 + 2.0 ** -23 * l.abs()).all())


@pytest.mark.parametrize("rows,Hq,H,D", [(1, 8, 2, 128), (8, 4, 1, 64), (90, 2, 2, 128), (70, 4, 1, 64)])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 24, 2.0 ** 26])
def test_scores_of_any_size_below_the_limit_give_numbers(rows, Hq, H, D, size):
    """One key's score is +-size and the others' a part of it: where the gap to the next is above the bound of the scores'
    own error, the output is that key's value (or that of the keys of equal score), to f16's and bf16's half steps."""
    n = 300
    b = Batch([n], [rows], Hq, H, D, 64, seed=33, kg=2.0 ** -8, vg=2.0 ** -8)
    j = torch.arange(n)
    slots = (b.table[0].long()[j // 64] * 64 + j % 64).to(DEV)
    # scores size * (1, 1/2, 1/4, ...) over and over, and zero: powers of two are values of the cache
    k = (0.75 * 2.0 ** -(j % 5).float()).view(-1, 1, 1).expand(n, H, D).to(torch.bfloat16).contiguous().to(DEV)
    v = torch.randn((n, H, D), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    fq.fp8q_kv4_append(b.cache, k, v, slots)
    for sign in (1.0, -1.0):
        b.q.copy_((sign * (1.0 - torch.arange(rows, device=DEV) / 256.0)).view(-1, 1, 1).expand_as(b.q))
        sm = float(np.float32(size / (0.75 * D)))
        out, lse = b.call(sm_scale=sm)
        o, l, a, e, big = attention(b, 0, sm)
        # equal keys have equal scores, so only the largest score's keys are left, with equal weights; sums of up to n
        tol = 2 * (2.0 ** -11 + n * 2.0 ** -24) * a + 2.0 ** -8 * o.abs()
        assert bool(((out.double() - o).abs() <= tol).all())
        d = 2 * (D + 4) * 2.0 ** -24 * e
        assert bool(((lse.double() - l).abs() <= d + 2.0 ** -11 + n * 2.0 ** -24 + 2.0 ** -23 * l.abs()).all())


@pytest.mark.parametrize("rows,q_start", [(1, False), (3, True), (90, True)])
def test_sequences_that_are_all_empty_need_no_page(rows, q_start):
    cache = fq.KV4Cache.empty(2, 2, 16, 128)
    q = torch.randn((2 * rows + 1, 8, 128), device=DEV).to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
    start = torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device=DEV) if q_start else None
    table = torch.zeros((2, 0), dtype=torch.int32, device=DEV)
    for ws in (None, torch.zeros(fq.fp8q_kv4_attention_workspace_size(cache, 2, q.shape[0], 8, rows), dtype=torch.uint8, device=DEV)):
        fq.fp8q_kv4_attention(q, cache, table, torch.zeros(2, dtype=torch.int32, device=DEV), start, rows, out=out, lse=lse,
                              workspace=ws)
        assert bool((out[:-1] == 0).all()) and bool((out[-1] == 7.0).all())
        assert bool((lse[:-1] == -math.inf).all()) and bool((lse[-1] == 7.0).all())


def inside(T, H, D):
    """A buffer of fives, views of it [T, H, D] (token-major, head-major), and whether all outside a view is as it was."""
    for shape, cut in (((T + 2, H + 3, D + 8), lambda x: x[1:T + 1, 2:H + 2, :D]),
                       ((H + 2, T + 3, D + 16), lambda x: x[1:H + 1, 2:T + 2, 8:D + 8].transpose(0, 1))):
        base = torch.full(shape, 5.0, dtype=torch.bfloat16, device=DEV)
        untouched = torch.ones(shape, dtype=torch.bool, device=DEV)
        cut(untouched).fill_(False)
        yield cut(base), lambda: bool((base[untouched] == 5.0).all())


@pytest.mark.parametrize("rows,Hq,H,D", [([3, 66], 8, 2, 128), ([1, 2], 8, 2, 128), ([1, 2], 6, 2, 64), ([90, 7], 4, 4, 64)])
def test_attention_writes_nothing_beside_a_strided_output(rows, Hq, H, D):
    b = Batch([70, 410], rows, Hq, H, D, 16, seed=41)
    want, _ = b.call()
    for out, untouched in inside(sum(rows), Hq, D):
        b.call(out=out)
        assert torch.equal(out, want) and untouched()


@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (64, 6), (64, 24)])
def test_rotation_and_read_back_write_nothing_beside_a_strided_output(D, R):
    T, H = 37, 3
    x = torch.randn((T, H, D), device=DEV).to(torch.bfloat16)
    positions, freq = torch.arange(T, device=DEV), fq.fp8q_rope_frequencies(R)
    cache, slots = fq.KV4Cache.empty(4, H, 16, D, 0.004, 0.004), torch.arange(T, device=DEV)
    fq.fp8q_kv4_append(cache, x, x, slots)
    want, (k, v) = fq.fp8q_rope(x, positions, freq), fq.fp8q_kv4_read(cache, slots)
    for (out, untouched), (other, as_well) in zip(inside(T, H, D), inside(T, H, D)):
        assert torch.equal(fq.fp8q_rope(x, positions, freq, out=out), want) and untouched()
        fq.fp8q_kv4_read(cache, slots, out=(out, other))
        assert torch.equal(out, k) and torch.equal(other, v) and untouched() and as_well()
