"""Rotary positions and the 4-bit KV cache without a GPU: what the C entry points refuse before touching CUDA, what
the binding refuses before it calls them, and the rotary frequencies (host code) against their formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_amax_b200 as fq
from fp8_w8a8_quantized_amax_b200 import build as fbuild
from tests import _kv4 as O
from tests.test_binding_checks import CUDA0, CUDA1, Lib, T

P, BAD = 0x10000, 0x10001
BF, U8, F32, F64, I32, I64 = (torch.bfloat16, torch.uint8, torch.float32, torch.float64, torch.int32, torch.int64)
CPU = torch.device("cpu")
# a valid call reaches the device: there it succeeds or fails by the machine, here there is none
VALID = fq.ERR_CUDA

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="dummy addresses must not reach a device")


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fq.lib()


# ------------------------------------------------------------ frequencies ---

def plain(rot, theta, kind=None, factor=1.0, low=1.0, high=4.0, orig=0.0):
    out = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if kind == "linear":
            f /= factor
        elif kind == "llama3":
            wave = 2 * math.pi / f
            if wave > orig / low:
                f /= factor
            elif wave >= orig / high:
                smooth = (orig / wave - low) / (high - low)
                f = (1 - smooth) * f / factor + smooth * f
        elif kind == "yarn":
            at = lambda n: rot * math.log(orig / (n * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
            ramp = min(1.0, max(0.0, (i - a) / ((b - a) or 0.001)))
            f = f / factor * ramp + f * (1 - ramp)
        out.append(f)
    return np.array(out)


@pytest.mark.parametrize("rot,theta,scaling", [
    (128, 500000.0, None),
    (2, 10000.0, None),
    (64, 10000.0, {"type": "linear", "factor": 4.0}),
    (128, 500000.0, {"type": "llama3", "factor": 8.0, "low": 1.0, "high": 4.0, "original_max_position": 8192.0}),
    (128, 500000.0, {"type": "llama3", "factor": 32.0, "original_max_position": 8192.0}),
    (128, 10000.0, {"type": "yarn", "factor": 16.0, "original_max_position": 4096.0}),
    (64, 1e6, {"type": "yarn", "factor": 4.0, "low": 2.0, "high": 16.0, "original_max_position": 32768.0}),
])
def test_frequencies(L, rot, theta, scaling):
    got = fq.fp8q_rope_frequencies(rot, theta, scaling, device="cpu").numpy()
    kw = {}
    if scaling:
        kw = dict(kind=scaling["type"], factor=scaling["factor"], orig=scaling.get("original_max_position", 0.0),
                  low=scaling.get("low", 1.0), high=scaling.get("high", 32.0 if scaling["type"] == "yarn" else 4.0))
    ref = plain(rot, theta, **kw)
    assert got.shape == (rot // 2,)
    # pow and log are within a unit in the last place each; llama3's blend subtracts numbers of like size
    assert np.all(np.abs(got - ref) <= 1e-13 * ref)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=-2), dict(rot_dim=7), dict(rot_dim=1 << 20), dict(theta=1.0), dict(theta=float("nan")),
    dict(theta=float("inf")),
    dict(scaling={"type": "linear", "factor": 0.5}), dict(scaling={"type": "linear", "factor": float("nan")}),
    dict(scaling={"type": "llama3", "factor": 8.0}),                                    # no original length
    dict(scaling={"type": "llama3", "factor": 8.0, "low": 4.0, "high": 4.0, "original_max_position": 8192}),
    dict(scaling={"type": "llama3", "factor": 8.0, "low": 0.0, "high": 4.0, "original_max_position": 8192}),
    dict(scaling={"type": "yarn", "factor": 8.0, "low": 40.0, "original_max_position": 8192}),
])
def test_frequencies_refusals(L, kw):
    a = dict(rot_dim=128, theta=10000.0, scaling=None)
    a.update(kw)
    with pytest.raises(fq.FP8QError) as e:
        fq.fp8q_rope_frequencies(device="cpu", **a)
    assert e.value.status == fq.ERR_INVALID_ARG


def test_unknown_scaling(L):
    with pytest.raises(ValueError):
        fq.fp8q_rope_frequencies(128, scaling={"type": "other", "factor": 2.0}, device="cpu")
    s = fq._RopeScaling(9, 2.0, 1.0, 4.0, 8192.0)
    buf = (ctypes.c_double * 64)()
    assert L.fp8q_rope_frequencies(ctypes.addressof(buf), 128, 1e4, ctypes.byref(s)) == fq.ERR_INVALID_ARG
    assert L.fp8q_rope_frequencies(None, 128, 1e4, None) == fq.ERR_INVALID_ARG


# ----------------------------------------------------------- C entry points ---

def rope(L, x=P, T=4, H=8, D=128, xt=1024, xh=128, pos=P, freq=P, rot=128, flags=0, m=1.0, y=P + (1 << 20), yt=1024,
         yh=128):
    return L.fp8q_rope(x, T, H, D, xt, xh, pos, freq, rot, flags, m, y, yt, yh, None)


INV, UNS, MIS = fq.ERR_INVALID_ARG, fq.ERR_UNSUPPORTED, fq.ERR_MISALIGNED


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(), VALID), (dict(T=0, x=None, y=None, pos=None, freq=None), fq.OK),
    (dict(y=P), VALID),                                          # in place
    (dict(y=P, yt=2048), INV), (dict(y=P, yh=256, yt=4096), INV),    # in place with other strides
    (dict(y=P, T=1, yt=99999), VALID),                           # one token has no token stride
    (dict(x=P + 2), VALID), (dict(x=BAD), MIS), (dict(y=(1 << 20) + 1), MIS),
    (dict(pos=P + 4), MIS), (dict(freq=P + 4), MIS),
    (dict(T=-1), INV), (dict(H=0), INV), (dict(D=0), INV), (dict(rot=0), INV), (dict(rot=130), INV),
    (dict(rot=63), INV), (dict(flags=4), INV), (dict(flags=3), VALID), (dict(flags=-1), INV),
    (dict(m=0.0), INV), (dict(m=-1.0), INV), (dict(m=float("nan")), INV), (dict(m=float("inf")), INV),
    (dict(x=None), INV), (dict(y=None), INV), (dict(pos=None), INV), (dict(freq=None), INV),
    (dict(xt=-1), INV), (dict(xh=-8), INV), (dict(xt=0, xh=0), VALID),      # a broadcast input
    (dict(yt=0), INV), (dict(yh=64), INV), (dict(yt=1023), INV),            # rows that overlap
    (dict(yt=128, yh=512), VALID), (dict(yt=128, yh=511), INV),             # head-major
    (dict(T=1 << 31, xt=0, H=1, yt=128), UNS), (dict(T=1 << 30, H=8, yt=1024), UNS),
])
def test_rope_arguments(L, kw, want):
    assert rope(L, **kw) == want


def cache(**kw):
    a = dict(k_pages=P, v_pages=P, num_pages=10, page_size=64, kv_heads=8, head_dim=128, k_scale=0.01, v_scale=0.01)
    a.update(kw)
    return fq._CacheStruct(*(a[n] for n, _ in fq._CacheStruct._fields_))


CACHES = [
    (dict(k_pages=None), INV), (dict(v_pages=None), INV), (dict(k_pages=P + 8), MIS), (dict(v_pages=P + 4), MIS),
    (dict(num_pages=0), INV), (dict(num_pages=-1), INV), (dict(num_pages=1 << 31), UNS),
    (dict(page_size=0), INV), (dict(page_size=48), INV), (dict(page_size=8), UNS), (dict(page_size=512), UNS),
    (dict(page_size=-64), INV), (dict(kv_heads=0), INV), (dict(kv_heads=5000), UNS),
    (dict(head_dim=96), UNS), (dict(head_dim=0), UNS), (dict(head_dim=256), UNS),
    (dict(k_scale=0.0), INV), (dict(v_scale=-1.0), INV), (dict(k_scale=float("nan")), INV),
    (dict(v_scale=float("inf")), INV),
]


def append(L, c=None, k=P, kt=1024, kh=128, v=P, vt=1024, vh=128, slots=P, T=4, pos=P, freq=P, rot=128, flags=0, m=1.0):
    return L.fp8q_kv4_append(ctypes.byref(c or cache()), k, kt, kh, v, vt, vh, slots, T, pos, freq, rot, flags, m, None)


def read(L, c=None, slots=P, T=4, k=P, kt=1024, kh=128, v=P, vt=1024, vh=128):
    return L.fp8q_kv4_read(ctypes.byref(c or cache()), slots, T, k, kt, kh, v, vt, vh, None)


def attend(L, c=None, q=P, qt=4096, qh=128, T=6, Hq=32, table=P, ts=16, mp=16, kv=P, qs=P, B=3, mq=4, sm=0.1, causal=1,
           window=0, o=P, ot=4096, oh=128, lse=None, ws=P, wsb=1 << 30):
    return L.fp8q_kv4_attention(ctypes.byref(c or cache()), q, qt, qh, T, Hq, table, ts, mp, kv, qs, B, mq, sm, causal,
                                window, o, ot, oh, lse, ws, wsb, None)


@no_gpu
@pytest.mark.parametrize("kw,want", CACHES)
def test_every_entry_point_checks_the_cache(L, kw, want):
    c = cache(**kw)
    assert append(L, c) == want and read(L, c) == want and attend(L, c) == want
    assert append(L, c, T=0) == want and read(L, c, T=0) == want
    assert L.fp8q_kv4_attention_workspace_size(ctypes.byref(c), 3, 3, 32, 1) == 0


def test_no_cache(L):
    assert L.fp8q_kv4_append(None, P, 0, 0, P, 0, 0, P, 1, None, None, 0, 0, 1.0, None) == INV
    assert L.fp8q_kv4_read(None, P, 1, P, 0, 0, P, 0, 0, None) == INV
    assert L.fp8q_kv4_attention_workspace_size(None, 1, 1, 1, 1) == 0


@pytest.mark.parametrize("page,heads,D,want", [(16, 1, 128, 1152), (64, 8, 128, 36864), (256, 2, 64, 18432),
                                               (48, 1, 128, 0), (8, 1, 128, 0), (64, 0, 128, 0), (64, 1, 100, 0)])
def test_page_bytes(L, page, heads, D, want):
    assert fq.fp8q_kv4_page_bytes(page, heads, D) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(), VALID), (dict(T=0, k=None, v=None, slots=None), fq.OK), (dict(T=-1), INV),
    (dict(pos=None, freq=None), VALID), (dict(pos=None), INV), (dict(freq=None), INV),
    (dict(k=None), INV), (dict(v=None), INV), (dict(slots=None), INV),
    (dict(k=P + 8), MIS), (dict(v=P + 2), MIS), (dict(slots=P + 4), MIS), (dict(kt=1028), MIS), (dict(vh=132), MIS),
    (dict(kt=-8), INV), (dict(kt=0), VALID),
    (dict(rot=136), INV), (dict(rot=12), UNS), (dict(rot=8), VALID), (dict(rot=0), INV),
    (dict(flags=1), VALID), (dict(flags=2), INV), (dict(flags=8), INV), (dict(m=0.0), INV),
    (dict(T=1 << 30), UNS),
])
def test_append_arguments(L, kw, want):
    assert append(L, **kw) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(), VALID), (dict(T=0, k=None, v=None, slots=None), fq.OK), (dict(T=-1), INV),
    (dict(k=None), INV), (dict(slots=None), INV), (dict(k=P + 8), MIS), (dict(vt=1028), MIS),
    (dict(kt=0), INV), (dict(vh=64), INV), (dict(kt=128, kh=512), VALID), (dict(T=1 << 30), UNS),
])
def test_read_arguments(L, kw, want):
    assert read(L, **kw) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(), VALID), (dict(T=0, q=None, o=None), fq.OK), (dict(B=0, table=None, kv=None), fq.OK),
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(Hq=0), INV), (dict(Hq=33), INV), (dict(mq=0), INV), (dict(mp=-1), INV),
    (dict(window=-1), INV), (dict(causal=2), INV), (dict(causal=0), VALID),
    (dict(sm=0.0), INV), (dict(sm=float("nan")), INV), (dict(sm=float("inf")), INV), (dict(sm=-1.0), INV),
    (dict(q=None), INV), (dict(o=None), INV), (dict(table=None), INV), (dict(kv=None), INV),
    (dict(q=P + 8), MIS), (dict(o=P + 8), MIS), (dict(table=P + 2), MIS), (dict(kv=P + 2), MIS), (dict(qs=P + 2), MIS),
    (dict(lse=P + 2), MIS), (dict(lse=P), VALID), (dict(qt=4100), MIS), (dict(oh=132, ot=8192), MIS),
    (dict(ot=0), INV), (dict(oh=64), INV), (dict(ts=15), INV), (dict(B=1, ts=0), VALID),
    (dict(ws=None), INV), (dict(ws=P + 8), MIS),
    (dict(qs=None), INV),                                      # one row per sequence: max_q_len is 1
    (dict(qs=None, mq=1), VALID), (dict(qs=None, mq=1, T=2), INV),
    (dict(c=cache(k_scale=1e20), sm=1e20), INV), (dict(c=cache(k_scale=1e-20), sm=1e20), VALID),
    (dict(B=70000, T=70000), UNS), (dict(mp=1 << 30, ts=1 << 30), UNS), (dict(mp=(1 << 25) - 1, ts=1 << 25), UNS),
    (dict(mp=1 << 24, ts=1 << 24), VALID), (dict(B=60000, T=60000, mq=5000), UNS), (dict(T=1 << 27, Hq=32, ot=4096), UNS),
])
def test_attention_arguments(L, kw, want):
    assert attend(L, **kw) == want


# ------------------------------------------------------------------ binding ---

class S(T):
    """The stand-in with what the cache's binding reads besides."""

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]


@pytest.fixture
def lib(monkeypatch):
    rec = Lib()
    monkeypatch.setattr(fq, "lib", lambda: rec)
    monkeypatch.setattr(fq, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(fq, "_current_device", lambda: 0)
    return rec


def a_cache(page=32, H=2, D=128, dev=CUDA0):
    t = S((5, H, page * D * 9 // 16), U8, device=dev)
    return fq.KV4Cache(t, t, page, D, 0.01, 0.01)


def refused(lib, name, f, **bad):
    for key, values in bad.items():
        for v in values:
            lib.calls.clear()
            with pytest.raises(ValueError):
                f(**{key: v})
            assert name not in lib.calls, (key, v)


def test_binding_cache(lib):
    good = S((5, 2, 32 * 72), U8)
    fq.KV4Cache(good, good, 32, 128)
    for bad in (S((5, 2, 32 * 72), U8, device=CPU), S((5, 2, 32 * 72), F32), S((5, 2, 32 * 64), U8), S((10, 2304), U8),
                S((4, 2, 32 * 72), U8), S((5, 2, 32 * 72), U8, contiguous=False), S((5, 2, 32 * 72), U8, device=CUDA1)):
        with pytest.raises(ValueError):
            fq.KV4Cache(good, bad, 32, 128)
    with pytest.raises(ValueError):
        fq.KV4Cache(S((5, 2, 32 * 64), U8), S((5, 2, 32 * 64), U8), 32, 128)


@pytest.mark.parametrize("name", ["k_scale", "v_scale", "k_pages", "v_pages", "page_size", "head_dim", "num_pages"])
def test_a_cache_does_not_change_behind_its_calls(lib, name):
    cache = a_cache()
    was = getattr(cache, name)
    with pytest.raises(AttributeError, match=name):
        setattr(cache, name, was)
    assert getattr(cache, name) is was


def test_binding_rope(lib):
    base = dict(x=S((6, 4, 128), BF), positions=S((6,), I64), freq=S((64,), F64), out=S((6, 4, 128), BF))
    call = lambda **kw: fq.fp8q_rope(**{**base, **kw})  # noqa: E731
    call()
    call(x=S((6, 4, 128), BF, strides=(9999, 256, 1)))
    assert lib.calls == ["fp8q_rope"] * 2
    refused(lib, "fp8q_rope", call,
            x=[S((6, 4, 128), BF, device=CPU), S((6, 4, 128), F32), S((6, 512), BF), S((6, 4, 128), BF, strides=(1, 6, 24))],
            positions=[S((5,), I64), S((6,), I32), S((6,), I64, device=CPU), S((6,), I64, contiguous=False), S((6, 1), I64)],
            freq=[S((64,), F32), S((64,), F64, device=CUDA1), S((64,), F64, contiguous=False)],
            out=[S((6, 4, 64), BF), S((6, 4, 128), F32), S((6, 4, 128), BF, device=CUDA1)])


def test_binding_append_and_read(lib):
    base = dict(cache=a_cache(), k=S((6, 2, 128), BF), v=S((6, 2, 128), BF), slots=S((6,), I64), positions=S((6,), I64),
                freq=S((64,), F64))
    call = lambda **kw: fq.fp8q_kv4_append(**{**base, **kw})  # noqa: E731
    call()
    call(positions=None, freq=None)
    assert lib.calls == ["fp8q_kv4_append"] * 2
    heads = [S((6, 3, 128), BF), S((6, 2, 64), BF), S((6, 2, 128), F32), S((6, 2, 128), BF, device=CUDA1), S((6, 256), BF)]
    refused(lib, "fp8q_kv4_append", call, k=heads, v=heads + [S((5, 2, 128), BF)],
            slots=[S((5,), I64), S((6,), I32), S((6,), I64, device=CPU)], positions=[None, S((7,), I64)],
            freq=[None, S((64,), F32)])
    out = (S((6, 2, 128), BF), S((6, 2, 128), BF))
    fq.fp8q_kv4_read(base["cache"], base["slots"], out=out)
    for bad in (dict(slots=S((6,), I32)), dict(out=(out[0], S((5, 2, 128), BF))), dict(out=(S((6, 2, 128), F32), out[1]))):
        with pytest.raises(ValueError):
            fq.fp8q_kv4_read(**{**dict(cache=base["cache"], slots=base["slots"], out=out), **bad})


def test_binding_attention(lib):
    base = dict(q=S((7, 8, 128), BF), cache=a_cache(), page_table=S((3, 9), I32), kv_len=S((3,), I32),
                q_start=S((4,), I32), max_q_len=4, out=S((7, 8, 128), BF), lse=S((7, 8), F32),
                workspace=S((64,), U8))
    call = lambda **kw: fq.fp8q_kv4_attention(**{**base, **kw})  # noqa: E731
    call()
    call(q_start=None, lse=None)
    assert lib.calls.count("fp8q_kv4_attention") == 2
    refused(lib, "fp8q_kv4_attention", call,
            q=[S((7, 8, 64), BF), S((7, 8, 128), F32), S((7, 1024), BF), S((7, 8, 128), BF, device=CUDA1)],
            page_table=[S((3, 9), I64), S((27,), I32), S((3, 9), I32, device=CPU), S((3, 9), I32, strides=(1, 3))],
            kv_len=[S((4,), I32), S((3,), I64), S((3,), I32, device=CPU)],
            q_start=[S((3,), I32), S((4,), I64)],
            out=[S((7, 8, 64), BF), S((6, 8, 128), BF), S((7, 8, 128), F32)],
            lse=[S((7, 8), F64), S((7, 7), F32), S((7, 8), F32, contiguous=False)],
            workspace=[S((64,), F32), S((64,), U8, device=CPU), S((64,), U8, device=CUDA1)])


# ------------------------------------------------------------------- oracle ---

def test_the_plain_form_quantizes_as_torch_casts():
    """The tests' own 64-bit form of the format, against torch's E4M3 cast and the definition's rounding properties."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 3, 128)) * 3
    codes, scales = O.quantize(x, 0.01)
    t = np.abs(x.astype(np.float32).reshape(40, 3, 8, 16)).max(-1) / (np.float32(6.0) * np.float32(0.01))
    want = torch.from_numpy(t).clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(scales, want)
    v = O.values(codes, scales, 0.01)
    step = O.E4M3[scales].repeat(16, -1) * np.float64(np.float32(0.01))
    # E2M1 steps are 1/2 up to 2, 1 up to 4, 2 up to 6 of the scale; past 6 it saturates (a scale rounded down by 2^-4)
    assert np.all(np.abs(v - x) <= step * (1.0 + 1e-6))
    small = np.abs(x) <= 2 * step
    assert np.all(np.abs(v - x)[small] <= 0.25 * step[small] * (1 + 1e-6))


def test_the_plain_form_rotates():
    x = np.arange(24.0).reshape(2, 2, 6)
    y = O.rotate(x, [1, 2], [math.pi / 2, math.pi])
    assert np.allclose(y[0, 0], [-2.0, -1.0, 0.0, -3.0, 4.0, 5.0])
    assert np.allclose(y[1, 0], [-12.0, 13.0, -14.0, 15.0, 16.0, 17.0])
    z = O.rotate(x, [1, 2], [math.pi / 2, math.pi], interleaved=True)
    assert np.allclose(z[0, 0], [-1.0, 0.0, -2.0, -3.0, 4.0, 5.0])
    assert np.allclose(O.rotate(O.rotate(x, [7, 9], [0.3, 0.1]), [7, 9], [0.3, 0.1], inverse=True), x)


def test_the_plain_form_attends():
    """Against torch's softmax in 64 bits on a dense problem."""
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((2, 9, 8)), rng.standard_normal((2, 9, 8))
    o, lse, _, _ = O.attention(q, k, v, 0.3, causal=True, window=4)
    tq, tk, tv = (torch.from_numpy(a) for a in (q, k, v))
    s = torch.einsum("nhd,hkd->nhk", tq, tk.repeat_interleave(2, 0)) * 0.3
    pos, j = torch.arange(4, 9)[:, None, None], torch.arange(9)[None, None]
    s = s.masked_fill((j > pos) | (j <= pos - 4), -math.inf)
    assert np.allclose(o, torch.einsum("nhk,hkd->nhd", s.softmax(-1), tv.repeat_interleave(2, 0)).numpy())
    assert np.allclose(lse, torch.logsumexp(s, -1).numpy())
    o, lse, _, _ = O.attention(q, k[:, :3], v[:, :3], 0.3)
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(np.isfinite(lse[2:]))


# ----------------------------------------------------------- the C++ calls ---

def test_cpp_binding_leaves_unexpected_operands_to_python(L):
    """Whatever is not a CUDA tensor of the expected kind: None, and nothing is called."""
    b = fq._binding
    x, i, f = torch.zeros(4, 2, 64, dtype=BF), torch.zeros(4, dtype=I64), torch.zeros(32, dtype=F64)
    c = cache(head_dim=64, kv_heads=2)
    at = ctypes.addressof(c)
    assert b.rope(x, i, f, 0, 1.0, x) is None                     # on the CPU
    assert b.rope(x, i, f, 0, 1.0) is None                        # too few
    assert b.rope(None, i, f, 0, 1.0, x) is None
    assert b.rope(S((4, 2, 64), BF), i, f, 0, 1.0, x) is None     # not a tensor
    assert b.append(at, 0, x, x, i, None, None, 0, 1.0) is None
    assert b.append("no address", 0, x, x, i, None, None, 0, 1.0) is None
    assert b.append(at, 1 << 70, x, x, i, None, None, 0, 1.0) is None
    assert b.read(at, 0, i, x, x) is None
    assert b.attention(at, 0, x, i, i, None, 1, 1.0, True, 0, x, None, x) is None
    sparse = torch.sparse_coo_tensor(torch.zeros(3, 1, dtype=I64), torch.ones(1, dtype=BF), (4, 2, 64))
    assert b.rope(sparse, i, f, 0, 1.0, x) is None


def test_package_fails_loudly_without_the_cpp_binding(monkeypatch, L):
    monkeypatch.setattr(fq, "BINDING_PATH", "/nonexistent/_kv4_binding.so")
    with pytest.raises(ImportError):
        fq._Binding().rope


# -------------------------------------------------------- empty page tables ---

@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(mp=0, ts=0, table=None), VALID), (dict(mp=0, ts=0), VALID), (dict(mp=0, ts=0, table=None, qs=None, mq=1), VALID),
    (dict(mp=0, ts=0, table=None, kv=None), INV), (dict(mp=1, ts=1, table=None), INV), (dict(mp=0, ts=-1, table=None), INV),
])
def test_attention_over_sequences_without_pages(L, kw, want):
    """A [B, 0] page table, as torch makes it for sequences that are all empty: no memory, and none is read."""
    assert torch.zeros((3, 0), dtype=I32).data_ptr() == 0
    assert attend(L, **kw) == want


# --------------------------------------------------- strides of any product ---

FAR = 1 << 40           # a stride; with 2^23 + 1 tokens the last one's offset is 2^63


@no_gpu
@pytest.mark.parametrize("T,t,h,want", [
    ((1 << 23) + 1, FAR, FAR, INV),                 # token 1 of head 0 is token 0 of head 1, past what 63 bits can tell
    ((1 << 8) + 1, FAR, 128, VALID), ((1 << 8) + 2, FAR, 128, INV),     # up to an offset of 2^48 elements
    (2, 1 << 48, 128, VALID), (2, (1 << 48) + 8, 128, INV), (2, (1 << 62), 128, INV),
    (1, (1 << 62), 128, VALID),                     # one token has no token stride
])
def test_offsets_stay_inside_63_bits(L, T, t, h, want):
    c = cache(kv_heads=2)
    assert rope(L, T=T, H=2, xt=0, xh=0, yt=t, yh=h) == want
    assert rope(L, T=T, H=2, xt=t, xh=h, yt=256, yh=128) == want
    assert append(L, c, T=T, kt=t, kh=h, vt=256) == want and append(L, c, T=T, vt=t, vh=h, kt=256) == want
    assert read(L, c, T=T, kt=t, kh=h, vt=256) == want and read(L, c, T=T, vt=t, vh=h, kt=256) == want
    assert attend(L, c, T=T, Hq=2, ot=t, oh=h, qt=0) == want and attend(L, c, T=T, Hq=2, qt=t, qh=h, ot=256) == want


# ------------------------------------------------------------ whole numbers ---

def test_binding_whole_numbers(lib, monkeypatch):
    """Numbers past 64 bits are refused, not cut to what is left of them (a window of 2^64 + 5 to one of 5); numpy's whole
    numbers are taken, others are not."""
    seen = []
    monkeypatch.setattr(fq, "_call", lambda dev, name, *args: seen.append(args))
    base = dict(q=S((7, 8, 128), BF), cache=a_cache(), page_table=S((3, 9), I32), kv_len=S((3,), I32),
                q_start=S((4,), I32), max_q_len=4, out=S((7, 8, 128), BF), workspace=S((64,), U8))
    call = lambda **kw: fq.fp8q_kv4_attention(**{**base, **kw})  # noqa: E731
    for bad in (2 ** 63, 2 ** 64 + 5, -2 ** 63 - 1):
        for name in ("window", "max_q_len"):
            with pytest.raises(ValueError, match=name):
                call(**{name: bad})
        with pytest.raises(ValueError):
            fq.fp8q_kv4_page_bytes(bad, 8, 128)
    with pytest.raises(TypeError):
        call(window=5.0)
    assert not seen
    call(window=np.int64(2 ** 63 - 1), max_q_len=np.int32(4), sm_scale=np.float32(0.125))
    assert 2 ** 63 - 1 in seen[0]
    assert all(not isinstance(a, np.generic) for a in seen[0])
