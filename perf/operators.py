"""What is measured of the 4-bit KV cache's operators: rotary positions, appending rotated keys and values to a paged
E2M1 cache, and attention over it.  `run` computes each in its plain form (elementary torch operations) where `own` is
false, and calls the library's kernels where it is true.

Cache format: for each (page, head) one slab of page_size rows of D/2 code bytes (E2M1, the even element in the low
nibble), then page_size rows of D/16 E4M3 scale bytes (one per 16 elements); a value is code * scale * g with one
static fp32 g per cache (k_scale, v_scale).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
THETA = 500000.0                       # Llama 3


# ------------------------------------------------------------------ cases ---

def _rope(name, tokens, heads, dim, rot, interleaved=False, inverse=False, far=8192, fused=0):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "inverse": inverse, "far": far, "fused": fused}


def _append(name, tokens, heads, dim, page, rot, interleaved=False, far=8192, skip=0.0, fused=0):
    return {"name": name, "op": "append", "tokens": tokens, "heads": heads, "dim": dim, "page": page, "rot": rot,
            "interleaved": interleaved, "far": far, "skip": skip, "fused": fused}


def _attn(name, seqs, q_max, kv_max, q_heads, kv_heads, dim, page, kv_min=1.0, causal=True, window=0, pad=0):
    return {"name": name, "op": "attention", "seqs": seqs, "q_max": q_max, "kv_max": kv_max, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "kv_min": kv_min, "causal": causal, "window": window,
            "pad": pad}


def listed():
    return [
        # queries and keys of a decode step of Llama-3.1-70B (64 + 8 heads), inside the fused qkv rows
        _rope("rope_decode_70b", 8, 72, 128, 128, far=131072, fused=80),
        # a prompt of Llama-3.1-8B (32 + 8 heads)
        _rope("rope_prompt_8b", 8192, 40, 128, 128, fused=48),
        # interleaved pairs in half of a 64-wide head, rotated back, an odd number of tokens
        _rope("rope_part_inverse", 777, 13, 64, 32, interleaved=True, inverse=True, far=1 << 20),
        # the new tokens of a batch of 64, two of them padding
        _append("append_decode_8b", 64, 8, 128, 16, 128, skip=0.03, far=131072, fused=48),
        # a prompt's keys and values
        _append("append_prompt_8b", 8192, 8, 128, 64, 128, fused=48),
        # part of a 64-wide head, interleaved, a ragged number of tokens
        _append("append_part", 1235, 5, 64, 32, 32, interleaved=True, skip=0.1),
        # one user's next token early in a conversation: latency
        _attn("attn_one_short_8b", 1, 1, 500, 32, 8, 128, 16),
        # a full batch of ragged conversations
        _attn("attn_batch_8b", 64, 1, 8192, 32, 8, 128, 64, kv_min=0.05),
        # one token after a 128K context (Llama-3.2-3B, three query heads to a key head)
        _attn("attn_long_3b", 1, 1, 131072, 24, 8, 128, 128),
        # a few drafted tokens a sequence, eight query heads to a key head, a sliding window, padding rows
        _attn("attn_draft_70b", 16, 4, 6000, 64, 8, 128, 32, kv_min=0.3, window=4096, pad=3),
        # the second part of a prompt after a cached first one
        _attn("attn_chunk_8b", 1, 2048, 8192, 32, 8, 128, 64),
        # short prompts of odd lengths together, 64-wide heads
        _attn("attn_ragged_64", 5, 611, 1900, 20, 4, 64, 16, kv_min=0.2, pad=7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention"])
    dim = rng.choice([64, 128, 128])
    if op == "rope":
        heads = rng.randint(1, 72)
        rot = dim if rng.random() < 0.6 else rng.choice([8, 16, 24, 32, 40, 48, dim // 2])
        tokens = _log_int(rng, 1, 8192 * 40 // heads if heads > 40 else 8192)
        c = _rope("", tokens, heads, dim, rot, rng.random() < 0.4, rng.random() < 0.3,
                  rng.choice([8192, 131072, 1 << 20]), rng.choice([0, heads + rng.randint(1, 8)]))
    elif op == "append":
        heads = rng.randint(1, 8)
        rot = dim if rng.random() < 0.6 else rng.choice([0, 8, 16, 24, 32, dim // 2])
        c = _append("", _log_int(rng, 1, 8192), heads, dim, rng.choice([16, 32, 64, 128, 256]), rot,
                    rng.random() < 0.4, rng.choice([8192, 131072, 1 << 20]), rng.choice([0.0, 0.1]),
                    rng.choice([0, 2 * heads + rng.randint(0, 9)]))
    else:
        kv_heads, group = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8])
        kind = rng.choice(["decode", "decode", "draft", "chunk"])
        page = rng.choice([16, 32, 64, 128, 256])
        if kind == "decode":
            kv = _log_int(rng, 1, 131072)
            seqs = _log_int(rng, 1, max(1, min(64, 64 * 8192 // kv)))
            q = 1
        elif kind == "draft":
            kv = _log_int(rng, 16, 16384)
            seqs = _log_int(rng, 1, max(1, min(32, 16 * 8192 // kv)))
            q = rng.randint(2, 16)
        else:
            kv = _log_int(rng, 64, 8192)
            q = _log_int(rng, 17, min(kv, 2048))
            seqs = rng.randint(1, max(1, min(6, 2048 * 8192 * 32 // (q * kv * kv_heads * group))))
        c = _attn("", seqs, q, kv, kv_heads * group, kv_heads, dim, page, rng.choice([0.05, 0.5, 1.0]),
                  rng.random() < 0.85, rng.choice([0, 0, 0, 1 + kv // 3]), rng.choice([0, 0, 5]))
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs ---

def _frequencies(rot, factor=8.0, low=1.0, high=4.0, original=8192.0):
    """Llama 3's rotary frequencies (radians per position): wave lengths past original / low are stretched by factor,
    those below original / high are kept, those between go over linearly."""
    out = []
    for i in range(rot // 2):
        f = THETA ** (-2.0 * i / rot)
        turns = original * f / (2.0 * math.pi)
        t = min(1.0, max(0.0, (turns - low) / (high - low)))
        out.append((1.0 - t) * f / factor + t * f)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _rows(gen, tokens, heads, dim, fused, at):
    """[tokens, heads, dim] bf16, with a few larger channels as keys have; where `fused`, a part of wider rows."""
    wide = max(fused, heads + at)
    x = torch.randn((tokens, wide, dim), generator=gen, device=DEV)
    x *= 1.0 + 7.0 * (torch.rand((1, wide, dim), generator=gen, device=DEV) < 0.04)
    return x.to(torch.bfloat16)[:, at:at + heads]


def _encode(x, g):
    """fp32 [..., D] -> (codes uint8 [..., D/2], scales uint8 [..., D/16])."""
    shape = x.shape
    b = x.reshape(*shape[:-1], shape[-1] // 16, 16)
    g6 = float(np.float32(6.0) * np.float32(g))
    t = (b.abs().amax(-1) / torch.full((), g6, device=x.device)).clamp(max=448.0)
    sc = t.to(torch.float8_e4m3fn)
    s = (sc.float() * float(np.float32(g))).unsqueeze(-1)
    q = torch.where(s > 0, b / torch.where(s > 0, s, 1.0), 0.0)
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code | (torch.signbit(q).to(torch.uint8) << 3)).reshape(*shape[:-1], shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), sc.view(torch.uint8)


def _pairs():
    """[256, 2]: the two E2M1 values that a code byte holds."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    return torch.stack([v.repeat(16), v.repeat_interleave(16)], -1)


def _decode(codes, scales, g, lut):
    """The fp32 values that codes [..., D/2] and scales [..., D/16] stand for."""
    v = lut.index_select(0, codes.reshape(-1).int()).reshape(*scales.shape, 16)
    v = v * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return (v * float(np.float32(g))).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _parts(pages, page, dim):
    """Views of a cache tensor [pages, heads, bytes]: codes [pages, heads, page, D/2], scales [pages, heads, page, D/16]."""
    n, h, _ = pages.shape
    cut = page * dim // 2
    return pages[:, :, :cut].unflatten(2, (page, dim // 2)), pages[:, :, cut:].unflatten(2, (page, dim // 16))


def _lengths(case):
    """Per sequence (new tokens, tokens in the cache with them): spread over the case's ranges, the first the longest."""
    q, kv = [], []
    for b in range(case["seqs"]):
        u, w = 1.0 - (b * 0.6180339887) % 1.0, 1.0 - (b * 0.7548776662) % 1.0
        q.append(case["q_max"] if case["q_max"] == 1 else max(1, int(case["q_max"] * (0.4 + 0.6 * u))))
        kv.append(max(q[-1], int(case["kv_max"] * (case["kv_min"] + (1.0 - case["kv_min"]) * w))))
    return q, kv


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    D = case["dim"]
    s = dict(case)
    s["pairs"] = _pairs()
    if case["op"] in ("rope", "append"):
        T, H, rot = case["tokens"], case["heads"], case["rot"]
        s["freq"] = _frequencies(rot) if rot else None
        start = int(torch.randint(0, max(1, case["far"] - T), (1,), generator=host))
        s["positions"] = torch.arange(start, start + T, device=DEV)
        if case["op"] == "rope":
            s["x"] = _rows(gen, T, H, D, case["fused"], 0)
            if own:
                s["out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
            return s
        wide = case["fused"]
        both = _rows(gen, T, 2 * H, D, wide, max(0, wide - 2 * H))
        s["k"], s["v"] = both[:, :H], both[:, H:]
        page = case["page"]
        pages = (T + page - 1) // page + 3
        at = torch.randperm(pages, generator=gen, device=DEV)
        i = torch.arange(T, device=DEV)
        slots = at[i // page] * page + i % page
        s["slots"] = torch.where(torch.rand(T, generator=gen, device=DEV) < case["skip"], -1, slots)
        s["unused"] = at[-1] * page                                     # a slot of no token
        s["k_pages"] = torch.zeros((pages, H, page * D * 9 // 16), dtype=torch.uint8, device=DEV)
        s["v_pages"] = torch.zeros_like(s["k_pages"])
        s["k_scale"], s["v_scale"] = 2.0 ** -6, 0.011
        if own:
            s["k_out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
            s["v_out"] = torch.empty_like(s["k_out"])
    else:
        B, H, page = case["seqs"], case["kv_heads"], case["page"]
        q, kv = _lengths(case)
        most = (max(kv) + page - 1) // page
        pages = sum((n + page - 1) // page for n in kv) + 2
        at = torch.randperm(pages, generator=gen, device=DEV).int()
        table = torch.zeros((B, most), dtype=torch.int32, device=DEV)
        used = 0
        for b, n in enumerate(kv):
            n = (n + page - 1) // page
            table[b, :n] = at[used:used + n]
            used += n
        s["page_table"] = table
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
        s["q_start"] = torch.tensor(np.concatenate([[0], np.cumsum(q)]), dtype=torch.int32, device=DEV)
        T = sum(q) + case["pad"]
        # where each new token stands in a [sequences, longest] rectangle
        s["place"] = torch.tensor([b * max(q) + i for b, n in enumerate(q) for i in range(n)], device=DEV)
        s["q"] = torch.randn((T, case["q_heads"], D), generator=gen, device=DEV).to(torch.bfloat16)
        s["k_scale"], s["v_scale"] = 0.0041, 2.0 ** -8
        for name in ("k", "v"):
            p = torch.empty((pages, H, page * D * 9 // 16), dtype=torch.uint8, device=DEV)
            codes, scales = _parts(p, page, D)
            chunk = max(1, (1 << 26) // (H * page * D))
            for i in range(0, pages, chunk):
                x = torch.randn((min(chunk, pages - i), H, page, D), generator=gen, device=DEV)
                if name == "k":
                    x *= 1.0 + 3.0 * (torch.arange(D, device=DEV) % 29 == 7)
                codes[i:i + chunk], scales[i:i + chunk] = _encode(x, s[name + "_scale"])
            s[name + "_pages"] = p
        # rows behind the last sequence are left as they were
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((T, case["q_heads"]), dtype=torch.float32, device=DEV)
        s["sm_scale"] = D ** -0.5
    if own:
        import fp8_w8a8_quantized_amax_b200 as fq
        s["cache"] = fq.KV4Cache(s["k_pages"], s["v_pages"], page_size=case["page"], head_dim=D,
                                 k_scale=s["k_scale"], v_scale=s["v_scale"])
        if case["op"] == "attention":
            need = fq.fp8q_kv4_attention_workspace_size(s["cache"], case["seqs"], T, case["q_heads"], case["q_max"])
            s["workspace"] = torch.zeros(max(16, need), dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------- plain forms ---

def _rotate(x, positions, freq, interleaved, inverse):
    """float64 [T, H, D] of x rotated by positions * freq."""
    x = x.double()
    R = 2 * freq.numel()
    a = (positions.double().unsqueeze(-1) * freq).unsqueeze(1)
    c, s = torch.cos(a), torch.sin(a)
    s = -s if inverse else s
    r, rest = x[..., :R], x[..., R:]
    x0, x1 = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :R // 2], r[..., R // 2:])
    y0, y1 = x0 * c - x1 * s, x1 * c + x0 * s
    y = torch.stack([y0, y1], -1).flatten(-2) if interleaved else torch.cat([y0, y1], -1)
    return torch.cat([y, rest], -1)


def _plain_append(s):
    page, D = s["page"], s["dim"]
    k = _rotate(s["k"], s["positions"], s["freq"], s["interleaved"], False) if s["rot"] else s["k"]
    keep = s["slots"] >= 0
    at = torch.where(keep, s["slots"], s["unused"])
    p, o = at // page, at % page
    back = []
    for x, pages, g in ((k.float(), s["k_pages"], s["k_scale"]), (s["v"].float(), s["v_pages"], s["v_scale"])):
        codes, scales = _parts(pages, page, D)
        codes[p, :, o], scales[p, :, o] = _encode(x, g)
        y = _decode(codes[p, :, o], scales[p, :, o], g, s["pairs"])
        back.append(torch.where(keep[:, None, None], y, 0.0).to(torch.bfloat16))
    return back


def _plain_attention(s):
    page, D, H, G = s["page"], s["dim"], s["kv_heads"], s["q_heads"] // s["kv_heads"]
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    B, qm = kv_len.numel(), s["q_max"]

    def gathered(pages, g):
        codes, scales = _parts(pages, page, D)
        at = s["page_table"].long()
        v = _decode(codes[at], scales[at], g, s["pairs"])                            # [B, pages, H, page, D]
        return v.transpose(1, 2).reshape(B, H, -1, D)

    k, v = gathered(s["k_pages"], s["k_scale"]), gathered(s["v_pages"], s["v_scale"])
    n = (q_start[1:] - q_start[:-1])[:, None]
    i = torch.arange(qm, device=DEV)[None]
    place = s["place"]
    tokens = place.numel()
    q = torch.zeros((B * qm, H * G, D), device=DEV)
    q[place] = s["q"][:tokens].float()
    q = q.reshape(B, qm, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * qm, D)
    w = torch.matmul(q, k.transpose(2, 3)) * s["sm_scale"]               # [B, H, G qm, kv]
    pos = (kv_len[:, None] - n + i)[:, None, :, None]
    j = torch.arange(k.shape[2], device=DEV)
    seen = (j < kv_len[:, None, None, None]).expand(B, 1, qm, -1)
    if s["causal"]:
        seen = seen & (j <= pos)
    if s["window"]:
        seen = seen & (j > pos - s["window"])
    w = w.reshape(B, H, G, qm, -1).masked_fill_(~seen.unsqueeze(2), -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-3e38)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.reshape(B, H, G * qm, -1), v).reshape(B, H, G, qm, D)
    o = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0)
    lse = (top + torch.log(total)).squeeze(-1)
    out, out_lse = torch.zeros_like(s["q"]), torch.zeros_like(s["lse"])
    out[:tokens] = o.permute(0, 3, 1, 2, 4).reshape(B * qm, H * G, D)[place].to(torch.bfloat16)
    out_lse[:tokens] = lse.permute(0, 3, 1, 2).reshape(B * qm, H * G)[place]
    return [out, out_lse]


def run(s):
    if own:
        import fp8_w8a8_quantized_amax_b200 as fq
        if s["op"] == "rope":
            return fq.fp8q_rope(s["x"], s["positions"], s["freq"], interleaved=s["interleaved"], inverse=s["inverse"],
                                out=s["out"])
        if s["op"] == "append":
            fq.fp8q_kv4_append(s["cache"], s["k"], s["v"], s["slots"], s["positions"] if s["rot"] else None,
                               s["freq"], interleaved=s["interleaved"])
            return list(fq.fp8q_kv4_read(s["cache"], s["slots"], out=(s["k_out"], s["v_out"])))
        fq.fp8q_kv4_attention(s["q"], s["cache"], s["page_table"], s["kv_len"], s["q_start"], s["q_max"],
                              sm_scale=s["sm_scale"], causal=s["causal"], window=s["window"], out=s["out"],
                              lse=s["lse"], workspace=s["workspace"])
        return [s["out"], s["lse"]]
    if s["op"] == "rope":
        return _rotate(s["x"], s["positions"], s["freq"], s["interleaved"], s["inverse"]).to(torch.bfloat16)
    return _plain_append(s) if s["op"] == "append" else _plain_attention(s)


# ------------------------------------------------------------------- work ---

def work(case):
    D = case["dim"]
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * D + 8 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    if case["op"] == "append":
        # read K and V, write their codes and scales; then read those and write the values they stand for
        n = 2 * case["tokens"] * case["heads"]
        return {"bytes": n * (2 * D + 2 * (D * 9 // 16) + 2 * D) + 24 * case["tokens"], "flops": 10 * n * D}
    pairs = read = rows = 0
    for q, kv in zip(*_lengths(case)):
        i = np.arange(kv - q, kv)                                       # positions of the new tokens
        last = i + 1 if case["causal"] else np.full(q, kv)
        first = np.maximum(0, i - case["window"] + 1) if case["window"] else np.zeros(q, int)
        pairs += int((last - first).sum())
        read += int(last.max() - first.min())
        rows += q
    bytes_ = read * case["kv_heads"] * 2 * (D * 9 // 16) + rows * case["q_heads"] * (4 * D + 4)
    return {"bytes": bytes_, "flops": 4 * D * pairs * case["q_heads"]}


# ------------------------------------------------------------------ exact ---

def _exact_rotate(x, positions, freq, interleaved, inverse):
    y = x.copy()
    half = freq.size
    turn = np.outer(positions.astype(np.float64), freq) * (-1.0 if inverse else 1.0)
    z = np.exp(1j * turn)[:, None, :]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    w = (x[..., a] + 1j * x[..., b]) * z
    y[..., a], y[..., b] = w.real, w.imag
    return y


def _nearest(values, x):
    """The index into ascending non-negative `values` nearest to each x >= 0; at a tie the even index."""
    mid = (values[1:] + values[:-1]) / 2
    low, high = np.searchsorted(mid, x, "left"), np.searchsorted(mid, x, "right")
    return np.where(low == high, low, np.where(low % 2 == 0, low, high))


def _exact_stored(x, g):
    """The float64 values that the cache holds for x [..., D] (fp32 steps where the definition rounds to fp32)."""
    e4m3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127])
    e2m1 = np.array(E2M1)
    g = np.float32(g)
    b = x.astype(np.float32).reshape(*x.shape[:-1], -1, 16)
    t = np.abs(b).max(-1) / (np.float32(6.0) * g)
    sc = e4m3[_nearest(e4m3, t.astype(np.float64))]
    s = (sc.astype(np.float32) * g)[..., None]
    q = np.divide(b, s, out=np.zeros_like(b), where=s > 0)
    v = np.copysign(e2m1[_nearest(e2m1, np.abs(q).astype(np.float64))], q)
    return (v * sc[..., None] * np.float64(g)).reshape(x.shape)


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    if case["op"] == "attention":
        return _exact_attention(s)
    to = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    positions = s["positions"].cpu().numpy()
    freq = s["freq"].cpu().numpy() if case["rot"] else None
    if case["op"] == "rope":
        return _exact_rotate(to(s["x"]), positions, freq, case["interleaved"], case["inverse"])
    k = _exact_rotate(to(s["k"]), positions, freq, case["interleaved"], False) if case["rot"] else to(s["k"])
    keep = (s["slots"].cpu().numpy() >= 0)[:, None, None]
    return [np.where(keep, _exact_stored(k, s["k_scale"]), 0.0),
            np.where(keep, _exact_stored(to(s["v"]), s["v_scale"]), 0.0)]


def _exact_attention(s):
    """One sequence and key head after the other, in float64."""
    page, D, H = s["page"], s["dim"], s["kv_heads"]
    G = s["q_heads"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=DEV)
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    cut = page * D // 2

    def values(pages, g, ids, h, n):
        slab = pages[ids, h]
        byte = slab[:, :cut].reshape(-1, D // 2).long()
        sc = slab[:, cut:].contiguous().view(torch.float8_e4m3fn).double().reshape(-1, D // 16)
        v = torch.stack([table[byte & 15], table[byte >> 4]], -1).reshape(-1, D // 16, 16) * sc[..., None]
        return v.reshape(-1, D)[:n] * float(np.float32(g))

    for b, n in enumerate(lens):
        r0, r1 = starts[b], starts[b + 1]
        if r1 == r0:
            continue
        ids = s["page_table"][b, :(n + page - 1) // page].long()
        pos = torch.arange(n - (r1 - r0), n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        hide = torch.zeros((r1 - r0, n), dtype=torch.bool, device=DEV)
        if s["causal"]:
            hide |= j > pos
        if s["window"]:
            hide |= j <= pos - s["window"]
        for h in range(H):
            k, v = values(s["k_pages"], s["k_scale"], ids, h, n), values(s["v_pages"], s["v_scale"], ids, h, n)
            for a in range(h * G, (h + 1) * G):
                w = (s["q"][r0:r1, a].double() @ k.T * s["sm_scale"]).masked_fill_(hide, -math.inf)
                l = torch.logsumexp(w, -1)
                lse[r0:r1, a] = l
                out[r0:r1, a] = torch.exp(w - l.clamp(min=-1e300)[:, None]) @ v
    return [out.cpu().numpy(), lse.cpu().numpy()]
