"""Cases of the operators around a paged KV cache: position rotation on the way into the
cache, a cache in 8 bits with a scale for each block and head, attention over it, and
attention with capped scores, a distance bias or a sliding window.

Four operators, each in its plain form (elementary torch operations in 32 bits) and, with
``own`` set, through the library's entry points:

* ``rope``      q and k rotated by position, k and v written to a bf16 pool
* ``rope_fp8``  the same into an E4M3 pool whose 16-token blocks hold one power-of-two
                scale for each kv head
* ``attend``    decode attention over such an E4M3 pool
* ``scored``    decode attention with a score cap, a distance bias or a window, over a bf16
                or a block-scaled E4M3 pool

A pool is ``[blocks, 16, kv heads, head dim]``; scales are one byte for each block and kv
head, standing for ``2 ** (byte - 127)`` (0: an empty block). Rotation frequencies are
64-bit fixed point, in units of 2^-64 turn for each position.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases
def _append(name, kind, seqs, new, first, last, hq, hkv, d, rot, pair, pad):
    """``seqs`` sequences get ``new`` tokens each, at positions spread over first..last;
    ``pad`` rows of the batch carry no token (slot -1)."""
    c = dict(kind=kind, seqs=seqs, new=new, first=first, last=last, hq=hq, hkv=hkv, d=d,
             rot=rot, interleaved=pair, pad=pad)
    return dict(c, name=name) if name else c


def _attend(name, kind, pool, seqs, nq, t_min, t_max, hq, hkv, d, cap=0.0, bias=False,
            window=0):
    c = dict(kind=kind, pool=pool, seqs=seqs, nq=nq, t_min=t_min, t_max=t_max, hq=hq, hkv=hkv,
             d=d, cap=cap, bias=bias, window=window)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request being decoded: the smallest call, where the launch counts
        _append("rope_one_token", "rope", 1, 1, 777, 777, 32, 8, 128, 128, False, 0),
        # a full serving batch with padding rows, far positions, adjacent-pair layout,
        # half of each head rotated
        _append("rope_batch_256", "rope", 247, 1, 100, 131000, 64, 8, 128, 64, True, 9),
        # a prompt chunk of several requests, ragged ends
        _append("rope_prompt_8190", "rope", 3, 2730, 0, 70000, 32, 8, 128, 128, False, 0),
        # one decode step of a batch of 64 into an 8-bit cache: most blocks partly filled
        _append("rope_fp8_decode_64", "rope_fp8", 64, 1, 500, 4100, 32, 8, 128, 128, False, 0),
        # a prompt chunk into an 8-bit cache: whole blocks, ragged ends
        _append("rope_fp8_prompt_8190", "rope_fp8", 3, 2730, 5, 9000, 64, 8, 128, 128, False, 0),
        # one short request over an 8-bit cache: latency
        _attend("fp8_one_request", "attend", "fp8", 1, 1, 333, 333, 32, 8, 128),
        # a layer's decode step over 64 requests of 512 to 4096 tokens
        _attend("fp8_decode_64", "attend", "fp8", 64, 1, 512, 4096, 32, 8, 128),
        # eight long contexts
        _attend("fp8_long_8", "attend", "fp8", 8, 1, 32768, 131072, 32, 8, 128),
        # verification of four draft tokens, 32 query rows for each kv head
        _attend("fp8_verify_128x4", "attend", "fp8", 128, 4, 256, 4096, 64, 8, 128),
        # capped scores over a bf16 cache
        _attend("cap_decode_64", "scored", "bf16", 64, 1, 512, 4096, 32, 8, 128, cap=50.0),
        # a sliding-window layer with capped scores at long contexts, draft tokens
        _attend("window_long_32x2", "scored", "bf16", 32, 2, 2048, 32768, 16, 8, 128, cap=30.0,
                window=1024),
        # distance bias over the 8-bit cache, a large batch with 8 query heads per kv head
        _attend("bias_fp8_256", "scored", "fp8", 256, 1, 300, 2500, 64, 8, 128, bias=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope_fp8", "attend", "scored"])
    if kind in ("rope", "rope_fp8"):
        d = 128 if kind == "rope_fp8" else rng.choice([64, 80, 96, 128])
        hkv = rng.choice([1, 2, 4, 5, 8])
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        rot = rng.choice([d, d, d // 2, d // 4])
        if rng.random() < 0.5:  # decode: one to four tokens of each sequence
            seqs, new = _spread(rng, 1, 300), rng.randint(1, 4)
        else:                   # prompt chunks
            seqs = rng.randint(1, 6)
            new = _spread(rng, 5, 8000 // seqs)
        first = rng.randint(0, 3000)
        last = first + _spread(rng, 1, 100000)
        return _append("", kind, seqs, new, first, last, hq, hkv, d, rot, rng.random() < 0.5,
                       rng.choice([0, 0, 3, 11]))
    pool = "fp8" if kind == "attend" else rng.choice(["bf16", "fp8"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    nq = rng.choice([1, 1, 2, 4])
    group = rng.choice([1, 2, 4, 5, 8])
    d = 128 if pool == "fp8" else rng.choice([64, 128])
    seqs = _spread(rng, 1, 256)
    t_max = _spread(rng, 20, min(131072, (600000 if pool == "fp8" else 300000) // seqs))
    t_min = max(1, int(t_max * rng.uniform(0.05, 1.0)))
    cap, bias, window = 0.0, False, 0
    if kind == "scored":
        cap, bias, window = rng.choice([(30.0, False, 0), (50.0, False, 1), (0.0, True, 0),
                                        (0.0, False, 1), (20.0, True, 1)])
        window = window and _spread(rng, 16, 4096)
    return _attend("", kind, pool, seqs, nq, t_min, t_max, hkv * group, hkv, d, cap, bias, window)


# ---------------------------------------------------------------- sizes that follow from a case
def _steps(n, lo, hi):
    """n whole numbers spread over lo..hi (over their logarithm), in no order."""
    u = (np.arange(1, n + 1) * 0.6180339887498949) % 1.0
    a, b = math.log(lo + 1.0), math.log(hi + 1.0)
    return np.clip(np.rint(np.exp(a + (b - a) * u) - 1.0), lo, hi).astype(np.int64)


def _lengths(case):
    t = _steps(case["seqs"], case["t_min"], case["t_max"])
    t[0] = case["t_max"]
    return t


def _seen(case):
    """(tokens that any query of a sequence sees, query-token pairs of a head)."""
    t, nq, w = _lengths(case), case["nq"], case["window"]
    hi = t[:, None] - nq + np.arange(nq)[None, :]          # last position of each query
    lo = np.maximum(hi - w + 1, 0) if w else np.zeros_like(hi)
    pairs = np.maximum(hi - lo + 1, 0)
    first = np.where(pairs > 0, lo, t[:, None]).min(axis=1)
    return int((t - first).sum()), int(pairs.sum())


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["kind"] in ("rope", "rope_fp8"):
        tokens = case["seqs"] * case["new"]
        rows = tokens + case["pad"]
        size = 1 if case["kind"] == "rope_fp8" else 2
        # q in and out, k and v in, k and v to the pool, slots and positions
        b = rows * (hq * d * 4 + 16) + tokens * 2 * hkv * d * (2 + size)
        return {"bytes": b, "flops": 3 * case["rot"] * (rows * hq + tokens * hkv)}
    tokens, pairs = _seen(case)
    rows = case["seqs"] * case["nq"]
    size = 1 if case["pool"] == "fp8" else 2
    b = 2 * tokens * hkv * d * size + 4 * rows * hq * d + 4 * tokens // BLOCK
    if case["pool"] == "fp8":
        b += 2 * hkv * tokens // BLOCK
    return {"bytes": b, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------- inputs
def _fp8_pool(blocks, hkv, d, gen):
    """Codes of normal values and block scales a few powers of two apart."""
    x = torch.randn((blocks, BLOCK, hkv, d), generator=gen, device="cuda").mul_(64)
    codes = x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.randint(119, 123, (blocks, hkv), generator=gen, device="cuda")
    return codes, scale.to(torch.uint8)


def _bf16(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _positions(case):
    """(position of each row, or -1 for padding; sequence of each row)."""
    start = _steps(case["seqs"], case["first"], case["last"])
    pos = (start[:, None] + np.arange(case["new"])[None, :]).reshape(-1)
    seq = np.repeat(np.arange(case["seqs"]), case["new"])
    none = np.full(case["pad"], -1, np.int64)
    return np.concatenate([pos, none]), np.concatenate([seq, none])


def _prepare_append(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    pos, seq = _positions(case)
    n = pos.size
    # only the blocks that the new tokens fall into are in this pool, in no order
    key = seq * (1 << 32) + pos // BLOCK
    used, block = np.unique(key[seq >= 0], return_inverse=True)
    blocks = used.size + 64
    place = rng.permutation(blocks)[block]
    slots = np.full(n, -1, np.int64)
    slots[seq >= 0] = place * BLOCK + pos[seq >= 0] % BLOCK
    freq = 10000.0 ** (-np.arange(0, case["rot"], 2) / case["rot"]) / (2 * math.pi)
    s = dict(case=case, q=_bf16((n, hq, d), gen), k=_bf16((n, hkv, d), gen),
             v=_bf16((n, hkv, d), gen),
             pos=torch.from_numpy(np.maximum(pos, 0)).cuda(), slots=torch.from_numpy(slots).cuda(),
             turns=torch.tensor([int(f * 2.0 ** 64) for f in freq], dtype=torch.int64).cuda())
    s["q_out"] = torch.empty_like(s["q"])
    # one more block than the pool has takes the plain form's padding rows
    if case["kind"] == "rope_fp8":
        s["k_all"], s["k_scale_all"] = _fp8_pool(blocks + 1, hkv, d, gen)
        s["v_all"], s["v_scale_all"] = _fp8_pool(blocks + 1, hkv, d, gen)
        s["k_scale"], s["v_scale"] = s["k_scale_all"][:blocks], s["v_scale_all"][:blocks]
    else:
        s["k_all"] = _bf16((blocks + 1, BLOCK, hkv, d), gen)
        s["v_all"] = _bf16((blocks + 1, BLOCK, hkv, d), gen)
    s["k_cache"], s["v_cache"] = s["k_all"][:blocks], s["v_all"][:blocks]
    return s


def _prepare_attend(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    hq, hkv, d, nq = case["hq"], case["hkv"], case["d"], case["nq"]
    lens = _lengths(case)
    nb = -(-lens // BLOCK)
    blocks, mb = int(nb.sum()) + 16, int(nb.max())
    order = rng.permutation(blocks)
    tables = np.full((lens.size, mb), -1, np.int32)
    tables[np.arange(mb)[None, :] < nb[:, None]] = order[:int(nb.sum())]
    s = dict(case=case, q=_bf16((lens.size * nq, hq, d), gen), scale=1.0 / math.sqrt(d),
             tables=torch.from_numpy(tables).cuda(),
             lens=torch.from_numpy(lens.astype(np.int32)).cuda(), slopes=None)
    s["out"] = torch.empty_like(s["q"])
    if case["pool"] == "fp8":
        s["k_cache"], s["k_scale"] = _fp8_pool(blocks, hkv, d, gen)
        s["v_cache"], s["v_scale"] = _fp8_pool(blocks, hkv, d, gen)
    else:
        s["k_cache"] = _bf16((blocks, BLOCK, hkv, d), gen)
        s["v_cache"] = _bf16((blocks, BLOCK, hkv, d), gen)
        s["k_scale"] = s["v_scale"] = None
    if case["bias"]:  # the usual geometric slopes: 2^(-8 i / heads)
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)],
                                   dtype=torch.float32, device="cuda")
    return s


def prepare(case, seed):
    if case["kind"] in ("rope", "rope_fp8"):
        return _prepare_append(case, seed)
    return _prepare_attend(case, seed)


# ---------------------------------------------------------------- plain forms
def _rotated(x, cos, sin, interleaved):
    """x [rows, heads, d] in 32 bits, its first 2 * cos.shape[-1] dims rotated."""
    h = cos.shape[-1]
    x = x.float()
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((y, x[..., 2 * h:]), dim=-1)


def _angles(s):
    """cos and sin of each row's angles: the turns wrap in 64-bit integers, so far
    positions lose nothing; the functions are taken in 64 bits."""
    turns = (s["pos"][:, None] * s["turns"][None, :]).double() * (2.0 * math.pi / 2.0 ** 64)
    return torch.cos(turns).float(), torch.sin(turns).float()


def _scale_code(amax):
    """The smallest power of two (as its byte) that brings amax to 448 or below."""
    m, e = torch.frexp(amax)          # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, (e + 127).clamp(1, 254), torch.ones_like(e))


def _two_to(code):
    return torch.exp2((code.to(torch.int32) - 127).double()).float()


def _append_scaled(x, block, offset, codes, scale):
    """Rows x [n, heads, d] into block-scaled codes, in place: a block started by this call
    takes the scale of its new rows; one that is continued keeps the larger of its scale
    and that, its earlier codes rounded to the new scale."""
    heads = scale.shape[1]
    amax = x.abs().amax(dim=-1)
    new = torch.zeros_like(scale, dtype=torch.int32)
    new.scatter_reduce_(0, block[:, None].expand(-1, heads), _scale_code(amax), "amax")
    fresh = torch.zeros(scale.shape[0], dtype=torch.int32, device=x.device)
    fresh.scatter_reduce_(0, block, (offset == 0).int(), "amax")
    old = torch.where(fresh[:, None] > 0, 0, scale.int())
    code = torch.maximum(old, new)
    grown = torch.where(old > 0, _two_to(old - code + 127), 1.0)
    touched = codes[block].view(torch.float8_e4m3fn).float() * grown[block][:, None, :, None]
    codes[block] = touched.to(torch.float8_e4m3fn).view(torch.uint8)
    y = x / _two_to(code[block])[..., None]
    codes[block, offset] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(torch.where(new > 0, code, scale.int()))


def _plain_append(s):
    case = s["case"]
    cos, sin = _angles(s)
    s["q_out"].copy_(_rotated(s["q"], cos, sin, case["interleaved"]))
    k = _rotated(s["k"], cos, sin, case["interleaved"])
    spare = s["k_cache"].shape[0]
    block = torch.where(s["slots"] < 0, spare, s["slots"] // BLOCK)
    offset = torch.where(s["slots"] < 0, 0, s["slots"] % BLOCK)
    if case["kind"] == "rope_fp8":
        _append_scaled(k, block, offset, s["k_all"], s["k_scale_all"])
        _append_scaled(s["v"].float(), block, offset, s["v_all"], s["v_scale_all"])
    else:
        s["k_all"][block, offset] = k.to(torch.bfloat16)
        s["v_all"][block, offset] = s["v"]


def _plain_attend(s):
    case = s["case"]
    seqs, nq, hq, hkv, d = (case[k] for k in ("seqs", "nq", "hq", "hkv", "d"))
    tables, lens = s["tables"].long().clamp(min=0), s["lens"].long()
    t = torch.arange(tables.shape[1] * BLOCK, device="cuda")
    inside = (t[None, :] < lens[:, None])[:, :, None, None]

    def gathered(cache, scale):
        if scale is None:
            x = cache[tables].float()
        else:
            x = cache[tables].view(torch.float8_e4m3fn).float()
            x = x * _two_to(scale[tables])[:, :, None, :, None]
        return torch.where(inside, x.reshape(seqs, -1, hkv, d), 0.0)

    q = s["q"].float().view(seqs, nq, hkv, hq // hkv, d)
    x = torch.einsum("snhgd,sthd->shgnt", q, gathered(s["k_cache"], s["k_scale"])) * s["scale"]
    last = lens[:, None] - nq + torch.arange(nq, device="cuda")[None, :]      # [seqs, nq]
    far = (t[None, None, :] - last[:, :, None])                               # <= 0 where seen
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    if s["slopes"] is not None:
        x = x + s["slopes"].view(1, hkv, -1, 1, 1) * far[:, None, None].float()
    seen = far <= 0
    if case["window"]:
        seen = seen & (far > -case["window"])
    x = torch.where(seen[:, None, None], x, -torch.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(dim=-1)
    o = torch.einsum("shgnt,sthd->snhgd", p, gathered(s["v_cache"], s["v_scale"]))
    total = total.permute(0, 3, 1, 2)[..., None]
    s["out"].copy_(torch.where(total > 0, o / total, 0.0).reshape(seqs * nq, hq, d))


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if case["kind"] in ("rope", "rope_fp8"):
        if own:
            import paged_kv_cache_101_gb300 as pkv
            if case["kind"] == "rope_fp8":
                pkv.rope_kv_append_fp8_block(
                    s["q"], s["k"], s["v"], s["pos"], s["turns"], s["slots"], s["k_cache"],
                    s["v_cache"], s["k_scale"], s["v_scale"], s["q_out"],
                    interleaved=case["interleaved"])
            else:
                pkv.rope_kv_append(
                    s["q"], s["k"], s["v"], s["pos"], s["turns"], s["slots"], s["k_cache"],
                    s["v_cache"], s["q_out"], interleaved=case["interleaved"])
        else:
            _plain_append(s)
        if case["kind"] == "rope":
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        values = {n: s[n].view(torch.float8_e4m3fn) for n in ("k_cache", "v_cache")}
        return {"q": s["q_out"], **values,
                "k_scale": s["k_scale"].view(torch.float8_e8m0fnu),
                "v_scale": s["v_scale"].view(torch.float8_e8m0fnu)}
    if own:
        import paged_kv_cache_101_gb300 as pkv
        if case["kind"] == "attend":
            pkv.paged_decode_attention_fp8_block(
                s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["tables"],
                s["lens"], case["nq"], s["scale"], s["out"])
        else:
            pkv.paged_decode_attention_scored(
                s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], case["nq"],
                s["scale"], s["out"], softcap=case["cap"], alibi_slopes=s["slopes"],
                window=case["window"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        _plain_attend(s)
    return s["out"]


# ---------------------------------------------------------------- the definition in 64 bits
def _value(code):
    """The numbers that E4M3 codes stand for: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = code.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    return torch.where(c >= 128, -mag, mag)


def _nearest(y):
    """The E4M3 value nearest to y, ties to the even mantissa, at most 448 in magnitude."""
    mag = y.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(y) * torch.round(mag / step) * step


def _exact_rope(x, pos, freq, interleaved):
    angle = 2 * math.pi * torch.remainder(pos.double()[:, None] * freq[None, :], 1.0)
    z = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    h = freq.numel()
    head = x[..., :2 * h].double()
    pairs = (head.unflatten(-1, (h, 2)) if interleaved
             else head.unflatten(-1, (2, h)).transpose(-1, -2)).contiguous()
    w = torch.view_as_real(torch.view_as_complex(pairs) * z)
    w = w if interleaved else w.transpose(-1, -2)
    return torch.cat((w.flatten(-2), x[..., 2 * h:].double()), dim=-1)


def _exact_blocks(x, s, codes, scale):
    """Values and scales of the pool after the rows x, block by block."""
    values = _value(codes)
    exps = scale.double() - 127
    slots = s["slots"].cpu().numpy()
    order = {}
    for row, slot in enumerate(slots.tolist()):
        if slot >= 0:
            order.setdefault(slot // BLOCK, []).append((row, slot % BLOCK))
    ids = torch.tensor(list(order), device="cuda")
    count = max(len(v) for v in order.values())
    rows = torch.tensor([[r for r, _ in v] + [v[0][0]] * (count - len(v)) for v in order.values()],
                        device="cuda")
    offs = torch.tensor([[o for _, o in v] + [v[0][1]] * (count - len(v)) for v in order.values()],
                        device="cuda")
    amax = x[rows].abs().amax(dim=(1, 3))                            # [blocks, heads]
    need = torch.ceil(torch.log2(amax / E4M3_MAX))
    need = need + (amax > E4M3_MAX * torch.exp2(need)).double()
    need = need - (amax <= E4M3_MAX * torch.exp2(need - 1)).double()
    before = exps[ids]
    begun = (offs == 0).any(dim=1)[:, None]
    after = torch.where(begun, need, torch.maximum(before, need))
    kept = _nearest(values[ids] * torch.exp2(before - after)[:, None, :, None])
    values[ids] = torch.where(begun[..., None, None], values[ids], kept)
    values[ids[:, None].expand(-1, count).reshape(-1), offs.reshape(-1)] = _nearest(
        x[rows] * torch.exp2(-after)[:, None, :, None]).flatten(0, 1)
    exps[ids] = after
    return values, torch.exp2(exps)


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    freq = s["turns"].double() / 2.0 ** 64
    q = _exact_rope(s["q"], s["pos"], freq, case["interleaved"])
    k = _exact_rope(s["k"], s["pos"], freq, case["interleaved"])
    v = s["v"].double()
    if case["kind"] == "rope_fp8":
        kc, ks = _exact_blocks(k, s, s["k_cache"], s["k_scale"])
        vc, vs = _exact_blocks(v, s, s["v_cache"], s["v_scale"])
        return {"q": q, "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs}
    some = s["slots"] >= 0
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc.view(-1, *kc.shape[2:])[s["slots"][some]] = k[some]
    vc.view(-1, *vc.shape[2:])[s["slots"][some]] = v[some]
    return {"q": q, "k_cache": kc, "v_cache": vc}


def exact(case, seed):
    if case["kind"] in ("rope", "rope_fp8"):
        return _exact_append(case, seed)
    s = _prepare_attend(case, seed)
    nq, hq, hkv = case["nq"], case["hq"], case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(case).tolist()):
        ids = s["tables"][i, :-(-n // BLOCK)].long()
        k, v = s["k_cache"][ids], s["v_cache"][ids]
        if case["pool"] == "fp8":
            k = _value(k) * torch.exp2(s["k_scale"][ids].double() - 127)[:, None, :, None]
            v = _value(v) * torch.exp2(s["v_scale"][ids].double() - 127)[:, None, :, None]
        k = k.double().flatten(0, 1)[:n].transpose(0, 1)             # [heads, n, d]
        v = v.double().flatten(0, 1)[:n].transpose(0, 1)
        at = torch.arange(n, device="cuda")
        for j in range(nq):
            end = n - nq + j
            if end < 0:
                continue
            begin = max(0, end - case["window"] + 1) if case["window"] else 0
            x = torch.bmm(s["q"][i * nq + j].double().view(hkv, hq // hkv, -1),
                          k[:, begin:end + 1].transpose(1, 2)) * s["scale"]
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if s["slopes"] is not None:
                x = x - s["slopes"].double().view(hkv, -1, 1) * (end - at[begin:end + 1]).double()
            out[i * nq + j] = torch.bmm(torch.softmax(x, dim=-1),
                                        v[:, begin:end + 1]).reshape(hq, -1)
    return out
