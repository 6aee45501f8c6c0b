"""GPU checks of pkv_paged_decode_attention_scored and _fp8_block against attention in
64 bits.

Tolerance, with A = sum p |v| / sum p (the 64-bit reference with |v|): relative errors of
the weights move the output by at most their size times A. They are
 - bf16 pools: 2^-16 (a weight in two bf16 terms); E4M3 pools: 2^-11 (half a step of one f16), or
   where that is more 2^-31 absolute for a weight times 2^(its value scale - the row's
   largest value scale), the largest weight being 1 or more (f16's smallest step);
 - the score's absolute error, twice (numerator and sum): fp32 products and sums,
   2^-18 * max sum |q||k| * scale; the cap's tanh adds softcap * 2^-21, the distance
   bias |slope| * distance * 2^-22.
Then 2^-20 A for fp32 sums over the context, and the rounding to bf16 (2^-8) where the
output is bf16.
"""
import math

import numpy as np
import pytest

import ops_reference as R
import paged_kv_cache_101_gb300 as pkv
from gpu_helpers import bf16_dev, to_f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAN_CODE = 0x7F


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Batch:
    def __init__(self, lens, nq, G, Hkv, D, fp8, seed=0, window=0, extra=3, mb=None):
        rng = np.random.default_rng(seed + 7 * nq + G + Hkv + D)
        self.lens = np.array(lens, np.int32)
        self.nq, self.Hq, self.Hkv, self.D, self.fp8 = nq, G * Hkv, Hkv, D, fp8
        S = len(lens)
        nb = -(-np.maximum(self.lens, 0) // 16)
        blocks = int(nb.sum()) + extra
        self.mb = mb or max(1, int(nb.max()) + 1)
        order = rng.permutation(blocks)
        self.tables = np.full((S, self.mb), -1, np.int32)
        at = 0
        self.q = R.bf16(rng.standard_normal((S * nq, self.Hq, D)))
        shape = (blocks, 16, Hkv, D)
        if fp8:
            self.kc = np.full(shape, NAN_CODE, np.uint8)
            self.vc = np.full(shape, NAN_CODE, np.uint8)
            self.ks = rng.integers(118, 124, (blocks, Hkv), dtype=np.uint8)
            self.vs = rng.integers(116, 126, (blocks, Hkv), dtype=np.uint8)
        else:
            self.kc = np.full(shape, 0x7FC1, np.uint16)
            self.vc = np.full(shape, 0xFF80, np.uint16)     # -inf
            self.ks = self.vs = None
        for s, T in enumerate(self.lens):
            first = max(0, T - nq - window + 1) if window else 0
            for b in range(int(nb[s])):
                if window and 16 * b + 15 < first:
                    continue                 # wholly before the window: no block at all
                p = order[at]
                at += 1
                self.tables[s, b] = p
                lo, hi = max(0, first - 16 * b), min(16, int(T) - 16 * b)
                x = rng.standard_normal((2, hi - lo, Hkv, D))
                if fp8:
                    c = R.e4m3_code(x * 60)
                    self.kc[p, lo:hi], self.vc[p, lo:hi] = c[0], c[1]
                else:
                    c = R.bf16(x)
                    self.kc[p, lo:hi], self.vc[p, lo:hi] = c[0], c[1]
        self.scale = 1.0 / math.sqrt(D)

    def values(self):
        if self.fp8:
            return R.pool_values(self.kc, self.ks), R.pool_values(self.vc, self.vs)
        return R.value(self.kc), R.value(self.vc)

    def device(self):
        up = dev if self.fp8 else (lambda a: bf16_dev(a, torch))
        ks = dev(self.ks) if self.fp8 else None
        vs = dev(self.vs) if self.fp8 else None
        return (bf16_dev(self.q, torch), up(self.kc), up(self.vc), dev(self.tables),
                dev(self.lens), ks, vs)

    def call(self, out_dtype=torch.float32, softcap=0.0, slopes=None, window=0, ws=None):
        q, kc, vc, bt, cl, ks, vs = self.device()
        out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
        sl = None if slopes is None else dev(slopes.astype(np.float32))
        pkv.paged_decode_attention_scored(q, kc, vc, bt, cl, self.nq, self.scale, out,
                                          softcap=softcap, alibi_slopes=sl, window=window,
                                          k_scale=ks, v_scale=vs, ws=ws)
        torch.cuda.synchronize()
        return out

    def check(self, out, softcap=0.0, slopes=None, window=0):
        k, v = self.values()
        f32 = None if slopes is None else slopes.astype(np.float32).astype(np.float64)
        ref, mag, big, low = R.attention(
            R.value(self.q), k, v, self.tables, self.lens, self.nq,
            np.float64(np.float32(self.scale)), softcap, f32, window,
            v_exp=self.vs.astype(int) if self.fp8 else None)
        T = np.repeat(np.maximum(self.lens, 0), self.nq)[:, None]
        score = big * 2.0 ** -18 + softcap * 2.0 ** -21
        if slopes is not None:
            # distances that count: all for a bias that grows with it, else those whose
            # bias is over -100 (a weight of e^-100)
            near = 100 / np.maximum(np.abs(slopes), 1e-9)[None, :]
            reach = np.where(slopes[None, :] < 0, T, np.minimum(T, near))
            score = score + np.abs(slopes)[None, :] * reach * 2.0 ** -22
        weight = (2.0 ** -11 if self.fp8 else 2.0 ** -16) + 2.0 ** -20 + 2 * score
        bound = weight[..., None] * mag + 2.0 ** -31 * low
        if out.dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
        got = to_f64(out)
        bad = ~(np.abs(got - ref) <= bound + 1e-30)
        assert not bad.any(), (f"{bad.sum()} of {bad.size} beyond the bound, first "
                               f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {ref[bad][0]}, "
                               f"bound {bound[bad][0]}")


def slopes_of(Hq):
    return np.array([2.0 ** (-8.0 * (i + 1) / Hq) for i in range(Hq)], np.float32)


LENGTHS = [1, 15, 16, 17, 31, 32, 33, 48, 100, 257, 700, 0]
HEADS = [(1, 4, 8), (1, 1, 1), (1, 8, 8), (4, 8, 4), (2, 5, 3), (4, 16, 1), (3, 1, 2), (1, 64, 1),
         (4, 1, 6)]     # nq, G, Hkv


@pytest.mark.parametrize("fp8,D", [(False, 64), (False, 128), (True, 128)])
@pytest.mark.parametrize("nq,G,Hkv", HEADS)
def test_plain_scores(fp8, D, nq, G, Hkv):
    b = Batch(LENGTHS, nq, G, Hkv, D, fp8)
    b.check(b.call())
    b.check(b.call(torch.bfloat16))


@pytest.mark.parametrize("fp8,D", [(False, 64), (False, 128), (True, 128)])
@pytest.mark.parametrize("nq,G,Hkv", HEADS)
@pytest.mark.parametrize("cap,bias,window", [(30.0, False, 0), (0.0, True, 0), (0.0, False, 40),
                                             (5.0, True, 17), (0.0, True, 1), (50.0, False, 4096)])
def test_scores(fp8, D, nq, G, Hkv, cap, bias, window):
    b = Batch(LENGTHS, nq, G, Hkv, D, fp8, window=window)
    sl = slopes_of(b.Hq) if bias else None
    b.check(b.call(softcap=cap, slopes=sl, window=window), cap, sl, window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,G", [(1, 4), (4, 8), (2, 7)])
def test_long_sequences_are_split_and_joined(fp8, nq, G):
    b = Batch([4001, 3, 2500, 640], nq, G, 4, 128, fp8)
    b.check(b.call())
    b.check(b.call(softcap=20.0, window=1500), 20.0, None, 1500)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_short_sequences(fp8):
    rng = np.random.default_rng(3)
    b = Batch(rng.integers(0, 60, 500), 1, 2, 2, 128, fp8)
    b.check(b.call())


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_of_extreme_size(fp8):
    """Scores far apart: one token takes all the weight, wherever it stands, and the
    running maximum is raised late."""
    b = Batch([300, 77, 600], 2, 4, 2, 128, fp8)
    b.q = R.bf16(R.value(b.q) * 30)
    b.check(b.call())
    sl = -slopes_of(b.Hq) * 4                     # the farthest token is favoured
    b.check(b.call(slopes=sl), 0.0, sl)
    b.check(b.call(softcap=1e-3), 1e-3)           # all scores equal


def test_values_of_very_different_scales():
    """Value scales 2^-60 .. 2^40 from block to block, growing and shrinking."""
    b = Batch([400, 90], 1, 4, 2, 128, True)
    rng = np.random.default_rng(4)
    b.vs = rng.integers(67, 168, b.vs.shape, dtype=np.uint8)
    b.vs[b.tables[0, 3]] = 0                      # an empty block's byte: 2^-127
    b.check(b.call())


def test_queries_of_extreme_size():
    """E4M3 pools take any finite q: large, tiny, and a row of zeros."""
    b = Batch([50, 40, 30], 1, 4, 2, 128, True)
    q = R.value(b.q)
    q[0] *= 2.0 ** 100
    q[1] *= 2.0 ** -100
    q[2] = 0
    b.q = R.bf16(q)
    b.scale = 1.0
    # the first row's scores pick single tokens: compare by the definition's own limit
    out = to_f64(b.call())
    k, v = b.values()
    ref, mag, _, low = R.attention(R.value(b.q), k, v, b.tables, b.lens, 1, 1.0,
                                   v_exp=b.vs.astype(int))
    assert np.all(np.abs(out - ref) <= 2.0 ** -10 * mag + 2.0 ** -31 * low)


@pytest.mark.parametrize("fp8", [False, True])
def test_lengths_beyond_the_table_are_clamped(fp8):
    b = Batch([64, 30, 5], 1, 4, 2, 128, fp8, mb=4)
    b.lens = np.array([1000, 30, -5], np.int32)
    got = b.call()
    assert not got[2].any()
    b.check(got)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_outside_the_pool_read_zeros(fp8):
    b = Batch([100, 40], 1, 4, 2, 128, fp8)
    b.tables[0, 2] = len(b.kc)
    b.tables[1, 0] = -3
    ws = torch.zeros(pkv.workspace_size_scored(2, 1, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out = b.call(ws=ws)
    assert pkv.workspace_error(ws) == 8
    zero = np.zeros((1,) + b.kc.shape[1:], b.kc.dtype)
    b.kc, b.vc = np.concatenate([b.kc, zero]), np.concatenate([b.vc, zero])
    if fp8:
        byte = np.full((1, 2), 100, np.uint8)
        b.ks, b.vs = np.concatenate([b.ks, byte]), np.concatenate([b.vs, byte])
    b.tables[0, 2] = b.tables[1, 0] = len(b.kc) - 1
    b.check(out)


@pytest.mark.parametrize("fp8", [False, True])
def test_same_bits_twice_and_on_another_stream(fp8):
    b = Batch([900, 31, 250, 1], 2, 4, 4, 128, fp8)
    a = b.call(softcap=10.0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c = b.call(softcap=10.0)
    assert torch.equal(a, c) and torch.equal(a, b.call(softcap=10.0))


def test_against_the_plain_calls():
    """Without a cap, a bias and a window it is pkv_paged_decode_attention."""
    b = Batch([300, 64, 999], 2, 4, 2, 128, False)
    q, kc, vc, bt, cl, _, _ = b.device()
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    pkv.paged_decode_attention(q, kc, vc, bt, cl, 2, b.scale, out)
    assert torch.allclose(out, b.call(), rtol=1e-4, atol=1e-5)


def test_fp8_block_entry():
    b = Batch(LENGTHS, 1, 4, 8, 128, True)
    q, kc, vc, bt, cl, ks, vs = b.device()
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    pkv.paged_decode_attention_fp8_block(q, kc, vc, ks, vs, bt, cl, 1, b.scale, out)
    assert torch.equal(out, b.call())
