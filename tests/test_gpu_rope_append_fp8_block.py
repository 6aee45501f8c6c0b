"""GPU checks of pkv_rope_kv_append_fp8_block against its definition in 64 bits.

v is bf16, so its scales and codes are exact. k' is computed in fp32 within
e = 2^-21 (|x| + |y|) of the exact rotation (test_gpu_rope_append.py): its scale is
the exact one unless the block's largest magnitude lies within e of 448 * 2^k, and a
code's value is within half an E4M3 step of a number that is within e of the exact one:
|err| <= max(2^-4 |x|, 2^-10 scale) + 2 e.
"""
import numpy as np
import pytest

import ops_reference as R
import paged_kv_cache_101_gb300 as pkv
from gpu_helpers import bf16_dev, bf16_host
from test_gpu_rope_append import check_rotated, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Pools:
    """Device pools and their 64-bit twins (k through its exact rotation)."""

    def __init__(self, blocks, Hkv, D, seed, empty=True):
        rng = np.random.default_rng(seed)
        self.Hkv, self.D = Hkv, D
        self.codes = [rng.integers(0, 127, (blocks, 16, Hkv, D), dtype=np.uint8) for _ in "kv"]
        self.scale = [np.zeros((blocks, Hkv), np.uint8) if empty else
                      rng.integers(110, 130, (blocks, Hkv), dtype=np.uint8) for _ in "kv"]
        self.kc, self.vc = (dev(c) for c in self.codes)
        self.ks, self.vs = (dev(s) for s in self.scale)

    def append(self, k, v, pos, turns, slots, q=None, interleaved=False):
        n = len(slots)
        q_dev = None if q is None else bf16_dev(q, torch)
        out = None if q is None else torch.full_like(q_dev, float("nan"))
        before = self.kc.cpu().numpy(), self.ks.cpu().numpy()
        pkv.rope_kv_append_fp8_block(q_dev, bf16_dev(k, torch), bf16_dev(v, torch), dev(pos),
                                     dev(turns), dev(slots), self.kc, self.vc, self.ks, self.vs,
                                     out, interleaved=interleaved)
        torch.cuda.synchronize()
        # v: exact
        R.append_block(R.value(v), slots, self.codes[1], self.scale[1])
        assert np.array_equal(self.vs.cpu().numpy(), self.scale[1])
        assert np.array_equal(self.vc.cpu().numpy(), self.codes[1])
        # k: from the pool as it was, so that earlier roundings do not add up
        ref, mag = R.rotate(R.value(k), pos, turns, interleaved)
        codes, scale = before[0].copy(), before[1].copy()
        R.append_block(ref, slots, codes, scale)
        got_c, got_s = self.kc.cpu().numpy(), self.ks.cpu().numpy()
        assert np.array_equal(got_s, scale)      # (no borderline maximum in these inputs)
        w = (slots >= 0) & (slots < codes.shape[0] * 16)
        at = slots[w]
        got = R.pool_values(got_c, got_s)[at // 16, at % 16]
        sc = np.ldexp(1.0, scale[at // 16].astype(int) - 127)[..., None]
        fin = np.isfinite(ref[w])
        bound = np.maximum(2.0 ** -4 * np.abs(ref[w]), 2.0 ** -10 * sc) + mag[w] * 2.0 ** -20
        assert (np.abs(got - ref[w])[fin] <= bound[fin]).all()
        rest = np.ones(codes.shape[:2], bool)
        rest[at // 16, at % 16] = False
        assert np.array_equal(got_c[rest], codes[rest])
        if q is not None:
            qr, qm = R.rotate(R.value(q), pos, turns, interleaved)
            check_rotated(bf16_host(out), qr, qm, "q")
        assert n == 0 or self.ks.cpu().numpy()[at // 16].all()


def rows(rng, n, H, D, spread=0.0):
    x = rng.standard_normal((n, H, D)) * 2.0 ** (spread * rng.standard_normal((n, H, 1)))
    return R.bf16(x)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,D,r", [
    (1, 32, 8, 128, 128), (16, 4, 2, 128, 64), (17, 5, 5, 80, 80), (50, 3, 3, 72, 20),
    (7, 2, 1, 256, 256), (100, 8, 4, 128, 128), (33, 2, 2, 64, 16), (20, 3, 9, 128, 96),
    (1500, 4, 2, 128, 64), (4500, 2, 1, 128, 128), (1200, 2, 1, 64, 64)])
def test_one_run(n, Hq, Hkv, D, r, interleaved):
    """One sequence's chunk from position 5 on: a block continued, blocks started."""
    rng = np.random.default_rng(n + D + r)
    blocks = n // 16 + 4
    pool = Pools(blocks, Hkv, D, seed=n, empty=False)
    order = rng.permutation(blocks)
    pos = np.arange(5, 5 + n)
    slots = order[pos // 16] * 16 + pos % 16
    pool.append(rows(rng, n, Hkv, D, 2.0), rows(rng, n, Hkv, D, 2.0), pos,
                pkv.rotary_turns(r).numpy(), slots, rows(rng, n, Hq, D), interleaved)


def test_token_by_token():
    """Three sequences decoded together for 40 steps, magnitudes wandering by powers of
    two, so that scales grow inside blocks and restart with each block."""
    rng = np.random.default_rng(5)
    Hkv, D, S = 3, 128, 3
    pool = Pools(12, Hkv, D, seed=6)
    order = rng.permutation(12).reshape(S, 4)
    turns = pkv.rotary_turns(D).numpy()
    pos = np.array([0, 9, 15])
    for step in range(40):
        slots = np.array([order[s, pos[s] // 16] * 16 + pos[s] % 16 for s in range(S)])
        if step % 7 == 3:
            slots[1] = -1                       # a padding row among them
        size = 2.0 ** rng.integers(-6, 7, (S, Hkv, 1))
        pool.append(R.bf16(rng.standard_normal((S, Hkv, D)) * size),
                    R.bf16(rng.standard_normal((S, Hkv, D)) * size), pos, turns, slots)
        pos = pos + (slots >= 0)


@pytest.mark.parametrize("n,new", [(1100, 1), (1300, 3), (4200, 2)])
def test_large_batches_of_short_runs(n, new):
    """Many sequences with one to three tokens each: several runs in a CTA's window."""
    rng = np.random.default_rng(n)
    seqs = n // new
    pool = Pools(2 * seqs + 3, 2, 128, seed=n, empty=False)
    start = rng.integers(0, 20, seqs)
    order = rng.permutation(2 * seqs).reshape(seqs, 2)
    pos = (start[:, None] + np.arange(new)).reshape(-1)
    at = (start[:, None] + np.arange(new)) % 32
    slots = (np.take_along_axis(order, at // 16, 1) * 16 + at % 16).reshape(-1)
    slots[rng.integers(0, slots.size, 40)] = -1
    # a padding row inside a run would part its block's rows: pad whole sequences
    bad = (slots.reshape(seqs, new) < 0).any(axis=1)
    slots = np.where(np.repeat(bad, new), -1, slots)
    pool.append(rows(rng, slots.size, 2, 128, 1.0), rows(rng, slots.size, 2, 128, 1.0), pos,
                pkv.rotary_turns(128).numpy(), slots, rows(rng, slots.size, 2, 128))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,r", [(70, 8, 8, 128), (300, 5, 5, 64), (500, 9, 9, 48),
                                        (1000, 2, 1, 128), (250, 0, 3, 24)])
def test_decode_batches(n, Hq, Hkv, r, interleaved):
    """One token of each sequence, three steps: blocks begun and continued, scales that grow
    in some heads only, padding rows, and an infinity among the values."""
    rng = np.random.default_rng(n + r)
    pool = Pools(n + 2, Hkv, 128, seed=n, empty=False)
    turns = pkv.rotary_turns(r).numpy()
    block = rng.permutation(n + 2)[:n]
    at = rng.integers(0, 14, n)
    at[::5] = 0
    for step in range(3):
        slots = block * 16 + at + step
        slots[rng.integers(0, n, n // 20 + 1)] = -1
        size = 2.0 ** rng.integers(-4, 5, (n, Hkv, 1))
        k = R.bf16(rng.standard_normal((n, Hkv, 128)) * size)
        v = R.bf16(rng.standard_normal((n, Hkv, 128)) * size)
        v[n // 2, 0, 5] = 0x7F80
        pool.append(k, v, at + step + 1000 * np.arange(n), turns, slots,
                    rows(rng, n, Hq, 128) if Hq else None, interleaved)


def test_several_runs_and_padding():
    """Draft tokens of four sequences with padding behind each, one crossing a block."""
    rng = np.random.default_rng(8)
    pool = Pools(10, 2, 128, seed=9, empty=False)
    slots = np.array([3, 4, 5, -1, 30, 31, 64, 65, -1, -1, 127, -1, 96, 97, 98, 99, -1])
    n = len(slots)
    pool.append(rows(rng, n, 2, 128), rows(rng, n, 2, 128), np.arange(n) + 100,
                pkv.rotary_turns(128).numpy(), slots, rows(rng, n, 4, 128))


def test_odd_values():
    """Zeros, infinities, NaN, the smallest and largest numbers."""
    pool = Pools(6, 1, 64, seed=3)
    x = np.zeros((6, 1, 64), np.float32)
    x[1, 0, :4] = [np.inf, -np.inf, np.nan, 3.0]
    x[2, 0, :3] = [1e-40, 2.0 ** -133, -(2.0 ** -126)]
    x[3, 0, :2] = [3.38e38, -1.0]
    x[4, 0, :] = 448.0
    x[5, 0, :] = 450.0                                    # needs the next power of two
    slots = np.arange(6) * 16
    zero = np.zeros((6, 1, 64), np.uint16)
    pool.append(zero, R.bf16(x), np.zeros(6, np.int64), pkv.rotary_turns(64).numpy(), slots)
    vs = pool.vs.cpu().numpy()[:, 0]
    assert vs[0] == 1 and vs[4] == 127 and vs[5] == 128
    assert pool.vc.cpu().numpy()[1, 0, 0, :3].tolist() == [0x7e, 0xfe, 0x7f]


def test_a_grown_scale_rounds_earlier_rows_once():
    pool = Pools(1, 1, 64, seed=1)
    turns = pkv.rotary_turns(64).numpy()
    rng = np.random.default_rng(2)
    for t, size in enumerate([1.0, 0.01, 64.0, 1.0, 1e30, 1e-30]):
        x = R.bf16(rng.standard_normal((1, 1, 64)) * size)
        pool.append(x, x, np.array([t]), turns, np.array([t]))


def test_slots_past_the_pool_and_all_padding():
    rng = np.random.default_rng(12)
    pool = Pools(4, 2, 64, seed=13)
    x = rows(rng, 5, 2, 64)
    pool.append(x, x, np.arange(5), pkv.rotary_turns(64).numpy(),
                np.array([-1, 64, 65, 2 ** 62, -7]))
    assert not pool.ks.any() and not pool.vs.any()


def test_equal_slots_do_not_fault():
    """Unspecified contents, but nothing outside the named block changes."""
    rng = np.random.default_rng(14)
    pool = Pools(4, 2, 64, seed=15)
    x = bf16_dev(rows(rng, 40, 2, 64), torch)
    before = pool.kc.clone()
    pkv.rope_kv_append_fp8_block(None, x, x, dev(np.arange(40)), pkv.rotary_turns(64).cuda(),
                                 dev(np.full(40, 18)), pool.kc, pool.vc, pool.ks, pool.vs, None)
    torch.cuda.synchronize()
    assert torch.equal(before[[0, 2, 3]], pool.kc[[0, 2, 3]])
