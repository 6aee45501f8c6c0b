"""GPU checks of pkv_rope_kv_append against the rotation in 64 bits.

Tolerance. The kernel's angle is 64-bit fixed point, its upper 32 bits rounded to fp32
(2^-25 of half a turn, 9.4e-8 rad); sincospif errs by at most 2 ulp (2^-22); three fp32
roundings of terms of at most |x| + |y| follow: together under 2^-21 (|x| + |y|). The
result is rounded once to bf16: 2^-8 relative. So every element is within
2^-8 (|ref| + e) + e, e = 2^-21 (|x| + |y|). v, and all that is not written, is exact.
"""
import numpy as np
import pytest

import ops_reference as R
import paged_kv_cache_101_gb300 as pkv
from gpu_helpers import bf16_dev, bf16_host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check_rotated(got_bits, ref, mag, what):
    got = R.value(got_bits)
    e = mag * 2.0 ** -21
    bound = 2.0 ** -8 * (np.abs(ref) + e) + e
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} beyond the bound"


class Case:
    def __init__(self, n, Hq, Hkv, D, r, seed=0, blocks=None, first=0, pad=(), positions=None):
        rng = np.random.default_rng(seed + 31 * n + D + r)
        self.n, self.Hq, self.Hkv, self.D = n, Hq, Hkv, D
        self.q = R.bf16(rng.standard_normal((n, Hq, D)))
        self.k = R.bf16(rng.standard_normal((n, Hkv, D)))
        self.v = R.bf16(rng.standard_normal((n, Hkv, D)))
        blocks = blocks or n // 16 + 3
        self.kc = R.bf16(rng.standard_normal((blocks, 16, Hkv, D)))
        self.vc = R.bf16(rng.standard_normal((blocks, 16, Hkv, D)))
        self.slots = rng.permutation(blocks * 16)[:n].astype(np.int64)
        self.slots[list(pad)] = -1
        self.pos = (np.arange(n) * 37 + first if positions is None
                    else np.asarray(positions)).astype(np.int64)
        self.turns = pkv.rotary_turns(r).numpy()

    def check(self, q_out, kc, vc, interleaved, scale=1.0, rotate_q=True):
        if rotate_q:
            ref, mag = R.rotate(R.value(self.q), self.pos, self.turns, interleaved, scale)
            check_rotated(bf16_host(q_out), ref, mag, "q")
        ref, mag = R.rotate(R.value(self.k), self.pos, self.turns, interleaved, scale)
        w = (self.slots >= 0) & (self.slots < self.kc.shape[0] * 16)
        flat = bf16_host(kc).reshape(-1, self.Hkv, self.D)
        check_rotated(flat[self.slots[w]], ref[w], mag[w], "k")
        want_v = self.vc.reshape(-1, self.Hkv, self.D).copy()
        want_v[self.slots[w]] = self.v[w]
        assert np.array_equal(bf16_host(vc).reshape(want_v.shape), want_v)
        keep = np.ones(flat.shape[0], bool)
        keep[self.slots[w]] = False
        assert np.array_equal(flat[keep], self.kc.reshape(flat.shape)[keep])


def run(c, interleaved, scale=1.0):
    kc, vc = bf16_dev(c.kc, torch), bf16_dev(c.vc, torch)
    q = bf16_dev(c.q, torch)
    q_out = torch.full_like(q, float("nan"))
    pkv.rope_kv_append(q, bf16_dev(c.k, torch), bf16_dev(c.v, torch), dev(c.pos), dev(c.turns),
                       dev(c.slots), kc, vc, q_out, interleaved=interleaved, rotary_scale=scale)
    torch.cuda.synchronize()
    assert np.array_equal(bf16_host(q), c.q)
    c.check(q_out, kc, vc, interleaved, scale)
    return q_out, kc, vc


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,D,r", [
    (1, 32, 8, 128, 128), (1, 1, 1, 8, 2), (5, 8, 2, 64, 64), (33, 7, 7, 80, 80),
    (19, 6, 3, 96, 24), (64, 64, 8, 128, 64), (17, 5, 5, 72, 40), (3, 2, 1, 256, 256),
    (2, 4, 2, 1024, 1024), (9, 4, 2, 24, 6), (11, 3, 1, 80, 20), (1000, 16, 2, 64, 32),
    (6, 9, 3, 136, 112), (1500, 4, 2, 128, 128), (1025, 3, 1, 80, 64), (2, 3, 1, 512, 512),
    (4, 2, 1, 520, 64)])
def test_rotation_and_append(n, Hq, Hkv, D, r, interleaved):
    run(Case(n, Hq, Hkv, D, r, pad=(0, n // 2) if n > 4 else ()), interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,D,r", [(1300, 1, 1, 96, 24), (2443, 3, 1, 24, 6),
                                          (1217, 4, 2, 80, 42), (1300, 1, 1, 136, 130),
                                          (9001, 1, 1, 24, 6), (1900, 2, 1, 1024, 1000)])
def test_many_rows_of_odd_dims(n, Hq, Hkv, D, r, interleaved):
    """Dims that no vector form takes, several rows to a block of threads."""
    run(Case(n, Hq, Hkv, D, r, pad=(0, 1, n // 2, n - 1), positions=np.arange(n) * 7919 - 5),
        interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    pos = [0, 1, -1, 131071, 10 ** 6 + 7, 2 ** 31 - 1, 2 ** 31 + 5, -(2 ** 40) + 3, 2 ** 52 + 1,
           2 ** 63 - 1]
    run(Case(len(pos), 4, 2, 128, 128, positions=pos), interleaved)


def test_rotary_scale():
    run(Case(12, 4, 2, 128, 96), False, scale=1.25)


def test_slots_past_the_pool_are_skipped():
    c = Case(8, 4, 2, 64, 64)
    c.slots[2] = c.kc.shape[0] * 16
    c.slots[5] = 2 ** 62
    run(c, False)


def test_slices_of_one_projection():
    """q, k and v as column ranges of one [n, (Hq + 2 Hkv) * D] tensor."""
    c = Case(21, 8, 2, 64, 64)
    whole = np.concatenate([c.q.reshape(21, -1), c.k.reshape(21, -1), c.v.reshape(21, -1)], axis=1)
    t = bf16_dev(whole, torch)
    q, k, v = (x.unflatten(1, (-1, 64)) for x in t.split([8 * 64, 2 * 64, 2 * 64], dim=1))
    assert not q.is_contiguous() and q.data_ptr() == t.data_ptr()
    kc, vc = bf16_dev(c.kc, torch), bf16_dev(c.vc, torch)
    q_out = torch.empty((21, 8, 64), dtype=torch.bfloat16, device="cuda")
    pkv.rope_kv_append(q, k, v, dev(c.pos), dev(c.turns), dev(c.slots), kc, vc, q_out)
    torch.cuda.synchronize()
    assert np.array_equal(bf16_host(t), whole)
    c.check(q_out, kc, vc, False)


@pytest.mark.parametrize("interleaved,r", [(False, 128), (False, 32), (True, 128), (True, 40)])
def test_in_place(interleaved, r):
    c = Case(37, 12, 4, 128, r)
    a, _, _ = run(c, interleaved)
    q, kc, vc = bf16_dev(c.q, torch), bf16_dev(c.kc, torch), bf16_dev(c.vc, torch)
    pkv.rope_kv_append(q, bf16_dev(c.k, torch), bf16_dev(c.v, torch), dev(c.pos), dev(c.turns),
                       dev(c.slots), kc, vc, q, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), q.view(torch.int16))


def test_keys_and_values_only():
    c = Case(20, 4, 2, 64, 64)
    kc, vc = bf16_dev(c.kc, torch), bf16_dev(c.vc, torch)
    assert pkv.rope_kv_append(None, bf16_dev(c.k, torch), bf16_dev(c.v, torch), dev(c.pos),
                              dev(c.turns), dev(c.slots), kc, vc, None) is None
    torch.cuda.synchronize()
    c.check(None, kc, vc, False, rotate_q=False)


def test_empty_batch():
    c = Case(1, 4, 2, 64, 64)
    kc, vc = bf16_dev(c.kc, torch), bf16_dev(c.vc, torch)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = torch.empty(0, dtype=torch.int64, device="cuda")
    pkv.rope_kv_append(e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), i, dev(c.turns), i, kc, vc,
                       e(0, 4, 64))
    torch.cuda.synchronize()
    assert np.array_equal(bf16_host(kc), c.kc) and np.array_equal(bf16_host(vc), c.vc)


def test_plain_append_of_unrotated_rows_agrees():
    """Position 0 turns nothing: the call is kv_append, bit for bit."""
    c = Case(40, 8, 2, 128, 128, positions=np.zeros(40))
    _, kc, vc = run(c, False)
    k2, v2 = bf16_dev(c.kc, torch), bf16_dev(c.vc, torch)
    pkv.kv_append(bf16_dev(c.k, torch), bf16_dev(c.v, torch), dev(c.slots), k2, v2)
    torch.cuda.synchronize()
    assert torch.equal(kc.view(torch.int16), k2.view(torch.int16))
    assert torch.equal(vc.view(torch.int16), v2.view(torch.int16))
