"""The operators used together, as a serving loop uses them: prompts and decode steps
written with their rotation into a paged pool (bf16, or block-scaled E4M3) that a block
manager hands out, and attention over it; a fork with copy-on-write; graph capture.

The reference keeps every token's exact rotated key and value; what the pool holds is
read back for the attention's own reference, so the bounds of test_gpu_scored.py apply
to it, and the pool's contents are checked against the exact keys by their own bounds
(test_gpu_rope_append*.py).
"""
import math

import numpy as np
import pytest

import ops_reference as R
import paged_kv_cache_101_gb300 as pkv
from gpu_helpers import bf16_dev, bf16_host, to_f64
from test_gpu_rope_append import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HQ, HKV, D = 8, 2, 128
TURNS = pkv.rotary_turns(D, base=500000.0)


class Server:
    """Pools, a block manager and the exact rows of every sequence."""

    def __init__(self, fp8, blocks=40, seed=0):
        self.fp8, self.rng = fp8, np.random.default_rng(seed)
        self.bm = pkv.BlockManager(blocks)
        shape = (blocks, 16, HKV, D)
        if fp8:
            self.kc = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
            self.ks = torch.zeros((blocks, HKV), dtype=torch.uint8, device="cuda")
            self.vc, self.vs = self.kc.clone(), self.ks.clone()
        else:
            self.kc = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            self.vc, self.ks, self.vs = self.kc.clone(), None, None
        self.turns = TURNS.cuda()
        self.k = {}

    def tokens(self, seqs, n):
        """n new tokens of each sequence: appended, then attended."""
        slots, copies = self.bm.append_batch(seqs, n)
        if copies:
            src, dst = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in zip(*copies))
            as_bf16 = (lambda t: t.view(torch.bfloat16)) if self.fp8 else (lambda t: t)
            pkv.copy_blocks(as_bf16(self.kc), as_bf16(self.vc), src, dst)
            if self.fp8:
                self.ks[dst.long()] = self.ks[src.long()]
                self.vs[dst.long()] = self.vs[src.long()]
        rows = n * len(seqs)
        pos = np.concatenate([np.arange(self.bm.length(s) - n, self.bm.length(s)) for s in seqs])
        q, k, v = (R.bf16(self.rng.standard_normal((rows, h, D))) for h in (HQ, HKV, HKV))
        exact, _ = R.rotate(R.value(k), pos, TURNS.numpy(), False)
        for i, s in enumerate(seqs):
            self.k.setdefault(s, []).append(exact[i * n:(i + 1) * n])
        self.q_exact, _ = R.rotate(R.value(q), pos, TURNS.numpy(), False)
        q_out = bf16_dev(q, torch)
        args = (q_out, bf16_dev(k, torch), bf16_dev(v, torch), dev(pos), self.turns, dev(slots),
                self.kc, self.vc)
        if self.fp8:
            pkv.rope_kv_append_fp8_block(*args, self.ks, self.vs, q_out)
        else:
            pkv.rope_kv_append(*args, q_out)
        return q_out

    def attend(self, seqs, nq, q, **kw):
        mb = max(-(-self.bm.length(s) // 16) for s in seqs)
        tables, lens = self.bm.block_tables(seqs, mb)
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        if self.fp8 and not kw:
            pkv.paged_decode_attention_fp8_block(q, self.kc, self.vc, self.ks, self.vs,
                                                 dev(tables), dev(lens), nq, 1 / math.sqrt(D), out)
        else:
            sl = kw.get("slopes")
            pkv.paged_decode_attention_scored(
                q, self.kc, self.vc, dev(tables), dev(lens), nq, 1 / math.sqrt(D), out,
                softcap=kw.get("softcap", 0.0), alibi_slopes=None if sl is None else dev(sl),
                window=kw.get("window", 0), k_scale=self.ks, v_scale=self.vs)
        torch.cuda.synchronize()
        self.check(seqs, nq, q, tables, lens, out, kw)
        return out

    def check(self, seqs, nq, q, tables, lens, out, kw):
        if self.fp8:
            scale = [np.ldexp(1.0, t.cpu().numpy().astype(int) - 127)[:, None, :, None]
                     for t in (self.ks, self.vs)]
            k, v = (R.e4m3_value(c.cpu().numpy()) * s for c, s in zip((self.kc, self.vc), scale))
            half, exps = 2.0 ** -4, self.vs.cpu().numpy().astype(int)
        else:
            k, v = R.value(bf16_host(self.kc)), R.value(bf16_host(self.vc))
            half, exps = 2.0 ** -8, None
        for i, s in enumerate(seqs):        # the pool holds the exact keys, rounded
            at = np.arange(lens[i])
            got = k[tables[i][at // 16], at % 16]
            want = np.concatenate(self.k[s])
            # E4M3: a row may be rounded once more for each growth of its block's scale,
            # each time within half a step (2^-4, or 2^-10 of a scale under 2^-5 here)
            times = 3 if self.fp8 else 1
            assert (np.abs(got - want) <= times * (half * np.abs(want) + 2.0 ** -15) + 2e-5).all()
        sl = kw.get("slopes")
        ref, mag, big, low = R.attention(to_f64(q), k, v, tables, lens, nq, 1 / math.sqrt(D),
                                         kw.get("softcap", 0.0), sl, kw.get("window", 0), exps)
        weight = (2.0 ** -11 if self.fp8 else 2.0 ** -16) + 2 * (big[..., None] * 2.0 ** -18
                                                                 + 2.0 ** -14) + 2.0 ** -20
        assert (np.abs(to_f64(out) - ref) <= weight * mag + 2.0 ** -31 * low).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_then_decode_steps(fp8):
    s = Server(fp8)
    for seq, n in ((0, 37), (1, 64), (2, 5)):
        assert s.bm.add_sequence(seq, 0)
        s.tokens([seq], n)
    for _ in range(20):
        s.attend([0, 1, 2], 1, s.tokens([0, 1, 2], 1))
    # four draft tokens, a window, a cap and a bias
    s.attend([2, 0], 4, s.tokens([2, 0], 4), window=30, softcap=20.0)
    slopes = np.array([2.0 ** -(i + 1) for i in range(HQ)], np.float32)
    s.attend([1, 2], 2, s.tokens([1, 2], 2), slopes=slopes)


@pytest.mark.parametrize("fp8", [False, True])
def test_fork_with_copy_on_write(fp8):
    s = Server(fp8, seed=4)
    s.bm.add_sequence(0, 0)
    s.tokens([0], 21)
    s.bm.fork(0, 1)
    s.k[1] = list(s.k[0])
    for _ in range(14):
        s.attend([0, 1], 1, s.tokens([0, 1], 1))


@pytest.mark.parametrize("fp8", [False, True])
def test_two_graphs_and_an_eager_call(fp8):
    """Append and attention captured twice without a workspace of their own, replayed on
    two streams at once next to an eager call: each result as when run alone."""
    s = Server(fp8, seed=9)
    s.bm.add_sequence(0, 0)
    s.tokens([0], 300)
    q = s.tokens([0], 1)
    alone = s.attend([0], 1, q, softcap=8.0)
    tables, lens = (dev(a) for a in s.bm.block_tables([0], 20))

    def attend(q, out):
        pkv.paged_decode_attention_scored(q, s.kc, s.vc, tables, lens, 1, 1 / math.sqrt(D), out,
                                          softcap=8.0, k_scale=s.ks, v_scale=s.vs)

    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(alone) for _ in range(3)]
    qs = [q.clone() for _ in range(3)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side[i]):
            for _ in range(5):
                attend(qs[i], outs[i])
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
        attend(qs[2], outs[2])
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, alone)


def test_a_captured_step_follows_its_inputs():
    """A captured append + attention replayed with new rows in the same buffers."""
    n = 3
    rng = np.random.default_rng(11)
    kc = torch.zeros((8, 16, HKV, D), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks = torch.zeros((8, HKV), dtype=torch.uint8, device="cuda")
    vs = torch.zeros_like(ks)
    q, k, v = (torch.zeros((n, h, D), dtype=torch.bfloat16, device="cuda") for h in (HQ, HKV, HKV))
    pos = torch.zeros(n, dtype=torch.int64, device="cuda")
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    tables = dev(np.array([[0, 3], [5, 1], [2, 7]], np.int32))
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(q)
    out = torch.empty((n, HQ, D), dtype=torch.float32, device="cuda")
    turns = TURNS.cuda()

    def step():
        pkv.rope_kv_append_fp8_block(q, k, v, pos, turns, slots, kc, vc, ks, vs, q_out)
        pkv.paged_decode_attention_fp8_block(q_out, kc, vc, ks, vs, tables, lens, 1, 0.1, out)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    eager = [t.clone() for t in (kc, vc, ks, vs)]
    for t in range(20):
        for x in (q, k, v):
            x.copy_(bf16_dev(R.bf16(rng.standard_normal(x.shape)), torch))
        pos.fill_(t)
        lens.fill_(t + 1)
        slots.copy_(tables[:, t // 16].long() * 16 + t % 16)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        # the same step, eagerly, on its own pools
        e_out = torch.empty_like(out)
        pkv.rope_kv_append_fp8_block(q, k, v, pos, turns, slots, eager[0], eager[1], eager[2],
                                     eager[3], q_out)
        pkv.paged_decode_attention_fp8_block(q_out, *eager, tables, lens, 1, 0.1, e_out)
        torch.cuda.synchronize()
        assert torch.equal(got, e_out)
        assert torch.equal(kc, eager[0]) and torch.equal(vs, eager[3])
