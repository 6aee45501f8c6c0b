"""The forms of the scored attention against attention in 64 bits, with the bounds of
test_gpu_scored.py. A table that is wide enough for long sequences brings the cells and
the merge; a narrow one, where there are few sequences, clusters that join in shared
memory (of one, two, four and eight blocks; with one and two on a multiprocessor)."""
import numpy as np
import pytest

import paged_kv_cache_101_gb300 as pkv
from test_gpu_scored import HEADS, LENGTHS, Batch, slopes_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

WIDE = 6000     # blocks: more than any cluster takes


@pytest.mark.parametrize("fp8,D", [(False, 64), (False, 128), (True, 128)])
@pytest.mark.parametrize("nq,G,Hkv", HEADS)
def test_wide_tables(fp8, D, nq, G, Hkv):
    b = Batch(LENGTHS, nq, G, Hkv, D, fp8, mb=WIDE)
    sl = slopes_of(b.Hq)
    b.check(b.call())
    b.check(b.call(torch.bfloat16, softcap=5.0, slopes=sl), 5.0, sl)


@pytest.mark.parametrize("fp8,D", [(False, 64), (False, 128), (True, 128)])
@pytest.mark.parametrize("nq,G", [(1, 4), (3, 4), (4, 8), (1, 64)])
@pytest.mark.parametrize("lens", [[1500], [1777, 0], [900, 33, 600, 1], [1000, 17] * 3,
                                  [801, 3, 0, 160, 640] * 4])
def test_clusters(fp8, D, nq, G, lens):
    """8 kv heads: 8 to 160 pairs of a sequence and a head."""
    b = Batch(lens, nq, G, 8, D, fp8)
    b.check(b.call())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 16, 17, 112, 113, 224, 225, 449, 897, 1793])
def test_one_head_of_one_sequence(fp8, T):
    """Shares of whole stages: some teams and some CTAs of the cluster have none."""
    b = Batch([T], 2, 4, 1, 128, fp8)
    b.check(b.call())
    b.check(b.call(window=100), 0.0, None, 100)


@pytest.mark.parametrize("fp8", [False, True])
def test_windows_of_more_pairs_than_multiprocessors(fp8):
    lens = [5000, 1100, 70, 0, 2048] * 4
    b = Batch(lens, 2, 2, 8, 128, fp8, window=900)
    b.check(b.call(softcap=30.0, window=900), 30.0, None, 900)


@pytest.mark.parametrize("mb", [None, WIDE])
@pytest.mark.parametrize("fp8", [False, True])
def test_scores_far_apart(fp8, mb):
    b = Batch([300, 77, 1200], 2, 4, 2, 128, fp8, mb=mb)
    sl = -slopes_of(b.Hq) * 4                     # the farthest token is favoured
    b.check(b.call(slopes=sl), 0.0, sl)


@pytest.mark.parametrize("mb", [None, WIDE])
def test_value_scales_far_apart(mb):
    """Shares of one sequence whose value scales are 2^-60 .. 2^40."""
    b = Batch([1400, 90], 1, 4, 2, 128, True, mb=mb)
    b.vs = np.random.default_rng(4).integers(67, 168, b.vs.shape, dtype=np.uint8)
    b.check(b.call())


@pytest.mark.parametrize("mb", [None, WIDE])
@pytest.mark.parametrize("fp8", [False, True])
def test_pages_outside_the_pool(fp8, mb):
    b = Batch([700, 40], 1, 4, 2, 128, fp8, mb=mb)
    b.tables[0, 2] = len(b.kc)
    b.tables[0, 40] = -2
    b.tables[1, 0] = 2 ** 31 - 1
    ws = torch.zeros(pkv.workspace_size_scored(2, 1, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out = b.call(ws=ws)
    assert pkv.workspace_error(ws) == 8
    zero = np.zeros((1,) + b.kc.shape[1:], b.kc.dtype)
    b.kc, b.vc = np.concatenate([b.kc, zero]), np.concatenate([b.vc, zero])
    if fp8:
        byte = np.full((1, 2), 100, np.uint8)
        b.ks, b.vs = np.concatenate([b.ks, byte]), np.concatenate([b.vs, byte])
    b.tables[0, 2] = b.tables[0, 40] = b.tables[1, 0] = len(b.kc) - 1
    b.check(out)


@pytest.mark.parametrize("mb", [None, WIDE])
def test_a_row_that_is_not_a_number_stays_alone(mb):
    """A NaN in one query row reaches that row's outputs only."""
    b = Batch([800, 90], 1, 4, 2, 128, False, mb=mb)
    clean = b.call()
    b.q = b.q.copy()
    b.q[0, 5] = 0x7FC0
    out = b.call()
    assert torch.isnan(out[0, 5]).all()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 5] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("mb", [None, WIDE])
def test_captured_beside_eager_calls(mb):
    """Two graphs and eager calls on two streams, each with its own workspace."""
    bs = [Batch([1200, 40], 1, 4, 4, 128, True, seed=i, mb=mb) for i in range(2)]
    want = [b.call() for b in bs]
    size = pkv.workspace_size_scored(2, 1, 16, 4, 128)
    graphs, outs, held = [], [], []
    for b in bs:
        q, kc, vc, bt, cl, ks, vs = b.device()
        out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        args = (q, kc, vc, ks, vs, bt, cl, 1, b.scale, out, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_decode_attention_fp8_block(*args)
        graphs.append(g)
        outs.append(out)
        held.append(args)
    side = torch.cuda.Stream()
    for _ in range(20):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    again = [b.call() for b in bs]
    torch.cuda.synchronize()
    for w, o, a in zip(want, outs, again):
        assert torch.equal(w, o) and torch.equal(w, a)


@pytest.mark.parametrize("mb", [None, WIDE])
@pytest.mark.parametrize("nq,G", [(1, 4), (4, 8)])
def test_a_small_workspace_is_refused_in_every_form(nq, G, mb):
    b = Batch([300, 40], nq, G, 4, 128, True, mb=mb)
    size = pkv.workspace_size_scored(2, nq, 4 * G, 4, 128)
    b.check(b.call(ws=torch.zeros(size, dtype=torch.uint8, device="cuda")))
    with pytest.raises(pkv.PkvError):
        b.call(ws=torch.zeros(size - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("nq,G", [(1, 4), (4, 8)])
def test_short_sequences_with_a_cell_each(nq, G):
    """More pairs of a sequence and a head than clusters take, up to 32 blocks, none and one."""
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 500, 80)
    lens[:3] = 0, 1, 512
    b = Batch(lens, nq, G, 8, 128, True)
    b.check(b.call())
    sl = slopes_of(b.Hq)
    b.check(b.call(torch.bfloat16, softcap=20.0, slopes=sl), 20.0, sl)
    bb = Batch(lens, nq, G, 8, 64, False)
    bb.check(bb.call())


def test_rows_behind_the_batch_stay():
    """Nothing is written behind the last row, in any form."""
    for mb in (None, WIDE):
        for lens in ([700, 33], [900] * 3, list(range(0, 400, 5))):
            b = Batch(lens, 1, 4, 8, 128, True, mb=mb)
            q, kc, vc, bt, cl, ks, vs = b.device()
            n = q.shape[0]
            out = torch.full((n + 8,) + tuple(q.shape[1:]), 7.0, dtype=torch.float32, device="cuda")
            pkv.paged_decode_attention_fp8_block(q, kc, vc, ks, vs, bt, cl, 1, b.scale, out[:n])
            torch.cuda.synchronize()
            assert (out[n:] == 7.0).all()
            b.check(out[:n])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,G,S,top", [(1, 4, 170, 128), (1, 2, 470, 256), (4, 8, 125, 500)])
def test_cells_of_several_short_sequences(fp8, nq, G, S, top):
    """More pairs of a sequence and a head group than cells; empty ones, runs of them, and
    single long ones among tiny ones."""
    rng = np.random.default_rng(S)
    lens = rng.integers(0, top + 1, S)
    lens[rng.integers(0, S, S // 5)] = 0
    lens[:4] = 0, 0, top, 1
    lens[-3:] = top, 0, 0
    for ls in (lens, np.where(np.arange(S) % 40 == 7, top, np.minimum(lens, 3))):
        b = Batch(ls, nq, G, 8, 128, fp8)
        b.check(b.call())
    b = Batch(np.zeros(S, int), nq, G, 8, 128, fp8)
    assert not b.call().any()
    one = np.zeros(S, int)
    one[S // 2] = top
    b = Batch(one, nq, G, 8, 128, fp8)
    b.check(b.call())
