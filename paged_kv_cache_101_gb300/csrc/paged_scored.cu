// paged_scored.cu -- paged decode attention with capped scores, a distance bias or
// a sliding window, over bf16 or block-scaled E4M3 pools.
//
// Mathematics. For query j of a sequence of T tokens at position p = T - nq + j,
//   x_t = cap(scale <q, k_t>) + slope (t - p),  out = sum_t 2^(y_t - m) v_t / sum_t 2^(y_t - m),
// y = x log2(e), over p - window < t <= p, with a running maximum m (raised only when
// a score passes it by more than a fixed lead; exact, since the sum uses the same m).
// cap(z) = c tanh(z / c) = c (1 - 2 / (1 + 2^(2 z log2(e) / c))): one ex2 and one
// reciprocal, absolute error 2^-22 c.
//
// Work. One unit is a 16-token block of a group of HG kv heads. Three forms, by rules on
// the sizes that plan_scored explains:
//  - cut: the units of all sequences (from the first block that any of the sequence's
//    windows touches) lie end to end, and the persistent grid cuts them into equal
//    cells. A sequence inside one cell is finished in place; one cut by a cell's border
//    leaves its partials (m, l, acc) in the workspace for the merge kernel;
//  - whole: a cell is a sequence of a head group, or as many as an equal share comes to;
//  - joined: a cluster of CTAs has a sequence and a kv head (scored_join_kernel).
// All depend on the sizes only, so results are deterministic.
//
// Staging. A producer warp brings whole blocks of the group's heads by TMA (one box
// for K, one for V: whole rows of the pool, contiguous where HG is all heads) into a
// ring of shared-memory stages; the other warps consume, one kv head each (two or
// four warps a head above 16 rows).
//
// Bounds. Up to 8 rows a head: HBM where the context is long, else what stands around the
// stream (lengths, tables and first blocks, three trips to memory one after the other; the
// merge's launch and three more): about 12 us a call. E4M3, 8 kv heads, 4 rows on one GB300:
// 8 sequences of 32768 to 131072 tokens 196 us, 6.73 TB/s, 99% of the measured copy
// bandwidth; 64 of 512 to 4096 46.4 us, 74%; one of 333 7.3 us (joined). bf16, capped, 64 of
// 512 to 4096: 75.3 us, 91%. At 32 rows a head the consumers' instructions: 128 sequences of
// 256 to 4096 tokens 116 us, 3.3 TB/s, issue slots 51%, ALU 45%, tensor pipe 38% busy.
//
// E4M3 pools. Codes become f16 (exact) on their way from shared memory to the tensor
// cores. (mma.sync takes E4M3 operands too, but on sm_103a the compiler turns that
// into the same conversions for every product and fp32 additions: 661 warp
// instructions for two blocks of a head with 4 rows against about half of it here.)
// A query row is scaled by a power of two and held in f16: bf16's 8 significant bits
// fit, so only elements below 2^-28 of the row's largest lose bits. A softmax weight,
// times its block's value scale over the row's largest so far, is held in f16
// (relative error at most 2^-11, steps of 2^-31 of the largest weight for the
// smallest). A block's key scale multiplies its scores.
//
// Order. A segment's blocks are taken from the newest to the oldest: weights tend to
// fall with distance (a distance bias makes sure of it), so the running maximum
// settles at once instead of rising all along.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "pkv_cells.cuh"
#include "pkv_common.cuh"
#include "pkv_ops_internal.h"

namespace pkv {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// Blocks of a stage. A wait for a barrier that has long completed costs a warp 83 cycles,
// and as much again goes into headers and hand-backs: E4M3 blocks come in pairs (two bf16
// blocks would leave too few stages).
constexpr __host__ __device__ int stage_blocks(bool fp8) { return fp8 ? 2 : 1; }

// One stage's n blocks b, b - 1: their sequence, what part they play in its segment (F_*),
// and the scale bytes of their heads.
struct Header {
    int32_t s, b, T, hg;
    int32_t flags, cell, slot, n;
    uint8_t ks[2][8], vs[2][8];
};
static_assert(sizeof(Header) == 64, "four 16-byte words");

// A team's ring, and which of all cells is the team's.
struct Ring {
    uint8_t *stages;
    Header *hdr;
    uint64_t *full, *empty;
    int cell;
};


__device__ __forceinline__ Ring carve(uint8_t *raw, const ScoredParams &p, int rings, int team)
{
    const DecodeParams &d = p.d;
    uint8_t *base = raw + (-smem_u32(raw) & 1023u);  // (as an offset: it stays a shared address)
    const int all = rings * d.nst, mine = team * d.nst;
    Ring r;
    r.stages = base + size_t(mine) * d.stage_bytes;
    r.hdr = reinterpret_cast<Header *>(base + size_t(all) * d.stage_bytes) + mine;
    r.full = reinterpret_cast<uint64_t *>(base + size_t(all) * (d.stage_bytes + sizeof(Header))) +
             2 * mine;
    r.empty = r.full + d.nst;
    r.cell = team * int(gridDim.x) + int(blockIdx.x);
    return r;
}

// The queries of the teams' consumer warps, behind the rings.
__device__ __forceinline__ uint8_t *query_fragments(uint8_t *raw, const ScoredParams &p, int rings)
{
    return raw + (-smem_u32(raw) & 1023u) +
           size_t(rings * p.d.nst) * (p.d.stage_bytes + sizeof(Header) + 16);
}

// Position in the ring.
struct Turn {
    uint32_t st = 0, phase = 0;
    __device__ __forceinline__ void next(int nst)
    {
        if (++st == uint32_t(nst)) {
            st = 0;
            phase ^= 1u;
        }
    }
};

struct Span {
    int T;   // tokens (clamped to the table)
    int b0;  // first block that a query's window touches
    int nb;  // blocks from there (taken from the last to the first)
};

__device__ __forceinline__ int first_seen(const ScoredParams &p, int T)
{
    const int f = T - p.d.nq - p.window + 1;
    return p.window > 0 && f > 0 ? f : 0;
}

__device__ __forceinline__ Span span(const ScoredParams &p, int s)
{
    Span r;
    r.T = seq_tokens(p.d, s);
    r.b0 = first_seen(p, r.T) / kBlockSize;
    r.nb = (r.T + kBlockSize - 1) / kBlockSize - r.b0;
    return r;
}

// What a CTA of a cluster (the joined form) takes: stages' worth [lo, hi) of the blocks of
// sequence s and head h, counted from the newest.
struct Share {
    int s, h, rank, lo, hi;
    Span sp;
};

template <bool FP8>
__device__ __forceinline__ Share share(const ScoredParams &p)
{
    constexpr int BL = stage_blocks(FP8);
    Share h;
    const int id = int(blockIdx.x) / p.cluster;
    h.rank = int(blockIdx.x) - id * p.cluster;
    h.h = id / p.d.S;
    h.s = id - h.h * p.d.S;
    h.sp = span(p, h.s);
    const int n = (h.sp.nb + BL - 1) / BL;
    h.lo = int(int64_t(n) * h.rank / p.cluster);
    h.hi = int(int64_t(n) * (h.rank + 1) / p.cluster);
    return h;
}

// 2^e; 0 below the normal range.
__device__ __forceinline__ float two_to(int e)
{
    return e < -126 ? 0.f : __uint_as_float(uint32_t(e + 127) << 23);
}

// ------------------------------------------------------------------ producer
// The blocks of a segment from the newest down, 32 at a time, a lane each: table entries
// and, for block-scaled pools, their heads' scale bytes. The batch behind the current one
// is on its way: its entries are asked for when the current batch starts, its scales (they
// need the entries) when half of that is used. An entry outside the pool is flagged and
// becomes the block past the pool's end, which TMA reads as zeros (the smallest scale).
template <bool FP8>
struct Blocks {
    int tab = -1, phys = 0;             // lane l: block tab - l
    uint2 ks, vs;
    int next_tab = -1, next_phys = 0;   // the batch behind it (-1: none)
    uint2 next_ks, next_vs;
    bool scaled = false;                // has next its scales?

    __device__ __forceinline__ int entry(const ScoredParams &p, int s, int top, int b0, int lane)
    {
        return top - lane >= b0 ? __ldg(p.d.block_tables + int64_t(s) * p.d.MB + top - lane) : 0;
    }
    __device__ __forceinline__ void scales(const ScoredParams &p, int hg, int &id, uint2 &k, uint2 &v)
    {
        const DecodeParams &d = p.d;
        if (id < 0 || id >= d.num_blocks) {
            atomicOr(d.ws + kWsErr, kErrBadBlock);
            id = int(d.num_blocks);
        }
        if (!FP8)
            return;
        k = v = make_uint2(0x01010101u, 0x01010101u);
        if (id >= d.num_blocks)
            return;
        const int64_t at = int64_t(id) * d.Hkv + hg * d.HG;
        const uint8_t *kp = p.k_scale + at, *vp = p.v_scale + at;
        if (p.scale_vec && d.HG == 8) {
            k = __ldg(reinterpret_cast<const uint2 *>(kp));
            v = __ldg(reinterpret_cast<const uint2 *>(vp));
        } else if (p.scale_vec && d.HG == 4) {
            k.x = __ldg(reinterpret_cast<const uint32_t *>(kp));
            v.x = __ldg(reinterpret_cast<const uint32_t *>(vp));
        } else if (p.scale_vec && d.HG == 2) {
            k.x = __ldg(reinterpret_cast<const uint16_t *>(kp));
            v.x = __ldg(reinterpret_cast<const uint16_t *>(vp));
        } else {
            uint32_t kb[8], vb[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                kb[h] = h < d.HG ? __ldg(kp + h) : 0u;
                vb[h] = h < d.HG ? __ldg(vp + h) : 0u;
            }
            k = make_uint2(kb[0] | kb[1] << 8 | kb[2] << 16 | kb[3] << 24,
                           kb[4] | kb[5] << 8 | kb[6] << 16 | kb[7] << 24);
            v = make_uint2(vb[0] | vb[1] << 8 | vb[2] << 16 | vb[3] << 24,
                           vb[4] | vb[5] << 8 | vb[6] << 16 | vb[7] << 24);
        }
    }
    // another segment
    __device__ __forceinline__ void reset() { tab = next_tab = -1; }
    // blocks b .. b - n + 1 are the next ones taken (all n before them were the same)
    __device__ __forceinline__ void reach(const ScoredParams &p, int s, int hg, int b, int n,
                                          int b0, int lane)
    {
        if (tab < 0 || b - n < tab - 32) {
            if (next_tab == b) {
                if (!scaled)
                    scales(p, hg, next_phys, next_ks, next_vs);
                phys = next_phys;
                ks = next_ks;
                vs = next_vs;
            } else {
                phys = entry(p, s, b, b0, lane);
                scales(p, hg, phys, ks, vs);
            }
            tab = b;
            next_tab = tab - 32 >= b0 ? tab - 32 : -1;
            scaled = false;
            if (next_tab >= 0)
                next_phys = entry(p, s, next_tab, b0, lane);
        } else if (next_tab >= 0 && !scaled && b <= tab - 16) {
            scales(p, hg, next_phys, next_ks, next_vs);
            scaled = true;
        }
    }
};

template <bool FP8>
__device__ void producer(const CUtensorMap *kmap, const CUtensorMap *vmap, const ScoredParams &p,
                         const Ring &ring, int lane)
{
    constexpr int BL = stage_blocks(FP8);
    const DecodeParams &d = p.d;
    const int S = d.S;
    int64_t total = 0;
    if (p.whole != kOwnCells) {
#pragma unroll 8
        for (int s = lane; s < S; s += 32)
            total += span(p, s).nb;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            total += __shfl_xor_sync(kFull, total, o);
    }
    Cells C;
    C.F = C.F1 = int64_t(d.n_hg) * total;
    C.F2 = 0;
    C.G = p.cells;
    C.NT = 0;
    if (ring.cell == 0 && lane == 0 && !p.whole) {
        d.ws[kWsUnits] = uint32_t(total);
        d.ws[kWsDense] = C.F >= C.G ? 1u : 0u;
    }
    int64_t a, e;
    if (p.whole == kOwnCells) {
        a = 0;
        e = ring.cell < p.cells ? span(p, ring.cell % S).nb : 0;
    } else {
        a = C.start(ring.cell);
        e = C.start(int64_t(ring.cell) + 1);
    }
    Turn turn;
    uint32_t issued = 0;
    bool ok = true;

    // wait until the next stage is free
    auto acquire = [&]() -> bool {
        if (issued < uint32_t(d.nst))
            return true;
        int w = 1;
        if (lane == 0)
            w = mbar_wait(smem_u32(&ring.empty[turn.st]), turn.phase ^ 1u, kWaitLimitNs);
        return __shfl_sync(kFull, w, 0) != 0;
    };

    if (a < e) {
        int hg, s = 0, b = 0;
        if (p.whole == kOwnCells) {
            hg = ring.cell / S;
            s = ring.cell - hg * S;
        } else {
            // the sequence that holds unit `rest` of its head group
            hg = int(a / total);
            int64_t rest = a - int64_t(hg) * total;
            for (int s0 = 0; s0 < S; s0 += 32) {
                const int mine = s0 + lane < S ? span(p, s0 + lane).nb : 0;
                int64_t incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t v = __shfl_up_sync(kFull, incl, o);
                    if (lane >= o)
                        incl += v;
                }
                const unsigned past = __ballot_sync(kFull, incl > rest);
                if (past) {
                    const int src = __ffs(past) - 1;
                    s = s0 + src;
                    b = int(rest - __shfl_sync(kFull, incl - mine, src));
                    break;
                }
                rest -= __shfl_sync(kFull, incl, 31);
            }
        }
        Span sp = span(p, s);
        const auto next_sequence = [&] {
            do {
                if (++s == S) {
                    s = 0;
                    ++hg;
                }
                sp = span(p, s);
            } while (sp.nb == 0);
        };
        // borders inside a sequence move to its start or, from the middle on, to its end
        const auto end_at_border = [&](int64_t u) {
            if (p.whole == kRoundedCells && u < e && u + sp.nb > e)
                e = 2 * (e - u) >= sp.nb ? u + sp.nb : u;
        };
        if (p.whole == kRoundedCells && b > 0) {
            a += 2 * b >= sp.nb ? sp.nb - b : -b;
            if (2 * b >= sp.nb && a < e)
                next_sequence();
            b = 0;
        }
        end_at_border(a);
        b = sp.b0 + sp.nb - 1 - b;  // the newest block comes first
        const uint64_t policy = policy_evict_first();
        bool opens = true;        // no segment of this cell ended yet
        bool from_top = false;    // the segment opens its sequence
        Blocks<FP8> blk;
        for (int64_t u = a; u < e;) {
            const int b_top = sp.b0 + sp.nb - 1;
            const int n = BL == 2 && u + 1 < e && b > sp.b0 ? 2 : 1;
            blk.reach(p, s, hg, b, n, sp.b0, lane);
            const int src = blk.tab - b;
            int block[BL];
            uint2 ks[BL], vs[BL];
#pragma unroll
            for (int k = 0; k < BL; ++k) {
                block[k] = __shfl_sync(kFull, blk.phys, src + k);
                if (FP8) {
                    ks[k].x = __shfl_sync(kFull, blk.ks.x, src + k);
                    ks[k].y = __shfl_sync(kFull, blk.ks.y, src + k);
                    vs[k].x = __shfl_sync(kFull, blk.vs.x, src + k);
                    vs[k].y = __shfl_sync(kFull, blk.vs.y, src + k);
                }
            }
            const bool first = u == a || b == b_top;
            if (first)
                from_top = b == b_top;
            const bool ends = b - n < sp.b0, last = u + n == e || ends;
            if (!(ok = acquire()))
                break;
            if (lane == 0) {
                // the merge's record: cell (and slot) of the sequence's first piece,
                // cell of its last
                if (!p.whole) {
                    int2 *rec = d.pieces + int64_t(s) * d.n_hg + hg;
                    if (b == b_top)
                        rec->x = ring.cell * 2 + (opens ? 0 : 1);
                    if (ends)
                        rec->y = ring.cell;
                }
                const int flags = (first ? F_FIRST : 0) | (last ? F_LAST : 0) |
                                  (ends && from_top ? F_DIRECT : 0);
                uint4 *h = reinterpret_cast<uint4 *>(&ring.hdr[turn.st]);
                h[0] = make_uint4(s, b, sp.T, hg);
                h[1] = make_uint4(flags, ring.cell, opens ? 0 : 1, n);
                if constexpr (FP8) {
                    h[2] = make_uint4(ks[0].x, ks[0].y, ks[1].x, ks[1].y);
                    h[3] = make_uint4(vs[0].x, vs[0].y, vs[1].x, vs[1].y);
                }
                const uint32_t bytes = uint32_t(d.stage_bytes / BL);
                const uint32_t bar = smem_u32(&ring.full[turn.st]);
                mbar_arrive_expect_tx(bar, uint32_t(n) * bytes);
                uint32_t dst = smem_u32(ring.stages) + turn.st * uint32_t(d.stage_bytes);
#pragma unroll
                for (int k = 0; k < BL; ++k, dst += bytes)
                    if (k < n) {
                        tma_load_5d_hint(dst, kmap, bar, 0, 0, 0, hg * d.HG, block[k], policy);
                        tma_load_5d_hint(dst + bytes / 2, vmap, bar, 0, 0, 0, hg * d.HG, block[k],
                                         policy);
                    }
            }
            __syncwarp();
            ++issued;
            turn.next(d.nst);
            u += n;
            b -= n;
            if (last)
                opens = false;
            if (b < sp.b0 && u < e) {
                next_sequence();
                end_at_border(u);
                b = sp.b0 + sp.nb - 1;
                blk.reset();
            }
        }
    }
    if (ok && (ok = acquire()) && lane == 0) {
        ring.hdr[turn.st].flags = F_END;
        mbar_arrive(smem_u32(&ring.full[turn.st]));
    }
    if (!ok && lane == 0) {
        atomicOr(d.ws + kWsErr, kErrProducerWait);
        // wait (bounded) for every copy that may still be in flight
        const uint32_t n = issued < uint32_t(d.nst) ? issued : uint32_t(d.nst);
        for (uint32_t k = 0; k < n; ++k) {
            if (turn.st == 0) {
                turn.st = uint32_t(d.nst);
                turn.phase ^= 1u;
            }
            --turn.st;
            if (!mbar_wait(smem_u32(&ring.full[turn.st]), turn.phase, kWaitLimitNs))
                atomicOr(d.ws + kWsErr, kErrDrainWait);
        }
    }
}

// The joined form's producer: lane t has the stages of team t, so that a turn of all teams
// costs one stage's instructions. A turn's table entries are asked for two turns ahead, the
// scale bytes that they point to one turn ahead.
template <bool FP8>
__device__ void produce_share(const CUtensorMap *kmap, const CUtensorMap *vmap,
                              const ScoredParams &p, const Ring &ring, const Share &part, int lane)
{
    constexpr int BL = stage_blocks(FP8);
    const DecodeParams &d = p.d;
    const int T = p.teams, n = part.hi - part.lo;
    const int32_t *table = d.block_tables + int64_t(part.s) * d.MB;
    const int top = part.sp.b0 + part.sp.nb - 1 - part.lo * BL;  // the share's newest block
    const uint64_t policy = policy_evict_first();
    const bool works = lane < T;
    const uint32_t bytes = uint32_t(d.stage_bytes / BL);
    int id[BL], id2[BL];
    uint32_t ks[BL], vs[BL];

    // blocks of stage i: top - BL i and the one before it
    const auto entries = [&](int i, int (&e)[BL]) {
#pragma unroll
        for (int k = 0; k < BL; ++k) {
            const int b = top - BL * i - k;
            e[k] = works && i < n && b >= part.sp.b0 ? __ldg(table + b) : 0;
        }
    };
    const auto scales = [&](int (&e)[BL]) {
#pragma unroll
        for (int k = 0; k < BL; ++k) {
            ks[k] = vs[k] = 1u;
            if (e[k] < 0 || e[k] >= d.num_blocks) {
                atomicOr(d.ws + kWsErr, kErrBadBlock);
                e[k] = int(d.num_blocks);  // past the tensor's end: zeros
            } else if (FP8) {
                const int64_t at = int64_t(e[k]) * d.Hkv + part.h;
                ks[k] = __ldg(p.k_scale + at);
                vs[k] = __ldg(p.v_scale + at);
            }
        }
    };
    entries(lane, id);
    entries(lane + T, id2);
    scales(id);
    const int depth = d.nst / T;  // turns in the ring
    int slot = 0;                 // of this turn
    uint32_t phase = 0;
    bool ok = true;
    int turn = 0;
    for (int i = lane; i - lane < n; i += T, ++turn) {
        const bool mine = works && i < n;
        const int st = slot * T + lane;
        if (mine && turn >= depth)
            ok = mbar_wait(smem_u32(&ring.empty[st]), phase ^ 1u, kWaitLimitNs);
        if (!__all_sync(kFull, ok)) {
            ok = false;
            break;
        }
        if (mine) {
            const uint32_t bar = smem_u32(&ring.full[st]);
            const int b = top - BL * i, nb = b - part.sp.b0 + 1 < BL ? b - part.sp.b0 + 1 : BL;
            uint4 *h = reinterpret_cast<uint4 *>(&ring.hdr[st]);
            h[0] = make_uint4(part.s, b, part.sp.T, part.h);
            h[1] = make_uint4((turn == 0 ? F_FIRST : 0) | (i + T >= n ? F_LAST : 0), 0, 0, nb);
            if constexpr (FP8) {
                h[2] = make_uint4(ks[0], 0, ks[BL - 1], 0);
                h[3] = make_uint4(vs[0], 0, vs[BL - 1], 0);
            }
            mbar_arrive_expect_tx(bar, uint32_t(nb) * bytes);
            uint32_t dst = smem_u32(ring.stages) + uint32_t(st) * uint32_t(d.stage_bytes);
#pragma unroll
            for (int k = 0; k < BL; ++k, dst += bytes)
                if (k < nb) {
                    tma_load_5d_hint(dst, kmap, bar, 0, 0, 0, part.h, id[k], policy);
                    tma_load_5d_hint(dst + bytes / 2, vmap, bar, 0, 0, 0, part.h, id[k], policy);
                }
        }
#pragma unroll
        for (int k = 0; k < BL; ++k)
            id[k] = id2[k];
        entries(i + 2 * T, id2);
        scales(id);
        if (++slot == depth) {
            slot = 0;
            phase ^= 1u;
        }
    }
    if (!ok && works) {
        if (lane == 0)
            atomicOr(d.ws + kWsErr, kErrProducerWait);
        // wait (bounded) for every copy that may still be in flight: the lane's stages of the
        // last `depth` turns
        for (int k = 0; k < depth && k < turn; ++k) {
            if (slot == 0) {
                slot = depth;
                phase ^= 1u;
            }
            --slot;
            if (lane + (turn - 1 - k) * T < n &&
                !mbar_wait(smem_u32(&ring.full[slot * T + lane]), phase, kWaitLimitNs))
                atomicOr(d.ws + kWsErr, kErrDrainWait);
        }
    }
}

// ------------------------------------------------------------------ consumers
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 of what a weight may reach before the running maximum is raised
constexpr float kLead = 8.f;
// E4M3: weights are scaled by 2^6 (at most 2^14 with the lead; f16 ends at 2^16)
constexpr int kWeightBits = 6;

// Sequence id % S of head group id / S, where it has no token: zeros for its heads.
template <int D>
__device__ __forceinline__ void clear_empty(const ScoredParams &p, int64_t id, int tid, int threads)
{
    const DecodeParams &d = p.d;
    const int hg = int(id / d.S), s = int(id - int64_t(hg) * d.S);
    if (seq_tokens(d, s) > 0)
        return;
    const int row = d.HG * d.G * D / (d.out_f32 ? 4 : 8);  // 16-byte words
    for (int e = tid; e < d.nq * row; e += threads) {
        const int j = e / row;
        static_cast<uint4 *>(d.out)[((int64_t(s) * d.nq + j) * d.n_hg + hg) * row + e - j * row] =
            make_uint4(0, 0, 0, 0);
    }
}

// Partials of the joined form: (m, l) and output sums of row r of team t at t rows_pad + r.
struct Partials {
    float2 *ml;
    float *acc;
    // floats of a row: four more than the head, so that a warp's stores meet no bank twice
    template <int D>
    static __device__ __forceinline__ constexpr int stride()
    {
        return D + 4;
    }
};

// The rows of a warp: NT n-tiles of 8, a lane holding rows 2 tq and 2 tq + 1 of each,
// tokens g and g + 8 of each of up to BL blocks.
// Above 16 rows a head takes several warps (WPH) of 16 rows. Those wait for their own
// results most of the time (with 8 warps on an SM the issue slots were 38% busy, the tensor
// cores 26%), so an SM has twelve of them (128 sequences x 4 queries: 166.6 -> 137.8 us, and
// 116 since), in teams of up to four with a ring, a producer
// warp and a cell each. The registers for that come from the producers (setmaxnreg) and
// from the queries, which a warp keeps in shared memory.
constexpr __host__ __device__ bool teams_of(int wph) { return wph > 1; }
constexpr int kTeamWarps = 12, kMaxTeams = 4, kMaxCluster = 8;
constexpr int kTeamThreads = 32 * (kTeamWarps + kMaxTeams);
constexpr int kLaunchRegs = 128, kConsumerRegs = 144, kProducerRegs = 80;
static_assert(kTeamWarps * kConsumerRegs + kMaxTeams * kProducerRegs <=
                  (kTeamWarps + kMaxTeams) * kLaunchRegs,
              "a block shares out the registers that it was launched with");

template <int D, bool FP8, int NT, int WPH, bool JOIN>
__device__ void consumer(const ScoredParams &p, const Ring &ring, int cw, int lane, uint8_t *qs,
                         int team, const Partials &joins)
{
    constexpr bool QS = teams_of(WPH);  // queries in shared memory
    constexpr int RL = 2 * NT;       // rows of a lane
    constexpr int BL = stage_blocks(FP8);  // two chains hide each other's waits
    constexpr int NH = FP8 ? 1 : D / 64;
    constexpr int KS = D / 16;       // k-steps of the scores
    constexpr int MT = D / 16;       // 16-dim m-tiles of the output
    const DecodeParams &d = p.d;
    const int hl = cw / WPH, r0 = (cw % WPH) * 8 * NT;
    const int g = lane >> 2, tq = lane & 3;
    // ldmatrix rows inside a [16 tokens][8 x 16 bytes] tile, 128-byte swizzle: where the lane
    // finds chunk 0 or 1; chunks 2i or 2i + 1 are at that address ^ 32 i
    const int k_tok = (lane & 7) + ((lane >> 3) & 1) * 8, k_chunk = lane >> 4;
    const int v_tok = (lane & 7) + ((lane >> 4) & 1) * 8, v_chunk = (lane >> 3) & 1;
    const int sw = lane & 7;
    const uint32_t k_at = smem_u32(ring.stages) + uint32_t(hl * NH * kTileBytes + k_tok * 128 +
                                                           ((k_chunk ^ sw) << 4));
    const uint32_t v_at =
        smem_u32(ring.stages) +
        uint32_t((d.HG + hl) * NH * kTileBytes + v_tok * 128 + ((v_chunk ^ sw) << 4));
    const uint32_t block_bytes = uint32_t(2 * d.HG * NH * kTileBytes);

    uint32_t qf[NT][QS ? 1 : KS][2];
    float acc[MT][NT][4];
    float m_r[RL], l_r[RL], mul[RL], slope[RL];
    int row_j[RL];  // query index of each row (the last one for rows past the end)
    int e_max = 0;  // E4M3: the largest value-scale byte so far
    const auto row_of = [&](int i) { return r0 + 8 * (i >> 1) + 2 * tq + (i & 1); };
#pragma unroll
    for (int i = 0; i < RL; ++i) {
        const int j = row_of(i) / d.G;
        row_j[i] = j < d.nq ? j : d.nq - 1;
        slope[i] = 0.f;
        mul[i] = p.mul;
    }
    Turn turn;
    if (JOIN)
        turn.st = uint32_t(team);
    for (;;) {
        if (!mbar_wait(smem_u32(&ring.full[turn.st]), turn.phase, kWaitLimitNs)) {
            if (lane == 0)
                atomicOr(d.ws + kWsErr, kErrConsumerWait);
            return;
        }
        const Header *h = &ring.hdr[turn.st];
        const int flags = h->flags;
        if (flags & F_END)
            break;
        const int s = h->s, T = h->T, blk = h->b, kvh = h->hg * d.HG + hl;
        const bool two = BL == 2 && h->n == 2;
        const int e_cell = h->cell, e_slot = h->slot;

        if (flags & F_FIRST) {
            // ---- a new segment: empty state, its queries
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                m_r[i] = -INFINITY;
                l_r[i] = 0.f;
                if (p.slopes) {
                    const int row = row_of(i), j = row / d.G;
                    slope[i] = row < d.rows ? __ldg(p.slopes + kvh * d.G + row - j * d.G) *
                                                  1.4426950408889634f
                                            : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[i][nt][c] = 0.f;
            e_max = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = r0 + 8 * nt + g;  // column g of the tile
                const int j = row / d.G;
                const bool valid = row < d.rows;
                const uint16_t *q =
                    d.q + ((int64_t(s) * d.nq + j) * d.Hq + int64_t(kvh) * d.G + row - j * d.G) * D;
                uint32_t qw[KS][2];
                if constexpr (FP8) {
                    // k-step ks is 16-byte chunk ks of a code row: lane tq holds dims
                    // 16 ks + 4 tq .. + 3 (k 2tq, 2tq + 1, 2tq + 8, 2tq + 9)
                    float top = 0.f;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const uint2 w = valid ? __ldg(reinterpret_cast<const uint2 *>(
                                                    q + 16 * ks + 4 * tq))
                                              : make_uint2(0, 0);
                        qw[ks][0] = w.x;
                        qw[ks][1] = w.y;
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16lo_f32(w.x)), fabsf(bf16hi_f32(w.x))),
                                               fmaxf(fabsf(bf16lo_f32(w.y)), fabsf(bf16hi_f32(w.y)))));
                    }
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
                    // the row's largest element comes to 2^14 .. 2^15
                    int e = int(__float_as_uint(top) >> 23) - 127 - 14;
                    e = top == 0.f ? 0 : max(e, -119);
                    const float f = two_to(-e);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            qw[ks][c] =
                                pack_f16x2(bf16lo_f32(qw[ks][c]) * f, bf16hi_f32(qw[ks][c]) * f);
                    // the factors of the lane's own rows; not a number where a row holds an
                    // infinity (its products overflow f16)
                    const float back = e > 113 ? NAN : two_to(e);
                    mul[2 * nt] = p.mul * __shfl_sync(kFull, back, 8 * tq);
                    mul[2 * nt + 1] = p.mul * __shfl_sync(kFull, back, 8 * tq + 4);
                } else {
                    const uint32_t *w = reinterpret_cast<const uint32_t *>(q);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        qw[ks][0] = valid ? __ldg(w + ks * 8 + tq) : 0u;
                        qw[ks][1] = valid ? __ldg(w + ks * 8 + 4 + tq) : 0u;
                    }
                }
                if constexpr (QS) {
                    // (every lane reads back its own words)
#pragma unroll
                    for (int i = 0; i < KS / 2; ++i)
                        reinterpret_cast<uint4 *>(qs)[(i * NT + nt) * 32 + lane] = make_uint4(
                            qw[2 * i][0], qw[2 * i][1], qw[2 * i + 1][0], qw[2 * i + 1][1]);
                } else {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            qf[nt][ks][c] = qw[ks][c];
                }
            }
        }

        // ---- scores S^T[token][row] (of whatever is there, where a second block is missing:
        //      those are masked below)
        float sc[BL][NT][4];
        const uint32_t stage = turn.st * uint32_t(d.stage_bytes);
#pragma unroll
        for (int k = 0; k < BL; ++k) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    sc[k][nt][c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {  // k-steps 2i, 2i + 1
            uint32_t b[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if constexpr (QS) {
                    const uint4 w = reinterpret_cast<const uint4 *>(qs)[(i * NT + nt) * 32 + lane];
                    b[nt][0] = w.x;
                    b[nt][1] = w.y;
                    b[nt][2] = w.z;
                    b[nt][3] = w.w;
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        b[nt][c] = qf[nt][2 * i + (c >> 1)][c & 1];
                }
            }
#pragma unroll
            for (int k = 0; k < BL; ++k) {
                uint32_t a0[4], a1[4];
                if constexpr (FP8) {
                    // one ldmatrix brings chunks 2i and 2i + 1 of all 16 tokens
                    uint32_t r[4];
                    ldsm_x4((k_at + stage + k * block_bytes) ^ uint32_t(32 * i), r);
                    e4m3x4_to_f16x2x2(r[0], a0[0], a0[2]);
                    e4m3x4_to_f16x2x2(r[1], a0[1], a0[3]);
                    e4m3x4_to_f16x2x2(r[2], a1[0], a1[2]);
                    e4m3x4_to_f16x2x2(r[3], a1[1], a1[3]);
                } else {
                    const uint32_t at = k_at + stage + uint32_t((i >> 1) * kTileBytes);
                    ldsm_x4(at ^ uint32_t(64 * (i & 1)), a0);
                    ldsm_x4(at ^ uint32_t(64 * (i & 1) + 32), a1);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (FP8) {
                        mma_f16_16816(sc[k][nt], a0, b[nt][0], b[nt][1]);
                        mma_f16_16816(sc[k][nt], a1, b[nt][2], b[nt][3]);
                    } else {
                        mma_bf16_16816(sc[k][nt], a0, b[nt][0], b[nt][1]);
                        mma_bf16_16816(sc[k][nt], a1, b[nt][2], b[nt][3]);
                    }
                }
            }
        }

        // ---- into y = x log2(e): x[k][i][c] is row i, block b - k, token g + 8 c
        float x[BL][RL][2];
        const int t0 = blk * kBlockSize;                          // the newer block
        const int t_low = two ? t0 - kBlockSize : t0;           // the step's first token
        const int first = first_seen(p, T);
        // are all tokens of the step seen by all rows?
        const bool masked = t0 + kBlockSize - 1 > T - d.nq || (p.window > 0 && t_low < T - p.window);
#pragma unroll
        for (int k = 0; k < BL; ++k) {
            const float kf = FP8 ? __uint_as_float(uint32_t(h->ks[k][hl]) << 23) : 1.f;
#pragma unroll
            for (int i = 0; i < RL; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    x[k][i][c] = sc[k][i >> 1][2 * c + (i & 1)] * (FP8 ? kf * mul[i] : mul[i]);
        }
        if (p.cap_log2 > 0.f) {
#pragma unroll
            for (int k = 0; k < BL; ++k)
#pragma unroll
                for (int i = 0; i < RL; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        x[k][i][c] = fmaf(-2.f * p.cap_log2, rcp(1.f + ex2(x[k][i][c])), p.cap_log2);
        }
        if (p.slopes) {
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                const float far = float(t0 + g - (T - d.nq + row_j[i]));
#pragma unroll
                for (int k = 0; k < BL; ++k)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        x[k][i][c] = fmaf(slope[i], far + float(8 * c - 16 * k), x[k][i][c]);
            }
        }
        if (__builtin_expect(masked, 0)) {
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                const int pos = T - d.nq + row_j[i];
                const int low = p.window > 0 ? pos - p.window : -1;  // the last one not seen
#pragma unroll
                for (int k = 0; k < BL; ++k)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int t = t0 - 16 * k + 8 * c + g;
                        if (t > pos || t <= low)
                            x[k][i][c] = -INFINITY;
                    }
            }
        }
        if (BL == 2 && !two) {
#pragma unroll
            for (int i = 0; i < RL; ++i)
                x[BL - 1][i][0] = x[BL - 1][i][1] = -INFINITY;
        }

        // ---- running maximum; the accumulator follows it (and the largest value scale)
        bool lead = false;
        float top[RL];
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            top[i] = fmaxf(x[0][i][0], x[0][i][1]);
            if (BL == 2)
                top[i] = fmaxf(top[i], fmaxf(x[BL - 1][i][0], x[BL - 1][i][1]));
            lead |= top[i] > m_r[i] + kLead;
        }
        int ev[2] = {0, 0}, e_new = 0;
        if constexpr (FP8) {
            ev[0] = h->vs[0][hl];
            ev[1] = two ? h->vs[1][hl] : 0;
            e_new = max(e_max, max(ev[0], ev[1]));
        }
        if (__any_sync(kFull, lead) || e_new > e_max) {
            float corr[RL];
            const float fe = FP8 ? two_to(e_max - e_new) : 1.f;
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                float t = top[i];
                t = fmaxf(t, __shfl_xor_sync(kFull, t, 4));
                t = fmaxf(t, __shfl_xor_sync(kFull, t, 8));
                t = fmaxf(t, __shfl_xor_sync(kFull, t, 16));
                const float mn = fmaxf(m_r[i], t);
                const float c = ex2(m_r[i] - (mn == -INFINITY ? 0.f : mn));
                m_r[i] = mn;
                l_r[i] *= c;
                corr[i] = c * fe;
            }
            e_max = e_new;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[mt][nt][c] *= corr[2 * nt + (c & 1)];
        }
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            const float mu = m_r[i] == -INFINITY ? 0.f : m_r[i];
#pragma unroll
            for (int k = 0; k < BL; ++k)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    x[k][i][c] = ex2(x[k][i][c] - mu);
                    l_r[i] += x[k][i][c];
                }
        }

        // ---- O^T[d][row] += V^T[d][token] P^T[token][row], P transposed into B
        //      fragments: bf16 as hi + lo, f16 (E4M3) with the block's value scale
        uint32_t ph[BL][NT][2], pl[NT][2];
#pragma unroll
        for (int k = 0; k < BL; ++k) {
            const float f = FP8 ? two_to(ev[k] - e_max + kWeightBits) : 1.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float a = x[k][2 * nt][c], bb = x[k][2 * nt + 1][c];
                    if constexpr (FP8) {
                        ph[k][nt][c] = movmatrix_trans(pack_f16x2(a * f, bb * f));
                    } else {
                        const uint32_t hi = pack_bf16x2(a, bb);
                        ph[k][nt][c] = movmatrix_trans(hi);
                        pl[nt][c] = movmatrix_trans(
                            pack_bf16x2(a - bf16lo_f32(hi), bb - bf16hi_f32(hi)));
                    }
                }
        }
        // tokens that no row of the sequence sees are zeroed in V too (stale slots may
        // hold anything)
        const bool edge = t_low < first || t0 + kBlockSize > T;
        auto pv = [&](auto is_edge) {
            constexpr bool EDGE = decltype(is_edge)::value;
#pragma unroll
            for (int k = 0; k < BL; ++k) {
                if (k == 1 && !two)
                    break;
                uint32_t keep[2] = {kFull, kFull};
                if constexpr (EDGE) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int t = t0 - 16 * k + 8 * c + 2 * tq;
                        keep[c] = (t >= first && t < T ? 0x0000ffffu : 0u) |
                                  (t + 1 >= first && t + 1 < T ? 0xffff0000u : 0u);
                    }
                }
                const uint32_t vb = v_at + stage + k * block_bytes;
                if constexpr (FP8) {
                    // chunks 2i and 2i + 1: a lane gets tokens 2tq, 2tq + 1 of the code pair
                    // (dims 2g, 2g + 1). Even dims (bytes 0, 2) make m-tile 2i, odd ones
                    // m-tile 2i + 1; M-rows g + 8 are 16 dims on.
#pragma unroll
                    for (int i = 0; i < MT / 2; ++i) {
                        uint32_t r[4], ae[4], ao[4];
                        ldsm_x4_trans(vb ^ uint32_t(32 * i), r);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            e4m3x4_to_f16x2x2(__byte_perm(r[m], 0u, 0x3120), ae[m], ao[m]);
                            if constexpr (EDGE) {
                                ae[m] &= keep[m >> 1];
                                ao[m] &= keep[m >> 1];
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16_16816(acc[2 * i][nt], ae, ph[k][nt][0], ph[k][nt][1]);
                            mma_f16_16816(acc[2 * i + 1][nt], ao, ph[k][nt][0], ph[k][nt][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t a[4];
                        ldsm_x4_trans((vb + uint32_t((i >> 2) * kTileBytes)) ^
                                          uint32_t(32 * (i & 3)),
                                      a);
                        if constexpr (EDGE) {
                            a[0] &= keep[0];
                            a[1] &= keep[0];
                            a[2] &= keep[1];
                            a[3] &= keep[1];
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_bf16_16816(acc[i][nt], a, ph[k][nt][0], ph[k][nt][1]);
                            mma_bf16_16816(acc[i][nt], a, pl[nt][0], pl[nt][1]);
                        }
                    }
                }
            }
        };
        if (__builtin_expect(edge, 0))
            pv(std::true_type());
        else
            pv(std::false_type());

        // ---- the stage goes back to the producer
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&ring.empty[turn.st]));
        if (JOIN) {  // every p.teams'th stage (there are as many at least)
            turn.st += uint32_t(p.teams);
            if (turn.st >= uint32_t(d.nst)) {
                turn.st -= uint32_t(d.nst);
                turn.phase ^= 1u;
            }
        } else {
            turn.next(d.nst);
        }

        if (JOIN && (flags & F_LAST)) {
            // ---- the team's end: its partial, for the join
            const float vf = FP8 ? ldexpf(1.f, e_max - 127 - kWeightBits) : 1.f;
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                float l = l_r[i];
                l += __shfl_xor_sync(kFull, l, 4);
                l += __shfl_xor_sync(kFull, l, 8);
                l += __shfl_xor_sync(kFull, l, 16);
                const int row = team * d.rows_pad + row_of(i);
                if (g == 0)
                    joins.ml[row] = make_float2(m_r[i], l);
                float *o = joins.acc + row * Partials::stride<D>();
#pragma unroll
                for (int mt = 0; mt < MT; mt += FP8 ? 2 : 1)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float v0 = acc[mt][i >> 1][2 * c + (i & 1)] * vf;
                        if constexpr (FP8) {
                            const float v1 = acc[mt + 1][i >> 1][2 * c + (i & 1)] * vf;
                            *reinterpret_cast<float2 *>(o + 16 * mt + 16 * c + 2 * g) =
                                make_float2(v0, v1);
                        } else {
                            o[16 * mt + 8 * c + g] = v0;
                        }
                    }
            }
            return;
        }
        if (!JOIN && (flags & F_LAST)) {
            // ---- the segment's end: full row sums, then the output or a partial
            const bool direct = flags & F_DIRECT;
            const float vf = FP8 ? ldexpf(1.f, e_max - 127 - kWeightBits) : 1.f;
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                float l = l_r[i];
                l += __shfl_xor_sync(kFull, l, 4);
                l += __shfl_xor_sync(kFull, l, 8);
                l += __shfl_xor_sync(kFull, l, 16);
                const int row = row_of(i);
                if (row >= d.rows)
                    continue;
                const int j = row / d.G;
                const int64_t o =
                    ((int64_t(s) * d.nq + j) * d.Hq + int64_t(kvh) * d.G + row - j * d.G) * D;
                const int64_t part = ((int64_t(e_cell) * 2 + e_slot) * d.HG + hl) * d.rows + row;
                const float f = (direct ? (l == 0.f ? 0.f : 1.f / l) : 1.f) * vf;
                if (!direct && g == 0)
                    *reinterpret_cast<float2 *>(d.ml + part * 2) = make_float2(m_r[i], l);
                float *pf = direct ? static_cast<float *>(d.out) + o : d.part + part * D;
                const bool as_bf16 = direct && !d.out_f32;
                __nv_bfloat16 *pb = static_cast<__nv_bfloat16 *>(d.out) + o;
#pragma unroll
                for (int mt = 0; mt < MT; mt += FP8 ? 2 : 1)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float v0 = acc[mt][i >> 1][2 * c + (i & 1)] * f;
                        if constexpr (FP8) {
                            // dims 2g, 2g + 1 of the chunk: the even and the odd m-tile
                            const float v1 = acc[mt + 1][i >> 1][2 * c + (i & 1)] * f;
                            const int dim = 16 * mt + 16 * c + 2 * g;
                            if (as_bf16)
                                *reinterpret_cast<uint32_t *>(pb + dim) = pack_bf16x2(v0, v1);
                            else
                                *reinterpret_cast<float2 *>(pf + dim) = make_float2(v0, v1);
                        } else {
                            const int dim = 16 * mt + 8 * c + g;
                            if (as_bf16)
                                pb[dim] = __float2bfloat16_rn(v0);
                            else
                                pf[dim] = v0;
                        }
                    }
            }
        }
    }
}

constexpr int kConsumers = 8;

template <int D, bool FP8, int NT, int WPH>
__global__ void __launch_bounds__(teams_of(WPH) ? kTeamThreads : 32 * (kConsumers + 1), 1)
    scored_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ ScoredParams p)
{
    constexpr bool TEAMS = teams_of(WPH);
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // consumer warps of a team lie together; producers behind all of them
    const bool produces = warp >= (TEAMS ? kTeamWarps : p.d.ncw);
    const int team = !TEAMS ? 0 : produces ? warp - kTeamWarps : warp / p.d.ncw;
    const Ring ring = carve(smem_raw, p, p.teams, team);
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
        for (int t = 0; t < p.teams; ++t)
            for (int i = 0; i < p.d.nst; ++i) {
                mbar_init(smem_u32(&ring.full[2 * t * p.d.nst + i]), 1);
                mbar_init(smem_u32(&ring.empty[2 * t * p.d.nst + i]), uint32_t(p.d.ncw));
            }
        fence_mbar_init();
    }
    // the kernel before this one on the stream may still write q or the pools
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    if (produces) {
        if constexpr (TEAMS)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        if (team < p.teams)
            producer<FP8>(&kmap, &vmap, p, ring, lane);
    } else {
        if constexpr (TEAMS)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
        if (team < p.teams) {
            const int cw = TEAMS ? warp - team * p.d.ncw : warp;
            if (p.whole)  // (otherwise the merge does it)
                for (int64_t id = ring.cell; id < int64_t(p.d.S) * p.d.n_hg; id += p.cells)
                    clear_empty<D>(p, id, cw * 32 + lane, 32 * p.d.ncw);
            consumer<D, FP8, NT, WPH, false>(
                p, ring, cw, lane, query_fragments(smem_raw, p, p.teams) + warp * (NT * D * 16), 0,
                Partials{});
        }
    }
}

// Adds one of n partials (m, l, a) to (M, L, A), M the largest m of all. One without a
// weight (a row that sees none of its tokens) leaves nothing to add.
__device__ __forceinline__ void add_partial(float M, float2 ml, float4 a, float &L, float4 &A)
{
    if (ml.y == 0.f)
        return;
    const float w = ml.x == M ? 1.f : ex2(ml.x - M);
    L = fmaf(w, ml.y, L);
    A.x = fmaf(w, a.x, A.x);
    A.y = fmaf(w, a.y, A.y);
    A.z = fmaf(w, a.z, A.z);
    A.w = fmaf(w, a.w, A.w);
}

// Elements 4c .. 4c + 3 of an output row: the sums A over L (zeros where nothing was seen).
template <int D>
__device__ __forceinline__ void write_row(const ScoredParams &p, int s, int kvh, int row, int c,
                                          float L, float4 A)
{
    const DecodeParams &d = p.d;
    const float f = L == 0.f ? 0.f : 1.f / L;
    A = make_float4(A.x * f, A.y * f, A.z * f, A.w * f);
    const int j = row / d.G;
    const int64_t o = ((int64_t(s) * d.nq + j) * d.Hq + int64_t(kvh) * d.G + row - j * d.G) * D +
                      4 * c;
    if (d.out_f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(d.out) + o) = A;
    else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(d.out) + o) =
            make_uint2(pack_bf16x2(A.x, A.y), pack_bf16x2(A.z, A.w));
}

// ------------------------------------------------------------------ merge
// Joins the partials of few rows (launch_merge has the other cases): WPR
// warps have a row, an equal share of its pieces each. Bound by three trips to memory, the
// lengths and records, the partials, the output, of as many CTAs as are resident.
template <int D, int WPR>
__global__ void __launch_bounds__(256)
    scored_merge_kernel(const __grid_constant__ ScoredParams p)
{
    __shared__ float4 s_acc[8][32];
    __shared__ float2 s_ml[8];
    const DecodeParams &d = p.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
    const int rows = d.HG * d.rows;  // of a sequence and head group
    const int64_t id = int64_t(blockIdx.x) * (8 / WPR) + warp / WPR;
    const int pair = int(id / rows), r = int(id - int64_t(pair) * rows);
    const int s = pair / d.n_hg, hg = pair - s * d.n_hg;
    const int hl = r / d.rows, row = r - hl * d.rows;
    const bool here = s < d.S;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the pieces kb .. ke of the sequence; one piece: finished in place. (A record that is none
    // of this call's, after a main kernel that gave up, names no cells: nothing to join.)
    const int2 rec = here ? __ldcg(d.pieces + int64_t(s) * d.n_hg + hg) : make_int2(0, 0);
    const bool empty = here && span(p, s).nb == 0;
    const bool dense = __ldcg(d.ws + kWsDense) != 0u;
    const int kb = rec.x >> 1, ke = rec.y;
    const bool joins = here && !empty && kb >= 0 && ke > kb && ke < p.cells;
    Cells C{};
    if (joins && !dense) {  // fewer units than cells: some cells are empty and hold nothing
        C.F = C.F1 = int64_t(d.n_hg) * int64_t(__ldcg(d.ws + kWsUnits));
        C.G = p.cells;
    }
    const int np = joins ? ke - kb + 1 : 0, n1 = np * (sub + 1) / WPR;
    float M = -INFINITY, L = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int PB = WPR == 1 ? 4 : 8;  // pieces at a time
    for (int k0 = np * sub / WPR; k0 < n1; k0 += PB) {
        const int64_t cell = int64_t(kb) + k0 + lane;
        int64_t at = -1;  // the lane's partial row
        if (lane < PB && k0 + lane < n1 && (dense || !C.empty(cell)))
            at = (cell * 2 + (k0 + lane == 0 ? (rec.x & 1) : 0)) * rows + r;
        const float2 ml = at >= 0 ? __ldcg(reinterpret_cast<const float2 *>(d.ml) + at)
                                  : make_float2(-INFINITY, 0.f);
        float4 v[PB];
#pragma unroll
        for (int k = 0; k < PB; ++k) {
            const int64_t from = __shfl_sync(kFull, at, k);
            v[k] = from >= 0 && lane * 4 < D
                       ? __ldcg(reinterpret_cast<const float4 *>(d.part + from * D + lane * 4))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float m = ml.x;
#pragma unroll
        for (int o = PB / 2; o >= 1; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        m = fmaxf(__shfl_sync(kFull, m, 0), M);
        const float f = M == m ? 1.f : ex2(M - m);
        M = m;
        L *= f;
        A = make_float4(A.x * f, A.y * f, A.z * f, A.w * f);
#pragma unroll
        for (int k = 0; k < PB; ++k)
            add_partial(M,
                        make_float2(__shfl_sync(kFull, ml.x, k), __shfl_sync(kFull, ml.y, k)),
                        v[k], L, A);
    }
    if (lane == 0)
        s_ml[warp] = make_float2(M, L);
    s_acc[warp][lane] = A;
    __syncthreads();
    if (sub != 0 || lane * 4 >= D || !(joins || empty))
        return;
    for (int k = 0; k < WPR; ++k)
        M = fmaxf(M, s_ml[warp + k].x);
    L = 0.f;
    A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < WPR; ++k)
        add_partial(M, s_ml[warp + k], s_acc[warp + k][lane], L, A);
    write_row<D>(p, s, hg * d.HG + hl, row, lane, L, A);
}

// The joined form, for few and short sequences: a cluster of CTAs has one sequence and kv
// head, a CTA an equal share of its blocks, and the teams of a CTA (a warp each up to 16
// rows) take the stages of one ring in turn, each with a state of its own. The teams'
// states are joined in shared memory, the CTAs' through the cluster's shared memory. Bound
// by the chain of trips to memory (length, table entry, block) and one warp's time for a
// stage, 1.3 us: one sequence of 333 tokens, 8 kv heads, E4M3, 7.3 us (10.4 us cut).
constexpr int kJoinThreads = 256;  // seven consumer warps at most, one producer

__device__ __forceinline__ uint32_t in_rank(uint32_t addr, int rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 cluster_f2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ float4 cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

template <int D, bool FP8, int NT, int WPH>
__global__ void __launch_bounds__(kJoinThreads, NT == 1 ? 2 : 1)
    scored_join_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ ScoredParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const DecodeParams &d = p.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = p.teams * WPH;
    const Ring ring = carve(smem_raw, p, 1, 0);
    uint8_t *qs = query_fragments(smem_raw, p, 1);
    Partials joins;
    joins.acc = reinterpret_cast<float *>(qs + (teams_of(WPH) ? n_warps * NT * D * 16 : 0));
    joins.ml = reinterpret_cast<float2 *>(joins.acc +
                                          p.teams * d.rows_pad * Partials::stride<D>());
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
        for (int i = 0; i < d.nst; ++i) {
            mbar_init(smem_u32(&ring.full[i]), 1);
            mbar_init(smem_u32(&ring.empty[i]), WPH);
        }
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < p.teams * d.rows_pad; i += kJoinThreads)
        joins.ml[i] = make_float2(-INFINITY, 0.f);
    // the kernel before this one on the stream may still write q or the pools
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    const Share part = share<FP8>(p);
    if (warp == n_warps) {
        produce_share<FP8>(&kmap, &vmap, p, ring, part, lane);
    } else if (warp < n_warps) {
        const int team = warp / WPH;
        if (team < part.hi - part.lo)
            consumer<D, FP8, NT, WPH, true>(p, ring, warp % WPH, lane, qs + warp * (NT * D * 16),
                                            team, joins);
    }
    __syncthreads();

    // ---- the teams' partials: one for the CTA (the teams' first), or the output
    constexpr int DQ = D / 4;
    for (int i0 = 0; i0 < d.rows * DQ; i0 += kJoinThreads) {
        const int i = i0 + threadIdx.x, row = i / DQ, c = i % DQ;
        float M = -INFINITY, L = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < d.rows) {
            for (int t = 0; t < p.teams; ++t)
                M = fmaxf(M, joins.ml[t * d.rows_pad + row].x);
            for (int t = 0; t < p.teams; ++t) {
                const int r = t * d.rows_pad + row;
                add_partial(M, joins.ml[r],
                            *reinterpret_cast<const float4 *>(joins.acc +
                                                              r * Partials::stride<D>() + 4 * c),
                            L, A);
            }
            if (p.cluster == 1)
                write_row<D>(p, part.s, part.h, row, c, L, A);
        }
        if (p.cluster > 1) {
            __syncthreads();  // (all of a row have read its (m, l); 256 threads have whole rows)
            if (row < d.rows) {
                *reinterpret_cast<float4 *>(joins.acc + row * Partials::stride<D>() + 4 * c) = A;
                if (c == 0)
                    joins.ml[row] = make_float2(M, L);
            }
        }
    }
    if (p.cluster == 1)
        return;

    // ---- the CTAs' partials: each CTA joins and writes a part of the rows' elements
    cluster_barrier();
    const int n = d.rows * DQ, hi = int(int64_t(n) * (part.rank + 1) / p.cluster);
    for (int i = int(int64_t(n) * part.rank / p.cluster) + threadIdx.x; i < hi; i += kJoinThreads) {
        const int row = i / DQ, c = i % DQ;
        const uint32_t ml = smem_u32(joins.ml + row);
        const uint32_t acc = smem_u32(joins.acc + row * Partials::stride<D>() + 4 * c);
        float2 m[kMaxCluster];
        float4 a[kMaxCluster];
        float M = -INFINITY, L = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            if (r < p.cluster) {
                m[r] = cluster_f2(in_rank(ml, r));
                a[r] = cluster_f4(in_rank(acc, r));
            }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            if (r < p.cluster)
                M = fmaxf(M, m[r].x);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            if (r < p.cluster)
                add_partial(M, m[r], a[r], L, A);
        write_row<D>(p, part.s, part.h, row, c, L, A);
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

template <int D, bool FP8, int NT, int WPH>
cudaError_t launch_one(const ScoredPlan &pl, const ScoredParams &p, const CUtensorMap &kmap,
                       const CUtensorMap &vmap, cudaStream_t stream)
{
    const auto kern = pl.cluster ? scored_join_kernel<D, FP8, NT, WPH> : scored_kernel<D, FP8, NT, WPH>;
    cudaError_t e;
    if (teams_of(WPH) && !pl.cluster) {
        // the warps share out kLaunchRegs a thread: with fewer they would wait forever
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess)
            return e;
        if (fa.numRegs < kLaunchRegs)
            return cudaErrorLaunchOutOfResources;
    }
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(pl.smem));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(pl.ctas));
    cfg.blockDim = dim3(unsigned(pl.threads));
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(pl.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pl.cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p);
    if (e != cudaSuccess)
        return e;
    if (pl.whole || pl.cluster)
        return cudaGetLastError();
    // The merge. GB300, E4M3, 8 kv heads. Where a sequence has eight pieces or more on average,
    // eight or four warps a row while the rows are few; eight warps / four / launch_merge,
    // launches included, in us: 1 sequence of 8000 tokens with 32 rows a head (256 rows in
    // all) 30.8/34.5/65.8, 3 with 16 (384) 34.5/36.1/53.2, 5 (640) 43.2/40.2/49.8, 8 (1024)
    // 50.1/46.4/51.6, 5 with 32 (1280) 51.2/49.3/53.4, 8 (2048) 66.9/62.3/62.9, 16 with 16
    // (2048) 77.3/72.1/69.8. With fewer pieces one warp a row while those all fit; one warp /
    // launch_merge: 64 sequences of 512 to 4096 with 4 rows (2048) 46.2/46.9, 256 of 300 to
    // 2500 with 8 (16384) 98.8/96.0, 128 of 256 to 4096 with 32 (32768) 121.9/116.3.
    const int64_t pairs = int64_t(p.d.S) * p.d.n_hg, rows = pairs * p.d.HG * p.d.rows;
    const bool few = pairs * 8 > pl.grid;  // pieces
    if (rows > (few ? 4096 : 1536))
        return launch_merge(pl, p.d, stream);
    const int warps = few ? 1 : rows <= 512 ? 8 : 4;
    const auto merge = few ? scored_merge_kernel<D, 1>
                           : warps == 8 ? scored_merge_kernel<D, 8> : scored_merge_kernel<D, 4>;
    cfg.gridDim = dim3(unsigned((rows * warps + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge, p);
}

}  // namespace

// The joined form of a plan, where it is the faster one: it saves the second launch, the
// walk over all sequences and the partials' way through memory, but its work is balanced
// only inside a sequence and its CTAs stream no faster than their few warps compute. GB300,
// E4M3, 8 kv heads, 4 rows, equal lengths, launch included, joined / cells in us:
//   1 sequence of 333, 1000, 4000, 8000 tokens   15.2/19.1  15.3/22.6  18.8/31.6  21.7/33.8
//   4                 1000, 4000, 8000           17.1/22.7  21.6/28.9  29.5/34.1
//   16 (1 CTA each)   1000, 2000, 4000, 8000     22.2/28.2  27.2/33.3  42.0/42.6  69.6/64.1
//   32 (2 on an SM)   333, 1000, 2000, 4000      19.0/26.1  29.2/33.9  45.0/44.0  75.4/63.5
// So with one CTA on an SM up to half of the blocks a team at which both take as long (a
// batch may hold one long sequence among short ones); with two up to 9: bf16 pools, 32
// sequences of 2048 to 32768 tokens with a window of 1024 (66 blocks on 7 teams) take
// 31.5/30.0.
static bool plan_joined(int S, int Hkv, int MB, int num_sms, int smem_optin, ScoredPlan *pl)
{
    ScoredPlan P = *pl;
    const int BL = stage_blocks(P.kv8);
    const int64_t pairs = int64_t(S) * Hkv;  // of a sequence and a kv head
    P.n_hg = Hkv;
    P.teams = (kJoinThreads / 32 - 1) / P.wph;
    P.threads = kJoinThreads;
    P.stage_bytes = BL * 2 * (P.kv8 ? 1 : P.D / 64) * kTileBytes;
    // two CTAs share an SM where one each would not do (up to 8 rows: registers)
    P.ctas_per_sm = pairs <= num_sms ? 1 : 2;
    if (pairs > int64_t(P.ntw == 1 ? 2 : 1) * num_sms)
        return false;
    // as many CTAs a pair as have work and fit (an eighth of a chip's part may be left over by
    // clusters of eight: 16 of them took two rounds, 8 did not)
    P.cluster = 1;
    while (P.cluster < kMaxCluster && MB > P.cluster * P.teams * BL &&
           pairs * P.cluster * 2 <= (P.cluster == 4 ? num_sms * 5 / 8 : num_sms))
        P.cluster *= 2;
    if (MB > P.cluster * P.teams * (P.ctas_per_sm == 1 ? 16 : 9))
        return false;
    P.grid = P.ctas = int(pairs) * P.cluster;
    const int extra = P.teams * (P.rows_pad * ((P.D + 4) * 4 + 8) +
                                 (teams_of(P.wph) ? P.wph * P.ntw * P.D * 16 : 0));
    const int per_stage = P.stage_bytes + int(sizeof(Header)) + 16;
    const int budget = P.ctas_per_sm == 1 ? smem_optin : (smem_optin + 1024) / 2 - 1024;
    // whole turns of the teams, so that a stage is always the same team's: another team that
    // is a turn ahead would take an old phase of its barrier for the new one
    P.nst = std::min(2, (budget - 1024 - extra) / per_stage / P.teams) * P.teams;
    if (P.nst < P.teams)
        return false;
    P.smem = 1024 + size_t(P.nst) * per_stage + extra;
    P.ws_bytes = kWsHeaderBytes;
    *pl = P;
    return true;
}

int plan_scored(int S, int nq, int Hq, int Hkv, int D, int MB, int num_sms, int smem_optin,
                int fp8, ScoredPlan *pl)
{
    ScoredPlan P{};
    P.D = D;
    P.kv8 = fp8;
    P.G = Hq / Hkv;
    P.rows = P.G * nq;
    // up to 16 rows a warp
    const int tiles = (P.rows + 7) / 8;
    P.ntw = tiles == 1 ? 1 : 2;
    P.wph = tiles <= 2 ? 1 : tiles <= 4 ? 2 : 4;
    P.rows_pad = P.wph * P.ntw * 8;
    P.HG = 1;
    if (plan_joined(S, Hkv, MB, num_sms, smem_optin, &P)) {
        *pl = P;
        return 0;
    }
    const bool teams = teams_of(P.wph);
    const auto teams_with = [&](int h) {
        return teams ? std::min(kMaxTeams, kTeamWarps / (h * P.wph)) : 1;
    };
    // heads of a group: one team has as many as possible, several teams the smallest group
    // that gives the most consumer warps. 3 kv heads, 32 rows, 2 teams of 3 heads / 4 of one:
    // 125 sequences of a tenth to all of 2000 tokens 61.8/75.2 us, 300 103/120; but 30 of 800
    // 37.0/32.3 (cells of a few blocks)
    for (int h = 1; h <= std::min((teams ? kTeamWarps : kConsumers) / P.wph, Hkv); ++h)
        if (Hkv % h == 0 && teams_with(h) * h > teams_with(P.HG) * P.HG)
            P.HG = h;
    P.n_hg = Hkv / P.HG;
    const int ncw = P.HG * P.wph;
    P.teams = teams_with(P.HG);
    P.threads = teams ? kTeamThreads : 32 * (1 + ncw);
    const int block_bytes = 2 * P.HG * (fp8 ? 1 : D / 64) * kTileBytes;
    P.stage_bytes = stage_blocks(fp8) * block_bytes;
    // few heads: several CTAs share an SM, so that as many warps hide each other's waits
    P.ctas_per_sm = teams ? 1 : std::min(4, std::max(1, kConsumers / ncw));
    const int per_stage = P.stage_bytes + int(sizeof(Header)) + 16;
    const int queries = teams ? P.teams * ncw * P.ntw * D * 16 : 0;
    const int budget = P.ctas_per_sm == 1 ? smem_optin : (smem_optin + 1024) / P.ctas_per_sm - 1024;
    P.nst = std::min(16, (budget - 1024 - queries) / per_stage / P.teams);
    if (P.nst < 2)
        return -1;
    P.smem = 1024 + size_t(P.teams) * P.nst * per_stage + queries;
    const int cap = P.ctas_per_sm * num_sms * P.teams;  // cells at most
    const int64_t units = int64_t(P.n_hg) * S;
    P.ctas = int(std::min<int64_t>(P.ctas_per_sm * num_sms, std::min<int64_t>(units, cap) * MB));
    P.grid = P.ctas * P.teams;
    // Short sequences that have a cell each: no walk over the batch, no pieces to join, but no
    // balance between long and short ones either. GB300, E4M3, 8 kv heads, 4 rows, equal
    // lengths, launches included, whole / cut in us: 40 sequences of 64, 256, 512, 1024 tokens
    // 15.4/20.8 22.6/26.1 31.0/29.4 47.6/37.7; 150 of them (all cells) 18.2/27.2 28.9/38.6
    // 40.2/50.5 63.9/74.7. Half of the length at which both take as long, as above.
    if (units <= cap && MB <= (2 * units >= cap ? 32 : 16)) {
        P.whole = kOwnCells;
        P.grid = P.n_hg * S;
        P.ctas = std::min(P.ctas_per_sm * num_sms, P.grid);
    }
    // More short sequences than cells: borders that move to the ends of sequences leave cells
    // that differ by a sequence at most, and nothing to join. The same, rounded / cut: 160
    // sequences (152 cells) of 64, 256, 512 tokens 24.3/26.8 39.2/37.2 59.4/50.3, of a tenth
    // to all of that 21.2/27.4 30.2/32.5 40.5/42.9; 600 of 64, 256, 512, 1024 34.5/43.0
    // 70.7/77.2 116/124 211/218, ragged 36.5/42.0 53.3/60.0 82.9/81.8 141/136. 32 rows a head
    // (more to join): 130 sequences (456 cells, 520 units) of 64, 256, 512, 1024 29.3/41.2
    // 47.0/59.7 68.8/73.5 113/102; 310 39.4/56.6 70.5/90.8 112/126 192/196.
    if (units > cap && MB <= (teams ? 32 : units >= 3 * int64_t(cap) ? 16 : 8))
        P.whole = kRoundedCells;
    P.off_rec = kWsHeaderBytes;
    P.off_ml = P.off_rec + round_up(size_t(S) * P.n_hg * 8, 256);
    P.off_part = P.off_ml + round_up(size_t(cap) * 2 * P.HG * P.rows * 2 * 4, 256);
    P.ws_bytes = P.off_part + round_up(size_t(cap) * 2 * P.HG * P.rows * size_t(D) * 4, 256);
    *pl = P;
    return 0;
}

cudaError_t launch_scored(const ScoredPlan &pl, const ScoredParams &p, const CUtensorMap &kmap,
                          const CUtensorMap &vmap, cudaStream_t stream)
{
    if (pl.kv8) {
        if (pl.wph == 4)
            return launch_one<128, true, 2, 4>(pl, p, kmap, vmap, stream);
        if (pl.wph == 2)
            return launch_one<128, true, 2, 2>(pl, p, kmap, vmap, stream);
        if (pl.ntw == 2)
            return launch_one<128, true, 2, 1>(pl, p, kmap, vmap, stream);
        return launch_one<128, true, 1, 1>(pl, p, kmap, vmap, stream);
    }
    if (pl.D == 64) {
        if (pl.wph == 4)
            return launch_one<64, false, 2, 4>(pl, p, kmap, vmap, stream);
        if (pl.wph == 2)
            return launch_one<64, false, 2, 2>(pl, p, kmap, vmap, stream);
        if (pl.ntw == 2)
            return launch_one<64, false, 2, 1>(pl, p, kmap, vmap, stream);
        return launch_one<64, false, 1, 1>(pl, p, kmap, vmap, stream);
    }
    if (pl.wph == 4)
        return launch_one<128, false, 2, 4>(pl, p, kmap, vmap, stream);
    if (pl.wph == 2)
        return launch_one<128, false, 2, 2>(pl, p, kmap, vmap, stream);
    if (pl.ntw == 2)
        return launch_one<128, false, 2, 1>(pl, p, kmap, vmap, stream);
    return launch_one<128, false, 1, 1>(pl, p, kmap, vmap, stream);
}

}  // namespace pkv
