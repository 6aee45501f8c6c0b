// pkv_ops_internal.h -- parameters and launchers of the operators of include/pkv_ops.h,
// shared by their host side (ops_api.cu) and their kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pkv_internal.h"
#include "pkv_ops.h"

namespace pkv {

// How a head's elements are reached: kHalf and kPairs move 16-byte vectors (the
// rotated part cut at vector boundaries); kScalar takes any even rotary_dim.
enum RopeForm { kHalf = 0, kPairs = 1, kScalar = 2 };

struct RopeParams {
    const uint16_t *q, *k, *v;             // bf16 rows
    int64_t q_stride, k_stride, v_stride;  // elements between rows
    const int64_t *positions;
    const uint64_t *turns;                 // [r / 2] 2^-64 turn per position
    const int64_t *slots;
    uint16_t *q_out;
    void *k_cache, *v_cache;               // bf16 or E4M3 codes
    uint8_t *k_scale, *v_scale;            // block-scaled pools (null: bf16)
    int64_t n, total_slots;
    int Hq, Hkv, D, r;
    int interleaved;
    int units;                             // 16-dim units of a head
    float scale;
};

cudaError_t launch_rope_append(const RopeParams &p, RopeForm form, cudaStream_t stream);

constexpr int kMaxFp8BlockDim = 256;  // head_dim of the block-scaled append

// Cells that cut no sequence: cell c is sequence c % S of head group c / S, or the borders of
// equal cells move to the nearer end of the sequence that they fall into.
enum { kOwnCells = 1, kRoundedCells = 2 };

struct ScoredParams {
    DecodeParams d;          // the decode call's own parameters (the merge reads these)
    const uint8_t *k_scale;  // [num_blocks][Hkv] scale bytes (null: bf16 pools)
    const uint8_t *v_scale;
    const float *slopes;     // [Hq] or null
    float mul;               // to the log2 domain: scale log2(e), or 2 scale log2(e) / softcap
    float cap_log2;          // softcap log2(e); 0: none
    int window;              // 0: none
    int whole;               // as in the plan
    int teams, cells;        // as in the plan (cells: its grid)
    int cluster;             // as in the plan
    int scale_vec;           // the scale bytes of a block's 2, 4 or 8 heads are one aligned word
};

struct ScoredPlan : DecodePlan {  // (grid: the cells of the call)
    int whole;  // kOwnCells, kRoundedCells (no pieces, no merge) or 0
    int teams;  // cells that a CTA works on at a time, each with warps and a ring of its own
    int ctas;   // of the launch
    int cluster;  // joined form: CTAs of a sequence and kv head (0: not that form)
};

// The plan of a scored call (fp8: block-scaled pools), MB the most blocks that a
// sequence reads; 0, or -1 if unsupported.
int plan_scored(int S, int nq, int Hq, int Hkv, int D, int MB, int num_sms, int smem_optin,
                int fp8, ScoredPlan *plan);

cudaError_t launch_scored(const ScoredPlan &plan, const ScoredParams &p, const CUtensorMap &kmap,
                          const CUtensorMap &vmap, cudaStream_t stream);

}  // namespace pkv
