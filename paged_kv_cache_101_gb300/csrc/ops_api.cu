// ops_api.cu -- the extern "C" entry points of include/pkv_ops.h: host checks,
// plans, tensor maps and launches.
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "pkv_ops_internal.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// SM count and shared-memory limit of the current device, read once per device.
struct DeviceLimits {
    int sms = 0, smem = 0;
};

cudaError_t device_limits(DeviceLimits *out)
{
    static std::mutex mu;
    static DeviceLimits known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    DeviceLimits &d = known[dev];
    if (d.sms == 0) {
        int sms = 0, smem = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) !=
                cudaSuccess)
            return e;
        d.smem = smem;
        d.sms = sms;
    }
    *out = d;
    return cudaSuccess;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static std::mutex mu;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::lock_guard<std::mutex> lk(mu);
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}

// A pool as boxes of one block's 16 tokens of `heads` kv heads, in shared memory
// [head][128-byte column half][token][128 bytes] with the 128-byte swizzle: bf16
// (64-element columns) or E4M3 codes (one 128-byte row per head).
bool encode_pool(CUtensorMap *map, const void *base, int64_t num_blocks, int Hkv, int D, int heads,
                 bool fp8)
{
    const auto encode = tensor_map_encoder();
    if (!encode)
        return false;
    const cuuint64_t size = fp8 ? 1 : 2, cols = 128 / size;
    const cuuint64_t halves = cuuint64_t(D) / cols, head = cuuint64_t(D) * size;
    const cuuint64_t token = head * Hkv;
    const cuuint64_t dims[5] = {cols, 16, halves, cuuint64_t(Hkv), cuuint64_t(num_blocks)};
    const cuuint64_t strides[4] = {token, 128, head, 16 * token};
    const cuuint32_t box[5] = {cuuint32_t(cols), 16, cuuint32_t(halves), cuuint32_t(heads), 1};
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    return encode(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                  const_cast<void *>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------------ rotation + append
pkv_status rope_append(pkv::RopeParams &p, int64_t num_blocks, bool fp8, void *stream)
{
    if (p.n < 0 || num_blocks < 1 || p.Hq < 0 || p.Hkv < 1 || p.D < 1 || p.r < 2 || p.r > p.D ||
        p.r % 2 != 0)
        return PKV_ERR_SHAPE;
    if (p.n == 0)
        return PKV_OK;
    if (!p.k || !p.v || !p.positions || !p.turns || !p.slots || !p.k_cache || !p.v_cache ||
        (p.Hq > 0 && (!p.q || !p.q_out)) || (p.Hq == 0 && (p.q || p.q_out)) ||
        (fp8 && (!p.k_scale || !p.v_scale)))
        return PKV_ERR_NULL;
    const int max_dim = fp8 ? pkv::kMaxFp8BlockDim : 1024;
    if (p.D % 8 != 0)
        return PKV_ERR_UNSUPPORTED;
    if (p.D > max_dim || p.Hkv > 1024 || p.Hq > 65536 || p.n > (int64_t(1) << 30) ||
        num_blocks > (int64_t(1) << 40) || !isfinite(p.scale))
        return PKV_ERR_RANGE;
    if (fp8 && p.n > INT32_MAX / (1 + 2 * ((p.Hkv + 7) / 8)))
        return PKV_ERR_RANGE;  // the grid
    const int64_t kv_row = int64_t(p.Hkv) * p.D, q_row = int64_t(p.Hq) * p.D;
    if (p.k_stride < kv_row || p.v_stride < kv_row || (p.Hq > 0 && p.q_stride < q_row))
        return PKV_ERR_SHAPE;
    const size_t cache_align = fp8 ? 8 : 16;
    if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.q_out, 16) ||
        !aligned(p.k_cache, cache_align) || !aligned(p.v_cache, cache_align) ||
        !aligned(p.positions, 8) || !aligned(p.turns, 8) || !aligned(p.slots, 8) ||
        p.q_stride % 8 != 0 || p.k_stride % 8 != 0 || p.v_stride % 8 != 0)
        return PKV_ERR_ALIGN;
    const pkv::RopeForm form = p.interleaved ? (p.r % 8 == 0 ? pkv::kPairs : pkv::kScalar)
                                             : (p.r % 16 == 0 ? pkv::kHalf : pkv::kScalar);
    if (p.Hq > 0 && p.q == p.q_out) {
        if (p.q_stride != q_row)
            return PKV_ERR_SHAPE;
        // a scalar unit reads pairs that another unit writes
        if (form == pkv::kScalar)
            return PKV_ERR_UNSUPPORTED;
    }
    p.total_slots = num_blocks * pkv::kBlockSize;
    p.units = form == pkv::kHalf ? p.r / 16 + (p.D - p.r + 15) / 16 : (p.D + 15) / 16;
    return pkv::launch_rope_append(p, form, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

// ------------------------------------------------------------------ scored attention
constexpr int kMaxTableWidth = 1 << 26;

pkv_status check_scored_geometry(int32_t num_seqs, int32_t nq, int32_t Hq, int32_t Hkv, int32_t D)
{
    if (num_seqs < 0 || nq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
        return PKV_ERR_SHAPE;
    if ((D != 64 && D != 128) || nq > 4 || (Hq / Hkv) * nq > pkv::kMaxRows)
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

pkv_status scored_attention(const void *q, const void *k_cache, const void *v_cache,
                            int64_t num_blocks, const uint8_t *k_scale, const uint8_t *v_scale,
                            const int32_t *block_tables, int32_t max_blocks_per_seq,
                            const int32_t *context_lens, int32_t num_seqs, int32_t nq,
                            int32_t Hq, int32_t Hkv, int32_t D, float scale, float softcap,
                            const float *slopes, int32_t window, void *out, int32_t out_dtype,
                            void *workspace, size_t workspace_bytes, void *stream)
{
    const pkv_status st = check_scored_geometry(num_seqs, nq, Hq, Hkv, D);
    if (st != PKV_OK)
        return st;
    if ((k_scale == nullptr) != (v_scale == nullptr))
        return PKV_ERR_NULL;
    const bool fp8 = k_scale != nullptr;
    if (fp8 && D != 128)
        return PKV_ERR_UNSUPPORTED;
    if (num_blocks < 1 || max_blocks_per_seq < 1)
        return PKV_ERR_SHAPE;
    if (out_dtype != PKV_BF16 && out_dtype != PKV_FP32)
        return PKV_ERR_DTYPE;
    constexpr float kLog2e = 1.4426950408889634f;
    const float mul = softcap > 0.f ? 2.f * scale * kLog2e / softcap : scale * kLog2e;
    if (!(softcap >= 0.f) || !isfinite(softcap) || (softcap > 0.f && !isfinite(mul)) || window < 0)
        return PKV_ERR_RANGE;
    if (num_seqs == 0)
        return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
        return PKV_ERR_NULL;
    if (!workspace)
        return PKV_ERR_WORKSPACE;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(slopes, 4) ||
        !aligned(workspace, 256))
        return PKV_ERR_ALIGN;
    if (max_blocks_per_seq > kMaxTableWidth || num_blocks > 0x7fffffffLL || num_seqs > (1 << 24) ||
        Hkv > 65535)
        return PKV_ERR_RANGE;
    DeviceLimits dev;
    if (device_limits(&dev) != cudaSuccess)
        return PKV_ERR_CUDA;
    pkv::ScoredPlan pl;
    // a window that reaches back over the longest possible context hides nothing; one that
    // does not bounds the blocks a sequence reads
    if (int64_t(window) >= int64_t(max_blocks_per_seq) * pkv::kBlockSize)
        window = 0;
    const int most_blocks =
        window > 0 ? int(std::min<int64_t>(max_blocks_per_seq,
                                           (int64_t(window) + nq + 2 * pkv::kBlockSize - 3) /
                                               pkv::kBlockSize))
                   : max_blocks_per_seq;
    if (pkv::plan_scored(num_seqs, nq, Hq, Hkv, D, most_blocks, dev.sms, dev.smem, fp8, &pl) != 0)
        return PKV_ERR_UNSUPPORTED;
    if (workspace_bytes < pkv_workspace_size_scored(num_seqs, nq, Hq, Hkv, D))
        return PKV_ERR_WORKSPACE;
    CUtensorMap kmap, vmap;
    if (!encode_pool(&kmap, k_cache, num_blocks, Hkv, D, pl.HG, fp8) ||
        !encode_pool(&vmap, v_cache, num_blocks, Hkv, D, pl.HG, fp8))
        return PKV_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    pkv::ScoredParams p;
    memset(&p, 0, sizeof p);
    p.d.q = static_cast<const uint16_t *>(q);
    p.d.out = out;
    p.d.block_tables = block_tables;
    p.d.context_lens = context_lens;
    p.d.ws = reinterpret_cast<uint32_t *>(ws);
    p.d.pieces = reinterpret_cast<int2 *>(ws + pl.off_rec);
    p.d.ml = reinterpret_cast<float *>(ws + pl.off_ml);
    p.d.part = reinterpret_cast<float *>(ws + pl.off_part);
    p.d.num_blocks = num_blocks;
    p.d.S = num_seqs;
    p.d.MB = max_blocks_per_seq;
    p.d.nq = nq;
    p.d.Hq = Hq;
    p.d.Hkv = Hkv;
    p.d.G = pl.G;
    p.d.rows = pl.rows;
    p.d.rows_pad = pl.rows_pad;
    p.d.HG = pl.HG;
    p.d.n_hg = pl.n_hg;
    p.d.out_f32 = out_dtype == PKV_FP32;
    p.d.stage_bytes = pl.stage_bytes;
    p.d.nst = pl.nst;
    p.d.ncw = pl.HG * pl.wph;
    p.d.total_q = num_seqs * nq;
    p.d.table_rows = num_seqs;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.slopes = slopes;
    p.mul = mul;
    p.cap_log2 = softcap * kLog2e;
    p.window = window;
    p.whole = pl.whole;
    p.teams = pl.teams;
    p.cells = pl.grid;
    p.cluster = pl.cluster;
    p.scale_vec = fp8 && (pl.HG == 8 || pl.HG == 4 || pl.HG == 2) &&
                  aligned(k_scale, pl.HG) && aligned(v_scale, pl.HG);
    return pkv::launch_scored(pl, p, kmap, vmap, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

}  // namespace

extern "C" {

pkv_status pkv_rotary_turns(int32_t rotary_dim, double base, int32_t kind, double factor,
                            double original_length, double low, double high, uint64_t *turns)
{
    if (!turns)
        return PKV_ERR_NULL;
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || (kind == PKV_ROPE_BASE && rotary_dim < 4))
        return PKV_ERR_SHAPE;
    if (kind < PKV_ROPE_PLAIN || kind > PKV_ROPE_RAMP)
        return PKV_ERR_UNSUPPORTED;
    const auto positive = [](double x) { return x > 0.0 && isfinite(x); };
    if (!positive(base) || (kind != PKV_ROPE_PLAIN && !positive(factor)))
        return PKV_ERR_RANGE;
    if (kind == PKV_ROPE_RAMP &&
        (!positive(original_length) || !isfinite(low) || !isfinite(high) || !(high > low)))
        return PKV_ERR_RANGE;
    if (kind == PKV_ROPE_BASE)
        base *= pow(factor, double(rotary_dim) / (rotary_dim - 2));
    for (int32_t i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rotary_dim) / (2.0 * M_PI);
        if (kind == PKV_ROPE_LINEAR)
            f /= factor;
        if (kind == PKV_ROPE_RAMP) {
            double keep = (original_length * f - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = keep * f + (1.0 - keep) * f / factor;
        }
        // whole turns change nothing at whole positions
        turns[i] = uint64_t((f - floor(f)) * 0x1p64);
    }
    return PKV_OK;
}

pkv_status pkv_rope_kv_append(const void *q, int64_t q_stride, const void *k_new,
                              int64_t k_stride, const void *v_new, int64_t v_stride,
                              const int64_t *positions, const uint64_t *turns,
                              const int64_t *slot_mapping, int64_t n_new, void *q_out,
                              void *k_cache, void *v_cache, int64_t num_blocks,
                              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                              int32_t rotary_dim, int32_t interleaved, float rotary_scale,
                              void *stream)
{
    pkv::RopeParams p{static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k_new),
                      static_cast<const uint16_t *>(v_new), q_stride, k_stride, v_stride,
                      positions, turns, slot_mapping, static_cast<uint16_t *>(q_out), k_cache,
                      v_cache, nullptr, nullptr, n_new, 0, num_q_heads, num_kv_heads, head_dim,
                      rotary_dim, interleaved, 0, rotary_scale};
    return rope_append(p, num_blocks, false, stream);
}

pkv_status pkv_rope_kv_append_fp8_block(
    const void *q, int64_t q_stride, const void *k_new, int64_t k_stride, const void *v_new,
    int64_t v_stride, const int64_t *positions, const uint64_t *turns,
    const int64_t *slot_mapping, int64_t n_new, void *q_out, void *k_cache, void *v_cache,
    uint8_t *k_scale, uint8_t *v_scale, int64_t num_blocks, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
    float rotary_scale, void *stream)
{
    pkv::RopeParams p{static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k_new),
                      static_cast<const uint16_t *>(v_new), q_stride, k_stride, v_stride,
                      positions, turns, slot_mapping, static_cast<uint16_t *>(q_out), k_cache,
                      v_cache, k_scale, v_scale, n_new, 0, num_q_heads, num_kv_heads, head_dim,
                      rotary_dim, interleaved, 0, rotary_scale};
    return rope_append(p, num_blocks, true, stream);
}

size_t pkv_workspace_size_scored(int32_t num_seqs, int32_t n_query_per_seq, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim)
{
    if (check_scored_geometry(num_seqs, n_query_per_seq, num_q_heads, num_kv_heads, head_dim) !=
        PKV_OK)
        return 0;
    if (num_seqs == 0)
        return 256;
    DeviceLimits dev;
    if (device_limits(&dev) != cudaSuccess)
        return 0;
    // the larger of the two pool types, at the widest table (the forms for narrow ones need
    // less, and otherwise the width plays no part)
    size_t bytes = 0;
    for (int fp8 = 0; fp8 < 2; ++fp8) {
        pkv::ScoredPlan pl;
        if ((fp8 && head_dim != 128) ||
            pkv::plan_scored(num_seqs, n_query_per_seq, num_q_heads, num_kv_heads, head_dim,
                             kMaxTableWidth, dev.sms, dev.smem, fp8, &pl) != 0)
            continue;
        bytes = pl.ws_bytes > bytes ? pl.ws_bytes : bytes;
    }
    return bytes;
}

pkv_status pkv_paged_decode_attention_scored(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    const uint8_t *k_scale, const uint8_t *v_scale, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
    int32_t n_query_per_seq, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    float scale, float softcap, const float *alibi_slopes, int32_t window, void *out,
    int32_t out_dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    return scored_attention(q, k_cache, v_cache, num_blocks, k_scale, v_scale, block_tables,
                            max_blocks_per_seq, context_lens, num_seqs, n_query_per_seq,
                            num_q_heads, num_kv_heads, head_dim, scale, softcap, alibi_slopes,
                            window, out, out_dtype, workspace, workspace_bytes, stream);
}

pkv_status pkv_paged_decode_attention_fp8_block(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    const uint8_t *k_scale, const uint8_t *v_scale, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
    int32_t n_query_per_seq, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    float scale, void *out, int32_t out_dtype, void *workspace, size_t workspace_bytes,
    void *stream)
{
    if (num_seqs > 0 && (!k_scale || !v_scale))
        return PKV_ERR_NULL;
    if (head_dim != 128)
        return PKV_ERR_UNSUPPORTED;
    return scored_attention(q, k_cache, v_cache, num_blocks, k_scale, v_scale, block_tables,
                            max_blocks_per_seq, context_lens, num_seqs, n_query_per_seq,
                            num_q_heads, num_kv_heads, head_dim, scale, 0.f, nullptr, 0, out,
                            out_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
