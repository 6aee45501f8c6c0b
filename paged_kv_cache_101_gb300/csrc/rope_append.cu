// rope_append.cu -- rotate the step's queries and keys by their positions and
// write keys and values into the paged pool (bf16, or E4M3 with one scale for each
// block and kv head).
//
// Mathematics. Pair j of a head at position p turns by a = 2 pi frac(p f_j), f_j in
// turns per position: (x, y) -> (x cos a - y sin a, y cos a + x sin a). f_j is kept
// as a 64-bit fraction of a turn, so p * f_j modulo 2^64 is the angle's fraction of
// a turn exactly (one integer multiplication does the range reduction that a
// floating product loses at far positions); its upper 32 bits go to sincospif, an
// error of 2^-24 of half a turn, well under bf16's rounding of the result.
//
// Work. A unit is up to 16 dims of one head of one row: the two 16-byte vectors
// that hold both members of eight pairs, so a thread turns what it loads and may
// write it back in place. Sines and cosines are computed once per row (shared
// memory) and used by all its heads.
#include <cfloat>

#include "pkv_common.cuh"
#include "pkv_ops_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;  // head_dim <= 1024

__device__ __forceinline__ float2 turn(int64_t position, uint64_t turns, float scale)
{
    const uint64_t t = uint64_t(position) * turns;
    // the fraction of a turn in [-1/2, 1/2), in half turns
    const float x = float(int32_t(uint32_t(t >> 32))) * 0x1p-31f;
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * scale, s * scale);
}

// The dims of unit u of a head: 8 from `d0`, 8 from `d1` (d1 = D: none).
template <int FORM>
__device__ __forceinline__ void unit_dims(int u, int r, int D, int &d0, int &d1)
{
    if (FORM == kHalf && u < r / 16) {
        d0 = 8 * u;
        d1 = 8 * u + r / 2;
    } else {
        d0 = FORM == kHalf ? r + 16 * (u - r / 16) : 16 * u;
        d1 = d0 + 8;
    }
}

__device__ __forceinline__ void unpack8(uint4 w, float *x)
{
    x[0] = bf16lo_f32(w.x);
    x[1] = bf16hi_f32(w.x);
    x[2] = bf16lo_f32(w.y);
    x[3] = bf16hi_f32(w.y);
    x[4] = bf16lo_f32(w.z);
    x[5] = bf16hi_f32(w.z);
    x[6] = bf16lo_f32(w.w);
    x[7] = bf16hi_f32(w.w);
}

// The 16 values of unit u of the head at `src`, plain (rows of v).
template <int FORM>
__device__ __forceinline__ void load_unit(const uint16_t *src, int d0, int d1, int D, float *x)
{
    unpack8(*reinterpret_cast<const uint4 *>(src + d0), x);
    if (d1 < D)
        unpack8(*reinterpret_cast<const uint4 *>(src + d1), x + 8);
    else
#pragma unroll
        for (int i = 8; i < 16; ++i)
            x[i] = 0.f;
}

// The same, rotated by the row's `trig` (cos, sin of each pair).
template <int FORM>
__device__ __forceinline__ void load_rotated(const uint16_t *src, int u, int d0, int d1,
                                             const RopeParams &p, const float2 *trig, float *x)
{
    load_unit<FORM>(src, d0, d1, p.D, x);
    if (FORM == kHalf) {
        if (u < p.r / 16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 t = trig[d0 + i];
                const float a = x[i], b = x[i + 8];
                x[i] = a * t.x - b * t.y;
                x[i + 8] = b * t.x + a * t.y;
            }
        }
    } else if (FORM == kPairs) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const int d = (i < 8 ? d0 : d1 - 8) + i;
            if (d < p.r) {
                const float2 t = trig[d / 2];
                const float a = x[i], b = x[i + 1];
                x[i] = a * t.x - b * t.y;
                x[i + 1] = b * t.x + a * t.y;
            }
        }
    } else {
        const int h = p.r / 2;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int d = d0 + i;
            if (d < p.r) {  // r <= D: d is a dim of the head
                const bool second = p.interleaved ? (d & 1) : d >= h;
                const int j = p.interleaved ? d / 2 : (second ? d - h : d);
                const int o = p.interleaved ? d ^ 1 : (second ? j : d + h);
                const float2 t = trig[j];
                const float other = __uint_as_float(uint32_t(src[o]) << 16);
                x[i] = second ? x[i] * t.x + other * t.y : x[i] * t.x - other * t.y;
            }
        }
    }
}

__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void store_unit(uint16_t *dst, int d0, int d1, int D, const float *x)
{
    *reinterpret_cast<uint4 *>(dst + d0) = pack8(x);
    if (d1 < D)
        *reinterpret_cast<uint4 *>(dst + d1) = pack8(x + 8);
}

// Rotate the q heads of row i (all threads of the CTA; trig is in place).
template <int FORM>
__device__ __forceinline__ void rotate_q(const RopeParams &p, int64_t i, const float2 *trig)
{
    for (int e = threadIdx.x; e < p.Hq * p.units; e += kThreads) {
        const int h = e / p.units, u = e - h * p.units;
        int d0, d1;
        unit_dims<FORM>(u, p.r, p.D, d0, d1);
        float x[16];
        load_rotated<FORM>(p.q + i * p.q_stride + h * p.D, u, d0, d1, p, trig, x);
        store_unit(p.q_out + (i * p.Hq + h) * p.D, d0, d1, p.D, x);
    }
}

// bf16 pools: one CTA per row.
template <int FORM>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p)
{
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ float2 trig[kMaxPairs];
    const int64_t i = blockIdx.x;
    const int64_t pos = __ldg(p.positions + i);
    for (int j = threadIdx.x; j < p.r / 2; j += kThreads)
        trig[j] = turn(pos, __ldg(p.turns + j), p.scale);
    __syncthreads();
    rotate_q<FORM>(p, i, trig);
    const int64_t slot = __ldg(p.slots + i);
    if (slot < 0 || slot >= p.total_slots)
        return;
    for (int e = threadIdx.x; e < 2 * p.Hkv * p.units; e += kThreads) {
        int h = e / p.units;
        const int u = e - h * p.units;
        const bool is_v = h >= p.Hkv;
        h -= is_v ? p.Hkv : 0;
        int d0, d1;
        unit_dims<FORM>(u, p.r, p.D, d0, d1);
        float x[16];
        if (is_v)
            load_unit<FORM>(p.v + i * p.v_stride + h * p.D, d0, d1, p.D, x);
        else
            load_rotated<FORM>(p.k + i * p.k_stride + h * p.D, u, d0, d1, p, trig, x);
        store_unit(static_cast<uint16_t *>(is_v ? p.v_cache : p.k_cache) +
                       (slot * p.Hkv + h) * p.D,
                   d0, d1, p.D, x);
    }
}

__device__ __forceinline__ uint2 encode8(const float *x, float f)
{
    uint2 w;
    w.x = uint32_t(pack_e4m3x2(x[0] * f, x[1] * f)) |
          (uint32_t(pack_e4m3x2(x[2] * f, x[3] * f)) << 16);
    w.y = uint32_t(pack_e4m3x2(x[4] * f, x[5] * f)) |
          (uint32_t(pack_e4m3x2(x[6] * f, x[7] * f)) << 16);
    return w;
}

// 2^(byte difference); a difference below every code's range gives 0.
__device__ __forceinline__ float two_to(int e)
{
    return e < -126 ? 0.f : __uint_as_float(uint32_t(e + 127) << 23);
}

// Round eight codes to a scale 2^-e times larger (f = 2^e, e < 0).
__device__ __forceinline__ uint2 rescale8(uint2 w, float f)
{
    uint32_t h[4];
    e4m3x4_to_f16x2x2(w.x, h[0], h[1]);
    e4m3x4_to_f16x2x2(w.y, h[2], h[3]);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.f32.f16 %0, lo;\n\t"
            "cvt.f32.f16 %1, hi;\n\t}"
            : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
            : "r"(h[i]));
    return encode8(x, f);
}

// Block-scaled E4M3 pools. CTAs [0, n) rotate q; CTA n + i serves the block that row
// i opens in the batch (row i - 1 falls elsewhere): the run of up to 16 rows that
// fall into it, one warp for each (kv head, K or V). The warp finds the run's
// largest magnitude, settles the block's scale, rounds the block's earlier codes
// to it if it grew, and writes the run.
template <int FORM>
__global__ void __launch_bounds__(kThreads) rope_append_fp8_kernel(const RopeParams p)
{
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ float2 trig[kBlockSize * kMaxFp8BlockDim / 2];
    const int tid = threadIdx.x, half = p.r / 2;
    if (blockIdx.x < p.n && p.Hq > 0) {
        const int64_t i = blockIdx.x;
        const int64_t pos = __ldg(p.positions + i);
        for (int j = tid; j < half; j += kThreads)
            trig[j] = turn(pos, __ldg(p.turns + j), p.scale);
        __syncthreads();
        rotate_q<FORM>(p, i, trig);
        return;
    }
    const int64_t i0 = blockIdx.x - (p.Hq > 0 ? p.n : 0);
    auto block_of = [&](int64_t i) -> int64_t {
        const int64_t s = __ldg(p.slots + i);
        return s < 0 || s >= p.total_slots ? -1 : s / kBlockSize;
    };
    const int64_t block = block_of(i0);
    if (block < 0 || (i0 > 0 && block_of(i0 - 1) == block))
        return;
    int rows = 1;
    bool begun = __ldg(p.slots + i0) % kBlockSize == 0;
    while (rows < kBlockSize && i0 + rows < p.n && block_of(i0 + rows) == block) {
        begun |= __ldg(p.slots + i0 + rows) % kBlockSize == 0;
        ++rows;
    }
    for (int e = tid; e < rows * half; e += kThreads) {
        const int rr = e / half, j = e - rr * half;
        trig[e] = turn(__ldg(p.positions + i0 + rr), __ldg(p.turns + j), p.scale);
    }
    __syncthreads();

    const int warp = tid >> 5, lane = tid & 31;
    for (int task = warp; task < 2 * p.Hkv; task += kThreads / 32) {
        const bool is_v = task >= p.Hkv;
        const int h = is_v ? task - p.Hkv : task;
        uint8_t *codes = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) +
                         (block * kBlockSize * p.Hkv + h) * p.D;
        uint8_t *scale = (is_v ? p.v_scale : p.k_scale) + block * p.Hkv + h;
        auto value = [&](int rr, int u, int d0, int d1, float *x) {
            const int64_t i = i0 + rr;
            if (is_v)
                load_unit<FORM>(p.v + i * p.v_stride + h * p.D, d0, d1, p.D, x);
            else
                load_rotated<FORM>(p.k + i * p.k_stride + h * p.D, u, d0, d1, p, trig + rr * half, x);
        };
        float amax = 0.f;
        for (int e = lane; e < rows * p.units; e += 32) {
            const int rr = e / p.units, u = e - rr * p.units;
            int d0, d1;
            unit_dims<FORM>(u, p.r, p.D, d0, d1);
            float x[16];
            value(rr, u, d0, d1, x);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float a = fabsf(x[c]);
                amax = fmaxf(amax, a <= FLT_MAX ? a : 0.f);
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // the smallest byte with amax <= 448 * 2^(byte - 127): 448 = 1.75 * 2^8
        const uint32_t bits = __float_as_uint(amax);
        int code = int(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
        code = code < 1 ? 1 : code;
        const int old = begun ? 0 : *scale;
        code = old > code ? old : code;
        __syncwarp();  // every lane has read the scale
        if (lane == 0)
            *scale = uint8_t(code);
        if (old > 0 && code > old) {
            const float f = two_to(old - code);
            for (int e = lane; e < kBlockSize * (p.D / 8); e += 32) {
                const int rr = e / (p.D / 8), c = e - rr * (p.D / 8);
                uint2 *w = reinterpret_cast<uint2 *>(codes + int64_t(rr) * p.Hkv * p.D + 8 * c);
                *w = rescale8(*w, f);
            }
            __syncwarp();  // the new rows come after
        }
        const float inv = two_to(127 - code);
        for (int e = lane; e < rows * p.units; e += 32) {
            const int rr = e / p.units, u = e - rr * p.units;
            int d0, d1;
            unit_dims<FORM>(u, p.r, p.D, d0, d1);
            float x[16];
            value(rr, u, d0, d1, x);
            uint8_t *row = codes + (__ldg(p.slots + i0 + rr) % kBlockSize) * p.Hkv * p.D;
            *reinterpret_cast<uint2 *>(row + d0) = encode8(x, inv);
            if (d1 < p.D)
                *reinterpret_cast<uint2 *>(row + d1) = encode8(x + 8, inv);
        }
    }
}

template <int FORM>
cudaError_t launch(const RopeParams &p, cudaStream_t stream)
{
    if (p.k_scale) {
        const int64_t grid = p.Hq > 0 ? 2 * p.n : p.n;
        rope_append_fp8_kernel<FORM><<<unsigned(grid), kThreads, 0, stream>>>(p);
    } else {
        rope_append_kernel<FORM><<<unsigned(p.n), kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams &p, RopeForm form, cudaStream_t stream)
{
    if (form == kHalf)
        return launch<kHalf>(p, stream);
    if (form == kPairs)
        return launch<kPairs>(p, stream);
    return launch<kScalar>(p, stream);
}

}  // namespace pkv
