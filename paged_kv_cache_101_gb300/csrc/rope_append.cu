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
#include <algorithm>
#include <cfloat>

#include "pkv_common.cuh"
#include "pkv_ops_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xffffffffU;
constexpr int kMaxPairs = 512;  // head_dim <= 1024
constexpr int kSms = 152;       // what the choices by row count are made for

// Launched with programmatic serialization: wait for the kernel before this one on the
// stream, then let the one behind it start its own prologue.
__device__ __forceinline__ void begin_after_previous()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}

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

// A unit as it lies in memory (zeros where it has only eight dims).
struct Raw {
    uint4 a, b;
};

__device__ __forceinline__ Raw load_raw(const uint16_t *src, int d0, int d1, int D)
{
    Raw w;
    w.a = *reinterpret_cast<const uint4 *>(src + d0);
    w.b = d1 < D ? *reinterpret_cast<const uint4 *>(src + d1) : make_uint4(0, 0, 0, 0);
    return w;
}

__device__ __forceinline__ void unpack16(const Raw &w, float *x)
{
    unpack8(w.a, x);
    unpack8(w.b, x + 8);
}

// Where pair j's cosine and sine stand: the units' c-th pairs side by side, so that the
// lanes of a warp, each at another unit, read from different banks.
__device__ __forceinline__ int trig_at(int j, int half) { return (j & 7) * ((half + 7) / 8) + j / 8; }

// Rotate a unit's values by the row's `trig` (cos, sin of each pair); kScalar reads the
// partners at `src`.
template <int FORM>
__device__ __forceinline__ void rotate_unit(const uint16_t *src, int u, int d0, const RopeParams &p,
                                            const float2 *trig, float *x)
{
    if (FORM == kHalf) {
        if (u < p.r / 16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 t = trig[trig_at(8 * u + i, p.r / 2)];
                const float a = x[i], b = x[i + 8];
                x[i] = a * t.x - b * t.y;
                x[i + 8] = b * t.x + a * t.y;
            }
        }
    } else if (FORM == kPairs) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            if (d0 + i < p.r) {  // the unit's dims follow one another
                const float2 t = trig[trig_at((d0 + i) / 2, p.r / 2)];
                const float a = x[i], b = x[i + 1];
                x[i] = a * t.x - b * t.y;
                x[i + 1] = b * t.x + a * t.y;
            }
        }
    } else if (p.interleaved) {  // (as kPairs; the rotated part may end inside a vector)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            if (d0 + i < p.r) {
                const float2 t = trig[trig_at((d0 + i) / 2, p.r / 2)];
                const float a = x[i], b = x[i + 1];
                x[i] = a * t.x - b * t.y;
                x[i + 1] = b * t.x + a * t.y;
            }
        }
    } else {
        // halves of h dims: partners h dims away, in other vectors; four at a time where
        // h allows it
        const int h = p.r / 2;
        const auto turn_one = [&](int i, float other) {
            const int d = d0 + i;
            const bool second = d >= h;
            const float2 t = trig[trig_at(second ? d - h : d, h)];
            x[i] = second ? x[i] * t.x + other * t.y : x[i] * t.x - other * t.y;
        };
        if (h % 4 == 0) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (d0 + i < p.r) {
                    const int d = d0 + i;
                    const uint2 w = *reinterpret_cast<const uint2 *>(src + (d >= h ? d - h : d + h));
                    turn_one(i, bf16lo_f32(w.x));
                    turn_one(i + 1, bf16hi_f32(w.x));
                    turn_one(i + 2, bf16lo_f32(w.y));
                    turn_one(i + 3, bf16hi_f32(w.y));
                }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int d = d0 + i;
                if (d < p.r)  // r <= D: d is a dim of the head
                    turn_one(i, __uint_as_float(uint32_t(src[d >= h ? d - h : d + h]) << 16));
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
        const uint16_t *src = p.q + i * p.q_stride + h * p.D;
        float x[16];
        unpack16(load_raw(src, d0, d1, p.D), x);
        rotate_unit<FORM>(src, u, d0, p, trig, x);
        store_unit(p.q_out + (i * p.Hq + h) * p.D, d0, d1, p.D, x);
    }
}

// Any rotary_dim and head_dim: a CTA has `rows` rows, their sines and cosines in shared
// memory: one row, or as many as its threads have units for where the rows still fill the
// GPU (four CTAs an SM). 3,438 rows of 6 heads of 96 dims, 24 of them rotated: 18.9 us with
// a row each, 7.0 us with five; 64 rows of 48 heads of 80 dims 3.9 us. Bound by the 2-byte
// loads of the partners: 8,000 rows of 48 heads of 80 dims 48 us, 2.6 TB/s.
template <int FORM>
__global__ void __launch_bounds__(kThreads) rope_append_any_kernel(const RopeParams p, int rows)
{
    begin_after_previous();
    __shared__ float2 trig[kMaxPairs + 8];
    const int half = p.r / 2, pitch = (half + 7) / 8 * 8;
    const int64_t i0 = int64_t(blockIdx.x) * rows;
    rows = p.n - i0 < rows ? int(p.n - i0) : rows;
    for (int e = threadIdx.x; e < rows * half; e += kThreads) {
        const int rr = e / half, j = e - rr * half;
        trig[rr * pitch + trig_at(j, half)] =
            turn(__ldg(p.positions + i0 + rr), __ldg(p.turns + j), p.scale);
    }
    __syncthreads();
    const int per = (p.Hq + 2 * p.Hkv) * p.units;  // of q, k and v
    for (int e = threadIdx.x; e < rows * per; e += kThreads) {
        const int rr = e / per, f = e - rr * per;
        const int64_t i = i0 + rr;
        int h = f / p.units;
        const int u = f - h * p.units;
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
        h -= is_v ? p.Hq + p.Hkv : is_q ? 0 : p.Hq;
        const uint16_t *src;
        uint16_t *dst;
        if (is_q) {
            src = p.q + i * p.q_stride + h * p.D;
            dst = p.q_out + (i * p.Hq + h) * p.D;
        } else {
            const int64_t slot = __ldg(p.slots + i);
            if (slot < 0 || slot >= p.total_slots)
                continue;
            src = is_v ? p.v + i * p.v_stride + h * p.D : p.k + i * p.k_stride + h * p.D;
            dst = static_cast<uint16_t *>(is_v ? p.v_cache : p.k_cache) + (slot * p.Hkv + h) * p.D;
        }
        int d0, d1;
        unit_dims<FORM>(u, p.r, p.D, d0, d1);
        float x[16];
        unpack16(load_raw(src, d0, d1, p.D), x);
        if (!is_v)
            rotate_unit<FORM>(src, u, d0, p, trig + rr * pitch, x);
        store_unit(dst, d0, d1, p.D, x);
    }
}

// Vector forms with at most 32 units a head: `split` warps of a CTA share a row, each
// taking every split-th group of heads. A lane keeps one unit of its head, so its
// eight sines and cosines stay in registers for all heads of the row; no shared
// memory, no barrier, kAhead heads' loads in flight a lane. KV: k and v as well (the
// block-scaled append runs this for q alone).
// kAhead: three where three CTAs share an SM (80 registers), eight beside the block-scaled
// append, which has 128 anyway. 8,190 rows of 64 q and 8 kv heads, block-scaled, 3 / 4 / 6 / 8 /
// 10 heads ahead: 61.0 / 57.7 / 56.3 / 54.3 / 55.7 us (53.3 with the first ones asked for before
// the sines); 8,190 of 32 and 8, bf16, 3 with three CTAs, 6 or 8 with two: 33.4 / 35.2 / 38.0.
template <int FORM, bool KV, int kAhead>
__device__ __forceinline__ void rotate_row(const RopeParams &p, int64_t i, int part, int split,
                                           int lane)
{
    const int per = 32 / p.units;  // heads of one group
    const int u = lane % p.units, sub = lane / p.units;
    int d0, d1;
    unit_dims<FORM>(u, p.r, p.D, d0, d1);
    const bool two = d1 < p.D;
    const int64_t slot = KV ? __ldg(p.slots + i) : -1;
    const bool stored = slot >= 0 && slot < p.total_slots;
    const int64_t pos = __ldg(p.positions + i);
    // groups of q heads, then of k's and v's (of one kind each: the choice is the warp's)
    const int nq = (p.Hq + per - 1) / per, nk = KV ? (p.Hkv + per - 1) / per : 0;
    const int groups = nq + (stored ? 2 * nk : 0);
    const bool turns = FORM == kHalf ? u < p.r / 16 : 16 * u < p.r;
    uint4 a[kAhead], b[kAhead];
    uint16_t *to[kAhead];
    bool rot[kAhead];
    const auto load = [&](int g0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            int group = g0 + k * split, heads = p.Hq;
            const uint16_t *from = p.q + i * p.q_stride;
            uint16_t *dst = p.q_out + i * p.Hq * p.D;
            const bool in = group < groups;
            rot[k] = turns;
            if (KV && group >= nq) {
                group -= nq;
                heads = p.Hkv;
                const bool is_v = group >= nk;
                group -= is_v ? nk : 0;
                from = is_v ? p.v + i * p.v_stride : p.k + i * p.k_stride;
                dst = static_cast<uint16_t *>(is_v ? p.v_cache : p.k_cache) + slot * p.Hkv * p.D;
                rot[k] = turns && !is_v;
            }
            const int h = group * per + sub;
            to[k] = in && sub < per && h < heads ? dst + h * p.D : nullptr;
            a[k] = b[k] = make_uint4(0, 0, 0, 0);
            if (to[k]) {
                a[k] = *reinterpret_cast<const uint4 *>(from + h * p.D + d0);
                if (two)
                    b[k] = *reinterpret_cast<const uint4 *>(from + h * p.D + d1);
            }
        }
    };
    load(part);  // on their way while the sines are computed
    float2 t[8];
    // pair 8 u + c is the unit's c-th in both layouts
    auto pair = [&](int c) {
        return turns && 8 * u + c < p.r / 2 ? turn(pos, __ldg(p.turns + 8 * u + c), p.scale)
                                            : make_float2(0.f, 0.f);
    };
    if (per == 4) {
        // four lanes hold the same unit of four heads: each computes two pairs for all
        const float2 lo = pair(sub), hi = pair(sub + 4);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float2 from = c < 4 ? lo : hi;
            t[c].x = __shfl_sync(kAll, from.x, (c & 3) * p.units + u);
            t[c].y = __shfl_sync(kAll, from.y, (c & 3) * p.units + u);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            t[c] = pair(c);
    }
    for (int g0 = part; g0 < groups; g0 += split * kAhead) {
        if (g0 != part)
            load(g0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (!to[k])
                continue;
            if (rot[k]) {
                float x[16];
                unpack8(a[k], x);
                unpack8(b[k], x + 8);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int m = FORM == kHalf ? c : 2 * c, n = FORM == kHalf ? c + 8 : 2 * c + 1;
                    if (FORM == kHalf || 8 * u + c < p.r / 2) {
                        const float v = x[m], w = x[n];
                        x[m] = v * t[c].x - w * t[c].y;
                        x[n] = w * t[c].x + v * t[c].y;
                    }
                }
                a[k] = pack8(x);
                b[k] = pack8(x + 8);
            }
            *reinterpret_cast<uint4 *>(to[k] + d0) = a[k];
            if (two)
                *reinterpret_cast<uint4 *>(to[k] + d1) = b[k];
        }
    }
}

// FEW: CTAs that are two an SM at most, with registers to load the first heads while the
// sines are computed: 256 rows of 64 q heads 4.5 -> 3.9 us; 320 (above it) 4.2 instead of 4.9.
template <int FORM, bool FEW>
__global__ void __launch_bounds__(kThreads, FEW ? 2 : 3) rope_append_kernel(const RopeParams p, int split)
{
    begin_after_previous();
    const int warp = threadIdx.x >> 5, rows = kThreads / 32 / split;
    const int64_t i = int64_t(blockIdx.x) * rows + warp / split;
    if (i < p.n)
        rotate_row<FORM, true, FEW ? 3 : 3>(p, i, warp % split, split, threadIdx.x & 31);
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

// Round a block's codes of one head to a larger scale (one warp; `vecs` 8-byte words a
// row). Not inlined: it happens a few times in a block's life, and its registers would
// be the run's.
__device__ __noinline__ void rescale_block(uint8_t *codes, int64_t row_bytes, int vecs, float f,
                                           int lane)
{
    for (int e0 = 0; e0 < kBlockSize * vecs; e0 += 8 * 32) {
        uint2 w[8], *to[8];  // eight loads wait together
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int e = e0 + 32 * k + lane, rr = e / vecs, c = e - rr * vecs;
            to[k] = reinterpret_cast<uint2 *>(codes + rr * row_bytes + 8 * c);
            if (rr < kBlockSize)
                w[k] = *to[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if ((e0 + 32 * k + lane) / vecs < kBlockSize)
                *to[k] = rescale8(w[k], f);
    }
}

// The smallest byte with amax <= 448 * 2^(byte - 127), 448 = 1.75 * 2^8, but at least `old`.
__device__ __forceinline__ int scale_code(float amax, int old)
{
    const uint32_t bits = __float_as_uint(amax);
    int code = int(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    code = code < 1 ? 1 : code;
    return old > code ? old : code;
}

// The scale byte of a block and head (`old`, 0: started here) once rows of largest finite
// magnitude amax join it: written where it changed, the codes so far rounded to it.
__device__ __forceinline__ int settle(float amax, int old, uint8_t *codes, uint8_t *scale,
                                      int64_t row_bytes, int vecs, int lane)
{
    const int code = scale_code(amax, old);
    __syncwarp();  // every lane has read the old byte
    if (lane == 0 && code != old)
        *scale = uint8_t(code);
    if (old > 0 && code > old) {
        rescale_block(codes, row_bytes, vecs, two_to(old - code), lane);
        __syncwarp();  // the new rows come after
    }
    return code;
}

// Where pass after pass of a warp over a run's units stands: unit u of row rr.
struct UnitAt {
    int rr, u, step_r, step_u, units;
    __device__ __forceinline__ UnitAt(int lane, int units_)
        : rr(lane / units_), u(lane - lane / units_ * units_), step_r(32 / units_),
          step_u(32 - 32 / units_ * units_), units(units_)
    {
    }
    __device__ __forceinline__ void next()
    {
        rr += step_r;
        u += step_u;
        if (u >= units) {
            u -= units;
            ++rr;
        }
    }
};

// One run: up to 16 rows from i0 that fall into one block, for head h of K or V, by one
// warp. It holds the run in registers, finds its largest magnitude, settles the block's
// scale, rounds the block's earlier codes to it if it grew, and writes the run. Lane
// l0 + r brings the slot of row i0 + r; `raw` the run's rows, pass by pass; trig its
// sines and cosines; `old` the block's scale byte (0: the run starts the block).
template <int FORM, int PASSES>
__device__ __forceinline__ void append_run(const RopeParams &p, const Raw (&raw)[PASSES], int64_t i0,
                                           int rows, int64_t block, int old, int64_t slot,
                                           int l0, bool is_v, int h, const float2 *trig,
                                           const UnitAt &start, int lane)
{
    const int pitch = (p.r / 2 + 7) / 8 * 8;
    uint8_t *codes = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) +
                     (block * kBlockSize * p.Hkv + h) * p.D;
    uint8_t *scale = (is_v ? p.v_scale : p.k_scale) + block * p.Hkv + h;
    // pass k: unit e % units of row e / units of the run, e = lane + 32 k. The values are
    // computed twice, for the largest magnitude and for the codes: kept, they would take
    // 64 registers and with them half of the CTAs of an SM.
    auto values = [&](int k, int rr, int u, int d0, float *x) {
        unpack16(raw[k], x);
        if (!is_v)
            rotate_unit<FORM>(p.k + (i0 + rr) * p.k_stride + h * p.D, u, d0, p, trig + rr * pitch, x);
    };
    auto largest = [&](float below) {
        float amax = 0.f;
        UnitAt at = start;
#pragma unroll
        for (int k = 0; k < PASSES; ++k, at.next()) {
            if (at.rr < rows) {
                int d0, d1;
                unit_dims<FORM>(at.u, p.r, p.D, d0, d1);
                float x[16];
                values(k, at.rr, at.u, d0, x);
#pragma unroll
                for (int c = 0; c < 16; ++c)  // (fmaxf passes over NaN)
                    amax = fmaxf(amax, below == INFINITY || fabsf(x[c]) <= below ? fabsf(x[c]) : 0.f);
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
        return amax;
    };
    float amax = largest(INFINITY);
    if (__builtin_expect(amax == INFINITY, 0))
        amax = largest(FLT_MAX);  // an infinity among them: the largest finite one counts
    const int code = settle(amax, old, codes, scale, p.Hkv * p.D, p.D / 8, lane);
    const float inv = two_to(127 - code);
    const int offset = int(slot) & (kBlockSize - 1);  // slots in use are not negative
    UnitAt at = start;
#pragma unroll
    for (int k = 0; k < PASSES; ++k, at.next()) {
        const int to = __shfl_sync(kAll, offset, l0 + (at.rr < rows ? at.rr : 0));
        if (at.rr < rows) {
            int d0, d1;
            unit_dims<FORM>(at.u, p.r, p.D, d0, d1);
            float x[16];
            values(k, at.rr, at.u, d0, x);
            uint8_t *row = codes + to * p.Hkv * p.D;
            *reinterpret_cast<uint2 *>(row + d0) = encode8(x, inv);
            if (d1 < p.D)
                *reinterpret_cast<uint2 *>(row + d1) = encode8(x + 8, inv);
        }
    }
}

// The same for heads of 128 dims in vector form, eight units a row: lane l has unit l % 8
// of rows l / 8, l / 8 + 4, ..
template <int FORM>
__device__ __forceinline__ void append_run_128(const RopeParams &p, const Raw (&raw)[4], int rows,
                                               int64_t block, int old, int64_t slot, int l0,
                                               bool is_v, int h, const float2 *trig, int pitch,
                                               int lane)
{
    const int u = lane & 7, sub = lane >> 3;
    const int64_t row_bytes = int64_t(p.Hkv) * 128;
    uint8_t *codes = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) +
                     block * kBlockSize * row_bytes + h * 128;
    const int nu = pitch / 8;
    const int pairs = is_v ? 0 : FORM == kHalf ? (u < p.r / 16 ? 8 : 0)
                                               : min(max(p.r / 2 - 8 * u, 0), 8);
    auto values = [&](int k, float *x) {
        unpack16(raw[k], x);
        const float2 *t = trig + (4 * k + sub) * pitch + u;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int m = FORM == kHalf ? c : 2 * c, n = FORM == kHalf ? c + 8 : 2 * c + 1;
            if (c < pairs) {
                const float2 cs = t[c * nu];
                const float v = x[m], w = x[n];
                x[m] = v * cs.x - w * cs.y;
                x[n] = w * cs.x + v * cs.y;
            }
        }
    };
    auto largest = [&](float below) {
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (4 * k + sub < rows) {
                float x[16];
                values(k, x);
#pragma unroll
                for (int c = 0; c < 16; ++c)  // (fmaxf passes over NaN)
                    amax = fmaxf(amax, below == INFINITY || fabsf(x[c]) <= below ? fabsf(x[c]) : 0.f);
            }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
        return amax;
    };
    float amax = largest(INFINITY);
    if (__builtin_expect(amax == INFINITY, 0))
        amax = largest(FLT_MAX);  // an infinity among them: the largest finite one counts
    const int code = settle(amax, old, codes, (is_v ? p.v_scale : p.k_scale) + block * p.Hkv + h,
                            row_bytes, 16, lane);
    const float inv = two_to(127 - code);
    const int offset = int(slot) & (kBlockSize - 1);  // slots in use are not negative
    int d0, d1;
    unit_dims<FORM>(u, p.r, 128, d0, d1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int to = __shfl_sync(kAll, offset, (l0 + 4 * k + sub) & 31);
        if (4 * k + sub < rows) {
            float x[16];
            values(k, x);
            uint8_t *row = codes + to * row_bytes;
            *reinterpret_cast<uint2 *>(row + d0) = encode8(x, inv);
            *reinterpret_cast<uint2 *>(row + d1) = encode8(x + 8, inv);
        }
    }
}

// Runs of one row (a decode step's), heads of 128 dims in vector form: eight lanes have a
// head, a warp four heads of one row, a CTA eight heads of four rows at a time. Lane l has
// the block, slot and position of row `first` + l; `singles` the lanes whose row is a run.
// No barrier and no shared memory, unlike longer runs.
template <int FORM>
__device__ __forceinline__ void append_singles(const RopeParams &p, unsigned singles, int64_t first,
                                               int64_t mine, int64_t slot, int64_t pos, bool is_v,
                                               int h0, int warp, int lane)
{
    const int u = lane & 7, sub = lane >> 3;
    const int64_t row_bytes = int64_t(p.Hkv) * 128;
    const int h = h0 + (warp & 1) * 4 + sub;
    const bool ok = h < p.Hkv;
    int d0, d1;
    unit_dims<FORM>(u, p.r, 128, d0, d1);
    const int pairs = is_v ? 0 : FORM == kHalf ? (u < p.r / 16 ? 8 : 0)
                                               : min(max(p.r / 2 - 8 * u, 0), 8);
    for (int k = 0; singles != 0; ++k, singles &= singles - 1) {
        if ((k & 3) != warp >> 1)
            continue;
        const int l0 = __ffs(singles) - 1;
        const int64_t i = first + l0;
        const int64_t block = __shfl_sync(kAll, mine, l0);
        const int at = int(__shfl_sync(kAll, slot, l0)) & (kBlockSize - 1);
        const int64_t position = __shfl_sync(kAll, pos, l0);
        uint8_t *scale = (is_v ? p.v_scale : p.k_scale) + block * p.Hkv + h;
        int old = 0;
        Raw raw;
        raw.a = raw.b = make_uint4(0, 0, 0, 0);
        if (ok) {
            if (at != 0)
                old = *scale;
            raw = load_raw((is_v ? p.v + i * p.v_stride : p.k + i * p.k_stride) + h * 128, d0, d1,
                           128);
        }
        float2 t[8];
        if (!is_v) {
            // four lanes have the same unit of four heads: each computes two pairs for all
            const float2 lo = sub < pairs ? turn(position, __ldg(p.turns + 8 * u + sub), p.scale)
                                          : make_float2(0.f, 0.f);
            const float2 hi = sub + 4 < pairs
                                  ? turn(position, __ldg(p.turns + 8 * u + sub + 4), p.scale)
                                  : make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float2 from = c < 4 ? lo : hi;
                t[c].x = __shfl_sync(kAll, from.x, (c & 3) * 8 + u);
                t[c].y = __shfl_sync(kAll, from.y, (c & 3) * 8 + u);
            }
        }
        float x[16];
        unpack16(raw, x);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int m = FORM == kHalf ? c : 2 * c, n = FORM == kHalf ? c + 8 : 2 * c + 1;
            if (c < pairs) {
                const float v = x[m], w = x[n];
                x[m] = v * t[c].x - w * t[c].y;
                x[n] = w * t[c].x + v * t[c].y;
            }
        }
        float amax = 0.f;  // of the finite ones
#pragma unroll
        for (int c = 0; c < 16; ++c)
            amax = fmaxf(amax, fabsf(x[c]) <= FLT_MAX ? fabsf(x[c]) : 0.f);
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
        const int code = scale_code(amax, old);
        uint8_t *codes = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) +
                         block * kBlockSize * row_bytes + h * 128;
        __syncwarp();  // every lane has read the old byte
        if (ok && u == 0 && code != old)
            *scale = uint8_t(code);
        // heads whose scale grew: the whole warp rounds their codes so far to it
        for (unsigned grew = __ballot_sync(kAll, ok && u == 0 && old > 0 && code > old); grew != 0;
             grew &= grew - 1) {
            const int from = __ffs(grew) - 1;
            const int64_t to = __shfl_sync(kAll, int64_t(reinterpret_cast<uintptr_t>(codes)),
                                           from);
            rescale_block(reinterpret_cast<uint8_t *>(to), row_bytes, 16,
                          two_to(__shfl_sync(kAll, old - code, from)), lane);
        }
        __syncwarp();  // the new rows come after
        if (ok) {
            const float inv = two_to(127 - code);
            uint8_t *row = codes + at * row_bytes;
            *reinterpret_cast<uint2 *>(row + d0) = encode8(x, inv);
            *reinterpret_cast<uint2 *>(row + d1) = encode8(x + 8, inv);
        }
    }
}

// Block-scaled E4M3 pools. `q_ctas` CTAs rotate q. Of the others, CTA (w, y) serves the
// runs that start in the `window` rows from w * window on (a row starts one where the
// row before it falls into another block), for eight heads of K (y even) or V, a warp
// each. A prompt has a run in 16 rows, and a CTA that finds none still costs its slot on an
// SM: 8,190 rows, K and V alone, 42.3 us with eight rows looked at one after another, 24.9 us
// with one look at eight, 18.8 us at sixteen. SINGLES: runs of one row apart, many at a time
// (256 rows of a decode step, 32 q and 8 kv heads, 8.7 -> 4.4 us, 1000 rows 18.9 -> 7.7); not
// for prompts, where the code beside it costs 8,190 rows 53.0 -> 55.1 us. Bound by the latency
// of slots, then rows, then stores while rows are few (64 rows with q 3.3 us); at 8,190 rows
// of 64 q and 8 kv heads 53.0 us, 88% of the measured copy bandwidth.
// PASSES 0: heads of 128 dims in vector form.
template <int FORM, int PASSES, bool SINGLES = false>
__global__ void __launch_bounds__(kThreads, PASSES == 8 ? 1 : 2)
    rope_append_fp8_kernel(const RopeParams p, int split, int64_t q_ctas, int window)
{
    begin_after_previous();
    __shared__ float2 trig[kBlockSize * (kMaxFp8BlockDim / 2 + 8)];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = p.r / 2;
    // the two kinds of CTAs are spread evenly over the grid, so that those that wait on
    // latency run beside those that wait on bandwidth
    const int64_t q_before = int64_t(blockIdx.x) * q_ctas / gridDim.x;
    if ((int64_t(blockIdx.x) + 1) * q_ctas / gridDim.x > q_before) {
        if constexpr (FORM != kScalar) {
            const int64_t i = q_before * (kThreads / 32 / split) + warp / split;
            if (i < p.n)
                rotate_row<FORM, false, 8>(p, i, warp % split, split, lane);
        } else {
            const int64_t i = q_before;
            const int64_t pos = __ldg(p.positions + i);
            for (int j = tid; j < half; j += kThreads)
                trig[trig_at(j, half)] = turn(pos, __ldg(p.turns + j), p.scale);
            __syncthreads();
            rotate_q<FORM>(p, i, trig);
        }
        return;
    }
    const int groups = (p.Hkv + 7) / 8;
    const int64_t at = blockIdx.x - q_before;
    const int64_t w = at / (2 * groups);
    const int y = int(at - w * (2 * groups));
    const bool is_v = y & 1;
    const int h = (y >> 1) * 8 + warp;
    const uint64_t turns0 = __ldg(p.turns + tid % half);
    const int pitch = (half + 7) / 8 * 8;
    const UnitAt start(lane, p.units);
    // lane l: slot and position of row w * window + l - 1 (the row before the window, the
    // window, and the rows that its last run may reach)
    const int64_t first = w * window - 1;
    const bool in = first + lane >= 0 && first + lane < p.n && lane <= window + kBlockSize - 1;
    const int64_t slot = in ? __ldg(p.slots + first + lane) : -1;
    const int64_t pos = in && !is_v ? __ldg(p.positions + first + lane) : 0;
    const int64_t mine = slot < 0 || slot >= p.total_slots ? -1 : slot / kBlockSize;
    const int64_t before = __shfl_up_sync(kAll, mine, 1);
    unsigned opens = __ballot_sync(kAll, lane >= 1 && lane <= window && mine >= 0 && mine != before);
    if constexpr (SINGLES) {
        const int64_t after = __shfl_down_sync(kAll, mine, 1);
        const unsigned singles = opens & __ballot_sync(kAll, mine != after);
        append_singles<FORM>(p, singles, first, mine, slot, pos, is_v, (y >> 1) * 8, warp, lane);
        opens &= ~singles;
    }
    for (unsigned left = opens; left != 0; left &= left - 1) {
        const int l0 = __ffs(left) - 1;  // the run's first row is lane l0's
        const int64_t i0 = first + l0;
        const int64_t block = __shfl_sync(kAll, mine, l0);
        const unsigned same = __ballot_sync(kAll, mine == block) >> l0;
        const int rows = min(same == kAll ? 32 : __ffs(~same) - 1, kBlockSize);
        const bool begun = __ballot_sync(kAll, lane >= l0 && lane < l0 + rows &&
                                                          slot % kBlockSize == 0) != 0;
        // the run's rows and scale are on their way while the sines are computed
        Raw raw[PASSES ? PASSES : 4];
        int old = 0;
        if (h < p.Hkv) {
            if (!begun)
                old = (is_v ? p.v_scale : p.k_scale)[block * p.Hkv + h];
            const int64_t stride = is_v ? p.v_stride : p.k_stride;
            const uint16_t *src = (is_v ? p.v : p.k) + i0 * stride + h * p.D;
            if constexpr (PASSES == 0) {
                int d0, d1;
                unit_dims<FORM>(lane & 7, p.r, 128, d0, d1);
                src += (lane >> 3) * stride;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    raw[k].a = raw[k].b = make_uint4(0, 0, 0, 0);
                    if (4 * k + (lane >> 3) < rows)
                        raw[k] = load_raw(src + 4 * k * stride, d0, d1, 128);
                }
            }
            UnitAt at = start;
#pragma unroll
            for (int k = 0; k < PASSES; ++k, at.next())
                if (at.rr < rows) {
                    int d0, d1;
                    unit_dims<FORM>(at.u, p.r, p.D, d0, d1);
                    raw[k] = load_raw(src + at.rr * stride, d0, d1, p.D);
                }
        }
        if (!is_v) {
            __syncthreads();  // the run before is written
            for (int e0 = 0; e0 < rows * half; e0 += kThreads) {
                const int e = e0 + tid, rr = e / half, j = e - rr * half;
                const int64_t at_row = __shfl_sync(kAll, pos, l0 + (rr < rows ? rr : 0));
                if (rr < rows)
                    trig[rr * pitch + trig_at(j, half)] =
                        turn(at_row, e0 == 0 ? turns0 : __ldg(p.turns + j), p.scale);
            }
            __syncthreads();
        }
        if (h >= p.Hkv)
            continue;
        if constexpr (PASSES == 0)
            append_run_128<FORM>(p, raw, rows, block, old, slot, l0, is_v, h, trig, pitch, lane);
        else
            append_run<FORM, PASSES>(p, raw, i0, rows, block, old, slot, l0, is_v, h, trig, start,
                                     lane);
    }
}

// A launch whose start may overlap the end of the kernel before it on the stream (the
// kernels wait before they touch memory).
template <typename... K, typename... A>
cudaError_t launch_overlapped(void (*kern)(K...), int64_t grid, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int FORM>
cudaError_t launch(const RopeParams &p, cudaStream_t stream)
{
    constexpr int kWarps = kThreads / 32;
    // Warps of a row: as many as leave two CTAs an SM or fewer, and two at least (each warp of
    // a row computes its sines and cosines again). 600 rows of 32 q and 8 kv heads, 8 / 4 / 2
    // warps: 5.4 / 3.6 / 3.7 us; 1000: 7.4 / - / 4.8; 8,190, 1 / 2 / 4 warps: 34.9 / 33.8 / 36.9
    // (33.4 now, 88% of the measured copy bandwidth).
    int split = p.n <= 2 * kSms ? kWarps : p.n <= 4 * kSms ? 4 : 2, window = 0;
    if (p.k_scale) {
        // With the windows' CTAs beside them (eight kv heads or fewer); one warp once rows are
        // many, for the append's own arithmetic fills the issue slots (8,190 rows, 1 / 2 / 4
        // warps: 65.7 / 69.6 / 78.5 us, an earlier form). Windows of 2 / 4 / 8 at 8 or 4 warps,
        // 400 rows of 32 q and 8 kv heads: 6.2 / - / 4.6 us where each is a run, 6.7 / - / 6.1
        // in runs of four, 7.9 / - / 6.6 in one sequence; 128: 3.5 / 3.5 / 4.3, 4.1 / 4.0 / 5.8,
        // 6.0 / 6.0 / 6.0.
        const int64_t full = 2 * kSms;
        window = p.n <= full * 2 / 3 ? 4 : p.n < 4096 ? 8 : 16;
        split = p.n <= full * 2 / 3 ? kWarps : p.n <= full * 4 / 3 ? 4 : p.n <= full * 2 ? 2 : 1;
    }
    const int rows = kWarps / split;
    const int64_t row_ctas = (p.n + rows - 1) / rows;
    if (p.k_scale) {
        const int64_t q_ctas = p.Hq == 0 ? 0 : FORM == kScalar ? p.n : row_ctas;
        const int64_t grid = q_ctas + (p.n + window - 1) / window * 2 * ((p.Hkv + 7) / 8);
        if constexpr (FORM != kScalar) {
            if (p.D == 128)
                return launch_overlapped(p.n < 4096 ? rope_append_fp8_kernel<FORM, 0, true>
                                                    : rope_append_fp8_kernel<FORM, 0>,
                                         grid, stream, p, split, q_ctas, window);
        }
        if (p.units * kBlockSize <= 32 * 4)
            return launch_overlapped(rope_append_fp8_kernel<FORM, 4>, grid, stream, p, split,
                                     q_ctas, window);
        return launch_overlapped(rope_append_fp8_kernel<FORM, 8>, grid, stream, p, split, q_ctas,
                                 window);
    }
    if constexpr (FORM != kScalar) {
        if (p.units <= 32)
            return launch_overlapped(row_ctas <= 2 * kSms ? rope_append_kernel<FORM, true>
                                                     : rope_append_kernel<FORM, false>,
                                     row_ctas, stream, p, split);
    }
    const int per = (p.Hq + 2 * p.Hkv) * p.units, pitch = (p.r / 2 + 7) / 8 * 8;
    const int64_t many = std::min<int64_t>(std::min(kThreads / per, kMaxPairs / pitch), p.n / (4 * kSms));
    const int any_rows = many > 1 ? int(many) : 1;
    return launch_overlapped(rope_append_any_kernel<FORM>, (p.n + any_rows - 1) / any_rows, stream, p,
                             any_rows);
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
