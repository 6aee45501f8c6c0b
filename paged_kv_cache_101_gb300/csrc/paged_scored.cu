// paged_scored.cu -- paged decode attention with capped scores, a distance bias or
// a sliding window, over bf16 or block-scaled E4M3 pools.
//
// The simplest form: one CTA per (sequence, kv head) walks the sequence's blocks;
// scores, softmax statistics and the accumulator live in shared memory in fp32.
#include <cuda_bf16.h>

#include <algorithm>

#include "pkv_common.cuh"
#include "pkv_ops_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float e4m3_value(uint8_t c)
{
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(c, lo, hi);
    float f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(lo));
    return f;
}

__global__ void __launch_bounds__(kThreads) scored_simple_kernel(const ScoredParams p, const void *kc,
                                                                 const void *vc, int D)
{
    extern __shared__ float sm[];
    const DecodeParams &d = p.d;
    const int R = d.rows, s = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    float *q = sm, *acc = q + R * D, *k = acc + R * D, *v = k + 16 * D, *x = v + 16 * D;
    float *m = x + R * 16, *l = m + R, *corr = l + R;
    int T = d.context_lens[s];
    T = min(max(T, 0), d.MB * kBlockSize);
    for (int e = tid; e < R * D; e += kThreads) {
        const int row = e / D, j = row / d.G, g = row - j * d.G;
        q[e] = __uint_as_float(uint32_t(d.q[((int64_t(s) * d.nq + j) * d.Hq + h * d.G + g) * D + e % D]) << 16);
        acc[e] = 0.f;
    }
    for (int r = tid; r < R; r += kThreads) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    const int first = p.window ? max(0, T - d.nq - p.window + 1) : 0;
    for (int b = first / kBlockSize; b * kBlockSize < T; ++b) {
        const int phys = d.block_tables[int64_t(s) * d.MB + b];
        const bool ok = phys >= 0 && phys < d.num_blocks;
        if (!ok && tid == 0)
            atomicOr(d.ws, kErrBadBlock);
        __syncthreads();
        for (int e = tid; e < 16 * D; e += kThreads) {
            const int t = b * kBlockSize + e / D;
            const int64_t at = ((int64_t(phys) * kBlockSize + e / D) * d.Hkv + h) * D + e % D;
            float kv = 0.f, vv = 0.f;
            if (ok && t < T && t >= first) {
                if (p.k_scale) {
                    const int64_t sc = int64_t(phys) * d.Hkv + h;
                    kv = ldexpf(e4m3_value(static_cast<const uint8_t *>(kc)[at]), int(p.k_scale[sc]) - 127);
                    vv = ldexpf(e4m3_value(static_cast<const uint8_t *>(vc)[at]), int(p.v_scale[sc]) - 127);
                } else {
                    kv = __uint_as_float(uint32_t(static_cast<const uint16_t *>(kc)[at]) << 16);
                    vv = __uint_as_float(uint32_t(static_cast<const uint16_t *>(vc)[at]) << 16);
                }
            }
            k[e] = kv;
            v[e] = vv;
        }
        __syncthreads();
        for (int e = tid; e < R * 16; e += kThreads) {
            const int row = e / 16, t = b * kBlockSize + e % 16, j = row / d.G;
            const int pos = T - d.nq + j;
            float y = 0.f;
            for (int c = 0; c < D; ++c)
                y = fmaf(q[row * D + c], k[(e % 16) * D + c], y);
            y *= p.scale;
            if (p.softcap > 0.f)
                y = p.softcap * tanhf(y / p.softcap);
            if (p.slopes)
                y += p.slopes[h * d.G + row - j * d.G] * float(t - pos);
            const bool seen = t <= pos && (!p.window || t > pos - p.window);
            x[e] = seen ? y : -INFINITY;
        }
        __syncthreads();
        for (int r = tid; r < R; r += kThreads) {
            float top = m[r];
            for (int c = 0; c < 16; ++c)
                top = fmaxf(top, x[r * 16 + c]);
            const float mu = top == -INFINITY ? 0.f : top;
            corr[r] = expf(m[r] - mu);
            float sum = 0.f;
            for (int c = 0; c < 16; ++c) {
                x[r * 16 + c] = expf(x[r * 16 + c] - mu);
                sum += x[r * 16 + c];
            }
            l[r] = l[r] * corr[r] + sum;
            m[r] = top;
        }
        __syncthreads();
        for (int e = tid; e < R * D; e += kThreads) {
            float a = acc[e] * corr[e / D];
            for (int c = 0; c < 16; ++c)
                a = fmaf(x[e / D * 16 + c], v[c * D + e % D], a);
            acc[e] = a;
        }
    }
    __syncthreads();
    for (int e = tid; e < R * D; e += kThreads) {
        const int row = e / D, j = row / d.G, g = row - j * d.G;
        const int64_t o = ((int64_t(s) * d.nq + j) * d.Hq + h * d.G + g) * D + e % D;
        const float y = l[row] > 0.f ? acc[e] / l[row] : (l[row] == 0.f ? 0.f : l[row]);
        if (d.out_f32)
            static_cast<float *>(d.out)[o] = y;
        else
            static_cast<__nv_bfloat16 *>(d.out)[o] = __float2bfloat16_rn(y);
    }
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace

int plan_scored(int S, int nq, int Hq, int Hkv, int D, int MB, int num_sms, int smem_optin,
                int fp8, DecodePlan *pl)
{
    (void)MB;
    (void)num_sms;
    DecodePlan P{};
    P.D = D;
    P.kv8 = fp8;
    P.G = Hq / Hkv;
    P.rows = P.G * nq;
    P.HG = 1;
    P.n_hg = Hkv;
    P.wph = 1;
    P.smem = size_t(2 * P.rows * D + 32 * D + P.rows * 19) * 4;
    if (int(P.smem) > smem_optin || Hkv > 65535)
        return -1;
    P.off_rec = kWsHeaderBytes;
    P.off_ml = P.off_rec + round_up(size_t(S) * P.n_hg * 8, 256);
    P.off_part = P.off_ml;
    P.ws_bytes = P.off_part;
    *pl = P;
    return 0;
}

cudaError_t launch_scored(const DecodePlan &pl, const ScoredParams &p, const void *kc,
                          const void *vc, cudaStream_t stream)
{
    cudaError_t e = cudaFuncSetAttribute(scored_simple_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, int(pl.smem));
    if (e != cudaSuccess)
        return e;
    scored_simple_kernel<<<dim3(unsigned(p.d.S), unsigned(p.d.Hkv)), kThreads, pl.smem, stream>>>(
        p, kc, vc, pl.D);
    return cudaGetLastError();
}

}  // namespace pkv
