// RMS norm of the residual stream, fused with the stream's addition and with an 8-bit output, and its backward pass.
//
//   s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w            (row by row, fp32 inside)
//   8-bit output: scale = max(amax |y|, 1e-30) / 448 per row or per 128 channels, code = e4m3(y / scale).
// The norm reads the sum before it is rounded to the stream's type; a NaN in a group makes its scale NaN.
//
// Backward, with xhat = s rstd and gw = w dy:
//   dx = ds + rstd (gw - xhat mean(gw xhat)),   dw = sum over rows of dy xhat,
// where ds is the gradient that reaches s by the residual path (s feeds the next layer too); dx is the gradient of
// x and of r alike.  The 8-bit rounding passes gradients straight through.
//
// All of it is bound by HBM: every operand is read once and written once, a row stays in registers between its sum
// and its output, and 8 channels per thread (16 bytes of bf16) are one access.
#pragma once

#include "gdn_kv.cuh"

namespace gdn {

struct NormParams {
    const void* x;
    const void* res;       // or null
    const float* weight;   // [d]
    void* s;               // x + res, or null
    void* y;
    float* y_scale;        // 8-bit output
    float* rstd;           // [rows] or null
    long long rows;
    int d;
    float eps;
};

template <typename T> __device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
    Vec16<__nv_bfloat16>::get(*reinterpret_cast<const uint4*>(p), x);
}
template <> __device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float (&x)[8]);
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                              pack_bf16x2(x[6], x[7]));
}
template <> __device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Reduction over the threads of a row: a warp's by shuffles; with several warps also through sm, in warp order, so
// that every thread gets the same bits.  `sm` is free again at the next call with the other buffer.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int warps, float* sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? max_nan(v, w) : v + w;
    }
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sm[0];
    for (int w = 1; w < warps; ++w) v = MAX ? max_nan(v, sm[w]) : v + sm[w];
    return v;
}

enum NormOut : int { NORM_SAME = 0, NORM_ROW = 1, NORM_GROUP = 2 };
constexpr int kNormGroup = 128;

// blockDim = (threads of a row, rows of a block; more than one row only with one warp a row).  NV units of 8 channels
// per thread.
template <typename T, int NV, int OUT>
__global__ void __launch_bounds__(512) gdn_add_rmsnorm_kernel(const NormParams p) {
    __shared__ float sm[2][32];
    const int tpr = blockDim.x, warps = tpr >> 5;
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.rows) return;  // whole warps; a block of several warps a row has one row
    const int units = p.d >> 3;
    const long long base = row * p.d;
    float s[NV][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = threadIdx.x + i * tpr;
        if (u < units) {
            load8<T>(static_cast<const T*>(p.x) + base + 8 * u, s[i]);
            if (p.res) {
                float r[8];
                load8<T>(static_cast<const T*>(p.res) + base + 8 * u, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[i][e] += r[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[i][e] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = threadIdx.x + i * tpr;
        if (p.s && u < units) store8<T>(static_cast<T*>(p.s) + base + 8 * u, s[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += s[i][e] * s[i][e];
    }
    const float rstd = 1.f / sqrtf(row_reduce<false>(sum, warps, sm[0]) / (float)p.d + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = threadIdx.x + i * tpr;
        if (u < units) {
            float w[8];
            load8<float>(p.weight + 8 * u, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[i][e] = s[i][e] * rstd * w[e];
            if (OUT == NORM_SAME) store8<T>(static_cast<T*>(p.y) + base + 8 * u, s[i]);
        }
        if (OUT != NORM_SAME) {
            if (OUT == NORM_GROUP) amax = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(s[i][e]));
            if (OUT == NORM_GROUP) {
                // 128 channels are 16 neighbouring threads of one unit (d is a multiple of 128)
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                if (u < units) {
                    const float top = max_nan(amax, 1e-30f), inv = 448.f / top;
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + base + 8 * u) =
                        make_uint2(pack_e4m3x4(s[i][0] * inv, s[i][1] * inv, s[i][2] * inv, s[i][3] * inv),
                                   pack_e4m3x4(s[i][4] * inv, s[i][5] * inv, s[i][6] * inv, s[i][7] * inv));
                    if ((u & 15) == 0) p.y_scale[row * (p.d / kNormGroup) + (u >> 4)] = top / 448.f;
                }
            }
        }
    }
    if (OUT == NORM_ROW) {
        const float top = max_nan(row_reduce<true>(amax, warps, sm[1]), 1e-30f), inv = 448.f / top;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * tpr;
            if (u < units)
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + base + 8 * u) =
                    make_uint2(pack_e4m3x4(s[i][0] * inv, s[i][1] * inv, s[i][2] * inv, s[i][3] * inv),
                               pack_e4m3x4(s[i][4] * inv, s[i][5] * inv, s[i][6] * inv, s[i][7] * inv));
        }
        if (threadIdx.x == 0) p.y_scale[row] = top / 448.f;
    }
}

// ------------------------------------------------------------------------------------------ backward
struct NormBwdParams {
    const void* dy;
    const void* s;
    const float* weight;
    const float* rstd;
    const void* ds;  // or null
    void* dx;
    float* part;     // [parts][d] column sums of the blocks' rows
    float* dweight;  // [d]
    long long rows;
    int d, parts;
};

// At most this many blocks' column sums: two per SM.
constexpr int kNormBwdParts = 296;
inline int norm_bwd_parts(long long rows) { return (int)(rows < kNormBwdParts ? rows : kNormBwdParts); }

// Block b takes rows b, b + gridDim.x, ...; a thread owns the same channels in every row, so its dw stay in registers.
template <typename T, int NV>
__global__ void __launch_bounds__(512) gdn_add_rmsnorm_bwd_kernel(const NormBwdParams p) {
    __shared__ float sm[2][32];
    const int tpr = blockDim.x, warps = tpr >> 5, units = p.d >> 3;
    float dw[NV][8] = {};
    int buf = 0;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const long long base = row * p.d;
        const float rstd = p.rstd[row];
        float x[NV][8], gw[NV][8];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * tpr;
            if (u < units) {
                load8<T>(static_cast<const T*>(p.s) + base + 8 * u, x[i]);
                load8<T>(static_cast<const T*>(p.dy) + base + 8 * u, gw[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = gw[i][e] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * tpr;
            float w[8] = {};
            if (u < units) load8<float>(p.weight + 8 * u, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[i][e] *= rstd;
                dw[i][e] += gw[i][e] * x[i][e];
                gw[i][e] *= w[e];
                sum += gw[i][e] * x[i][e];
            }
        }
        const float mean = row_reduce<false>(sum, warps, sm[buf]) / (float)p.d;
        buf ^= 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * tpr;
            if (u < units) {
                float r[8] = {};
                if (p.ds) load8<T>(static_cast<const T*>(p.ds) + base + 8 * u, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] += rstd * (gw[i][e] - x[i][e] * mean);
                store8<T>(static_cast<T*>(p.dx) + base + 8 * u, r);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = threadIdx.x + i * tpr;
        if (u < units) store8<float>(p.part + (long long)blockIdx.x * p.d + 8 * u, dw[i]);
    }
}

// Column sums of the blocks' sums, in a fixed order: 32 channels per block, 8 warps that take every eighth row.
__global__ void __launch_bounds__(256) gdn_add_rmsnorm_dw_kernel(const NormBwdParams p) {
    __shared__ float sm[8][33];
    cudaGridDependencySynchronize();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < p.d)
        for (int i = warp; i < p.parts; i += 8) v += p.part[(long long)i * p.d + c];
    sm[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < p.d) {
#pragma unroll
        for (int w = 1; w < 8; ++w) v += sm[w][lane];
        p.dweight[c] = v;
    }
}

}  // namespace gdn
