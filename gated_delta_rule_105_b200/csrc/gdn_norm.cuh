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
// and its output, and 8 channels per thread (16 bytes of bf16) are one access.  Measured at 16384 rows of 4096 bf16
// channels: forward with 128-channel scales 79 to 84 us (5.8 TB/s), backward 100 us (5.4 TB/s); 48 rows of 2048: 15 us, of which
// the host's call is 11.
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
    int stages;  // of the ring
};

// Largest magnitude of three, NaN if one is NaN.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 8 channels as four pairs.
struct F8 {
    float2 v[4];
};
template <typename T> __device__ __forceinline__ F8 load_f8(const T* p);
template <> __device__ __forceinline__ F8 load_f8<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    return r;
}
template <> __device__ __forceinline__ F8 load_f8<float>(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    return F8{{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}
template <typename T> __device__ __forceinline__ void store_f8(T* p, const F8& x);
template <> __device__ __forceinline__ void store_f8<__nv_bfloat16>(__nv_bfloat16* p, const F8& x) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x.v[0].x, x.v[0].y), pack_bf16x2(x.v[1].x, x.v[1].y),
                                              pack_bf16x2(x.v[2].x, x.v[2].y), pack_bf16x2(x.v[3].x, x.v[3].y));
}
template <> __device__ __forceinline__ void store_f8<float>(float* p, const F8& x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
}
__device__ __forceinline__ void store_e4m3(uint8_t* p, const F8& x, float f) {
    const float2 ff = make_float2(f, f);
    const float2 a = mul2(x.v[0], ff), b = mul2(x.v[1], ff), c = mul2(x.v[2], ff), d = mul2(x.v[3], ff);
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_e4m3x4(a.x, a.y, b.x, b.y), pack_e4m3x4(c.x, c.y, d.x, d.y));
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
    // up to 16 warps; what lies behind the last one's value is 0 (see the kernels' start)
    const float4* q = reinterpret_cast<const float4*>(sm);
    v = 0.f;
    for (int w = 0; w < warps; w += 4) {
        const float4 x = q[w >> 2];
        v = MAX ? max_nan(max_abs_nan(x.x, x.y, x.z), max_nan(v, x.w)) : v + ((x.x + x.y) + (x.z + x.w));
    }
    return v;
}

// Rows ahead of the one in work lie in shared memory: every thread copies the 8-channel units that it will use itself
// (16-byte asynchronous copies), so no barrier stands between a copy and its use, and registers hold one row only.
// Operand o of stage st is at [st][row of the block][o][unit].
template <typename T, int OPS, int NV>
struct NormRing {
    uint8_t* base;      // this thread's first unit of stage 0, operand 0
    int stages;         // 1 to 4
    uint32_t op_bytes;  // one operand's row
    uint32_t st_bytes;  // one stage of the block

    __device__ __forceinline__ NormRing(uint8_t* smem, int d, int n) {
        stages = n;
        op_bytes = d * sizeof(T);
        st_bytes = op_bytes * OPS * blockDim.y;
        base = smem + threadIdx.y * (op_bytes * OPS) + threadIdx.x * 8 * sizeof(T);
    }
    __device__ __forceinline__ void fetch(int st, int o, const T* row, int units) const {
        const uint32_t dst = sm100_smem(base + st * st_bytes + o * op_bytes);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(row + threadIdx.x * 8);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((int)threadIdx.x + i * (int)blockDim.x < units) {
#pragma unroll
                for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
                    const uint32_t off = i * blockDim.x * 8 * sizeof(T) + 16 * k;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + off), "l"(src + off) : "memory");
                }
            }
    }
    // Unit i of operand o.
    __device__ __forceinline__ F8 get(int st, int o, int i) const {
        return load_f8<T>(reinterpret_cast<const T*>(base + st * st_bytes + o * op_bytes) + i * blockDim.x * 8);
    }
    __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // All but the newest stages - 1 groups have landed.
    __device__ __forceinline__ void wait() const {
        if (stages == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
        else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
        else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    static __device__ __forceinline__ uint32_t sm100_smem(const void* p) {
        return static_cast<uint32_t>(__cvta_generic_to_shared(p));
    }
};

enum NormOut : int { NORM_SAME = 0, NORM_ROW = 1, NORM_GROUP = 2 };
constexpr int kNormGroup = 128;

// blockDim = (threads of a row, rows at a time; more than one only with one warp a row).  NV units of 8 channels per
// thread.  Block b takes rows b, b + gridDim.x, ... (times rows at a time).
template <typename T, int NV, int OUT>
__global__ void __launch_bounds__(512) gdn_add_rmsnorm_kernel(const NormParams p) {
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ __align__(16) float sm[4][16];
    const int tpr = blockDim.x, warps = tpr >> 5, units = p.d >> 3;
    if (warps > 1) {
        if (threadIdx.x < 64) (&sm[0][0])[threadIdx.x] = 0.f;
        __syncthreads();
    }
    const float inv_d = 1.f / (float)p.d;
    const NormRing<T, 2, NV> ring(s_ring, p.d, p.stages);
    const long long first = (long long)blockIdx.x * blockDim.y + threadIdx.y, step = (long long)gridDim.x * blockDim.y;
    auto ask = [&](long long row, int st) {
        if (row < p.rows) {
            ring.fetch(st, 0, static_cast<const T*>(p.x) + row * p.d, units);
            if (p.res) ring.fetch(st, 1, static_cast<const T*>(p.res) + row * p.d, units);
        }
        ring.commit();
    };
    for (int i = 0; i < ring.stages - 1; ++i) ask(first + i * step, i);
    F8 wt[NV] = {};  // a thread's channels are the same in every row
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((int)threadIdx.x + i * tpr < units) wt[i] = load_f8<float>(p.weight + 8 * (threadIdx.x + i * tpr));
    int st = 0, st_in = ring.stages - 1, buf = 0;
    for (long long row = first; row < p.rows; row += step) {
        ask(row + (ring.stages - 1) * step, st_in);
        st_in = st_in + 1 == ring.stages ? 0 : st_in + 1;
        ring.wait();
        const long long base = row * p.d;
        F8 s[NV];
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * tpr;
            if (u < units) {
                s[i] = ring.get(st, 0, i);
                if (p.res) {
                    const F8 r = ring.get(st, 1, i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i].v[e] = add2(s[i].v[e], r.v[e]);
                }
                if (p.s) store_f8<T>(static_cast<T*>(p.s) + base + 8 * u, s[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum = fma2(s[i].v[e], s[i].v[e], sum);
            }
        }
        st = st + 1 == ring.stages ? 0 : st + 1;
        const float rstd = rsqrtf(fmaf(row_reduce<false>(sum.x + sum.y, warps, sm[buf]), inv_d, p.eps));
        if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
        const float2 rr = make_float2(rstd, rstd);
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * tpr;
            if (OUT == NORM_GROUP) amax = 0.f;
            if (u < units) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[i].v[e] = mul2(mul2(s[i].v[e], rr), wt[i].v[e]);
                    if (OUT != NORM_SAME) amax = max_abs_nan(amax, s[i].v[e].x, s[i].v[e].y);
                }
                if (OUT == NORM_SAME) store_f8<T>(static_cast<T*>(p.y) + base + 8 * u, s[i]);
            }
            if (OUT == NORM_GROUP) {
                // 128 channels are 16 neighbouring threads of one unit (d is a multiple of 128)
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                if (u < units) {
                    const float top = max_nan(amax, 1e-30f);
                    store_e4m3(static_cast<uint8_t*>(p.y) + base + 8 * u, s[i], 448.f / top);
                    if ((u & 15) == 0) p.y_scale[row * (p.d / kNormGroup) + (u >> 4)] = top / 448.f;
                }
            }
        }
        if (OUT == NORM_ROW) {
            const float top = max_nan(row_reduce<true>(amax, warps, sm[2 + buf]), 1e-30f), inv = 448.f / top;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = threadIdx.x + i * tpr;
                if (u < units) store_e4m3(static_cast<uint8_t*>(p.y) + base + 8 * u, s[i], inv);
            }
            if (threadIdx.x == 0) p.y_scale[row] = top / 448.f;
        }
        buf ^= 1;
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
    int stages;  // of the ring
};

// Block b takes rows b, b + gridDim.x, ...; a thread owns the same channels in every row, so its share of dw stays in
// registers.  blockDim = (threads of a row, rows at a time): with one warp a row a block works on several, whose
// dw are added through shared memory at the end.  A row's three operands are all asked for before the first is used.
template <typename T, int NV>
__global__ void __launch_bounds__(512) gdn_add_rmsnorm_bwd_kernel(const NormBwdParams p) {
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ __align__(16) float sm[2][16];
    const int tpr = blockDim.x, warps = tpr >> 5, units = p.d >> 3;
    if (warps > 1) {
        if (threadIdx.x < 32) (&sm[0][0])[threadIdx.x] = 0.f;
        __syncthreads();
    }
    const float inv_d = 1.f / (float)p.d;
    cudaTriggerProgrammaticLaunchCompletion();  // the sum kernel may be brought up meanwhile
    const NormRing<T, 3, NV> ring(s_ring, p.d, p.stages);
    const long long first = (long long)blockIdx.x * blockDim.y + threadIdx.y, step = (long long)gridDim.x * blockDim.y;
    auto ask = [&](long long row, int st) {
        if (row < p.rows) {
            ring.fetch(st, 0, static_cast<const T*>(p.s) + row * p.d, units);
            ring.fetch(st, 1, static_cast<const T*>(p.dy) + row * p.d, units);
            if (p.ds) ring.fetch(st, 2, static_cast<const T*>(p.ds) + row * p.d, units);
        }
        ring.commit();
    };
    for (int i = 0; i < ring.stages - 1; ++i) ask(first + i * step, i);
    F8 dw[NV] = {}, wt[NV] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((int)threadIdx.x + i * tpr < units) wt[i] = load_f8<float>(p.weight + 8 * (threadIdx.x + i * tpr));
    int st = 0, st_in = ring.stages - 1, buf = 0;
    float rstd = first < p.rows ? p.rstd[first] : 0.f;
    for (long long row = first; row < p.rows; row += step) {
        ask(row + (ring.stages - 1) * step, st_in);
        st_in = st_in + 1 == ring.stages ? 0 : st_in + 1;
        const float rstd_next = row + step < p.rows ? p.rstd[row + step] : 0.f;
        ring.wait();
        const long long base = row * p.d;
        const float2 rr = make_float2(rstd, rstd);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * tpr;
            if (u < units) {
                const F8 x = ring.get(st, 0, i), y = ring.get(st, 1, i);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 t = mul2(y.v[e], mul2(x.v[e], rr));
                    dw[i].v[e] = add2(dw[i].v[e], t);
                    sum = fma2(t, wt[i].v[e], sum);
                }
            }
        }
        // dx = ds + rstd w dy - x (rstd^2 mean)
        const float mean = row_reduce<false>(sum.x + sum.y, warps, sm[buf]) * inv_d, c = -rstd * rstd * mean;
        const float2 cc = make_float2(c, c);
        buf ^= 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * tpr;
            if (u < units) {
                const F8 x = ring.get(st, 0, i), y = ring.get(st, 1, i);
                F8 r = {};
                if (p.ds) r = ring.get(st, 2, i);
#pragma unroll
                for (int e = 0; e < 4; ++e) r.v[e] = fma2(x.v[e], cc, fma2(mul2(y.v[e], wt[i].v[e]), rr, r.v[e]));
                store_f8<T>(static_cast<T*>(p.dx) + base + 8 * u, r);
            }
        }
        st = st + 1 == ring.stages ? 0 : st + 1;
        rstd = rstd_next;
    }
    if (blockDim.y > 1) {
        __syncthreads();  // the ring is read; the rows' dw of a block take its place, [rows at a time - 1][d]
        float* s_dw = reinterpret_cast<float*>(s_ring);
        if (threadIdx.y > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = threadIdx.x + i * tpr;
                if (u < units) store_f8<float>(s_dw + (threadIdx.y - 1) * p.d + 8 * u, dw[i]);
            }
        }
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 0; y < (int)blockDim.y - 1; ++y)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = threadIdx.x + i * tpr;
                if (u < units) {
                    const F8 o = load_f8<float>(s_dw + y * p.d + 8 * u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dw[i].v[e] = add2(dw[i].v[e], o.v[e]);
                }
            }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = threadIdx.x + i * tpr;
        if (u < units) store_f8<float>(p.part + (long long)blockIdx.x * p.d + 8 * u, dw[i]);
    }
}

// Column sums of the blocks' sums, in a fixed order: 32 channels per block, warp w takes rows w, w + 32, ...
constexpr int kDwWarps = 32;
__global__ void __launch_bounds__(kDwWarps * 32) gdn_add_rmsnorm_dw_kernel(const NormBwdParams p) {
    __shared__ float sm[kDwWarps][33];
    cudaGridDependencySynchronize();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < p.d) {
#pragma unroll 4
        for (int i = warp; i < p.parts; i += kDwWarps) v += p.part[(long long)i * p.d + c];
    }
    sm[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < p.d) {
#pragma unroll
        for (int w = 1; w < kDwWarps; ++w) v += sm[w][lane];
        p.dweight[c] = v;
    }
}

}  // namespace gdn
