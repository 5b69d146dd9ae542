// The attention layer's paged key/value cache: layout, the 8-bit format, writing new tokens and reading rows back.
//
// Layout.  A pool of pages; page p holds `page` consecutive positions of one sequence for every KV head,
// [n_pages][Hkv][page][d], K and V apart.  block_table[n][i] names the page of sequence n's positions
// [i page, (i + 1) page).  Head before position, so that one (page, head) tile is one contiguous block: the
// attention kernels stream it without gaps, and one bulk copy or tensor-map box fetches it.
//
// 8-bit format.  A row x[d] (one token, one head) is stored as e4m3 codes and one scale byte b, value =
// code * 2^(b - 127), with the smallest exponent e = b - 127 that keeps |x| <= 448 * 2^e.  A power of two costs
// nothing in relative precision (e4m3 is itself a floating format), and it makes every stored value an exact bf16
// number -- 4 significant bits, and e is kept within [-117, 119] so that none leaves bf16's normal range -- so that
// attention over the 8-bit cache works on the same keys and values as over its read-back in a bf16 cache (results differ
// by the order of sums, and by the decode kernel's f16 form of Q), and quantisation has no rounding but the one to e4m3
// (x * 2^-e is exact).  A row that holds an infinity or a NaN gets byte 255, the NaN scale,
// and reads back as NaN throughout: non-finite values are kept visible, and the codes themselves are always finite.
#pragma once

#include <cuda_fp8.h>

#include "gdn_common.cuh"
#include "gdn_host.h"

namespace gdn {

constexpr int kScaleExpMin = -117, kScaleExpMax = 119;
constexpr unsigned kScaleNan = 255;

struct KvParams {
    void* k_cache;              // [n_pages][hkv][page][d] bf16 or e4m3
    void* v_cache;
    uint8_t* k_scale;           // [n_pages][hkv][page], 8-bit cache only
    uint8_t* v_scale;
    const int32_t* table;       // [n_seq][max_pages]
    const int32_t* seq_lens;    // [n_seq] positions in the cache, the new tokens among them
    const int32_t* cu;          // [n_seq + 1] or null (n_tok / n_seq tokens each)
    int n_tok, n_seq, n_pages, max_pages, hkv, d, page_log2;
};

// Sequence n's rows [start, start + T) among the packed new tokens and its length in the cache.  T < 0: not a valid
// sequence (the error word says why); nothing of it is read or written.
struct SeqSpan {
    int start, T, len;
};
__device__ __forceinline__ SeqSpan kv_span(const KvParams& p, int n, unsigned* err) {
    SeqSpan s;
    int end;
    if (p.cu) {
        s.start = p.cu[n];
        end = p.cu[n + 1];
        if (s.start < 0 || end < s.start || end > p.n_tok) {
            atomicOr(err, kErrSeqlens);
            s.T = -1;
            return s;
        }
    } else {
        const int T = p.n_tok / p.n_seq;
        s.start = n * T;
        end = s.start + T;
    }
    s.T = end - s.start;
    s.len = p.seq_lens[n];
    if (s.len < s.T || s.len > ((long long)p.max_pages << p.page_log2)) {
        atomicOr(err, kErrPages);
        s.T = -1;
    }
    return s;
}

// The sequence of packed row tau: the last n with cu[n] <= tau, found by the whole warp with 32 probes a step (one
// step up to 32 sequences, two up to 1024: dependent loads are what a small call spends its time on).  -1: the row
// lies behind the last sequence, or cu is not in order (then the error word says so).
__device__ __forceinline__ int kv_warp_find(const int32_t* cu, int n_seq, int tau, int& start, int& end, unsigned* err) {
    const int lane = threadIdx.x & 31;
    int lo = 0, size = n_seq;  // the answer is in [lo, lo + size)
    while (size > 1) {
        const int stride = (size + 31) >> 5;
        const int at = lo + lane * stride;
        const bool in = lane * stride < size && cu[at] <= tau;
        const int hits = __popc(__ballot_sync(0xffffffffu, in));
        const int step = max(hits - 1, 0);
        lo += step * stride;
        size = min(stride, size - step * stride);
    }
    start = cu[lo];
    end = cu[lo + 1];
    if (start < 0 || start > tau || end <= tau) {
        if (tau < cu[n_seq] && lane == 0) atomicOr(err, kErrSeqlens);
        return -1;
    }
    return lo;
}

// The same for the rows tau0 .. tau0 + nt - 1 (nt <= TPW) of a warp: lane t < nt gets row tau0 + t's sequence, n = -1 where it
// has none.
template <int TPW>
__device__ __forceinline__ void kv_warp_find_rows(const int32_t* cu, int n_seq, int tau0, int nt, int& n, int& start, int& end, unsigned* err) {
    int cn = -1, cs = 0, ce = 0;
    if (TPW == 1) {  // (every lane)
        n = kv_warp_find(cu, n_seq, tau0, start, end, err);
        return;
    }
    n = -1;
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
        if (t >= nt) break;
        if (cn < 0 || tau0 + t >= ce) cn = kv_warp_find(cu, n_seq, tau0 + t, cs, ce, err);
        if ((threadIdx.x & 31) == t) n = cn, start = cs, end = ce;
    }
}

// Page index of block-table entry i of sequence n, or -1 (error word set) when it names no page of the pool.
__device__ __forceinline__ int kv_page(const KvParams& p, int n, int i, unsigned* err) {
    const int pg = p.table[(long long)n * p.max_pages + i];
    if (pg < 0 || pg >= p.n_pages) {
        atomicOr(err, kErrPages);
        return -1;
    }
    return pg;
}

__device__ __forceinline__ float kv_scale_value(unsigned byte) {
    return byte == kScaleNan ? __int_as_float(0x7fc00000) : __int_as_float((int)(byte << 23));
}

// 16 bytes of input as floats: 8 bf16 or 4 fp32.
template <typename T> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Vec16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4& u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// Two fp32 operations per instruction, where a kernel would run out of issue slots first.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
// Four floats to four e4m3 codes (nearest, ties to even; finite values beyond 448 saturate).
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// ------------------------------------------------------------------------------------------ append
struct KvAppendParams {
    KvParams c;
    const void* x[2];        // new keys and values, [n_tok][hkv][d], token rows `stride` elements apart
    long long stride[2];
};

// One row chunk of a lane (N values of a row that LG lanes hold together) into the cache.
template <typename TIn, int D, bool E4M3>
__device__ __forceinline__ void kv_store_row(const KvParams& c, int which, long long row, int lane_in_row, const uint4& u) {
    constexpr int N = Vec16<TIn>::N, LG = D / N;
    float x[N];
    Vec16<TIn>::get(u, x);
    if (E4M3) {
        // the largest magnitude as an integer: the order of |x|'s bit patterns is the order of |x|, and infinities
        // and NaNs come out on top
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
        for (int o = LG / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool bad = top >= 0x7f800000u;
        // 448 = 1.75 * 2^8, so amax = 1.m * 2^a needs e = a - 8, one more when 1.m > 1.75
        int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = min(max(e, kScaleExpMin), kScaleExpMax);
        const float inv = bad ? 0.f : __int_as_float((127 - e) << 23);
        uint32_t code[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            code[i] = bad ? 0u : pack_e4m3x4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
        if (row < 0) return;
        uint8_t* dst = static_cast<uint8_t*>(which ? c.v_cache : c.k_cache) + row * D + lane_in_row * N;
        if (N == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[N / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(dst) = code[0];
        if (lane_in_row == 0) (which ? c.v_scale : c.k_scale)[row] = (uint8_t)(bad ? kScaleNan : (unsigned)(e + 127));
    } else {
        if (row < 0) return;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which ? c.v_cache : c.k_cache) + row * D + lane_in_row * N;
        if (N == 8) *reinterpret_cast<uint4*>(dst) = u;
        else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    }
}

constexpr int kKvWarps = 8, kKvBatch = 4;  // loads of K, and of V, that a lane has in flight

// One warp per TPW new tokens.  Their first K and V rows are loaded before the tokens' places in the cache are known (the
// search over cu_seqlens, the length and the block table are a chain of dependent loads that does not need them).  LG
// lanes hold one head's row, so the row maximum is log2(LG) shuffles and each head's codes leave as full sectors.
// Bound by HBM, and in small calls by the look-ups: 8 heads x 128, bf16 to e4m3, 75776 tokens 77 us (6.0 TB/s), 2048
// tokens 4.7 us.  More blocks per SM (48 registers), streaming loads and blocks of 4 warps change nothing.
template <typename TIn, int D, bool E4M3, int TPW>
__global__ void __launch_bounds__(kKvWarps * 32) gdn_kv_append_kernel(const KvAppendParams p, unsigned* err) {
    constexpr int N = Vec16<TIn>::N, LG = D / N, RPP = 32 / LG, PB = kKvBatch;  // rows per pass, passes per batch
    const int lane = threadIdx.x & 31;
    const int tau0 = (blockIdx.x * kKvWarps + (threadIdx.x >> 5)) * TPW, ntok = min(TPW, p.c.n_tok - tau0);
    if (ntok <= 0) return;
    const int tl = TPW == 1 ? 0 : lane;  // the token that this lane looks up
    // row r of the warp's ntok * hkv is head r mod hkv of token r / hkv
    const int hkv = p.c.hkv, nr = ntok * hkv, sub = lane / LG, col = lane % LG;
    auto token_of = [&](int r) {
        int t = 0;
#pragma unroll
        for (int i = 1; i < TPW; ++i) t += r >= i * hkv;
        return t;
    };
    const uint4* src[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) src[w] = reinterpret_cast<const uint4*>(static_cast<const TIn*>(p.x[w]) + tau0 * p.stride[w]);
    uint4 u[2][PB];
    auto load = [&](int r0) {
#pragma unroll
        for (int b = 0; b < PB; ++b) {
            const int r = r0 + b * RPP + sub, t = token_of(r);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint4* at = src[w] + (r0 + b * RPP) * LG + lane;  // row r, as if the tokens' rows had no gaps
                if (TPW > 1) at += t * (p.stride[w] * (int)sizeof(TIn) / 16 - hkv * LG);
                u[w][b] = r < nr ? *at : make_uint4(0, 0, 0, 0);
            }
        }
    };
    load(0);
    int n, start, end;
    if (p.c.cu) {
        kv_warp_find_rows<TPW>(p.c.cu, p.c.n_seq, tau0, ntok, n, start, end, err);
    } else {
        const int T = p.c.n_tok / p.c.n_seq;
        n = tl < ntok ? (tau0 + tl) / T : -1;
        start = n * T;
        end = start + T;
    }
    long long base = -1;  // of token tl: where it goes
    if (n >= 0) {
        const int len = p.c.seq_lens[n];
        if (end > p.c.n_tok || len < end - start || len > ((long long)p.c.max_pages << p.c.page_log2)) {
            atomicOr(err, end > p.c.n_tok ? kErrSeqlens : kErrPages);
        } else {
            const int pos = len - (end - (tau0 + tl));
            const int pg = kv_page(p.c, n, pos >> p.c.page_log2, err);
            if (pg >= 0) base = ((long long)pg * hkv << p.c.page_log2) + (pos & ((1 << p.c.page_log2) - 1));
        }
    }
    for (int r0 = 0; r0 < nr; r0 += PB * RPP) {
        if (r0 > 0) load(r0);
#pragma unroll
        for (int b = 0; b < PB; ++b) {
            const int r = r0 + b * RPP + sub, t = token_of(r);
            const long long at = TPW == 1 ? base : __shfl_sync(0xffffffffu, base, t);
            const long long row = r < nr && at >= 0 ? at + ((long long)(r - t * hkv) << p.c.page_log2) : -1;
#pragma unroll
            for (int w = 0; w < 2; ++w) kv_store_row<TIn, D, E4M3>(p.c, w, row, col, u[w][b]);
        }
    }
}

// ------------------------------------------------------------------------------------------ read back
struct KvReadParams {
    KvParams c;  // n_tok = rows of the output, cu = their sequences; seq_lens unused
    void* y[2];  // dense keys and values, [n_tok][hkv][d]
};

// One warp per TPW output tokens; a lane owns 8 channels of a head's row (16 bytes of bf16 output).  Bound by HBM once
// enough loads are in flight: 16 sequences of 16384, 4 heads x 128, e4m3 to bf16, 96 us (6.1 TB/s).
template <typename TOut, int D, bool E4M3, int TPW>
__global__ void __launch_bounds__(kKvWarps * 32) gdn_kv_read_kernel(const KvReadParams p, unsigned* err) {
    constexpr int LG = D / 8, RPP = 32 / LG, PB = kKvBatch;
    const int lane = threadIdx.x & 31;
    const int tau0 = (blockIdx.x * kKvWarps + (threadIdx.x >> 5)) * TPW, ntok = min(TPW, p.c.n_tok - tau0);
    if (ntok <= 0) return;
    const int tl = TPW == 1 ? 0 : lane;  // the token that this lane looks up
    int n, start, end;
    kv_warp_find_rows<TPW>(p.c.cu, p.c.n_seq, tau0, ntok, n, start, end, err);
    long long base = -1;  // of token tl: where it lies in the cache
    if (n >= 0) {
        const int pos = tau0 + tl - start;
        if (end > p.c.n_tok || (pos >> p.c.page_log2) >= p.c.max_pages) {
            atomicOr(err, end > p.c.n_tok ? kErrSeqlens : kErrPages);
        } else {
            const int pg = kv_page(p.c, n, pos >> p.c.page_log2, err);
            if (pg >= 0) base = ((long long)pg * p.c.hkv << p.c.page_log2) + (pos & ((1 << p.c.page_log2) - 1));
        }
    }
    // row r of the warp's ntok * hkv (head r mod hkv of token r / hkv) is row tau0 * hkv + r of the output
    const int hkv = p.c.hkv, nr = ntok * hkv, sub = lane / LG, col = (lane % LG) * 8;
    for (int r0 = 0; r0 < nr; r0 += PB * RPP) {
        uint4 u[2][PB];
        unsigned sc[2][PB];
        bool have[PB];
#pragma unroll
        for (int b = 0; b < PB; ++b) {
            const int r = r0 + b * RPP + sub;
            int t = 0;
#pragma unroll
            for (int i = 1; i < TPW; ++i) t += r >= i * hkv;
            const long long at = TPW == 1 ? base : __shfl_sync(0xffffffffu, base, t);
            const long long row = at + ((long long)(r - t * hkv) << p.c.page_log2);
            have[b] = r < nr && at >= 0;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint8_t* cache = static_cast<const uint8_t*>(w ? p.c.v_cache : p.c.k_cache);
                if (!have[b]) continue;
                if (E4M3) {
                    const uint2 c2 = *reinterpret_cast<const uint2*>(cache + row * D + col);
                    u[w][b] = make_uint4(c2.x, c2.y, 0, 0);
                    sc[w][b] = (w ? p.c.v_scale : p.c.k_scale)[row];
                } else {
                    u[w][b] = *reinterpret_cast<const uint4*>(cache + (row * D + col) * 2);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < PB; ++b) {
            const int r = r0 + b * RPP + sub;
            if (!have[b]) continue;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                TOut* dst = static_cast<TOut*>(p.y[w]) + ((long long)tau0 * hkv + r) * D + col;
                float x[8];
                if (E4M3) {
                    const float s = kv_scale_value(sc[w][b]);
                    const uint32_t c2[2] = {u[w][b].x, u[w][b].y};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __half2_raw h2 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c2[i >> 1] >> (16 * (i & 1))),
                                                                          __NV_E4M3);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                        x[2 * i] = f.x * s;
                        x[2 * i + 1] = f.y * s;
                    }
                } else {
                    Vec16<__nv_bfloat16>::get(u[w][b], x);
                }
                if (sizeof(TOut) == 2) {
                    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
                } else {
                    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
                    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
                }
            }
        }
    }
}

}  // namespace gdn
