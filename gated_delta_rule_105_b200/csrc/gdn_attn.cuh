// Attention of new tokens over the paged cache (gdn_kv.cuh): scheduling shared by the two kernels, the kernel for
// few query rows (decoding), and the kernel that joins split items.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j - max),   over keys j <= pos_i, and with a
//   window also j > pos_i - window;  pos_i is the new token's place in its sequence.
//
// Query heads share KV heads in groups of G, so the unit of work is an item: (sequence, KV head, group of query rows),
// where row r of a (sequence, KV head) is new token r / G and head r mod G of the group.  Every item streams its keys
// once in blocks of 128 to 384 (a unit).  All units of all items form one line, and each CTA takes an equal stretch of it
// whatever the sequences' lengths are: the split depends on device-side lengths only, so a captured graph replays
// with new lengths and nothing is read back.  A CTA ends up with whole items (written directly) and at most two parts
// of items, its first and its last, whose unnormalised sums, maxima and denominators go to the workspace; a join kernel
// adds the parts of an item in a fixed order.  The workspace is therefore a fixed size per CTA.
#pragma once

#include "gdn_kv.cuh"

// gdn_sm100.cuh defines one out-of-line function; declared static first, it stays local to this translation unit (the
// library's other one has its own).  It is not marked there: bench.py's record of DRAM traffic goes by that header's text.
namespace gdn {
namespace sm100 {
static __device__ __noinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                   unsigned* err, long long limit);
}
}  // namespace gdn
#include "gdn_sm100.cuh"

namespace gdn {

constexpr int kAttnSms = 148;  // B200

struct AttnParams {
    KvParams c;
    const __nv_bfloat16* q;  // [n_tok][hq][d], token rows q_stride elements apart
    long long q_stride;
    void* o;                 // [n_tok][hq][d]
    float* lse;              // [n_tok][hq] or null
    float scale_log2;        // scale * log2(e)
    int window;              // 0: none
    int G, hq;
    int o_f32;
    int debug_stall;         // diagnostic (gdn_debug_stall): 0 in every ordinary call
    int rows_lo, rows_hi;    // this kernel takes sequences with rows_lo < T G <= rows_hi
    int* desc;               // [grid][kDescInts], the split item that starts in this CTA, for the join kernel
    float* part;             // [grid][2][R][d] partial sums (chunk: [grid][2][row tile][d / 4][128][4])
    float* ml;               // [grid][2][R][2] maximum (base 2) and denominator
};
// sequence (-1: none), KV head, first row, rows, slot of the first part, number of CTAs it spans, the first token's row
constexpr int kDescInts = 8;

// Units of one (KV head, row group) of a sequence, from the first unit of keys that any of its rows sees.
struct AttnSpan {
    SeqSpan s;
    int rgs;      // row groups
    int u_first;  // first unit
    int units;    // per row group
};

template <int R, int UNIT>
__device__ __forceinline__ AttnSpan attn_span(const AttnParams& p, int n, unsigned* err) {
    AttnSpan a;
    a.s = kv_span(p.c, n, err);
    a.units = 0, a.rgs = 0, a.u_first = 0;
    const long long rows = (long long)a.s.T * p.G;
    if (a.s.T <= 0 || rows <= p.rows_lo || rows > p.rows_hi) return a;
    a.rgs = (int)((rows + R - 1) / R);
    const int lo = p.window > 0 ? max(0, a.s.len - a.s.T + 1 - p.window) : 0;
    a.u_first = lo / UNIT;
    a.units = (a.s.len + UNIT - 1) / UNIT - a.u_first;
    return a;
}

// Sum over the block (every thread gets it) and the exclusive prefix of each thread.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long v, long long& total, long long* sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sm[w];
        total += sm[w];
    }
    return before + x - v;
}

__device__ __forceinline__ void attn_store4(void* o, int f32, long long at, float4 a, float f) {
    if (f32) *reinterpret_cast<float4*>(static_cast<float*>(o) + at) = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
    else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(o) + at) = make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
}
__device__ __forceinline__ float attn_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------------------------------ few rows
// mma.sync kernel for up to 16 query rows per item.  Bound by the cache's bytes: tensor work is small, and what counts
// is that every warp keeps its loads in flight and spends few instructions per key.  Each warp has a ring of its own in
// shared memory, filled with 16-byte asynchronous copies a few steps ahead, and no barrier with the other warps until the
// item ends.  The order of the contraction index is free, so thread t of a quad takes 8 (16 in 8 bits) consecutive
// channels of its key as its share of several k-steps (Q is loaded in the same order), and for V the keys of a step are
// interleaved with byte permutes.  16-byte chunk c of row r lies at c ^ swizzle(r), which makes both reads free of bank
// conflicts: K's (rows 2i and 2i + 1, chunks 0-3 or 4-7) and V's (rows 2t + const, chunks 2i and 2i + 1).
// Measured, with the join: 64 sequences of up to 16384, 16 query and 4 KV heads x 128, e4m3: 139 to 147 us, 5.2 TB/s of
// cache; one sequence of 4096, 2 KV heads, bf16: 17 us, of which the host's call is 11.  What is left is instructions: the
// conversions of the 8-bit codes and the softmax of rows that the tile has and the item does not.  Two CTAs of 8 warps per
// SM where the registers allow it (one of 12 for 16 rows): 148 us against 155 with one.  That is 128 registers a thread; for
// e4m3 and d = 128 ptxas spills 60 bytes (stores; 96 of loads) there.
//   S[q][key]: A = Q (16 rows), B = K; thread (g, t) = (lane / 4, lane % 4) gets rows g, g + 8 and keys 2t, 2t + 1.
//   O^T[d][q]: A = V^T (16 channels x 16 keys), B = P^T, whose fragment is exactly S's: no shuffle in between.
template <int CH>  // chunks of a row; 4: two rows share the 128 bytes of all banks
__host__ __device__ constexpr uint32_t dec_swizzle(uint32_t r) {
    return CH == 4 ? (r >> 1) & 3u : ((((r >> 1) & 3u) ^ ((r & 1u) << 1)) << 1);
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// prmt in its default mode: selector nibbles of 8 and above give eight copies of the byte's sign bit (__byte_perm takes
// three bits of each nibble only).
__device__ __forceinline__ uint32_t permute(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
// Two e4m3 codes a and b, each below a byte of its own sign (`w` = code a, sign a, code b, sign b from low to high, one
// byte permute with sign replication), as a bf16 pair.  Shifted left by 4 and masked, sign, exponent and mantissa stand
// where bf16 has them; the biases (7 and 127) make that the value times 2^-120, subnormal codes included, and one exact
// multiplication undoes it.  0x7f, e4m3's NaN, would read as 480: the cache writer never stores it.
__device__ __forceinline__ uint32_t e4m3_signed_to_bf16x2(uint32_t w) {
    return mul_bf16x2((w << 4) & 0x87f087f0u, 0x7b807b80u);
}
// Codes 0, 1 or 2, 3 of a word.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, int hi) {
    return e4m3_signed_to_bf16x2(permute(w, 0, hi ? 0xb3a2 : 0x9180));
}
// The same codes as an f16 pair: one conversion instruction, but f16's range is too short for weights times values.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The scales 2^(byte - 127) of the two bytes of `w`; infinity for the NaN scale.
__device__ __forceinline__ float scale_lo(uint32_t w) { return __uint_as_float((w << 23) & 0x7f800000u); }
__device__ __forceinline__ float scale_hi(uint32_t w) { return __uint_as_float((w << 15) & 0x7f800000u); }
__device__ __forceinline__ bool bf16x2_nonfinite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ bool bf16x8_nonfinite(const uint4& u) {
    return bf16x2_nonfinite(u.x) || bf16x2_nonfinite(u.y) || bf16x2_nonfinite(u.z) || bf16x2_nonfinite(u.w);
}
// The pair with 0 in the place of a NaN or an infinity.
__device__ __forceinline__ uint32_t bf16x2_finite(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}
__device__ __forceinline__ uint4 bf16x8_finite(const uint4& u) {
    return make_uint4(bf16x2_finite(u.x), bf16x2_finite(u.y), bf16x2_finite(u.z), bf16x2_finite(u.w));
}
// Adds what bf16x2_finite() took out of a pair of values to a row's sums of their channels.
__device__ __forceinline__ void add_nonfinite(uint32_t w, float& lo, float& hi) {
    if ((w & 0x7f80u) == 0x7f80u) lo += __uint_as_float(w << 16);
    if ((w & 0x7f800000u) == 0x7f800000u) hi += __uint_as_float(w & 0xffff0000u);
}
// Row of the pool that holds position `key` of the sequence with this block table, KV head h (a bad page was reported when its
// rows were asked for, and read as page 0).
__device__ __forceinline__ long long attn_pool_row(const KvParams& c, const int32_t* table, int key, int h) {
    int pg = table[key >> c.page_log2];
    if ((unsigned)pg >= (unsigned)c.n_pages) pg = 0;
    return (((long long)pg * c.hkv + h) << c.page_log2) + (key & ((1 << c.page_log2) - 1));
}

// The running maximum is lazy: sums are scaled down only when a row's maximum has grown by more than 2^8.  What is taken off
// the scores is therefore 8 more than the maximum of that moment: no weight is ever above 1, and no finite value times a
// weight leaves fp32's range.  (Behind such a step the largest weight is 2^-8, which costs neither fp32 nor bf16 a bit.)
constexpr float kRescaleLog2 = 8.f;

template <int D, bool E4M3, int R> struct DecTraits {
    static constexpr int RB = D * (E4M3 ? 1 : 2);          // bytes of a row
    static constexpr int WARPS = RB == 256 ? 8 : R == 8 ? 8 : 12;
    static constexpr int CTAS = RB == 256 || R == 16 ? 1 : 2;  // per SM
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int KS = RB == 64 ? 32 : 16;          // keys of one warp step
    static constexpr int UNIT = KS * WARPS;
    static constexpr int KL = RB / 64;                     // 16-byte K reads per thread and 8 keys
    static constexpr int MT = D / 16;                      // channel tiles of 16
    static constexpr int RS = R / 8;                       // sets of 8 rows
    static constexpr int STAGE = 2 * KS * RB + (E4M3 ? 256 : 0);  // a multiple of 256: chunk numbers are XORed in place
    static constexpr int STAGES = 3;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int JOIN = WARPS * R * D * 4;         // in the ring's place once it is empty
    static constexpr size_t smem = (RING > JOIN ? RING : JOIN) + WARPS * R * 8 + 256;
};

template <int D, bool E4M3, int R>
__global__ void __launch_bounds__((DecTraits<D, E4M3, R>::THREADS), (DecTraits<D, E4M3, R>::CTAS))
gdn_attn_decode_kernel(const AttnParams p, unsigned* err) {
    using Tr = DecTraits<D, E4M3, R>;
    constexpr int kDecWarps = Tr::WARPS, kDecThreads = Tr::THREADS, KS = Tr::KS, UNIT = Tr::UNIT, KL = Tr::KL, MT = Tr::MT, RS = Tr::RS,
                  RB = Tr::RB, STAGES = Tr::STAGES, NT = KS / 8, KG = KS / 16;
    extern __shared__ __align__(256) uint8_t smem[];
    float* s_o = reinterpret_cast<float*>(smem);                  // [warps][R][D]
    float* s_ml = reinterpret_cast<float*>(smem + (Tr::RING > Tr::JOIN ? Tr::RING : Tr::JOIN));  // [warps][R][2]
    long long* s_scan = reinterpret_cast<long long*>(s_ml + kDecWarps * R * 2);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int cta = blockIdx.x, N = p.c.n_seq;

    cudaTriggerProgrammaticLaunchCompletion();  // the next kernel may be brought up while this one runs
    // this CTA's stretch [w0, w1) of all units, and the sequence it starts in
    long long W = 0;
    for (int base = 0; base < N; base += kDecThreads) {
        long long mine = 0, total;
        if (base + tid < N) {
            const AttnSpan a = attn_span<R, UNIT>(p, base + tid, err);
            mine = (long long)a.units * a.rgs * p.c.hkv;
        }
        block_scan<kDecThreads>(mine, total, s_scan);
        W += total;
    }
    const int grid = (int)min((long long)gridDim.x, W);  // CTAs that get a unit at all: no stretch is empty
    int* desc = p.desc + (long long)cta * kDescInts;
    if (tid == 0) desc[0] = -1;
    if (cta >= grid) return;
    const long long w0 = W * cta / grid, w1 = W * (cta + 1) / grid;
    long long seen = 0;
    for (int base = 0; base < N; base += kDecThreads) {
        long long mine = 0, total;
        if (base + tid < N) {
            const AttnSpan a = attn_span<R, UNIT>(p, base + tid, err);
            mine = (long long)a.units * a.rgs * p.c.hkv;
        }
        const long long before = seen + block_scan<kDecThreads>(mine, total, s_scan);
        if (before <= w0 && w0 < before + mine) {
            s_scan[16] = base + tid;
            s_scan[17] = before;
        }
        seen += total;
        if (seen > w0) break;
    }
    __syncthreads();
    int n = (int)s_scan[16];
    long long off = w0 - s_scan[17];  // units of sequence n before this CTA's place

    AttnSpan sp = attn_span<R, UNIT>(p, n, err);
    for (long long w = w0; w < w1;) {
        // next sequence with work, one by one (32 at a time: 147 us for 144 over 64 sequences, the hot loop spills)
        while (off >= (long long)sp.units * sp.rgs * p.c.hkv) {
            off = 0;
            sp = attn_span<R, UNIT>(p, ++n, err);
        }
        const int item = (int)(off / sp.units), x0 = (int)(off - (long long)item * sp.units);
        const int h = item / sp.rgs, rg = item - h * sp.rgs;
        const int cnt = (int)min((long long)(sp.units - x0), w1 - w);
        const int T = sp.s.T, len = sp.s.len;

        // ---- the item's query rows: A fragments, in K's channel order
        const int row_lo = rg * R + g, rows = T * p.G;
        // a0, a2 of rows g and (R = 16) a1, a3 of rows g + 8.  For the 8-bit cache Q becomes f16, each row divided by a
        // power of two (exact down to 2^-28 of the row's largest), since K's codes convert to f16 in one instruction.
        uint32_t qf[D / 16][4];
        float qscale[RS];
        int hi_[RS], lo_[RS];  // keys [lo_, hi_] that rows g and g + 8 see
#pragma unroll
        for (int r = 0; r < RS; ++r) {
            const int row = row_lo + 8 * r;
            const bool there = row < rows;
            const int tok = there ? row / p.G : 0, gh = there ? row - tok * p.G : 0;
            const int pos = len - T + tok;
            hi_[r] = there ? pos : -1;
            lo_[r] = p.window > 0 ? pos - p.window + 1 : 0;
            const __nv_bfloat16* q = p.q + (long long)(sp.s.start + tok) * p.q_stride + (h * p.G + gh) * D;
            qscale[r] = p.scale_log2;
            if (E4M3) {
                unsigned top = 0;
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint2 u = there ? *reinterpret_cast<const uint2*>(q + 64 * j + 16 * t + 4 * s) : make_uint2(0, 0);
                        qf[4 * j + s][r] = u.x;
                        qf[4 * j + s][2 + r] = u.y;
                        if (R == 8) qf[4 * j + s][1] = qf[4 * j + s][3] = 0;
                        top = max(max(top, u.x & 0x7fffu), (u.x >> 16) & 0x7fffu);
                        top = max(max(top, u.y & 0x7fffu), (u.y >> 16) & 0x7fffu);
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // largest magnitude into [2^14, 2^15); an infinity or a NaN makes the row's scores NaN
                const int e = min(max((int)(top >> 7) - 127 - 14, -100), 113);
                const float inv = __int_as_float((127 - e) << 23);
                qscale[r] = top >= 0x7f80u ? __int_as_float(0x7fc00000) : p.scale_log2 * __int_as_float((127 + e) << 23);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t u = qf[i][2 * half + r];
                        const __half2 hq = __floats2half2_rn(__uint_as_float(u << 16) * inv, __uint_as_float(u & 0xffff0000u) * inv);
                        qf[i][2 * half + r] = top >= 0x7f80u ? 0u : *reinterpret_cast<const uint32_t*>(&hq);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint4 u = there ? *reinterpret_cast<const uint4*>(q + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
                    qf[2 * j][r] = u.x;
                    qf[2 * j][2 + r] = u.y;
                    qf[2 * j + 1][r] = u.z;
                    qf[2 * j + 1][2 + r] = u.w;
                    if (R == 8) qf[2 * j][1] = qf[2 * j][3] = qf[2 * j + 1][1] = qf[2 * j + 1][3] = 0;
                }
            }
        }
        // keys that every row of the sequence sees: [full_lo, full_hi]
        const int full_hi = len - T, full_lo = p.window > 0 ? len - p.window : 0;

        float o[RS][MT][4] = {};
        float m[RS], l[RS];
#pragma unroll
        for (int r = 0; r < RS; ++r) m[r] = -INFINITY, l[r] = 0.f;
        const int k_begin = (sp.u_first + x0) * UNIT + warp * KS;
        const int32_t* table = p.c.table + (long long)n * p.c.max_pages;
        // This warp's ring.  A stage is KS rows of K, KS of V, and in 8 bits their scale bytes.
        // Block-table entries are looked up one step before their rows are asked for.
        int entry[KG];
        auto position = [&](int k0, int kg) { return min(k0 + 16 * kg, (len - 1) & ~15); };
        auto look = [&](int k0) {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) entry[kg] = table[position(k0, kg) >> p.c.page_log2];
        };
        // Byte offsets in a stage.  Rows c_row + i RPI of a copy differ from row c_row in the swizzle by a constant per i;
        // the rows of a K read do not differ at all, those of a V read by the key's parity.
        constexpr int CH = RB / 16, RPI = 32 / CH;  // chunks of a row, rows per copy instruction
        const int c_row = lane / CH, c_ch = lane % CH;
        const uint32_t c_off = c_row * RB + ((c_ch ^ dec_swizzle<CH>(c_row)) << 4);
        const uint32_t k_off = g * RB + ((t ^ dec_swizzle<CH>(g)) << 4);
        const uint32_t v_off = KS * RB + 2 * t * RB + (((CH == 4 ? g >> 1 : g) ^ dec_swizzle<CH>(2 * t)) << 4);
        const uint8_t* k_src = static_cast<const uint8_t*>(p.c.k_cache) + c_row * RB + c_ch * 16;
        const uint8_t* v_src = static_cast<const uint8_t*>(p.c.v_cache) + c_row * RB + c_ch * 16;
        const uint8_t* s_src = lane ? p.c.v_scale : p.c.k_scale;
        auto fetch = [&](int k0, uint32_t dst) {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) {
                int pg = entry[kg];
                if ((unsigned)pg >= (unsigned)p.c.n_pages) {
                    if (lane == 0) atomicOr(err, kErrPages);
                    pg = 0;
                }
                // row of the 16 keys in the pool (below 2^31: checked on the host)
                const int row = ((pg * p.c.hkv + h) << p.c.page_log2) + (position(k0, kg) & ((1 << p.c.page_log2) - 1));
                const long long off = (long long)row * RB;
#pragma unroll
                for (int i = 0; i < 16 / RPI; ++i) {
                    const uint32_t to = (dst + c_off) ^ (dec_swizzle<CH>(i * RPI) << 4);
                    copy16(to + (kg * 16 + i * RPI) * RB, k_src + off + i * RPI * RB);
                    copy16(to + (KS + kg * 16 + i * RPI) * RB, v_src + off + i * RPI * RB);
                }
                if (E4M3 && lane < 2) copy16(dst + 2 * KS * RB + lane * KS + kg * 16, s_src + row);
            }
        };
        auto shared16 = [&](uint32_t at) {
            uint4 u;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
            return u;
        };
        auto shared_u16 = [&](uint32_t at) {
            uint16_t u;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(at) : "memory");
            return (uint32_t)u;
        };
        const uint32_t ring = sm100::smem_u32(smem) + warp * STAGES * Tr::STAGE;
        uint32_t st = ring, st_in = ring + (STAGES - 1) * Tr::STAGE;  // the stage in use and the one to fill
        auto advance = [&](uint32_t& at) { at = at == ring + (STAGES - 1) * Tr::STAGE ? ring : at + Tr::STAGE; };
        // The first unit may begin before the first key that any row sees, where the block table may hold anything (pages that
        // the window has passed): those rows, which the mask hides, are taken from that key's page.  Later units begin behind it.
        const int first_key = p.window > 0 ? max(0, len - T + 1 - p.window) : 0;
#pragma unroll
        for (int kg = 0; kg < KG; ++kg) entry[kg] = table[max(position(k_begin, kg), first_key) >> p.c.page_log2];
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) {
            if (i < cnt) {
                fetch(k_begin + i * UNIT, ring + i * Tr::STAGE);
                look(k_begin + (i + 1) * UNIT);
            }
            copy_commit();
        }

        bool taken_out = false;  // the same in all of the warp
        for (int x = 0; x < cnt; ++x) {
            const int k0 = k_begin + x * UNIT;
            copy_wait<STAGES - 2>();
            __syncwarp();
            // every lane is done with the stage of the step before: it takes the rows of STAGES - 1 steps ahead
            if (x + STAGES - 1 < cnt) {
                fetch(k0 + (STAGES - 1) * UNIT, st_in);
                advance(st_in);
                look(k0 + STAGES * UNIT);
            }
            copy_commit();
            unsigned ksc[NT], vsc[NT];  // scale bytes of keys 2t, 2t + 1 of each 8
            if (E4M3) {
#pragma unroll
                for (int kt = 0; kt < NT; ++kt) {
                    ksc[kt] = shared_u16(st + 2 * t + 2 * KS * RB + 8 * kt);
                    vsc[kt] = shared_u16(st + 2 * t + 2 * KS * RB + KS + 8 * kt);
                }
            }
            // ---- scores
            float s[NT][2 * RS];
#pragma unroll
            for (int kt = 0; kt < NT; ++kt) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < KL; ++j) {
                    const uint4 kr = shared16(((st + k_off) ^ (64 * j)) + 8 * kt * RB);
                    const uint32_t kw[4] = {kr.x, kr.y, kr.z, kr.w};
                    if (E4M3) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t(&a)[4] = qf[4 * j + i];
                            uint32_t b0, b1;
                            e4m3x4_f16(kw[i], b0, b1);
                            mma_f16(c, a[0], a[1], a[2], a[3], b0, b1);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t(&a)[4] = qf[2 * j + i];
                            mma_bf16(c, a[0], a[1], a[2], a[3], kw[2 * i], kw[2 * i + 1]);
                        }
                    }
                }
                if (E4M3) {
                    const float ks[2] = {scale_lo(ksc[kt]), scale_hi(ksc[kt])};
                    const float nan[2] = {ks[0] - ks[0], ks[1] - ks[1]};  // 0, or NaN for the NaN scale
#pragma unroll
                    for (int i = 0; i < 2 * RS; ++i) s[kt][i] = fmaf(c[i] * qscale[i >> 1], ks[i & 1], nan[i & 1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * RS; ++i) s[kt][i] = c[i] * p.scale_log2;
                }
            }
            // ---- mask: only steps that some row does not see whole
            const bool edge = k0 < full_lo || k0 + KS - 1 > full_hi;
            if (edge) {
#pragma unroll
                for (int kt = 0; kt < NT; ++kt)
#pragma unroll
                    for (int i = 0; i < 2 * RS; ++i) {
                        const int key = k0 + 8 * kt + 2 * t + (i & 1);
                        if (key > hi_[i >> 1] || key < lo_[i >> 1]) s[kt][i] = -INFINITY;
                    }
            }
            // ---- running maximum
            float top[RS];
            bool grow = false;
#pragma unroll
            for (int r = 0; r < RS; ++r) {
                top[r] = -INFINITY;
#pragma unroll
                for (int kt = 0; kt < NT; ++kt) top[r] = fmaxf(top[r], fmaxf(s[kt][2 * r], s[kt][2 * r + 1]));
                grow = grow || top[r] > m[r];
            }
            if (__any_sync(0xffffffffu, grow)) {
                float f[RS];
#pragma unroll
                for (int r = 0; r < RS; ++r) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                    f[r] = 1.f;
                    if (top[r] > m[r]) {  // each row by itself, whatever the others need
                        const float up = top[r] + kRescaleLog2;
                        f[r] = m[r] == -INFINITY ? 0.f : exp2f(m[r] - up);
                        l[r] *= f[r];
                        m[r] = up;
                    }
                }
#pragma unroll
                for (int r = 0; r < RS; ++r) {
                    const float fa = __shfl_sync(0xffffffffu, f[r], 8 * t), fb = __shfl_sync(0xffffffffu, f[r], 8 * t + 4);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        o[r][i][0] *= fa, o[r][i][2] *= fa;
                        o[r][i][1] *= fb, o[r][i][3] *= fb;
                    }
                }
            }
            uint32_t pf[NT][RS];  // P^T fragments: rows g and g + 8, keys 2t, 2t + 1 of each 8
#pragma unroll
            for (int r = 0; r < RS; ++r) {
                const float mu = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
                for (int kt = 0; kt < NT; ++kt) {
                    float a = sm100::ex2_approx(s[kt][2 * r] - mu), b = sm100::ex2_approx(s[kt][2 * r + 1] - mu);
                    l[r] += a + b;
                    if (E4M3) {  // (the NaN scale's codes are 0: infinity times them is NaN)
                        a *= scale_lo(vsc[kt]);
                        b *= scale_hi(vsc[kt]);
                    }
                    pf[kt][r] = pack_bf16x2(a, b);
                }
            }
            if (E4M3 && edge) {  // a key that a row does not see adds nothing, whatever its scale says
#pragma unroll
                for (int kt = 0; kt < NT; ++kt)
#pragma unroll
                    for (int r = 0; r < RS; ++r) {
                        if (s[kt][2 * r] == -INFINITY) pf[kt][r] &= 0xffff0000u;
                        if (s[kt][2 * r + 1] == -INFINITY) pf[kt][r] &= 0xffffu;
                    }
            }
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) {
                // V rows of keys 2t, 2t + 1, 2t + 8, 2t + 9: 16 bytes each (8 of a row of 64 codes; two of one of 256 bytes)
                uint4 vr[4], vr2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t at = ((st + v_off) ^ (dec_swizzle<CH>(i & 1) << 4)) + (16 * kg + (i & 1) + 8 * (i >> 1)) * RB;
                    vr[i] = shared16(at);
                    if (CH == 4 && (g & 1)) vr[i].x = vr[i].z, vr[i].y = vr[i].w;
                    if (CH == 16) vr2[i] = shared16(at + 128);
                }
                // ---- a masked key's V may hold anything, and 0 * NaN is NaN: non-finite values are taken out here, and added
                // behind the last step to the rows that do see their key (8-bit codes are always finite)
                if (!E4M3 && edge) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool bad = bf16x8_nonfinite(vr[i]) || (CH == 16 && bf16x8_nonfinite(vr2[i]));
                        if (!__any_sync(0xffffffffu, bad)) continue;
                        taken_out = true;
                        vr[i] = bf16x8_finite(vr[i]);
                        if (CH == 16) vr2[i] = bf16x8_finite(vr2[i]);
                    }
                }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t a0, a1, a2, a3;
                    if (E4M3) {
                        // channels 2i, 2i + 1 of this thread's 16 (8): codes of both keys of a pair, each with its sign
                        const int wd = i >> 1;
                        auto word = [&](const uint4& u) { return wd == 0 ? u.x : wd == 1 ? u.y : wd == 2 ? u.z : u.w; };
                        const uint32_t x0 = word(vr[0]), x1 = word(vr[1]), x2 = word(vr[2]), x3 = word(vr[3]);
                        const unsigned sa = (i & 1) ? 0xe6a2 : 0xc480, sb = (i & 1) ? 0xf7b3 : 0xd591;
                        a0 = e4m3_signed_to_bf16x2(permute(x0, x1, sa));
                        a1 = e4m3_signed_to_bf16x2(permute(x0, x1, sb));
                        a2 = e4m3_signed_to_bf16x2(permute(x2, x3, sa));
                        a3 = e4m3_signed_to_bf16x2(permute(x2, x3, sb));
                    } else {
                        const int wd = i & 3;
                        auto word = [&](const uint4& u) { return wd == 0 ? u.x : wd == 1 ? u.y : wd == 2 ? u.z : u.w; };
                        const uint4(&vv)[4] = i < 4 ? vr : vr2;
                        const uint32_t x0 = word(vv[0]), x1 = word(vv[1]), x2 = word(vv[2]), x3 = word(vv[3]);
                        a0 = __byte_perm(x0, x1, 0x5410);
                        a1 = __byte_perm(x0, x1, 0x7632);
                        a2 = __byte_perm(x2, x3, 0x5410);
                        a3 = __byte_perm(x2, x3, 0x7632);
                    }
#pragma unroll
                    for (int r = 0; r < RS; ++r) mma_bf16(o[r][i], a0, a1, a2, a3, pf[2 * kg][r], pf[2 * kg + 1][r]);
                }
            }
            advance(st);
        }
        if (!E4M3 && taken_out) {
            // The rare case: this warp's steps with masked keys once more, from the cache.  A non-finite value reaches its own
            // channel of the rows that see its key, whatever their weight (and nothing else: not the denominators).
            int hi[RS][2], lo[RS][2];  // of this thread's sums: rows 2t, 2t + 1 of each 8
#pragma unroll
            for (int r = 0; r < RS; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    hi[r][c] = __shfl_sync(0xffffffffu, hi_[r], 8 * t + 4 * c);
                    lo[r][c] = __shfl_sync(0xffffffffu, lo_[r], 8 * t + 4 * c);
                }
#pragma unroll 1
            for (int x = 0; x < cnt; ++x) {
                const int k0 = k_begin + x * UNIT;
                if (k0 >= full_lo && k0 + KS - 1 <= full_hi) continue;
#pragma unroll 1
                for (int key = max(k0, first_key); key < min(k0 + KS, len); ++key) {
                    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.c.v_cache) + attn_pool_row(p.c, table, key, h) * D;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(v + 64 * (i >> 2) + 8 * g + 2 * (i & 3));
#pragma unroll
                        for (int r = 0; r < RS; ++r) {
                            if (key >= lo[r][0] && key <= hi[r][0]) add_nonfinite(w, o[r][i][0], o[r][i][2]);
                            if (key >= lo[r][1] && key <= hi[r][1]) add_nonfinite(w, o[r][i][1], o[r][i][3]);
                        }
                    }
                }
            }
        }
        __syncthreads();  // every warp's ring is read: the join takes its place

        // ---- join the warps
#pragma unroll
        for (int r = 0; r < RS; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (t == 0) {
                s_ml[(warp * R + g + 8 * r) * 2] = m[r];
                s_ml[(warp * R + g + 8 * r) * 2 + 1] = l[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RS; ++r) {
            float f[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int q = 2 * t + c + 8 * r;
                float mm = -INFINITY;
#pragma unroll
                for (int ww = 0; ww < kDecWarps; ++ww) mm = fmaxf(mm, s_ml[(ww * R + q) * 2]);
                const float mine = s_ml[(warp * R + q) * 2];
                f[c] = mine == -INFINITY ? 1.f : exp2f(mine - mm);  // no maximum: nothing seen, or a NaN to pass on
            }
            // channels 2i and 2i + 1 of this thread's share are neighbours
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int d = E4M3 ? (D / 8) * g + 2 * i : 64 * (i >> 2) + 8 * g + 2 * (i & 3);
                *reinterpret_cast<float2*>(&s_o[(warp * R + 2 * t + 8 * r) * D + d]) = make_float2(o[r][i][0] * f[0], o[r][i][2] * f[0]);
                *reinterpret_cast<float2*>(&s_o[(warp * R + 2 * t + 1 + 8 * r) * D + d]) = make_float2(o[r][i][1] * f[1], o[r][i][3] * f[1]);
            }
        }
        __syncthreads();
        const bool whole = cnt == sp.units;
        const int slot = w == w0 ? 0 : 1;
        for (int i = tid; i < R * D / 4; i += kDecThreads) {
            const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
            const int row = rg * R + r;
            if (row >= rows) continue;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int ww = 0; ww < kDecWarps; ++ww) mm = fmaxf(mm, s_ml[(ww * R + r) * 2]);
#pragma unroll
            for (int ww = 0; ww < kDecWarps; ++ww) {
                const float4 b = *reinterpret_cast<const float4*>(&s_o[(ww * R + r) * D + d]);
                a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
                const float mw = s_ml[(ww * R + r) * 2];
                ll += s_ml[(ww * R + r) * 2 + 1] * (mw == -INFINITY ? 1.f : exp2f(mw - mm));
            }
            if (whole) {
                const int tok = row / p.G, gh = row - tok * p.G;
                const long long at = (long long)(sp.s.start + tok) * p.hq + h * p.G + gh;
                attn_store4(p.o, p.o_f32, at * D + d, a, ll == 0.f ? 0.f : 1.f / ll);
                if (d == 0 && p.lse) p.lse[at] = attn_lse(mm, ll);
            } else {
                const long long at = ((long long)cta * 2 + slot) * R + r;
                reinterpret_cast<float4*>(p.part + at * D)[d / 4] = a;
                if (d == 0) {
                    p.ml[at * 2] = mm;
                    p.ml[at * 2 + 1] = ll;
                }
            }
        }
        if (!whole && x0 == 0 && tid == 0) {  // the item starts here and ends in a later CTA
            const long long end = w + sp.units;
            desc[0] = n;
            desc[1] = h;
            desc[2] = rg * R;
            desc[3] = min(R, rows - rg * R);
            desc[4] = slot;
            desc[5] = (int)((end * grid + W - 1) / W) - cta;  // up to the first CTA that begins at `end` or behind
            desc[6] = sp.s.start;
        }
        __syncthreads();
        w += cnt;
        off += cnt;
    }
}

// ------------------------------------------------------------------------------------------ joining split items
// Softmax parts combine like blocks do: by a common maximum, sums and denominators.  One launch joins the parts of both
// kernels.
//
// An item of the decode kernel has few rows and may have many parts (one long context shared out among all CTAs): a block
// takes one row, warp w its parts w, w + 8, ..., with a running maximum, and the warps' results combine the same way.
constexpr int kJoinWarps = 8;
struct JoinArrays {
    const int* desc;
    const float* part;
    const float* ml;
};
struct JoinParams {
    JoinArrays dec, tc;
    void* o;
    float* lse;
    int tc_blocks, dec_split;  // blocks for the chunk kernel's items, and for each of the decode kernel's
    int rows;                  // R of the decode kernel
    int G, hq, d, o_f32;
};

struct JoinRow {
    float4 a;
    float m, l;
    __device__ __forceinline__ void add(float4 v, float vm, float vl) {
        if (vm == -INFINITY && vl == 0.f) return;  // nothing seen there: its sums may not have been written
        const float nm = fmaxf(m, vm);
        // no maximum at all but a denominator: a NaN to pass on
        const float fa = m == -INFINITY ? 0.f : exp2f(m - nm), fv = vm == -INFINITY ? 1.f : exp2f(vm - nm);
        a.x = a.x * fa + v.x * fv, a.y = a.y * fa + v.y * fv, a.z = a.z * fa + v.z * fv, a.w = a.w * fa + v.w * fv;
        l = l * fa + vl * fv;
        m = nm;
    }
};

// An item of the chunk kernel has 256 rows, in the layout [row tile][d / 4][128 rows][4]: a block takes 32 of them, a lane
// one row, a warp NC groups of 4 channels, with a running maximum.  Everything of a part is asked for at once.
constexpr int kJoinTileBlocks = 8;  // blocks of an item
template <int NC>
__device__ __forceinline__ void join_tile(const JoinParams& p, int block) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = block / kJoinTileBlocks, r = block % kJoinTileBlocks * 32 + lane;  // row of the item
    const int4 d0 = reinterpret_cast<const int4*>(p.tc.desc)[c * 2], d1 = reinterpret_cast<const int4*>(p.tc.desc)[c * 2 + 1];
    if (d0.x < 0 || r - lane >= d0.w) return;
    const int h = d0.y, rows = d0.w, slot0 = d1.x, parts = d1.y, start = d1.z;
    const bool there = r < rows;
    constexpr int d4 = 8 * NC;  // groups of 4 channels
    const int warp_at = ((r >> 7) * d4 + warp * NC) * 128 + (r & 127);
    float m = -INFINITY, l = 0.f;
    float4 a[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
        const int slot = (c + k) * 2 + (k ? 0 : slot0);
        const float2 x = reinterpret_cast<const float2*>(p.tc.ml)[slot * 256 + r];
        float4 v[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j) v[j] = reinterpret_cast<const float4*>(p.tc.part)[(long long)slot * (256 * d4) + warp_at + j * 128];
        // a part that has seen nothing of a row may not have written its sums (what stands there is not used)
        if (x.x == -INFINITY && x.y == 0.f) continue;
        const float nm = fmaxf(m, x.x);
        // (no maximum at all but a denominator: a NaN to pass on)
        const float fa = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f(m - nm), fv = x.x == -INFINITY ? 1.f : exp2f(x.x - nm);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            a[j].x = fmaf(v[j].x, fv, a[j].x * fa), a[j].y = fmaf(v[j].y, fv, a[j].y * fa);
            a[j].z = fmaf(v[j].z, fv, a[j].z * fa), a[j].w = fmaf(v[j].w, fv, a[j].w * fa);
        }
        l = fmaf(x.y, fv, l * fa);
        m = nm;
    }
    if (!there) return;
    const int row = d0.z + r, tok = row / p.G, gh = row - tok * p.G;
    const long long at = (long long)(start + tok) * p.hq + h * p.G + gh;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int j = 0; j < NC; ++j) attn_store4(p.o, p.o_f32, at * p.d + (warp * NC + j) * 4, a[j], inv);
    if (warp == 0 && p.lse) p.lse[at] = attn_lse(m, l);
}

__global__ void __launch_bounds__(kJoinWarps * 32) gdn_attn_join_kernel(const JoinParams p) {
    __shared__ float4 s_a[kJoinWarps][32];
    __shared__ float2 s_ml[kJoinWarps];
    cudaGridDependencySynchronize();
    if ((int)blockIdx.x < p.tc_blocks) {  // the longer ones first
        if (p.d == 128) join_tile<4>(p, blockIdx.x);
        else join_tile<2>(p, blockIdx.x);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x - p.tc_blocks, c = b / p.dec_split, y = b - c * p.dec_split;
    const int4 d0 = reinterpret_cast<const int4*>(p.dec.desc)[c * 2], d1 = reinterpret_cast<const int4*>(p.dec.desc)[c * 2 + 1];
    if (d0.x < 0) return;
    const int h = d0.y, rows = d0.w, slot0 = d1.x, parts = d1.y, start = d1.z;
    const bool alone = parts <= kJoinWarps;  // few parts: a warp per row
    const int first = alone ? 0 : warp, step = alone ? 1 : kJoinWarps;
    const bool mine = lane * 4 < p.d;
    for (int r = alone ? y * kJoinWarps + warp : y; r < rows; r += alone ? p.dec_split * kJoinWarps : p.dec_split) {
        float4 v;
        float2 ml;
        auto ask = [&](int i) {
            v = make_float4(0.f, 0.f, 0.f, 0.f);
            ml = make_float2(-INFINITY, 0.f);
            if (i < parts) {
                const long long at = ((long long)(c + i) * 2 + (i ? 0 : slot0)) * p.rows + r;
                ml = *reinterpret_cast<const float2*>(p.dec.ml + at * 2);
                if (mine) v = *reinterpret_cast<const float4*>(p.dec.part + at * p.d + 4 * lane);
            }
        };
        JoinRow out{make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
        ask(first);
#pragma unroll 4
        for (int i = first; i < parts; i += step) {
            const float4 x = v;
            const float2 xm = ml;
            ask(i + step);
            out.add(x, xm.x, xm.y);
        }
        if (!alone) {
            __syncthreads();  // the row before has been read
            s_a[warp][lane] = out.a;
            if (lane == 0) s_ml[warp] = make_float2(out.m, out.l);
            __syncthreads();
            if (warp != 0) continue;
#pragma unroll
            for (int w = 1; w < kJoinWarps; ++w) out.add(s_a[w][lane], s_ml[w].x, s_ml[w].y);
        }
        const int row = d0.z + r, tok = row / p.G, gh = row - tok * p.G;
        const long long at = (long long)(start + tok) * p.hq + h * p.G + gh;
        if (mine) attn_store4(p.o, p.o_f32, at * p.d + 4 * lane, out.a, out.l == 0.f ? 0.f : 1.f / out.l);
        if (lane == 0 && p.lse) p.lse[at] = attn_lse(out.m, out.l);
    }
}

}  // namespace gdn
