// Attention of new tokens over the paged cache (gdn_kv.cuh): scheduling shared by the two kernels, the kernel for
// few query rows (decoding), and the kernel that joins split items.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j - max),   over keys j <= pos_i, and with a
//   window also j > pos_i - window;  pos_i is the new token's place in its sequence.
//
// Query heads share KV heads in groups of G, so the unit of work is an item: (sequence, KV head, group of query rows),
// where row r of a (sequence, KV head) is new token r / G and head r mod G of the group.  Every item streams its keys
// once in blocks of 128 or 256 (a unit).  All units of all items form one line, and each CTA takes an equal stretch of it
// whatever the sequences' lengths are: the split depends on device-side lengths only, so a captured graph replays
// with new lengths and nothing is read back.  A CTA ends up with whole items (written directly) and at most two parts
// of items, its first and its last, whose unnormalised sums, maxima and denominators go to the workspace; the join
// kernel adds the parts of an item in a fixed order.  The workspace is therefore a fixed size per CTA.
#pragma once

#include "gdn_kv.cuh"

// gdn_sm100.cuh defines one out-of-line function; declared static first, it stays local to this translation unit (the
// library's other one has its own).
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
    int rows_lo, rows_hi;    // this kernel takes sequences with rows_lo < T G <= rows_hi
    int* desc;               // [grid][kDescInts]: the split item that starts in this CTA, for the join kernel
    float* part;             // [grid][2][R][d] partial sums
    float* ml;               // [grid][2][R][2] maximum (base 2) and denominator
};
// n (-1: none), KV head, first row, rows, slot of the first part, number of CTAs it spans
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

// ------------------------------------------------------------------------------------------ few rows
// mma.sync kernel for up to 16 query rows per item.  Bound by the cache's bytes: tensor work is small, and what counts
// is that every warp keeps 16-byte loads in flight.  K and V go from global memory straight into the registers of
// the matrix instructions, without shared memory: the order of the contraction index is free, so thread t of a quad
// takes 8 (16 in 8 bits) consecutive channels of its key as its share of several k-steps (Q is loaded in the same
// order), and for V the keys of a step are interleaved with byte permutes.
//   S[q][key]: A = Q (16 rows), B = K; thread (g, t) = (lane / 4, lane % 4) gets rows g, g + 8 and keys 2t, 2t + 1.
//   O^T[d][q]: A = V^T (16 channels x 16 keys), B = P^T, whose fragment is exactly S's: no shuffle in between.
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
// e4m3 codes in the high bytes of both halves of `w` (low bytes: anything) as a bf16 pair.  The code's exponent and
// mantissa moved to bf16's place make the value times 2^-120 (biases 7 and 127), subnormal codes included, and one
// exact multiplication undoes that.  0x7f, e4m3's NaN, would read as 480: the cache writer never stores it.
__device__ __forceinline__ uint32_t e4m3_hi_to_bf16x2(uint32_t w) {
    const uint32_t s = w & 0x80008000u;
    return mul_bf16x2(((w >> 4) & 0x07f007f0u) | s, 0x7b807b80u);
}
// Codes 0, 1 and 2, 3 of a word.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, int hi) {
    return e4m3_hi_to_bf16x2(hi ? __byte_perm(w, 0, 0x3424) : __byte_perm(w, 0, 0x1404));
}
__device__ __forceinline__ bool bf16x2_nonfinite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

constexpr int kDecThreads = 256, kDecWarps = 8, kDecRows = 16;
constexpr float kRescaleLog2 = 8.f;  // the running maximum follows only when it would be off by more than 2^8

template <int D, bool E4M3> struct DecTraits {
    static constexpr int KS = (D == 128 && !E4M3) ? 16 : 32;  // keys of one warp step
    static constexpr int UNIT = KS * kDecWarps;
    static constexpr int KL = D * (E4M3 ? 1 : 2) / 64;        // 16-byte K loads per thread and 8 keys
    static constexpr int MT = D / 16;                         // channel tiles of 16
    static constexpr size_t smem = kDecWarps * kDecRows * D * 4 + kDecWarps * kDecRows * 8 + 256;
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(kDecThreads, D == 64 ? 2 : 1) gdn_attn_decode_kernel(const AttnParams p, unsigned* err) {
    using Tr = DecTraits<D, E4M3>;
    constexpr int KS = Tr::KS, UNIT = Tr::UNIT, KL = Tr::KL, MT = Tr::MT, R = kDecRows, NT = KS / 8, KG = KS / 16;
    extern __shared__ __align__(16) uint8_t smem[];
    float* s_o = reinterpret_cast<float*>(smem);                  // [warps][R][D]
    float* s_ml = s_o + kDecWarps * R * D;                        // [warps][R][2]
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
        while (off >= (long long)sp.units * sp.rgs * p.c.hkv) {  // next sequence with work
            off = 0;
            sp = attn_span<R, UNIT>(p, ++n, err);
        }
        const int item = (int)(off / sp.units), x0 = (int)(off - (long long)item * sp.units);
        const int h = item / sp.rgs, rg = item - h * sp.rgs;
        const int cnt = (int)min((long long)(sp.units - x0), w1 - w);
        const int T = sp.s.T, len = sp.s.len;

        // ---- the item's query rows: A fragments, in K's channel order
        const int row_lo = rg * R + g, rows = T * p.G;
        uint32_t qf[D / 16][4];
        int hi_[2], lo_[2];  // keys [lo_, hi_] that rows g and g + 8 see
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = row_lo + 8 * r;
            const bool there = row < rows;
            const int tok = there ? row / p.G : 0, gh = there ? row - tok * p.G : 0;
            const int pos = len - T + tok;
            hi_[r] = there ? pos : -1;
            lo_[r] = p.window > 0 ? pos - p.window + 1 : 0;
            const __nv_bfloat16* q = p.q + (long long)(sp.s.start + tok) * p.q_stride + (h * p.G + gh) * D;
            if (E4M3) {
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint2 u = there ? *reinterpret_cast<const uint2*>(q + 64 * j + 16 * t + 4 * s) : make_uint2(0, 0);
                        qf[4 * j + s][r] = u.x;
                        qf[4 * j + s][2 + r] = u.y;
                    }
            } else {
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint4 u = there ? *reinterpret_cast<const uint4*>(q + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
                    qf[2 * j][r] = u.x;
                    qf[2 * j][2 + r] = u.y;
                    qf[2 * j + 1][r] = u.z;
                    qf[2 * j + 1][2 + r] = u.w;
                }
            }
        }
        // keys that every row of the sequence sees: [full_lo, full_hi]
        const int full_hi = len - T, full_lo = p.window > 0 ? len - p.window : 0;

        float o[2][MT][4] = {};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        const int k_begin = (sp.u_first + x0) * UNIT + warp * KS;
        uint4 kr[NT][KL];
        uint4 vr[KG][4];        // bf16, D == 128: two chunks -> vr2
        uint4 vr2[KG][4];
        unsigned ksc[NT], vsc[NT];  // scale bytes of keys 2t, 2t + 1 of each 8
        constexpr int ESZ = E4M3 ? 1 : 2;

        auto page_row = [&](int k0) {  // row index of position k0 (a multiple of 16) in the pool
            const int kk = min(k0, len - 1) & ~15;
            int pg = p.c.table[(long long)n * p.c.max_pages + (kk >> p.c.page_log2)];
            if (pg < 0 || pg >= p.c.n_pages) {
                if (lane == 0) atomicOr(err, kErrPages);
                pg = 0;
            }
            return (((long long)pg * p.c.hkv + h) << p.c.page_log2) + (kk & ((1 << p.c.page_log2) - 1));
        };
        long long prow[KG];
        auto find = [&](int k0) {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) prow[kg] = page_row(k0 + 16 * kg);
        };
        auto load_k = [&]() {
#pragma unroll
            for (int kt = 0; kt < NT; ++kt) {
                const long long row = prow[kt >> 1] + 8 * (kt & 1);
                const uint8_t* base = static_cast<const uint8_t*>(p.c.k_cache) + (row + g) * (D * ESZ) + 16 * t;
#pragma unroll
                for (int j = 0; j < KL; ++j) kr[kt][j] = *reinterpret_cast<const uint4*>(base + 64 * j);
                if (E4M3) ksc[kt] = *reinterpret_cast<const uint16_t*>(p.c.k_scale + row + 2 * t);
            }
        };
        auto load_v = [&]() {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long row = prow[kg] + 2 * t + (i & 1) + 8 * (i >> 1);
                    const uint8_t* base = static_cast<const uint8_t*>(p.c.v_cache) + row * (D * ESZ);
                    if (E4M3 && D == 64) {
                        const uint2 u = *reinterpret_cast<const uint2*>(base + 8 * g);
                        vr[kg][i] = make_uint4(u.x, u.y, 0, 0);
                    } else {
                        vr[kg][i] = *reinterpret_cast<const uint4*>(base + 16 * g);
                    }
                    if (!E4M3 && D == 128) vr2[kg][i] = *reinterpret_cast<const uint4*>(base + 128 + 16 * g);
                }
                if (E4M3) {
                    vsc[2 * kg] = *reinterpret_cast<const uint16_t*>(p.c.v_scale + prow[kg] + 2 * t);
                    vsc[2 * kg + 1] = *reinterpret_cast<const uint16_t*>(p.c.v_scale + prow[kg] + 8 + 2 * t);
                }
            }
        };
        find(k_begin);
        load_k();
        load_v();

        for (int x = 0; x < cnt; ++x) {
            const int k0 = k_begin + x * UNIT;
            const bool more = x + 1 < cnt;
            // ---- scores
            float s[NT][4];
#pragma unroll
            for (int kt = 0; kt < NT; ++kt) {
                s[kt][0] = s[kt][1] = s[kt][2] = s[kt][3] = 0.f;
#pragma unroll
                for (int j = 0; j < KL; ++j) {
                    const uint32_t kw[4] = {kr[kt][j].x, kr[kt][j].y, kr[kt][j].z, kr[kt][j].w};
                    if (E4M3) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16(s[kt], qf[4 * j + i][0], qf[4 * j + i][1], qf[4 * j + i][2], qf[4 * j + i][3],
                                     e4m3_pair(kw[i], 0), e4m3_pair(kw[i], 1));
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            mma_bf16(s[kt], qf[2 * j + i][0], qf[2 * j + i][1], qf[2 * j + i][2], qf[2 * j + i][3],
                                     kw[2 * i], kw[2 * i + 1]);
                    }
                }
                const float c0 = E4M3 ? p.scale_log2 * kv_scale_value(ksc[kt] & 0xff) : p.scale_log2;
                const float c1 = E4M3 ? p.scale_log2 * kv_scale_value(ksc[kt] >> 8) : p.scale_log2;
                s[kt][0] *= c0, s[kt][1] *= c1, s[kt][2] *= c0, s[kt][3] *= c1;
            }
            // ---- the next step's keys
            if (more) {
                // V of this step is in registers already; prow moves on
                find(k0 + UNIT);
                load_k();
            }
            // ---- mask: only steps that some row does not see whole
            const bool edge = k0 < full_lo || k0 + KS - 1 > full_hi;
            if (edge) {
#pragma unroll
                for (int kt = 0; kt < NT; ++kt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = k0 + 8 * kt + 2 * t + (i & 1), r = i >> 1;
                        if (key > hi_[r] || key < lo_[r]) s[kt][i] = -INFINITY;
                    }
            }
            // ---- running maximum
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int kt = 0; kt < NT; ++kt) {
                top[0] = fmaxf(top[0], fmaxf(s[kt][0], s[kt][1]));
                top[1] = fmaxf(top[1], fmaxf(s[kt][2], s[kt][3]));
            }
            if (__any_sync(0xffffffffu, top[0] > m[0] + kRescaleLog2 || top[1] > m[1] + kRescaleLog2)) {
                float f[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                    const float nm = fmaxf(m[r], top[r]);
                    f[r] = m[r] == -INFINITY ? 0.f : exp2f(m[r] - nm);
                    l[r] *= f[r];
                    m[r] = nm;
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float fa = __shfl_sync(0xffffffffu, f[r], 8 * t), fb = __shfl_sync(0xffffffffu, f[r], 8 * t + 4);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        o[r][i][0] *= fa, o[r][i][2] *= fa;
                        o[r][i][1] *= fb, o[r][i][3] *= fb;
                    }
                }
            }
            const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
            uint32_t pf[NT][2];  // P^T fragments: rows g and g + 8, keys 2t, 2t + 1 of each 8
#pragma unroll
            for (int kt = 0; kt < NT; ++kt) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float a = sm100::ex2_approx(s[kt][2 * r] - mu[r]), b = sm100::ex2_approx(s[kt][2 * r + 1] - mu[r]);
                    l[r] += a + b;
                    if (E4M3) {
                        const float va = kv_scale_value(vsc[kt] & 0xff), vb = kv_scale_value(vsc[kt] >> 8);
                        // a key that this row does not see adds nothing, whatever its scale says
                        a = edge && s[kt][2 * r] == -INFINITY ? 0.f : a * va;
                        b = edge && s[kt][2 * r + 1] == -INFINITY ? 0.f : b * vb;
                    }
                    pf[kt][r] = pack_bf16x2(a, b);
                }
            }
            // ---- a masked key's V may hold anything, and 0 * NaN is NaN: non-finite values there are taken out, and
            // the rows that do see such a key get a NaN weight instead (8-bit codes are always finite)
            if (!E4M3 && edge) {
#pragma unroll
                for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        bool bad = bf16x2_nonfinite(vr[kg][i].x) || bf16x2_nonfinite(vr[kg][i].y) ||
                                   bf16x2_nonfinite(vr[kg][i].z) || bf16x2_nonfinite(vr[kg][i].w);
                        if (D == 128)
                            bad = bad || bf16x2_nonfinite(vr2[kg][i].x) || bf16x2_nonfinite(vr2[kg][i].y) ||
                                  bf16x2_nonfinite(vr2[kg][i].z) || bf16x2_nonfinite(vr2[kg][i].w);
                        if (!__any_sync(0xffffffffu, bad)) continue;
                        unsigned any = bad;  // over the eight threads that hold this key
                        any |= __shfl_xor_sync(0xffffffffu, any, 4);
                        any |= __shfl_xor_sync(0xffffffffu, any, 8);
                        any |= __shfl_xor_sync(0xffffffffu, any, 16);
                        if (any) {
                            vr[kg][i] = make_uint4(0, 0, 0, 0);
                            if (D == 128) vr2[kg][i] = make_uint4(0, 0, 0, 0);
                            const int kt = 2 * kg + (i >> 1), key = k0 + 8 * kt + 2 * t + (i & 1);
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                if (key <= hi_[r] && key >= lo_[r])
                                    pf[kt][r] = (i & 1) ? (pf[kt][r] & 0xffffu) | 0x7fc00000u : (pf[kt][r] & 0xffff0000u) | 0x7fc0u;
                        }
                    }
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) {
                const uint32_t b00 = pf[2 * kg][0], b01 = pf[2 * kg + 1][0], b10 = pf[2 * kg][1], b11 = pf[2 * kg + 1][1];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t a0, a1, a2, a3;
                    if (E4M3) {
                        // channels 2i, 2i + 1 of this thread's 16 (8): codes of both keys of a pair into one word
                        const int wd = i >> 1;
                        auto word = [&](const uint4& u) { return wd == 0 ? u.x : wd == 1 ? u.y : wd == 2 ? u.z : u.w; };
                        const uint32_t x0 = word(vr[kg][0]), x1 = word(vr[kg][1]), x2 = word(vr[kg][2]), x3 = word(vr[kg][3]);
                        const unsigned sa = (i & 1) ? 0x6020 : 0x4000, sb = (i & 1) ? 0x7030 : 0x5010;
                        a0 = e4m3_hi_to_bf16x2(__byte_perm(x0, x1, sa));
                        a1 = e4m3_hi_to_bf16x2(__byte_perm(x0, x1, sb));
                        a2 = e4m3_hi_to_bf16x2(__byte_perm(x2, x3, sa));
                        a3 = e4m3_hi_to_bf16x2(__byte_perm(x2, x3, sb));
                    } else {
                        const int wd = i & 3;
                        auto word = [&](const uint4& u) { return wd == 0 ? u.x : wd == 1 ? u.y : wd == 2 ? u.z : u.w; };
                        const uint4(&vv)[4] = i < 4 ? vr[kg] : vr2[kg];
                        const uint32_t x0 = word(vv[0]), x1 = word(vv[1]), x2 = word(vv[2]), x3 = word(vv[3]);
                        a0 = __byte_perm(x0, x1, 0x5410);
                        a1 = __byte_perm(x0, x1, 0x7632);
                        a2 = __byte_perm(x2, x3, 0x5410);
                        a3 = __byte_perm(x2, x3, 0x7632);
                    }
                    mma_bf16(o[0][i], a0, a1, a2, a3, b00, b01);
                    mma_bf16(o[1][i], a0, a1, a2, a3, b10, b11);
                }
            }
            if (more) load_v();
        }

        // ---- join the warps
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (t == 0) {
                s_ml[(warp * R + g + 8 * r) * 2] = m[r];
                s_ml[(warp * R + g + 8 * r) * 2 + 1] = l[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
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
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                if (p.o_f32) {
                    reinterpret_cast<float4*>(static_cast<float*>(p.o) + at * D)[d / 4] = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
                } else {
                    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * D)[d / 4] =
                        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
                }
                if (d == 0 && p.lse) p.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
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
            const int c1 = (int)((end * grid + W - 1) / W);  // first CTA whose stretch begins at `end` or behind
            desc[0] = n;
            desc[1] = h;
            desc[2] = rg * R;
            desc[3] = min(R, rows - rg * R);
            desc[4] = slot;
            desc[5] = c1 - cta;
            desc[6] = sp.s.start;
        }
        __syncthreads();
        w += cnt;
        off += cnt;
    }
}

// ------------------------------------------------------------------------------------------ joining split items
// Block (c, y) joins rows [y kJoinRows, (y + 1) kJoinRows) of the item that starts in CTA c and does not end there.
constexpr int kJoinRows = 8, kJoinThreads = 256;
struct JoinParams {
    const int* desc[2];
    const float* part[2];
    const float* ml[2];
    int grid[2];  // CTAs of each attention kernel (0: not launched)
    int rows[2];  // R of each
    void* o;
    float* lse;
    int G, hq, d, o_f32;
};

__global__ void __launch_bounds__(kJoinThreads) gdn_attn_join_kernel(const JoinParams p) {
    cudaGridDependencySynchronize();
    int c = blockIdx.x, which = 0;
    if (c >= p.grid[0]) c -= p.grid[0], which = 1;
    const int* desc = p.desc[which] + (long long)c * kDescInts;
    if (desc[0] < 0) return;
    const int h = desc[1], row0 = desc[2], rows = desc[3], slot0 = desc[4], parts = desc[5], start = desc[6], R = p.rows[which];
    const int tpr = p.d / 4, per = kJoinThreads / tpr;  // threads of a row, rows at a time
    const int d4 = threadIdx.x % tpr;
    for (int r = blockIdx.y * kJoinRows + threadIdx.x / tpr; r < min(rows, ((int)blockIdx.y + 1) * kJoinRows); r += per) {
        const float* ml = p.ml[which];
        float mm = -INFINITY;
        for (int i = 0; i < parts; ++i) mm = fmaxf(mm, ml[((((long long)(c + i) * 2 + (i ? 0 : slot0)) * R) + r) * 2]);
        float ll = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < parts; ++i) {
            const long long at = ((long long)(c + i) * 2 + (i ? 0 : slot0)) * R + r;
            const float mi = ml[at * 2];
            if (mi == -INFINITY && ml[at * 2 + 1] == 0.f) continue;  // nothing seen there: its sums are not written
            const float f = mi == -INFINITY ? 1.f : exp2f(mi - mm);
            const float4 b = reinterpret_cast<const float4*>(p.part[which] + at * p.d)[d4];
            ll += ml[at * 2 + 1] * f;
            a.x += b.x * f, a.y += b.y * f, a.z += b.z * f, a.w += b.w * f;
        }
        const int row = row0 + r, tok = row / p.G, gh = row - tok * p.G;
        const long long at = (long long)(start + tok) * p.hq + h * p.G + gh;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        if (p.o_f32) {
            reinterpret_cast<float4*>(static_cast<float*>(p.o) + at * p.d)[d4] = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        } else {
            reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * p.d)[d4] =
                make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        }
        if (d4 == 0 && p.lse) p.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
    }
}

}  // namespace gdn
