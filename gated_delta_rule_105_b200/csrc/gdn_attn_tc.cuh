// Paged attention for many query rows (chunks of prompts): tcgen05 kernel.  See gdn_attn.cuh for the operator, the items
// and how their units are shared out; here an item is 256 query rows of one (sequence, KV head) and a unit is a tile of
// 128 keys.
//
// Bound by the tensor core on paper (4 d flops per row and key); measured over three sequences of up to 16384 positions
// and 1000 new tokens, 16 query and 4 KV heads x 128, bf16: 321 to 330 us, 0.83 PFLOP/s.  A step of 64 keys takes a
// warpgroup 2150 cycles, of which its exponentials take 911 (512 if it had the SM's exp units to itself), rescaling and
// maximum 470, reading S 290 and waiting for it 420; exp units and tensor core are both busy 45% of the time.
//
// One CTA per SM.  The 256 rows are two tiles of 128 (the height of one MMA), each with its own softmax warpgroup.  Scores
// come in steps of 64 keys with two buffers per row tile: S of the next step is there before the softmax of this one is
// done, so neither the softmax nor the tensor core waits for the other's latency (one buffer of 128 keys: 347 us).
//   warp 0        loads K and V tiles: one tensor-map box per (page, 64 channels), a ring of stages each
//   warps 1, 2    issue S = Q K^T (both operands in shared memory) and O += P V (P in tensor memory), one per row tile
//   warp 3        bf16 cache: looks for non-finite V rows in tiles that are not wholly visible (see below)
//   warps 4 - 11  softmax: thread = row, the 64 scores of a step in registers, P back into the columns of S as bf16
//   warps 12 - 15 8-bit cache: codes of a tile (bulk copies, one per page) to exact bf16 in the swizzled layout
// Tensor memory: S/P of both tiles (2 x 2 x 64 columns) and O of both (2 x d).  The running maximum is lazy (kRescaleLog2):
// that O is scaled down is rare after the first steps; then the warp waits for the last P V and reads and writes its part
// of O itself.
//
// Masked keys.  A score that a row must not see is set to -inf before the maximum, so K may hold anything there.  For V a
// weight of 0 is not enough, 0 * NaN is NaN: in tiles that some row does not see whole, NaNs and infinities of V are zeroed in
// shared memory (in 8 bits the rows with the NaN scale) and their keys marked; a row that does see a marked key gets them
// at the end of its segment, each in its own channel, from the cache.
#pragma once

#include "gdn_attn.cuh"

namespace gdn {

constexpr int kTcRows = 256, kTcTile = 128, kTcStep = 64;

template <int D, bool E4M3> struct AttnTc {
    static constexpr int THREADS = E4M3 ? 512 : 384;
    static constexpr int NK = 2, NV = E4M3 ? 2 : 3, NR = E4M3 ? 2 : 0;  // K, V and raw stages
    static constexpr int HALF = kTcTile * 128;                          // 64 channels of 128 rows, bf16
    static constexpr int TILE = HALF * (D / 64);
    static constexpr int RAW = kTcTile * D;
    static constexpr int OFF_Q = 0, OFF_K = 2 * TILE, OFF_V = OFF_K + NK * TILE, OFF_RAW = OFF_V + NV * TILE;
    static constexpr int OFF_SC = OFF_RAW + NR * RAW;       // raw scale bytes
    static constexpr int OFF_CTL = OFF_SC + NR * kTcTile;   // barriers and the like
    static constexpr int CTL = 1024;
    static constexpr int BYTES = OFF_CTL + CTL + 1024;      // + alignment to 1024
    static_assert(BYTES <= 232448, "shared memory of a block");
};

struct AttnTcCtl {
    uint64_t q_full[2], k_full[3], k_empty[3], v_full[3], v_ready[3], v_empty[3], r_full[2], r_empty[2];
    uint64_t s_full[2][2], p_full[2][2], o_full[2][2], drain[2];  // [row tile][buffer of S]
    uint64_t stall;  // diagnostic only: nothing ever arrives on it (gdn_debug_stall)
    uint32_t tmem;
    volatile int abort_flag;
    uint32_t bad[3][4];  // marked keys of each V stage's tile
    uint8_t saw[256];    // whether a row has seen a marked key (its own thread writes and reads it)
    // where this CTA's stretch starts
    long long W, w0, w1;
    int n, h, rt, x;
};
static_assert(sizeof(AttnTcCtl) <= 1024, "control block");
// Used while the work is shared out, in Q's place.
struct TcScratch {
    long long scan[32];
    long long pre[257];
};

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            sm100::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(sm100::smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}
// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld16(uint32_t ta, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(ta)
        : "memory");
}
// gdn_sm100.cuh's bounded wait without its out-of-line part: a kernel that moves registers between its warpgroups
// (setmaxnreg) cannot call functions.
constexpr long long kTcStallCycles = 2000000LL;  // of the diagnostic wait: about 1 ms
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err,
                                        long long limit = sm100::kWaitLimitCycles) {
    if (sm100::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (*abort_flag) return false;
        if (sm100::mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > limit) {
            *abort_flag = 1;
            atomicOr(err, kErrTimeout);
            return false;
        }
    }
}
__device__ __forceinline__ bool tc_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
    return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_flag, err));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// MMAs whose descriptors are given by their low words (addresses); the high words are constants.  The issuing warp walks
// along whole, with the bases made uniform by a shuffle, so that the operands stay in uniform registers: built by one
// thread in vector registers they cost 85 cycles an instruction, more than the tensor core takes for it.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
template <uint32_t HI_A, uint32_t HI_B, uint32_t IDESC>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %6, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(accumulate), "n"(HI_A), "n"(HI_B), "r"(IDESC)
        : "memory");
}
template <uint32_t HI_B, uint32_t IDESC>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b64 db, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b), "r"(accumulate), "n"(HI_B), "r"(IDESC)
        : "memory");
}
// Descriptor words as gdn_sm100.cuh's umma_desc() has them: address and leading offset (low), stride offset, version and
// 128-byte swizzle (high).
__host__ __device__ constexpr uint32_t desc_low(uint32_t saddr, uint32_t lbo) { return ((saddr >> 4) & 0x3fffu) | (lbo >> 4) << 16; }
__host__ __device__ constexpr uint32_t desc_high(uint32_t sbo) { return (sbo >> 4) | 1u << 14 | 2u << 29; }

template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Key tiles [t0, t1) that rows [r0, r1) of a sequence see (r0 < r1 <= rows).
__device__ __forceinline__ void tile_range(const AttnParams& p, const SeqSpan& s, int r0, int r1, int& t0, int& t1) {
    const int base = s.len - s.T;
    t1 = (base + (r1 - 1) / p.G) / kTcTile + 1;
    t0 = p.window > 0 ? max(0, base + r0 / p.G - p.window + 1) / kTcTile : 0;
}
__device__ __forceinline__ int tc_units(const AttnParams& p, const SeqSpan& s, int rt) {
    int t0, t1;
    tile_range(p, s, rt * kTcRows, min(s.T * p.G, (rt + 1) * kTcRows), t0, t1);
    return t1 - t0;
}
// The sequence's span if this kernel takes it, T = 0 if not.
__device__ __forceinline__ SeqSpan tc_span(const AttnParams& p, int n, unsigned* err) {
    SeqSpan s = kv_span(p.c, n, err);
    if (s.T <= 0 || s.T * p.G <= p.rows_lo || s.T * p.G > p.rows_hi) s.T = 0;
    return s;
}

// A CTA's current segment: `cnt` tiles of an item from tile `tile0` on.  Every role walks the same segments.
struct TcSeg {
    SeqSpan s;
    int n, h, rt, x, units, cnt, rts;
    int tile0;       // first tile of the segment
    int pmin, pmax;  // positions of the item's first and last row
    long long w;

    __device__ __forceinline__ void item(const AttnParams& p, const AttnTcCtl* c) {
        const int rows = s.T * p.G, base = s.len - s.T;
        pmin = base + rt * kTcRows / p.G;
        pmax = base + (min(rows, (rt + 1) * kTcRows) - 1) / p.G;
        const int first = first_tile_of(p, pmin);
        units = pmax / kTcTile + 1 - first;
        tile0 = first + x;
        cnt = (int)min((long long)(units - x), c->w1 - w);
    }
    static __device__ __forceinline__ int first_tile_of(const AttnParams& p, int pos) {
        return p.window > 0 ? max(0, pos - p.window + 1) / kTcTile : 0;
    }
    // First key that any row of the item sees.
    __device__ __forceinline__ int first_key(const AttnParams& p) const { return p.window > 0 ? max(0, pmin - p.window + 1) : 0; }
    __device__ __forceinline__ void start(const AttnParams& p, const AttnTcCtl* c, unsigned* err) {
        n = c->n, h = c->h, rt = c->rt, x = c->x, w = c->w0;
        s = tc_span(p, n, err);
        rts = (s.T * p.G + kTcRows - 1) / kTcRows;
        item(p, c);
    }
    // Moves on; false when the stretch is done.
    __device__ __forceinline__ bool next(const AttnParams& p, const AttnTcCtl* c, unsigned* err) {
        w += cnt;
        if (w >= c->w1) return false;
        x = 0;
        if (++rt == rts) {
            rt = 0;
            if (++h == p.c.hkv) {
                h = 0;
                // the next sequence of this kernel, 32 at a time: hundreds of decoding ones may lie between two chunks
                unsigned some = 0;
                SeqSpan t;
                for (++n; n < p.c.n_seq; n += 32) {
                    const int at = n + (threadIdx.x & 31);
                    t.T = 0;
                    if (at < p.c.n_seq) t = tc_span(p, at, err);
                    some = __ballot_sync(0xffffffffu, t.T > 0);
                    if (some) break;
                }
                if (!some) return false;  // (there is one)
                const int l = __ffs(some) - 1;
                n += l;
                s.start = __shfl_sync(0xffffffffu, t.start, l);
                s.T = __shfl_sync(0xffffffffu, t.T, l);
                s.len = __shfl_sync(0xffffffffu, t.len, l);
                rts = (s.T * p.G + kTcRows - 1) / kTcRows;
            }
        }
        item(p, c);
        return true;
    }
    // Steps [a, b) of this segment that row tile i (0, 1) of the item takes part in, and the positions of its rows.
    __device__ __forceinline__ void active(const AttnParams& p, int i, int& a, int& b, int& lo, int& hi) const {
        const int rows = s.T * p.G, r0 = rt * kTcRows + i * kTcTile, base = s.len - s.T;
        constexpr int SPT = kTcTile / kTcStep;
        a = b = tile0 * SPT;
        lo = pmin, hi = pmax;
        if (r0 >= rows) return;
        lo = base + r0 / p.G;
        hi = base + (min(rows, r0 + kTcTile) - 1) / p.G;
        a = max(p.window > 0 ? max(0, lo - p.window + 1) / kTcStep : 0, tile0 * SPT);
        b = max(a, min(hi / kTcStep + 1, (tile0 + cnt) * SPT));
    }
    // Whether some row with a position in [lo, hi] does not see all keys of [k0, k0 + n).
    static __device__ __forceinline__ bool edge(const AttnParams& p, int k0, int n, int lo, int hi) {
        return k0 + n - 1 > lo || (p.window > 0 && k0 < hi - p.window + 1);
    }
};

// The rare case of a row at position `pos` that has seen marked keys in the segment: what was taken out of V goes to channels
// [c0, c0 + 32) of its sums o, whatever the keys' weights.  A row of the 8-bit cache with the NaN scale is NaN throughout.
// The chunk case of the head of the file with every value NaN takes 944 us.
template <int D, bool E4M3>
__device__ __forceinline__ void add_marked(const AttnParams& p, const TcSeg& g, int pos, int c0, float (&o)[32]) {
    if (E4M3) {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __int_as_float(0x7fc00000);
        return;
    }
    const int32_t* table = p.c.table + (long long)g.n * p.c.max_pages;
    const int first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
#pragma unroll 1
    for (int k0 = g.tile0 * kTcTile; k0 < (g.tile0 + g.cnt) * kTcTile; k0 += kTcTile) {
        if (!TcSeg::edge(p, k0, kTcTile, g.pmin, g.pmax)) continue;
#pragma unroll 1
        for (int key = max(k0, first); key <= min(k0 + kTcTile - 1, pos); ++key) {
            const uint4* v = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.c.v_cache) + attn_pool_row(p.c, table, key, g.h) * D + c0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint4 u = v[e];
                if (!bf16x8_nonfinite(u)) continue;
                add_nonfinite(u.x, o[8 * e], o[8 * e + 1]);
                add_nonfinite(u.y, o[8 * e + 2], o[8 * e + 3]);
                add_nonfinite(u.z, o[8 * e + 4], o[8 * e + 5]);
                add_nonfinite(u.w, o[8 * e + 6], o[8 * e + 7]);
            }
        }
    }
}

// Shares out the units and finds this CTA's first segment; false: nothing to do.  All threads.
template <int THREADS>
__device__ __forceinline__ bool tc_schedule(const AttnParams& p, AttnTcCtl* c, TcScratch* sc, unsigned* err) {
    const int tid = threadIdx.x, N = p.c.n_seq;
    int k = 1;  // threads per sequence
    while (k < 256 && k * 2 * N <= 256) k *= 2;
    const int per = 256 / k;
    auto mine_of = [&](int base) {
        long long mine = 0;
        const int n = base + tid / k;
        if (tid < 256 && n < N) {
            const SeqSpan s = tc_span(p, n, err);
            const int rts = (s.T * p.G + kTcRows - 1) / kTcRows;
            for (int rt = tid % k; rt < rts; rt += k) mine += tc_units(p, s, rt);
        }
        return mine * p.c.hkv;
    };
    long long W = 0, total = 0, before = 0;
    for (int base = 0; base < N; base += per) {  // once, up to 256 sequences
        before = block_scan<THREADS>(mine_of(base), total, sc->scan);
        W += total;
    }
    const int grid = (int)min((long long)gridDim.x, W), cta = blockIdx.x;
    if (cta >= grid) return false;
    const long long w0 = W * cta / grid, w1 = W * (cta + 1) / grid;
    long long seen = 0;
    for (int base = 0; base < N; base += per) {
        if (N > per) before = block_scan<THREADS>(mine_of(base), total, sc->scan);
        if (seen + total <= w0) {
            seen += total;
            continue;
        }
        if (tid < 256) sc->pre[tid] = seen + before;
        if (tid == 0) sc->pre[256] = seen + total;
        __syncthreads();
        if (tid < 256 && tid % k == 0 && sc->pre[tid] <= w0 && w0 < sc->pre[tid + k]) {
            c->n = base + tid / k;
            c->w0 = sc->pre[tid];        // for now: where the sequence starts
            c->w1 = sc->pre[tid + k] - sc->pre[tid];
        }
        break;
    }
    __syncthreads();
    const int n = c->n;
    const long long off = w0 - c->w0, per_head = c->w1 / p.c.hkv;
    const int h = (int)(off / per_head);
    const long long rem = off - h * per_head;
    const SeqSpan s = tc_span(p, n, err);
    const int rts = (s.T * p.G + kTcRows - 1) / kTcRows;
    long long at = 0;
    for (int base = 0; base < rts; base += THREADS) {
        const int rt = base + tid;
        const int u = rt < rts ? tc_units(p, s, rt) : 0;
        const long long before = at + block_scan<THREADS>(u, total, sc->scan);
        if (u > 0 && before <= rem && rem < before + u) {
            c->rt = rt;
            c->x = (int)(rem - before);
        }
        at += total;
        if (at > rem) break;
    }
    __syncthreads();
    if (tid == 0) c->h = h, c->W = W, c->w0 = w0, c->w1 = w1;
    __syncthreads();
    return true;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(AttnTc<D, E4M3>::THREADS, 1)
gdn_attn_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttnParams p,
                      unsigned* err) {
    using namespace sm100;
    using L = AttnTc<D, E4M3>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    AttnTcCtl* c = reinterpret_cast<AttnTcCtl*>(smem + L::OFF_CTL);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    cudaTriggerProgrammaticLaunchCompletion();  // the join kernel may be brought up meanwhile
    if (tid == 0) p.desc[blockIdx.x * kDescInts] = -1;
    if (!tc_schedule<L::THREADS>(p, c, reinterpret_cast<TcScratch*>(smem + L::OFF_Q), err)) {
        cudaGridDependencySynchronize();  // see the end of the kernel
        return;
    }
    if (warp == 1) tmem_alloc(&c->tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c->q_full[i], 128);
            for (int j = 0; j < 2; ++j) {
                mbar_init(&c->s_full[i][j], 1);
                mbar_init(&c->p_full[i][j], 128);
                mbar_init(&c->o_full[i][j], 1);
            }
            mbar_init(&c->drain[i], 1);
            if (i == 0) mbar_init(&c->stall, 1);
            mbar_init(&c->r_full[i], 1);
            mbar_init(&c->r_empty[i], 128);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&c->k_full[i], E4M3 ? 128 : 1);
            mbar_init(&c->k_empty[i], 2);
            mbar_init(&c->v_full[i], 1);
            mbar_init(&c->v_ready[i], E4M3 ? 128 : 32);
            mbar_init(&c->v_empty[i], 2);
            for (int j = 0; j < 4; ++j) c->bad[i][j] = 0;
        }
        c->abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem;
    volatile int* ab = &c->abort_flag;

    if (warp < 4) {
        reg_dec<E4M3 ? 88 : 128>();
        if (warp == 0) {
            // ---- loader.  Fill f of a ring of S stages: stage f % S, waits for the (f / S)-th release.
            const int npg = kTcTile >> p.c.page_log2, page = 1 << p.c.page_log2;
            const int boxes = npg * (E4M3 ? 1 : D / 64);
            const int i = lane % npg, hf = lane / npg;  // this lane's page of the tile and channel half
            int fk = 0, fv = 0, fr = 0;
            bool ok = true;
            TcSeg g;
            g.start(p, c, err);
            do {
                const int t0 = g.tile0;
                const int32_t* row = p.c.table + (long long)g.n * p.c.max_pages;
                // pages [first, pages) hold keys that the item sees; before them (the window has passed) and behind the
                // sequence's end the table may hold anything
                const int pages = (g.s.len + page - 1) >> p.c.page_log2, first = g.first_key(p) >> p.c.page_log2;
                auto look = [&](int tile) {  // this lane's page of a tile: -1 where there is none to load
                    const int at = tile * npg + i;
                    if (lane >= boxes || at < first || at >= pages) return -1;
                    const int pg = row[at];
                    if (pg >= 0 && pg < p.c.n_pages) return pg;
                    atomicOr(err, kErrPages);
                    return 0;
                };
                int pg = look(t0);
                for (int j = 0; ok && j < g.cnt; ++j) {
                    const int pg_next = j + 1 < g.cnt ? look(t0 + j + 1) : -1;
                    const int r0 = (pg * p.c.hkv + g.h) << p.c.page_log2;  // < 2^31 (checked on the host)
                    const uint32_t n = __popc(__ballot_sync(0xffffffffu, pg >= 0));
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (E4M3) {
                            const int st = fr % 2;
                            ok = ok && tc_warp_wait(&c->r_empty[st], ((fr / 2) & 1) ^ 1, ab, err);
                            if (!ok) break;
                            if (lane == 0) mbar_expect_tx(&c->r_full[st], n * page * (D + 1));
                            __syncwarp();
                            if (pg >= 0) {
                                const uint8_t* src = static_cast<const uint8_t*>(kv ? p.c.v_cache : p.c.k_cache);
                                const uint8_t* sc = kv ? p.c.v_scale : p.c.k_scale;
                                bulk_load(smem + L::OFF_RAW + st * L::RAW + i * page * D, src + (long long)r0 * D, page * D, &c->r_full[st]);
                                bulk_load(smem + L::OFF_SC + st * kTcTile + i * page, sc + r0, page, &c->r_full[st]);
                            }
                            ++fr;
                        } else {
                            int& f = kv ? fv : fk;
                            const int S = kv ? L::NV : L::NK, st = f % S;
                            uint64_t* full = kv ? &c->v_full[st] : &c->k_full[st];
                            ok = ok && tc_warp_wait(kv ? &c->v_empty[st] : &c->k_empty[st], ((f / S) & 1) ^ 1, ab, err);
                            if (!ok) break;
                            if (lane == 0) mbar_expect_tx(full, n * page * 128);
                            __syncwarp();
                            if (pg >= 0)
                                tma_load_2d(smem + (kv ? L::OFF_V : L::OFF_K) + st * L::TILE + hf * L::HALF + i * page * 128,
                                            kv ? &tm_v : &tm_k, full, hf * 64, r0);
                            ++f;
                        }
                    }
                    pg = pg_next;
                }
            } while (ok && g.next(p, c, err));
            if (!ok) {  // given up: let the copies in flight land before the CTA goes (each wait has its own limit)
                int zero = 0;
                if (E4M3) {
                    for (int f = max(0, fr - 2); f < fr; ++f) tc_wait(&c->r_full[f % 2], (f / 2) & 1, &zero, err);
                } else {
                    for (int f = max(0, fk - L::NK); f < fk; ++f) tc_wait(&c->k_full[f % L::NK], (f / L::NK) & 1, &zero, err);
                    for (int f = max(0, fv - L::NV); f < fv; ++f) tc_wait(&c->v_full[f % L::NV], (f / L::NV) & 1, &zero, err);
                }
            }
        } else if (warp < 3) {
            // ---- MMA issuers, one warp per row tile: while one waits for its P, the other's MMAs keep the tensor core busy
            constexpr uint32_t id_s = idesc_bf16(128, kTcStep, false, false), id_o = idesc_bf16(128, D, false, true);
            constexpr uint32_t hi = desc_high(1024);
            const int i = warp - 1;
            const uint32_t sq = uniform(desc_low(smem_u32(smem + L::OFF_Q + i * L::TILE), 16)),
                           ts = uniform(tmem + i * 128), to = uniform(tmem + 256 + i * 128);
            const uint32_t sk = desc_low(smem_u32(smem + L::OFF_K), 16), sv = desc_low(smem_u32(smem + L::OFF_V), L::HALF);
            int ck = 0, cv = 0, seg = 0;  // K and V tiles taken, segments
            uint32_t pp = 0;              // parity of the next P, a bit per buffer
            bool ok = true;
            // S = Q K^T of 64 keys into buffer h, O += P V of buffer h (by one lane)
            auto scores = [&](int h, uint32_t k0) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = ((ks >> 2) * L::HALF + (ks & 3) * 32) / 16;
                    mma_ss<hi, hi, id_s>(ts + h * kTcStep, sq + off, k0 + h * (kTcStep * 128 / 16) + off, ks > 0);
                }
                umma_commit(&c->s_full[i][h]);
            };
            auto values = [&](int h, uint32_t v0, uint32_t more) {
#pragma unroll
                for (int ks = 0; ks < kTcStep / 16; ++ks)
                    mma_ts<hi, id_o>(to, ts + h * kTcStep + ks * 8, v0 + (h * 4 + ks) * (2048 / 16), ks > 0 ? 1u : more);
                umma_commit(&c->o_full[i][h]);
            };
            TcSeg g;
            g.start(p, c, err);
            // Diagnostic: a wait that runs out.  It sets the error word and the abort flag, and this warp issues no MMA; every
            // other role then leaves through its own bounded waits, behind which it drains what it issued.
            if (p.debug_stall && i == 0) ok = __all_sync(0xffffffffu, tc_wait(&c->stall, 0, ab, err, kTcStallCycles));
            do {
                const int u0 = g.tile0 * 2, tiles = g.cnt;
                int a, b, plo, phi;
                g.active(p, i, a, b, plo, phi);
                ok = ok && tc_warp_wait(&c->q_full[i], seg & 1, ab, err) && tc_warp_wait(&c->k_full[ck % L::NK], (ck / L::NK) & 1, ab, err);
                if (!ok) break;
                tc_fence_after();
                {
                    const uint32_t k0 = uniform(sk + (ck % L::NK) * (L::TILE / 16));
                    if (elect_one()) {
                        // a row tile without steps here is told so too: no role gets a phase ahead of another
                        if (b == a) umma_commit(&c->o_full[i][0]);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (u0 + h >= a && u0 + h < b) scores(h, k0);
                        umma_commit(&c->k_empty[ck % L::NK]);
                    }
                    __syncwarp();
                    ++ck;
                }
                for (int t = 0; ok && t < tiles; ++t) {
                    // Of each step u: O += P V of u, then S of u + 2 into the same columns (in issue order).
                    const int stv = cv % L::NV, stk = ck % L::NK;
                    const bool more = t + 1 < tiles;
                    ok = tc_warp_wait(&c->v_ready[stv], (cv / L::NV) & 1, ab, err);
                    if (ok && more) ok = tc_warp_wait(&c->k_full[stk], (ck / L::NK) & 1, ab, err);
                    const uint32_t v0 = uniform(sv + stv * (L::TILE / 16)), k0 = uniform(sk + stk * (L::TILE / 16));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int u = u0 + 2 * t + h;
                        const bool pv = u >= a && u < b, qk = more && u + 2 >= a && u + 2 < b;
                        if (ok && pv) {
                            ok = tc_warp_wait(&c->p_full[i][h], (pp >> h) & 1, ab, err);
                            pp ^= 1u << h;
                        }
                        if (!ok) continue;
                        tc_fence_after();
                        if (elect_one()) {
                            if (pv) values(h, v0, u > a);
                            if (qk) scores(h, k0);
                            if (h == 1) {
                                umma_commit(&c->v_empty[stv]);
                                if (more) umma_commit(&c->k_empty[stk]);
                            }
                        }
                        __syncwarp();
                    }
                    ++cv;
                    if (more) ++ck;
                }
                ++seg;
            } while (ok && g.next(p, c, err));
            // every MMA has read its operands before the CTA goes
            if (elect_one()) umma_commit(&c->drain[i]);
            __syncwarp();
            int zero = 0;
            tc_warp_wait(&c->drain[i], 0, &zero, err);
        } else if (!E4M3) {
            // ---- NaNs and infinities of V, in tiles that are not wholly visible
            int cv = 0;
            bool ok = true;
            TcSeg g;
            g.start(p, c, err);
            do {
                const int f0 = g.tile0;
                for (int j = 0; ok && j < g.cnt; ++j, ++cv) {
                    const int st = cv % L::NV;
                    ok = tc_warp_wait(&c->v_full[st], (cv / L::NV) & 1, ab, err);
                    if (!ok) break;
                    if (TcSeg::edge(p, (f0 + j) * kTcTile, kTcTile, g.pmin, g.pmax)) {
                        uint8_t* v = smem + L::OFF_V + st * L::TILE;
                        // a thread looks at four rows whole
#pragma unroll 1
                        for (int rr = 0; rr < 4; ++rr) {
                            const int r = lane + 32 * rr;
                            bool bad = false;
                            for (int ch = 0; ch < D / 8; ++ch) {
                                uint4* at = reinterpret_cast<uint4*>(v + (ch >> 3) * L::HALF + sw128(r, ch & 7));
                                const uint4 u = *at;
                                if (bf16x8_nonfinite(u)) {
                                    *at = bf16x8_finite(u);
                                    bad = true;
                                }
                            }
                            const uint32_t m = __ballot_sync(0xffffffffu, bad);
                            if (lane == 0) c->bad[st][rr] = m;
                        }
                        fence_proxy_async();
                    }
                    mbar_arrive(&c->v_ready[st]);
                }
            } while (ok && g.next(p, c, err));
        }
    } else if (warp < 12) {
        // ---- softmax
        reg_inc<E4M3 ? 168 : 184>();
        const int i = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;  // row tile, row in it
        const uint32_t ts = tmem + i * 128 + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t to = tmem + 256 + i * 128 + ((uint32_t)((warp & 3) * 32) << 16);
        // a negative scale goes into Q's sign and a zero one into Q itself, so that larger S means larger score
        const float cs = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u, keep = p.scale_log2 == 0.f ? 0u : 0xffffffffu;
        uint32_t sp = 0, op = 0;  // parities of the next S and of the next finished P V, a bit per buffer
        int cv0 = 0;              // V tiles before this segment
        bool ok = true;
        TcSeg g;
        g.start(p, c, err);
        do {
            const int rows = g.s.T * p.G, row = g.rt * kTcRows + i * kTcTile + r;
            const bool there = row < rows;
            const int tok = there ? row / p.G : 0, gh = row - tok * p.G;
            const int pos = g.s.len - g.s.T + tok;
            {
                const uint4* q = reinterpret_cast<const uint4*>(p.q + (long long)(g.s.start + tok) * p.q_stride + (long long)(g.h * p.G + (there ? gh : 0)) * D);
                uint8_t* dst = smem + L::OFF_Q + i * L::TILE;
#pragma unroll
                for (int ch = 0; ch < D / 8; ++ch) {
                    uint4 u = there ? q[ch] : make_uint4(0, 0, 0, 0);
                    u.x = (u.x ^ flip) & keep, u.y = (u.y ^ flip) & keep, u.z = (u.z ^ flip) & keep, u.w = (u.w ^ flip) & keep;
                    *reinterpret_cast<uint4*>(dst + (ch >> 3) * L::HALF + sw128(r, ch & 7)) = u;
                }
                fence_proxy_async();
                mbar_arrive(&c->q_full[i]);
            }
            int a, b, plo, phi;  // this row tile's steps and positions
            g.active(p, i, a, b, plo, phi);
            c->saw[i * kTcTile + r] = 0;
            float m = -INFINITY, l = 0.f;
            for (int u = a; ok && u < b; ++u) {
                const uint32_t tb = ts + (u & 1) * kTcStep;
                ok = tc_warp_wait(&c->s_full[i][u & 1], (sp >> (u & 1)) & 1, ab, err);
                if (!ok) break;
                sp ^= 1u << (u & 1);
                tc_fence_after();
                float s[2][32];
                tmem_ld32(tb, s[0]);
                tmem_ld32(tb + 32, s[1]);
                tmem_wait_ld();
                const int k0 = u * kTcStep, chi = pos - k0, clo = p.window > 0 ? chi - p.window + 1 : 0;
                if (TcSeg::edge(p, k0, kTcStep, plo, phi)) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (q * 32 + e > chi || q * 32 + e < clo) s[q][e] = -INFINITY;
                }
                float top;
                {
                    float m4[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float* x = &s[q >> 1][(q & 1) * 16];
                        m4[q] = max3(x[0], x[1], x[2]);
#pragma unroll
                        for (int e = 3; e < 15; e += 2) m4[q] = max3(m4[q], x[e], x[e + 1]);
                        m4[q] = fmaxf(m4[q], x[15]);
                    }
                    top = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
                }
                // each row by itself: its result does not depend on the rows beside it
                const bool grow = (top - m) * cs > kRescaleLog2;
                if (__any_sync(0xffffffffu, grow)) {
                    float f = 1.f;
                    if (grow) {
                        f = m == -INFINITY ? 0.f : exp2f((m - top) * cs);
                        m = top;
                        l *= f;
                    }
                    if (u > a) {
                        // the step before's P V (that of the step before it is done, or S would not be here)
                        ok = tc_warp_wait(&c->o_full[i][(u - 1) & 1], ((op >> ((u - 1) & 1)) & 1) ^ 1, ab, err);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            uint32_t o[16];
                            tmem_ld16(to + q * 16, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16u(to + q * 16, o);
                        }
                    }
                }
                if (TcSeg::edge(p, (u >> 1) * kTcTile, kTcTile, g.pmin, g.pmax)) {
                    // marked keys (see the head of the file)
                    const int cv = cv0 + (u >> 1) - g.tile0, st = cv % L::NV;
                    ok = tc_warp_wait(&c->v_ready[st], (cv / L::NV) & 1, ab, err);
                    if (!ok) break;
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        const int lo = clo - 32 * q, hi = chi - 32 * q;  // bits [lo, hi] of this word
                        if (hi < 0 || lo > 31) continue;
                        const uint32_t seen = (0xffffffffu >> (31 - min(hi, 31))) & (0xffffffffu << max(lo, 0));
                        if (c->bad[st][(u & 1) * 2 + q] & seen) c->saw[i * kTcTile + r] = 1;
                    }
                    __syncwarp();
                }
                const float mc = m == -INFINITY ? 0.f : fmaf(m, cs, kRescaleLog2);
                const float2 c2 = make_float2(cs, cs), mc2 = make_float2(-mc, -mc);
                float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 x = fma2(make_float2(s[q][2 * e], s[q][2 * e + 1]), c2, mc2);
                        x.x = ex2_approx(x.x), x.y = ex2_approx(x.y);
                        l2[e & 1] = add2(l2[e & 1], x);
                        w[e] = pack_bf16x2(x.x, x.y);
                    }
                    tmem_st16u(tb + q * 16, w);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&c->p_full[i][u & 1]);
                op ^= 1u << (u & 1);
                l2[0] = add2(l2[0], l2[1]);
                l += l2[0].x + l2[0].y;
            }
            cv0 += g.cnt;
            if (!ok) break;
            // ---- the segment's result
            if (b == a) op ^= 1u;  // the issuer's word that there was nothing to do
            const int ob = b > a ? (b - 1) & 1 : 0;
            ok = tc_warp_wait(&c->o_full[i][ob], ((op >> ob) & 1) ^ 1, ab, err);
            if (!ok) break;
            tc_fence_after();
            const bool whole = g.cnt == g.units;
            const long long at = (long long)(g.s.start + tok) * p.hq + g.h * p.G + gh;
            const float m2 = m == -INFINITY ? -INFINITY : fmaf(m, cs, kRescaleLog2);
            // A part of an item goes to the workspace, for the join kernel.
            const long long slot = blockIdx.x * 2LL + (g.w == c->w0 ? 0 : 1);
            if (whole) {
                if (there && p.lse) p.lse[at] = attn_lse(m2, l);
            } else {
                if (there) reinterpret_cast<float2*>(p.ml)[slot * kTcRows + i * kTcTile + r] = make_float2(m2, l);
                if (i == 0 && r == 0 && g.x == 0) {  // the item starts here and ends in a later CTA
                    const long long grid = min((long long)gridDim.x, c->W), end = g.w + g.units;
                    int4* desc = reinterpret_cast<int4*>(p.desc) + blockIdx.x * 2;
                    desc[0] = make_int4(g.n, g.h, g.rt * kTcRows, min(kTcRows, rows - g.rt * kTcRows));
                    desc[1] = make_int4((int)(slot & 1), (int)((end * grid + c->W - 1) / c->W) - (int)blockIdx.x, g.s.start, 0);
                }
            }
            if (whole || b > a) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const bool saw = c->saw[i * kTcTile + r] != 0;
                float4* dst = reinterpret_cast<float4*>(p.part) + (slot * 2 + i) * (D / 4) * kTcTile + r;
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    float o[32];
                    tmem_ld32(to + q * 32, o);
                    tmem_wait_ld();
                    if (saw) add_marked<D, E4M3>(p, g, pos, q * 32, o);
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) dst[(q * 8 + e) * kTcTile] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else if (there) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            attn_store4(p.o, p.o_f32, at * D + q * 32 + e, make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]), inv);
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();  // O is free once the next Q (arrived after this) lets the issuer go on
        } while (ok && g.next(p, c, err));
        tmem_wait_st();  // (a role that gave up may have left some of O's behind)
    } else {
        // ---- 8-bit cache: codes to bf16.  Eight (D = 64: four) threads share a row, 16 codes each.
        reg_dec<88>();
        const int t128 = tid - 384;
        constexpr int TPR = D / 16, RPP = 128 / TPR;  // threads of a row, rows per pass
        const int col = t128 % TPR, r_in = t128 / TPR;
        int fr = 0, fk = 0, fv = 0;
        bool ok = true;
        TcSeg g;
        g.start(p, c, err);
        do {
            const int f0 = g.tile0;
            for (int j = 0; ok && j < g.cnt; ++j) {
                const bool edge = TcSeg::edge(p, (f0 + j) * kTcTile, kTcTile, g.pmin, g.pmax);
                // rows [unseen, valid) of the tile are keys that the item sees; the others' pages may not have been loaded
                const int valid = g.s.len - (f0 + j) * kTcTile, unseen = g.first_key(p) - (f0 + j) * kTcTile;
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    const int rs = fr % 2;
                    int& f = kv ? fv : fk;
                    const int S = kv ? L::NV : L::NK, st = f % S;
                    ok = tc_warp_wait(&c->r_full[rs], (fr / 2) & 1, ab, err) &&
                         tc_warp_wait(kv ? &c->v_empty[st] : &c->k_empty[st], ((f / S) & 1) ^ 1, ab, err);
                    if (!ok) break;
                    const uint8_t* raw = smem + L::OFF_RAW + rs * L::RAW;
                    const uint8_t* sc = smem + L::OFF_SC + rs * kTcTile;
                    uint8_t* dst = smem + (kv ? L::OFF_V : L::OFF_K) + st * L::TILE;
#pragma unroll 4
                    for (int pass = 0; pass < TPR; ++pass) {
                        const int r = pass * RPP + r_in;
                        const uint4 u = *reinterpret_cast<const uint4*>(raw + r * D + col * 16);
                        unsigned byte = sc[r];
                        // a value row that may be masked must be finite: one with the NaN scale is zeroed and marked
                        bool bad = false;
                        if (kv && edge) {
                            bad = byte == kScaleNan && r < valid && r >= unseen;
                            if (byte == kScaleNan || r >= valid || r < unseen) byte = 0;
                            const uint32_t hit = __ballot_sync(0xffffffffu, bad);
                            // the warp covers 32 / TPR neighbouring rows
                            uint32_t mark = 0;
#pragma unroll
                            for (int q = 0; q < 32 / TPR; ++q) mark |= ((hit >> (q * TPR)) & 1u) << q;
                            constexpr int RW = 32 / TPR;
                            uint8_t* bytes = reinterpret_cast<uint8_t*>(c->bad[st]);
                            // RW = 4 or 8 rows: a nibble or a byte of the mask
                            const int r0 = pass * RPP + (t128 >> 5) * RW;
                            if (RW == 8) {
                                if (lane == 0) bytes[r0 >> 3] = (uint8_t)mark;
                            } else if (lane == 0) {
                                // clear and set this nibble (its neighbour belongs to another warp)
                                atomicAnd(&c->bad[st][r0 >> 5], ~(0xfu << (r0 & 31)));
                                atomicOr(&c->bad[st][r0 >> 5], mark << (r0 & 31));
                            }
                        }
                        // 2^(byte - 127) as bf16: the byte is its exponent field (0 clears the row, 255 is NaN)
                        const uint32_t s1 = byte == kScaleNan ? 0x7fc0u : byte << 7, s2 = s1 | (s1 << 16);
                        const uint32_t cw[4] = {u.x, u.y, u.z, u.w};
                        uint32_t o[8];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            o[2 * q] = mul_bf16x2(e4m3_pair(cw[q], 0), s2);
                            o[2 * q + 1] = mul_bf16x2(e4m3_pair(cw[q], 1), s2);
                        }
                        uint8_t* line = dst + (col >> 2) * L::HALF;
                        *reinterpret_cast<uint4*>(line + sw128(r, (2 * col) & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(line + sw128(r, (2 * col + 1) & 7)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    fence_proxy_async();
                    mbar_arrive(&c->r_empty[rs]);
                    mbar_arrive(kv ? &c->v_ready[st] : &c->k_full[st]);
                    ++fr;
                    ++f;
                }
            }
        } while (ok && g.next(p, c, err));
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
    // with a decode kernel before this one on the stream: its results are complete when this kernel is
    cudaGridDependencySynchronize();
}

// 2-D map over the cache's rows [n_pages * hkv * page][d], box 64 channels x one page, 128-byte swizzle.
typedef CUresult (*AttnEncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                    const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline bool make_cache_map(CUtensorMap* map, const void* base, int d, long long rows, int page) {
    static const AttnEncodeTiled enc = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<AttnEncodeTiled>(ptr);
    }();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)d * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)page};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdn
