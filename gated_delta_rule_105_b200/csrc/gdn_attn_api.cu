// libgdn C ABI, the attention layer beside the token mixer: the paged key/value cache, attention over it, and the
// residual stream's RMS norm.  Host-side argument checks and launches.
#include <algorithm>
#include <cmath>

#include "gdn.h"
#include "gdn_attn.cuh"
#include "gdn_attn_tc.cuh"
#include "gdn_host.h"
#include "gdn_norm.cuh"
#include "gdn_prof.cuh"

namespace gdn {

// Launches `kern`; with `early` it may start while the launch before it on the stream still runs (programmatic stream
// serialisation): the kernel waits for that launch's memory with cudaGridDependencySynchronize().
template <typename... P, typename... A>
static cudaError_t launch_after(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool early,
                                const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

static gdn_status check_ptrs(std::initializer_list<const void*> required, std::initializer_list<const void*> optional) {
    for (const void* ptr : required) {
        if (!ptr) return fail(GDN_ERR_INVALID_ARG, "a required pointer is NULL");
        if (!aligned16(ptr)) return fail(GDN_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", ptr);
    }
    for (const void* ptr : optional)
        if (ptr && !aligned16(ptr)) return fail(GDN_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", ptr);
    return GDN_OK;
}

// The checks that every call on the paged cache shares; fills the layout.
static gdn_status check_cache(KvParams* c, const void* k_cache, const void* v_cache, const uint8_t* k_scale,
                              const uint8_t* v_scale, const int32_t* table, int n_tok, int n_seqs, int n_pages,
                              int max_pages, int page_size, int Hkv, int d, gdn_dtype cache_dt) {
    if (n_tok < 0) return fail(GDN_ERR_INVALID_ARG, "the number of tokens must be >= 0 (got %d)", n_tok);
    if (n_seqs < 1 || n_seqs > 65535) return fail(GDN_ERR_INVALID_ARG, "n_seqs must be in [1, 65535] (got %d)", n_seqs);
    if (n_pages < 1 || max_pages < 1)
        return fail(GDN_ERR_INVALID_ARG, "need n_pages >= 1 and max_pages >= 1 (got %d, %d)", n_pages, max_pages);
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return fail(GDN_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128 (got %d)", page_size);
    if (Hkv < 1 || Hkv > 1024) return fail(GDN_ERR_INVALID_ARG, "Hkv must be in [1, 1024] (got %d)", Hkv);
    if (d != 64 && d != 128) return fail(GDN_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", d);
    if (cache_dt != GDN_BF16 && cache_dt != GDN_E4M3)
        return fail(GDN_ERR_UNSUPPORTED, "the cache is GDN_BF16 or GDN_E4M3 (got %d)", (int)cache_dt);
    if ((long long)n_pages * Hkv * page_size > 0x7fffffffLL)
        return fail(GDN_ERR_UNSUPPORTED, "n_pages * Hkv * page_size must be below 2^31");
    // (the decode kernel looks up to four units of 384 keys past a sequence's end before it clamps the position)
    if ((long long)max_pages * page_size > 0x7fffffffLL - 4095)
        return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_size must be at most 2^31 - 4096");
    gdn_status st = check_ptrs({k_cache, v_cache, table}, {k_scale, v_scale});
    if (st != GDN_OK) return st;
    if (cache_dt == GDN_E4M3 && (!k_scale || !v_scale))
        return fail(GDN_ERR_INVALID_ARG, "an 8-bit cache needs k_scale and v_scale");
    if (cache_dt == GDN_BF16 && (k_scale || v_scale))
        return fail(GDN_ERR_INVALID_ARG, "k_scale and v_scale go with an 8-bit cache only");
    c->k_cache = const_cast<void*>(k_cache);
    c->v_cache = const_cast<void*>(v_cache);
    c->k_scale = const_cast<uint8_t*>(k_scale);
    c->v_scale = const_cast<uint8_t*>(v_scale);
    c->table = table;
    c->seq_lens = nullptr;
    c->cu = nullptr;
    c->n_tok = n_tok;
    c->n_seq = n_seqs;
    c->n_pages = n_pages;
    c->max_pages = max_pages;
    c->hkv = Hkv;
    c->d = d;
    c->page_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    return GDN_OK;
}

static gdn_status check_stride(const char* what, long long stride, long long width, int esize) {
    if (stride < width || stride * esize % 16 != 0)
        return fail(GDN_ERR_INVALID_ARG, "%s must be at least %lld elements and a multiple of 16 bytes (got %lld)", what,
                    width, stride);
    return GDN_OK;
}

// Tokens per warp of the cache's writing and reading-back kernels.  A warp has room for `batch` 16-byte-a-lane rows at a
// time; heads that do not fill it leave lanes idle and look-ups (a chain of dependent loads) unshared, so that several
// tokens share a warp then -- half as many where the cache's rows are bf16, twice as wide -- unless the call is too small to
// occupy the GPU with fewer warps.  Measured, one | 2 | 4 tokens a warp, us, d = 128:
//   75776 tokens, 2 heads, e4m3:  append 66.2 | 38.9 | 26.5,  read 33.9 | 23.6 | 21.6
//   75776 tokens, 4 heads, e4m3:  append 69.8 | 45.8 | 46.9,  read 45.5 | 39.0 | 40.1
//   75776 tokens, 8 heads, e4m3:  append 77.5 | 83.4 | 86.4,  read 73.7 | 75.3
//   75776 tokens, 4 heads, bf16:  append 48.4 | 49.4,         read 51.4 | 54.6
//    4096 tokens, 4 heads, e4m3:  append  6.3 |  5.0 |  5.9,  read  3.7 |  3.7 |  3.9
//    2048 tokens, 4 heads, e4m3:  append  4.4 |  4.3 |  5.9,  read  2.8 |  3.0 |  3.8
static int kv_tokens(const KvParams& c, int batch, bool e4m3) {
    if (c.n_tok < 16 * kAttnSms) return 1;
    if (!e4m3) batch /= 2;
    return c.hkv >= batch ? 1 : 2 * c.hkv >= batch ? 2 : 4;
}
template <typename TIn, int D, int TPW>
static void launch_append_rows(const KvAppendParams& p, bool e4m3, unsigned* err, cudaStream_t stream) {
    const unsigned grid = (p.c.n_tok + kKvWarps * TPW - 1LL) / (kKvWarps * TPW);
    if (e4m3) gdn_kv_append_kernel<TIn, D, true, TPW><<<grid, kKvWarps * 32, 0, stream>>>(p, err);
    else gdn_kv_append_kernel<TIn, D, false, TPW><<<grid, kKvWarps * 32, 0, stream>>>(p, err);
}
template <typename TIn, int D>
static void launch_append(const KvAppendParams& p, bool e4m3, unsigned* err, cudaStream_t stream) {
    const int t = kv_tokens(p.c, kKvBatch * 32 * Vec16<TIn>::N / D, e4m3);
    if (t == 1) launch_append_rows<TIn, D, 1>(p, e4m3, err, stream);
    else if (t == 2) launch_append_rows<TIn, D, 2>(p, e4m3, err, stream);
    else launch_append_rows<TIn, D, 4>(p, e4m3, err, stream);
}
template <typename TOut, int D, int TPW>
static void launch_read_rows(const KvReadParams& p, bool e4m3, unsigned* err, cudaStream_t stream) {
    const unsigned grid = (p.c.n_tok + kKvWarps * TPW - 1LL) / (kKvWarps * TPW);
    if (e4m3) gdn_kv_read_kernel<TOut, D, true, TPW><<<grid, kKvWarps * 32, 0, stream>>>(p, err);
    else gdn_kv_read_kernel<TOut, D, false, TPW><<<grid, kKvWarps * 32, 0, stream>>>(p, err);
}
template <typename TOut, int D>
static void launch_read(const KvReadParams& p, bool e4m3, unsigned* err, cudaStream_t stream) {
    const int t = kv_tokens(p.c, kKvBatch * 32 * 8 / D, e4m3);
    if (t == 1) launch_read_rows<TOut, D, 1>(p, e4m3, err, stream);
    else if (t == 2) launch_read_rows<TOut, D, 2>(p, e4m3, err, stream);
    else launch_read_rows<TOut, D, 4>(p, e4m3, err, stream);
}

// ---- attention
// Which kernels a call launches, and its workspace: a function of the sizes that the host knows.  Sequences of up to
// dec_max_rows() query rows per KV head belong to the decode kernel, longer ones to the chunk kernel.  Where every
// sequence has as many tokens (no cu_seqlens) or there is but one, one kernel takes the call; with no more tokens than
// sequences it is taken for decoding of one token each; else both run.  The decode kernel works on 8 rows at a time where
// that is enough (half the softmax and the accumulators), else on 16, reading an item's keys again for every 16.  Packed
// calls choose those rows as for one token a sequence, since only the device knows the lengths: what has more rows than
// that (several tokens a sequence; a chunk among slots that are mostly idle, n_tok <= n_seqs) reads its keys once per 8 or 16
// rows.  Such calls are right, and not measured here.
//
// The limit, measured with one token a sequence and 8 | 16 | 32 | 48 heads per KV head, us:
//   32 sequences of 8192, 4 KV heads, d = 128, bf16: decode  88 |  94 | 177 | 247, chunk 105 | 106 | 107 | 108
//   the same, e4m3:                                  decode  64 |  67 | 119 | 169, chunk 140 | 141 | 142 | 142
//   the same, d = 64, bf16:                          decode  52 |  53 |  91 | 128, chunk  91 |  92 |  92 |  92
//   2 sequences of 4096, 2 KV heads, d = 128, bf16:  decode  10 |  13 |  14 |  17, chunk  33 |  34 |  35 |  35
static int dec_max_rows(int d, bool e4m3) { return d * (e4m3 ? 1 : 2) <= 128 ? 32 : 16; }
struct AttnArrays {
    int grid;  // 0: this kernel is not launched
    size_t desc, ml, part;
};
struct AttnPlan {
    AttnArrays dec, tc;
    int limit;     // the decode kernel's largest row count
    int dec_rows;  // its rows at a time: 8 or 16
    size_t bytes;
};
static AttnPlan attn_plan(int n_tok, int n_seqs, bool packed, int G, int d, bool e4m3) {
    AttnPlan a = {};
    const int most = dec_max_rows(d, e4m3);
    a.limit = 0x7fffffff;
    if (n_tok <= n_seqs && G <= most) {
        a.dec.grid = 1;
    } else if (n_seqs == 1 || !packed) {
        if ((long long)(n_tok / n_seqs) * G <= most) a.dec.grid = 1;
        else a.tc.grid = 1, a.limit = 0;
    } else {
        a.dec.grid = a.tc.grid = 1;
        a.limit = most;
    }
    auto place = [&](AttnArrays& r, int grid, int rows) {
        if (!r.grid) return;
        r.grid = grid;
        r.desc = a.bytes;
        r.ml = r.desc + (size_t)grid * kDescInts * sizeof(int);
        r.part = r.ml + (size_t)grid * 2 * rows * 2 * sizeof(float);
        a.bytes = r.part + (size_t)grid * 2 * rows * d * sizeof(float);
    };
    a.dec_rows = (long long)G * (packed ? 1 : std::max(1, n_tok / n_seqs)) <= 8 ? 8 : 16;
    const bool two = a.dec_rows == 8 && (e4m3 || d == 64);  // CTAs per SM, as DecTraits has it
    place(a.dec, kAttnSms * (two ? 2 : 1), a.dec_rows);
    place(a.tc, kAttnSms, kTcRows);
    return a;
}

static void use_arrays(AttnParams& p, const AttnArrays& r, uint8_t* ws) {
    p.desc = reinterpret_cast<int*>(ws + r.desc);
    p.ml = reinterpret_cast<float*>(ws + r.ml);
    p.part = reinterpret_cast<float*>(ws + r.part);
}

template <int D, bool E4M3, int R>
static cudaError_t launch_decode(const AttnParams& p, int grid, unsigned* err, cudaStream_t stream) {
    using Tr = DecTraits<D, E4M3, R>;
    const cudaError_t e = allow_shared<&gdn_attn_decode_kernel<D, E4M3, R>>((int)Tr::smem);
    if (e != cudaSuccess) return e;
    gdn_attn_decode_kernel<D, E4M3, R><<<grid, Tr::THREADS, Tr::smem, stream>>>(p, err);
    return cudaGetLastError();
}

template <int D, bool E4M3>
static gdn_status launch_attn(AttnParams p, const AttnPlan& plan, uint8_t* ws, JoinParams& j, unsigned* err, cudaStream_t stream) {
    cudaError_t e;
    if (plan.dec.grid) {
        use_arrays(p, plan.dec, ws);
        p.rows_lo = 0;
        p.rows_hi = plan.limit;
        e = plan.dec_rows == 8 ? launch_decode<D, E4M3, 8>(p, plan.dec.grid, err, stream)
                               : launch_decode<D, E4M3, 16>(p, plan.dec.grid, err, stream);
        if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "attention decode kernel launch: %s", cudaGetErrorString(e));
        j.dec = {p.desc, p.part, p.ml};
    }
    if (plan.tc.grid) {
        use_arrays(p, plan.tc, ws);
        p.rows_lo = plan.dec.grid ? plan.limit : 0;
        p.rows_hi = 0x7fffffff;
        CUtensorMap mk = {}, mv = {};
        if (!E4M3) {
            const long long rows = ((long long)p.c.n_pages * p.c.hkv) << p.c.page_log2;
            if (!make_cache_map(&mk, p.c.k_cache, D, rows, 1 << p.c.page_log2) || !make_cache_map(&mv, p.c.v_cache, D, rows, 1 << p.c.page_log2))
                return fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled failed");
        }
        auto kern = gdn_attn_chunk_kernel<D, E4M3>;
        using L = AttnTc<D, E4M3>;
        e = allow_shared<&gdn_attn_chunk_kernel<D, E4M3>>(L::BYTES);
        if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        // beside a decode kernel it takes the SMs that that one leaves (and ends after it, for the join)
        e = launch_after(kern, dim3(plan.tc.grid), dim3(L::THREADS), L::BYTES, stream, plan.dec.grid > 0, mk, mv, p, err);
        if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "attention chunk kernel launch: %s", cudaGetErrorString(e));
        j.tc = {p.desc, p.part, p.ml};
    }
    j.rows = plan.dec_rows;
    // Blocks per decode item: one per row where items are so few that each has more parts than a block has warps, else two.
    // One sequence of 4096, 16 rows: 17.8 us with a block per row, 18.0 with two, 25.4 with one; 64 sequences of up to
    // 16384: 145.0, 143.0 and 143.1; 23 sequences beside a chunk: 57.9, 55.3 and 54.7.
    j.dec_split = (long long)p.c.n_seq * p.c.hkv * kJoinWarps < plan.dec.grid ? plan.dec_rows : 2;
    j.tc_blocks = plan.tc.grid * kJoinTileBlocks;
    e = launch_after(gdn_attn_join_kernel, dim3(j.tc_blocks + plan.dec.grid * j.dec_split), dim3(kJoinWarps * 32), 0, stream, true, j);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "attention join kernel launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

// ---- norm
// Launch shape: a warp per row of up to 512 channels, eight rows a block; else four units of 8 channels per thread, up to
// 512 threads.  512 threads per SM in all, and as many stages of the ring as fit, up to four.  Measured at 16384 rows of
// 4096 bf16 channels: two units per thread on 1024 threads (the same rows in flight, twice the warps to bring together
// per row) forward 98 us against 81, backward 142 against 103; six blocks per SM instead of four 89 and 123.
struct NormShape {
    dim3 block;
    int nv, grid, stages;
    size_t smem;
};
static NormShape norm_shape(long long rows, int d, int esize, int ops) {
    NormShape n;
    const int units = d / 8;
    const int tpr = units <= 64 ? 32 : std::min(512, ((units + 3) / 4 + 31) / 32 * 32);
    const int per = (units + tpr - 1) / tpr;
    n.nv = per <= 1 ? 1 : per <= 2 ? 2 : 4;
    n.block = dim3(tpr, tpr == 32 && units <= 64 ? 8 : 1);
    const int per_sm = std::max(1, 512 / (int)(n.block.x * n.block.y));
    n.grid = (int)std::min<long long>((rows + n.block.y - 1) / n.block.y, (long long)kAttnSms * per_sm);
    const size_t stage = (size_t)n.block.y * ops * d * esize, room = (size_t)224 * 1024 - 1024 * per_sm;
    n.stages = (int)std::max<size_t>(1, std::min<size_t>(4, room / per_sm / stage));
    n.smem = stage * n.stages;
    return n;
}

template <auto Kern, typename P>
static cudaError_t launch_norm_shape(const NormShape& n, const P& p, cudaStream_t stream) {
    const cudaError_t e = allow_shared<Kern>(224 * 1024);
    if (e != cudaSuccess) return e;
    Kern<<<n.grid, n.block, n.smem, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, int OUT>
static cudaError_t launch_norm(NormParams p, cudaStream_t stream) {
    const NormShape n = norm_shape(p.rows, p.d, sizeof(T), 2);
    p.stages = n.stages;
    return n.nv == 1   ? launch_norm_shape<&gdn_add_rmsnorm_kernel<T, 1, OUT>>(n, p, stream)
           : n.nv == 2 ? launch_norm_shape<&gdn_add_rmsnorm_kernel<T, 2, OUT>>(n, p, stream)
                       : launch_norm_shape<&gdn_add_rmsnorm_kernel<T, 4, OUT>>(n, p, stream);
}

template <typename T>
static cudaError_t launch_norm_bwd(NormBwdParams p, cudaStream_t stream) {
    const NormShape n = norm_shape(p.rows, p.d, sizeof(T), 3);
    p.stages = n.stages;
    p.parts = n.grid;
    const cudaError_t e = n.nv == 1   ? launch_norm_shape<&gdn_add_rmsnorm_bwd_kernel<T, 1>>(n, p, stream)
                          : n.nv == 2 ? launch_norm_shape<&gdn_add_rmsnorm_bwd_kernel<T, 2>>(n, p, stream)
                                      : launch_norm_shape<&gdn_add_rmsnorm_bwd_kernel<T, 4>>(n, p, stream);
    if (e != cudaSuccess) return e;
    return launch_after(gdn_add_rmsnorm_dw_kernel, dim3((p.d + 31) / 32), dim3(kDwWarps * 32), 0, stream, true, p);
}

static gdn_status check_norm(long long rows, int d, gdn_dtype dt) {
    if (rows < 0 || rows > 0x7fffffffLL) return fail(GDN_ERR_INVALID_ARG, "rows must be in [0, 2^31) (got %lld)", rows);
    if (d < 8 || d > 16384 || d % 8 != 0)
        return fail(GDN_ERR_UNSUPPORTED, "d must be a multiple of 8 in [8, 16384] (got %d)", d);
    if (dt != GDN_F32 && dt != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "unknown dtype %d", (int)dt);
    return GDN_OK;
}

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_kv_append(const void* k, const void* v, long long k_stride, long long v_stride, void* k_cache,
                         void* v_cache, uint8_t* k_scale, uint8_t* v_scale, const int32_t* block_table,
                         const int32_t* seq_lens, const int32_t* cu_seqlens, int n_tok, int n_seqs, int n_pages,
                         int max_pages, int page_size, int Hkv, int d, gdn_dtype dt, gdn_dtype cache_dt,
                         cudaStream_t stream) {
    clear_error();
    KvAppendParams p;
    gdn_status st = check_cache(&p.c, k_cache, v_cache, k_scale, v_scale, block_table, n_tok, n_seqs, n_pages, max_pages,
                                page_size, Hkv, d, cache_dt);
    if (st != GDN_OK) return st;
    if (dt != GDN_F32 && dt != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "k and v are GDN_F32 or GDN_BF16 (got %d)", (int)dt);
    if (n_tok == 0) return GDN_OK;
    if ((st = check_ptrs({k, v, seq_lens}, {cu_seqlens})) != GDN_OK) return st;
    const int esize = dt == GDN_F32 ? 4 : 2;
    if ((st = check_stride("k_stride", k_stride, (long long)Hkv * d, esize)) != GDN_OK) return st;
    if ((st = check_stride("v_stride", v_stride, (long long)Hkv * d, esize)) != GDN_OK) return st;
    if (!cu_seqlens && n_tok % n_seqs != 0)
        return fail(GDN_ERR_INVALID_ARG, "without cu_seqlens the tokens must divide evenly (%d over %d)", n_tok, n_seqs);
    unsigned* err = err_word_ptr(&st);
    if (!err) return st;
    p.c.seq_lens = seq_lens;
    p.c.cu = cu_seqlens;
    p.x[0] = k, p.x[1] = v;
    p.stride[0] = k_stride, p.stride[1] = v_stride;
    const bool e = cache_dt == GDN_E4M3;
    ProfScope prof(PK_KV_APPEND, stream);
    if (dt == GDN_F32) d == 64 ? launch_append<float, 64>(p, e, err, stream) : launch_append<float, 128>(p, e, err, stream);
    else d == 64 ? launch_append<__nv_bfloat16, 64>(p, e, err, stream) : launch_append<__nv_bfloat16, 128>(p, e, err, stream);
    prof.done();
    const cudaError_t ce = cudaGetLastError();
    if (ce != cudaSuccess) return fail(GDN_ERR_CUDA, "cache append kernel launch: %s", cudaGetErrorString(ce));
    return GDN_OK;
}

gdn_status gdn_kv_read(const void* k_cache, const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                       const int32_t* block_table, const int32_t* cu_seqlens, void* k, void* v, int n_rows, int n_seqs,
                       int n_pages, int max_pages, int page_size, int Hkv, int d, gdn_dtype cache_dt, gdn_dtype dt,
                       cudaStream_t stream) {
    clear_error();
    KvReadParams p;
    gdn_status st = check_cache(&p.c, k_cache, v_cache, k_scale, v_scale, block_table, n_rows, n_seqs, n_pages,
                                max_pages, page_size, Hkv, d, cache_dt);
    if (st != GDN_OK) return st;
    if (dt != GDN_F32 && dt != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "k and v are GDN_F32 or GDN_BF16 (got %d)", (int)dt);
    if (n_rows == 0) return GDN_OK;
    if ((st = check_ptrs({cu_seqlens, k, v}, {})) != GDN_OK) return st;
    unsigned* err = err_word_ptr(&st);
    if (!err) return st;
    p.c.cu = cu_seqlens;
    p.y[0] = k, p.y[1] = v;
    const bool e = cache_dt == GDN_E4M3;
    ProfScope prof(PK_KV_READ, stream);
    if (dt == GDN_F32) d == 64 ? launch_read<float, 64>(p, e, err, stream) : launch_read<float, 128>(p, e, err, stream);
    else d == 64 ? launch_read<__nv_bfloat16, 64>(p, e, err, stream) : launch_read<__nv_bfloat16, 128>(p, e, err, stream);
    prof.done();
    const cudaError_t ce = cudaGetLastError();
    if (ce != cudaSuccess) return fail(GDN_ERR_CUDA, "cache read kernel launch: %s", cudaGetErrorString(ce));
    return GDN_OK;
}

size_t gdn_paged_attn_workspace_bytes(int n_tok, int n_seqs, int Hq, int Hkv, int d) {
    if (n_tok < 1 || n_seqs < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (d != 64 && d != 128)) return 0;
    size_t most = 0;  // enough for a call with or without cu_seqlens, over either cache
    for (int i = 0; i < 4; ++i) most = std::max(most, attn_plan(n_tok, n_seqs, i & 1, Hq / Hkv, d, i & 2).bytes);
    return most;
}

gdn_status gdn_paged_attn_fwd(const void* q, long long q_stride, const void* k_cache, const void* v_cache,
                              const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table,
                              const int32_t* seq_lens, const int32_t* cu_seqlens, float scale, int window, void* o,
                              float* lse, int n_tok, int n_seqs, int n_pages, int max_pages, int page_size, int Hq,
                              int Hkv, int d, gdn_dtype cache_dt, gdn_dtype o_dt, void* workspace, size_t ws_bytes,
                              cudaStream_t stream) {
    clear_error();
    AttnParams p = {};
    gdn_status st = check_cache(&p.c, k_cache, v_cache, k_scale, v_scale, block_table, n_tok, n_seqs, n_pages, max_pages,
                                page_size, Hkv, d, cache_dt);
    if (st != GDN_OK) return st;
    if (Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > 256)
        return fail(GDN_ERR_INVALID_ARG, "Hq must be 1 to 256 times Hkv (got %d, %d)", Hq, Hkv);
    if (o_dt != GDN_F32 && o_dt != GDN_BF16) return fail(GDN_ERR_UNSUPPORTED, "o is GDN_F32 or GDN_BF16 (got %d)", (int)o_dt);
    if (!std::isfinite(scale * kLog2e)) return fail(GDN_ERR_INVALID_ARG, "scale is not finite, or too large");
    if (window < 0) return fail(GDN_ERR_INVALID_ARG, "window must be >= 0 (got %d)", window);
    if ((long long)n_tok * (Hq / Hkv) > 0x7fffff00LL) return fail(GDN_ERR_UNSUPPORTED, "too many query rows");
    if (n_tok == 0) return GDN_OK;
    if ((st = check_ptrs({q, seq_lens, o}, {cu_seqlens, lse, workspace})) != GDN_OK) return st;
    if ((st = check_stride("q_stride", q_stride, (long long)Hq * d, 2)) != GDN_OK) return st;
    if (!cu_seqlens && n_tok % n_seqs != 0)
        return fail(GDN_ERR_INVALID_ARG, "without cu_seqlens the tokens must divide evenly (%d over %d)", n_tok, n_seqs);
    const AttnPlan plan = attn_plan(n_tok, n_seqs, cu_seqlens != nullptr, Hq / Hkv, d, cache_dt == GDN_E4M3);
    if (!workspace || ws_bytes < plan.bytes)
        return fail(GDN_ERR_INVALID_ARG, "the attention needs %zu bytes of workspace (got %zu)", plan.bytes, ws_bytes);
    unsigned* err = err_word_ptr(&st);
    if (!err) return st;
    p.c.seq_lens = seq_lens;
    p.c.cu = cu_seqlens;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.q_stride = q_stride;
    p.o = o;
    p.lse = lse;
    p.scale_log2 = scale * kLog2e;
    p.window = window;
    p.G = Hq / Hkv;
    p.hq = Hq;
    p.o_f32 = o_dt == GDN_F32;
    p.debug_stall = debug_stall();
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    JoinParams j = {};
    j.o = o, j.lse = lse, j.G = p.G, j.hq = Hq, j.d = d, j.o_f32 = p.o_f32;
    ProfScope prof(PK_ATTN, stream);
    if (cache_dt == GDN_E4M3) st = d == 64 ? launch_attn<64, true>(p, plan, ws, j, err, stream) : launch_attn<128, true>(p, plan, ws, j, err, stream);
    else st = d == 64 ? launch_attn<64, false>(p, plan, ws, j, err, stream) : launch_attn<128, false>(p, plan, ws, j, err, stream);
    prof.done();
    return st;
}

gdn_status gdn_add_rmsnorm_fwd(const void* x, const void* residual, const float* weight, void* s, void* y,
                               float* y_scale, float* rstd, long long rows, int d, gdn_dtype dt, gdn_dtype y_dt,
                               int group, float eps, cudaStream_t stream) {
    clear_error();
    gdn_status st = check_norm(rows, d, dt);
    if (st != GDN_OK) return st;
    if (y_dt != dt && y_dt != GDN_E4M3)
        return fail(GDN_ERR_UNSUPPORTED, "y is GDN_E4M3 or has the input's dtype (got %d)", (int)y_dt);
    if (y_dt == GDN_E4M3) {
        if (group != 0 && group != kNormGroup)
            return fail(GDN_ERR_UNSUPPORTED, "group must be 0 (one scale per row) or %d (got %d)", kNormGroup, group);
        if (group && d % group != 0) return fail(GDN_ERR_UNSUPPORTED, "d must be a multiple of the group (got %d)", d);
    } else if (group != 0 || y_scale) {
        return fail(GDN_ERR_INVALID_ARG, "group and y_scale go with an 8-bit output only");
    }
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(GDN_ERR_INVALID_ARG, "eps must be >= 0");
    if (rows == 0) return GDN_OK;
    if ((st = check_ptrs({x, weight, y}, {residual, s, y_scale, rstd})) != GDN_OK) return st;
    if (y_dt == GDN_E4M3 && !y_scale) return fail(GDN_ERR_INVALID_ARG, "an 8-bit output needs y_scale");
    const NormParams p{x, residual, weight, s, y, y_scale, rstd, rows, d, eps, 0};
    ProfScope prof(PK_RMSNORM, stream);
    cudaError_t e;
    if (dt == GDN_F32)
        e = y_dt != GDN_E4M3 ? launch_norm<float, NORM_SAME>(p, stream)
            : group          ? launch_norm<float, NORM_GROUP>(p, stream)
                             : launch_norm<float, NORM_ROW>(p, stream);
    else
        e = y_dt != GDN_E4M3 ? launch_norm<__nv_bfloat16, NORM_SAME>(p, stream)
            : group          ? launch_norm<__nv_bfloat16, NORM_GROUP>(p, stream)
                             : launch_norm<__nv_bfloat16, NORM_ROW>(p, stream);
    prof.done();
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "norm kernel launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

size_t gdn_add_rmsnorm_bwd_workspace_bytes(long long rows, int d) {
    if (rows < 1 || d < 8 || d > 16384 || d % 8 != 0) return 0;
    return (size_t)norm_shape(rows, d, 4, 3).grid * d * sizeof(float);  // the grid does not depend on the type
}

gdn_status gdn_add_rmsnorm_bwd(const void* dy, const void* s, const float* weight, const float* rstd, const void* ds,
                               void* dx, float* dweight, long long rows, int d, gdn_dtype dt, void* workspace,
                               size_t ws_bytes, cudaStream_t stream) {
    clear_error();
    gdn_status st = check_norm(rows, d, dt);
    if (st != GDN_OK) return st;
    if ((st = check_ptrs({weight, dweight}, {workspace})) != GDN_OK) return st;
    if (rows == 0) {  // the gradient of no rows
        const cudaError_t e = cudaMemsetAsync(dweight, 0, (size_t)d * sizeof(float), stream);
        if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "norm backward: %s", cudaGetErrorString(e));
        return GDN_OK;
    }
    if ((st = check_ptrs({dy, s, rstd, dx}, {ds})) != GDN_OK) return st;
    const size_t need = gdn_add_rmsnorm_bwd_workspace_bytes(rows, d);
    if (!workspace || ws_bytes < need)
        return fail(GDN_ERR_INVALID_ARG, "the norm's backward pass needs %zu bytes of workspace (got %zu)", need, ws_bytes);
    const NormBwdParams p{dy, s, weight, rstd, ds, dx, static_cast<float*>(workspace), dweight, rows, d, 0, 0};
    ProfScope prof(PK_RMSNORM_BWD, stream);
    const cudaError_t e = dt == GDN_F32 ? launch_norm_bwd<float>(p, stream) : launch_norm_bwd<__nv_bfloat16>(p, stream);
    prof.done();
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "norm backward kernel launch: %s", cudaGetErrorString(e));
    return GDN_OK;
}

}  // extern "C"
