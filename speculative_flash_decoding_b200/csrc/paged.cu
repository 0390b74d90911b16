// Host side of the paged cache's entry points (alspec_paged_*): argument
// checks, tensor maps, workspace layout and launches.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "alspec.h"
#include "host.h"
#include "paged_kernels.cuh"

namespace alspec {
namespace {

int elem_size(int dtype) { return dtype == ALSPEC_F32 ? 4 : dtype == ALSPEC_BF16 ? 2 : 1; }

// The description without its pointers.
alspec_status check_shape(const alspec_paged_cache* c) {
    if (!c || c->reserved != 0) return ALSPEC_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->page_size < 1 || c->n_kv_heads < 1 || c->head_dim < 1)
        return ALSPEC_ERR_INVALID_ARG;
    if (c->dtype != ALSPEC_F32 && c->dtype != ALSPEC_BF16 && c->dtype != ALSPEC_E4M3)
        return ALSPEC_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return ALSPEC_ERR_UNSUPPORTED;
    if (c->page_size % 8 != 0) return ALSPEC_ERR_UNSUPPORTED;
    if (c->n_kv_heads > 65535) return ALSPEC_ERR_UNSUPPORTED;
    const bool contiguous = c->page_stride == 0 && c->head_stride == 0 && c->token_stride == 0;
    if (contiguous) {
        // The head and page strides of the contiguous layout stay below the
        // limits too: page_size * head_dim * heads fits 64 bits, and 2^40.
        const double bytes = (double)c->n_kv_heads * c->page_size * c->head_dim *
                             elem_size(c->dtype);
        return bytes < 1099511627776.0 ? ALSPEC_OK : ALSPEC_ERR_UNSUPPORTED;
    }
    for (const int64_t s : {c->page_stride, c->head_stride, c->token_stride}) {
        if (s < c->head_dim || s >= ((int64_t)1 << 40)) return ALSPEC_ERR_INVALID_ARG;
        const int64_t bytes = s * elem_size(c->dtype);
        if (bytes % 16 != 0 || bytes >= ((int64_t)1 << 40)) return ALSPEC_ERR_INVALID_ARG;
    }
    return ALSPEC_OK;
}

alspec_status check_cache(const alspec_paged_cache* c) {
    const alspec_status st = check_shape(c);
    if (st != ALSPEC_OK) return st;
    if (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages))
        return ALSPEC_ERR_INVALID_ARG;
    if (c->dtype == ALSPEC_E4M3 &&
        (!c->k_scales || !c->v_scales || (reinterpret_cast<uintptr_t>(c->k_scales) & 3u) ||
         (reinterpret_cast<uintptr_t>(c->v_scales) & 3u)))
        return ALSPEC_ERR_INVALID_ARG;
    return ALSPEC_OK;
}

PageLayout layout_of(const alspec_paged_cache& c) {
    PageLayout l{};
    if (c.page_stride == 0) {
        l.token_stride = c.head_dim;
        l.head_stride = (long long)c.page_size * c.head_dim;
        l.page_stride = l.head_stride * c.n_kv_heads;
    } else {
        l.page_stride = c.page_stride;
        l.head_stride = c.head_stride;
        l.token_stride = c.token_stride;
    }
    l.n_pages = c.n_pages;
    l.page_size = c.page_size;
    l.hkv = c.n_kv_heads;
    return l;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool table_ok(const int32_t* table, int batch, int max_pages) {
    return table && aligned4(table) && batch >= 1 && max_pages >= 1;
}

// Tokens a page table row can name, kept so far below 2^31 that tile
// arithmetic does not pass it.
int table_tokens(int max_pages, int page_size) {
    return (int)std::min<long long>((long long)max_pages * page_size, (1ll << 31) - 4096);
}

// A programmatic launch: every kernel of this file waits for the kernel ahead
// before it touches memory.
template <typename P>
alspec_status launch(void (*fn)(P), dim3 blocks, unsigned threads, int smem, void* stream,
                     const P& p) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = blocks;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr = programmatic_launch();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return ok(cudaLaunchKernelEx(&cfg, fn, p)) ? ALSPEC_OK : ALSPEC_ERR_CUDA;
}

// ------------------------------------------------------------ append, gather

using AppendFn = void (*)(AppendParams);
using GatherFn = void (*)(GatherParams);

template <int D>
AppendFn append_for(int src, int dst) {
    if (src == ALSPEC_F32)
        return dst == ALSPEC_F32    ? paged_append_kernel<kF32, kF32, D>
               : dst == ALSPEC_BF16 ? paged_append_kernel<kF32, kBf16, D>
                                    : paged_append_kernel<kF32, kE4m3, D>;
    return dst == ALSPEC_F32    ? paged_append_kernel<kBf16, kF32, D>
           : dst == ALSPEC_BF16 ? paged_append_kernel<kBf16, kBf16, D>
                                : paged_append_kernel<kBf16, kE4m3, D>;
}

template <int D>
GatherFn gather_for(int src, int dst) {
    if (dst == ALSPEC_F32)
        return src == ALSPEC_F32    ? paged_gather_kernel<kF32, kF32, D>
               : src == ALSPEC_BF16 ? paged_gather_kernel<kBf16, kF32, D>
                                    : paged_gather_kernel<kE4m3, kF32, D>;
    return src == ALSPEC_F32    ? paged_gather_kernel<kF32, kBf16, D>
           : src == ALSPEC_BF16 ? paged_gather_kernel<kBf16, kBf16, D>
                                : paged_gather_kernel<kE4m3, kBf16, D>;
}

// ------------------------------------------------------------ decode

using PagedFn = void (*)(PagedParams);

struct PagedKernel {
    PagedFn fn;
    int threads, smem, part_floats;
    int tile, box;  // tokens of a tile, rows of a TMA box
};

template <int T, int D, int BOX>
PagedKernel paged_kernel(int box) {
    using C = PagedCfg<T, D, BOX>;
    return PagedKernel{paged_decode_kernel<T, D, BOX>, C::kThreads, C::kSmemBytes, C::PART, C::TT,
                       box};
}

// `box`: the largest power of two that divides a page; a box takes that, up
// to a tile.  Rows of up to 128 bytes lie the same way whatever the box.
template <int T, int D>
PagedKernel paged_kernel_box(int box) {
    using C = PagedCfg<T, D, 8>;
    box = std::min(box, C::TT);
    if constexpr (C::SEGS > 1) {
        if (box == 8) return paged_kernel<T, D, 8>(box);
        if (C::TT > 16 && box == 16) return paged_kernel<T, D, 16>(box);
    }
    return paged_kernel<T, D, C::TT>(box);
}

template <int D>
PagedKernel paged_kernel_type(int dtype, int out_dtype, int box) {
    return dtype == ALSPEC_F32        ? paged_kernel_box<kPagesF32, D>(box)
           : dtype == ALSPEC_E4M3
               ? (out_dtype == ALSPEC_BF16 ? paged_kernel_box<kPagesE4m3, D>(box)
                                           : paged_kernel_box<kPagesE4m3Wide, D>(box))
           : out_dtype == ALSPEC_BF16 ? paged_kernel_box<kPagesBf16, D>(box)
                                      : paged_kernel_box<kPagesBf16Wide, D>(box);
}

PagedKernel paged_kernel_for(const alspec_paged_cache& c, int out_dtype) {
    const int box = c.page_size & -c.page_size;
    return c.head_dim == 128 ? paged_kernel_type<128>(c.dtype, out_dtype, box)
                             : paged_kernel_type<64>(c.dtype, out_dtype, box);
}

// Workspace: the error word and one ticket per CTA, and two partials per CTA.
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t ticket_bytes(int ctas) { return align256((size_t)(kPagedTickets + ctas) * 4); }

size_t workspace_bytes_for(const PagedKernel& k, int ctas) {
    return ticket_bytes(ctas) + align256((size_t)ctas * 2 * k.part_floats * 4);
}

alspec_status check_heads(const alspec_paged_cache* c, int batch, int n_q_heads) {
    const alspec_status st = check_shape(c);
    if (st != ALSPEC_OK) return st;
    if (batch < 1 || n_q_heads < 1 || n_q_heads % c->n_kv_heads != 0)
        return ALSPEC_ERR_INVALID_ARG;
    if (batch > 65535 || n_q_heads > (1 << 20)) return ALSPEC_ERR_UNSUPPORTED;
    return ALSPEC_OK;
}

// A 5-D view (element, slot, 128-byte segment, KV head, page) of a pool (rows
// of 64 bytes: one segment); boxes of `box` slots with all their segments.
alspec_status encode_pages(CUtensorMap* map, const void* base, const alspec_paged_cache& c,
                           const PageLayout& l, int box) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const alspec_status st = tiled_map_encoder(&encode);
    if (st != ALSPEC_OK) return st;
    const int es = elem_size(c.dtype);
    const int row = c.head_dim * es, seg = std::min(row, 128);
    const cuuint64_t dims[5] = {(cuuint64_t)(seg / es), (cuuint64_t)c.page_size,
                                (cuuint64_t)(row / seg), (cuuint64_t)c.n_kv_heads,
                                (cuuint64_t)c.n_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)(l.token_stride * es), (cuuint64_t)seg,
                                   (cuuint64_t)(l.head_stride * es),
                                   (cuuint64_t)(l.page_stride * es)};
    const cuuint32_t boxes[5] = {(cuuint32_t)(seg / es), (cuuint32_t)box,
                                 (cuuint32_t)(row / seg), 1, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUresult r = encode(
        map,
        c.dtype == ALSPEC_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
        : c.dtype == ALSPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
        5, const_cast<void*>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
        row >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ALSPEC_OK : ALSPEC_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace alspec

using namespace alspec;

extern "C" {

alspec_status alspec_paged_append(const alspec_paged_cache* cache, const void* k, const void* v,
                                  int src_dtype, int64_t k_stride, int64_t v_stride,
                                  const int32_t* positions, const int32_t* seq_ids, int n_tokens,
                                  const int32_t* page_table, int batch, int max_pages,
                                  uint32_t* err, void* stream) {
    const alspec_status st = check_cache(cache);
    if (st != ALSPEC_OK) return st;
    if (src_dtype != ALSPEC_F32 && src_dtype != ALSPEC_BF16) return ALSPEC_ERR_INVALID_ARG;
    if (n_tokens < 0 || !table_ok(page_table, batch, max_pages) || !aligned4(err) ||
        !aligned4(positions) || !aligned4(seq_ids))
        return ALSPEC_ERR_INVALID_ARG;
    if (n_tokens == 0) return ALSPEC_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v) || !positions) return ALSPEC_ERR_INVALID_ARG;
    if (!seq_ids && n_tokens > batch) return ALSPEC_ERR_INVALID_ARG;
    const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
    const int64_t unit = 16 / elem_size(src_dtype);
    AppendParams p{};
    for (int w = 0; w < 2; ++w) {
        const int64_t s = w ? v_stride : k_stride;
        if (s != 0 && (s < row || s % unit != 0 || s >= ((int64_t)1 << 40)))
            return ALSPEC_ERR_INVALID_ARG;
        p.src_stride[w] = s ? s : row;
    }
    const int64_t rows = (int64_t)n_tokens * cache->n_kv_heads;
    if (rows > 0x40000000) return ALSPEC_ERR_UNSUPPORTED;
    const int per_block = kAppendThreads / (cache->head_dim / kAppendLane);
    const int64_t blocks = std::min<int64_t>((rows + per_block - 1) / per_block,
                                             (int64_t)kAppendCtas * sm_count_for_plan());
    p.lay = layout_of(*cache);
    p.pages[0] = cache->k_pages;
    p.pages[1] = cache->v_pages;
    p.scales[0] = cache->k_scales;
    p.scales[1] = cache->v_scales;
    p.src[0] = k;
    p.src[1] = v;
    p.positions = positions;
    p.seq_ids = seq_ids;
    p.table = page_table;
    p.n = n_tokens;
    p.batch = batch;
    p.max_pages = max_pages;
    p.err = err;
    const AppendFn fn = cache->head_dim == 128 ? append_for<128>(src_dtype, cache->dtype)
                                               : append_for<64>(src_dtype, cache->dtype);
    return launch(fn, (unsigned)blocks, kAppendThreads, 0, stream, p);
}

alspec_status alspec_paged_gather(const alspec_paged_cache* cache, const int32_t* page_table,
                                  int max_pages, const int32_t* seq_lens, int batch,
                                  int max_seq_len, int out_dtype, void* k_out, void* v_out,
                                  uint32_t* err, void* stream) {
    const alspec_status st = check_cache(cache);
    if (st != ALSPEC_OK) return st;
    if (out_dtype != ALSPEC_F32 && out_dtype != ALSPEC_BF16) return ALSPEC_ERR_INVALID_ARG;
    if (!table_ok(page_table, batch, max_pages) || !seq_lens || !aligned4(seq_lens) ||
        max_seq_len < 1 || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out) ||
        !aligned4(err))
        return ALSPEC_ERR_INVALID_ARG;
    GatherParams p{};
    if (max_seq_len > 0x7fffffff - kGatherRows) return ALSPEC_ERR_UNSUPPORTED;
    p.blocks_per_seq = (max_seq_len + kGatherRows - 1) / kGatherRows;
    const int64_t blocks = (int64_t)p.blocks_per_seq * batch;
    if (blocks > 0x7fffffff) return ALSPEC_ERR_UNSUPPORTED;
    p.lay = layout_of(*cache);
    p.pages[0] = cache->k_pages;
    p.pages[1] = cache->v_pages;
    p.scales[0] = cache->k_scales;
    p.scales[1] = cache->v_scales;
    p.table = page_table;
    p.lens = seq_lens;
    p.out[0] = k_out;
    p.out[1] = v_out;
    p.max_pages = max_pages;
    p.max_len = max_seq_len;
    p.err = err;
    const GatherFn fn = cache->head_dim == 128 ? gather_for<128>(cache->dtype, out_dtype)
                                               : gather_for<64>(cache->dtype, out_dtype);
    // A CTA for every head while eight an SM are not reached, else two for the
    // heads (8 x 16K-64K e4m3: 309 us, with one CTA a head 314, with one for
    // all 326; 50 tokens each of 64 sequences of a 64K capacity 143, 542, 81).
    const bool few = blocks < (int64_t)8 * sm_count_for_plan();
    return launch(fn, dim3((unsigned)blocks, (unsigned)std::min(cache->n_kv_heads, few ? 65535 : 2)),
                  kGatherThreads, 0, stream, p);
}

size_t alspec_paged_workspace_size(const alspec_paged_cache* cache, int batch, int n_q_heads) {
    if (check_heads(cache, batch, n_q_heads) != ALSPEC_OK) return 0;
    const PagedKernel k = paged_kernel_for(*cache, ALSPEC_F32);
    return workspace_bytes_for(k, sm_count_for_plan());
}

alspec_status alspec_paged_decode(const alspec_paged_cache* cache, const void* q, int64_t q_stride,
                                  int n_q_heads, const int32_t* page_table, int max_pages,
                                  const int32_t* seq_lens, int batch, int n_sink, int window,
                                  float scale, int out_dtype, void* out, float* lse,
                                  int timeout_ms, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    alspec_status st = check_heads(cache, batch, n_q_heads);
    if (st != ALSPEC_OK) return st;
    if ((st = check_cache(cache)) != ALSPEC_OK) return st;
    if (out_dtype != ALSPEC_F32 && out_dtype != ALSPEC_BF16) return ALSPEC_ERR_INVALID_ARG;
    if (!q || !aligned16(q) || !table_ok(page_table, batch, max_pages) || !seq_lens ||
        !aligned4(seq_lens) || !out || !aligned16(out) || !aligned4(lse) || n_sink < 0 ||
        window < 0 || timeout_ms < 0 || !std::isfinite(scale))
        return ALSPEC_ERR_INVALID_ARG;
    const int64_t row = (int64_t)n_q_heads * cache->head_dim;
    const int qsize = cache->dtype == ALSPEC_F32 ? 4 : 2;
    if (q_stride != 0 && (q_stride < row || q_stride * qsize % 16 != 0 ||
                          q_stride >= ((int64_t)1 << 40)))
        return ALSPEC_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace)) return ALSPEC_ERR_WORKSPACE;
    const PagedKernel kern = paged_kernel_for(*cache, out_dtype);
    const int group = n_q_heads / cache->n_kv_heads;
    const int blocks = (group + kHeadRows - 1) / kHeadRows;
    const int cap = table_tokens(max_pages, cache->page_size);
    // The running sums of a batch's costs (two a tile, one a run) are 32-bit,
    // and so is a place among those of a sequence's units.
    if (std::max<int64_t>(batch, (int64_t)cache->n_kv_heads * blocks) *
            (2 * ((int64_t)cap / kern.tile + 2) + 1) >=
        (1ll << 31))
        return ALSPEC_ERR_UNSUPPORTED;
    const int ctas = sm_count_for_plan();
    if (workspace_bytes < workspace_bytes_for(kern, ctas)) return ALSPEC_ERR_WORKSPACE;
    if ((st = smem_attr_once(reinterpret_cast<const void*>(kern.fn), kern.smem)) != ALSPEC_OK)
        return st;

    PagedParams p{};
    const PageLayout l = layout_of(*cache);
    p.box = kern.box;
    if ((st = encode_pages(&p.tk, cache->k_pages, *cache, l, p.box)) != ALSPEC_OK) return st;
    if ((st = encode_pages(&p.tv, cache->v_pages, *cache, l, p.box)) != ALSPEC_OK) return st;
    p.q = q;
    p.q_stride = q_stride ? q_stride : row;
    p.ks = cache->k_scales;
    p.vs = cache->v_scales;
    p.table = page_table;
    p.lens = seq_lens;
    p.batch = batch;
    p.hq = n_q_heads;
    p.hkv = cache->n_kv_heads;
    p.group = group;
    p.blocks = blocks;
    p.max_pages = max_pages;
    p.page_size = cache->page_size;
    p.n_pages = cache->n_pages;
    p.cap = cap;
    // No sequence is longer than cap, so neither term says more.
    p.S = std::min(n_sink, p.cap);
    p.W = std::min(window, p.cap);
    // t / page_size for t < 2^31: with 2^(k - 1) < page_size <= 2^k, mul =
    // ceil(2^(31 + k) / page_size) makes (t * mul) >> (31 + k) exact.
    unsigned k = 0;
    while ((1ull << k) < (unsigned long long)cache->page_size) ++k;
    p.page_mul = (unsigned)(((1ull << (31 + k)) + cache->page_size - 1) / cache->page_size);
    p.page_shift = k - 1;
    // A factor above zero keeps masked scores (-inf) what they are; the sign
    // goes to the queries.
    const double factor = 1.4426950408889634 *
                          (scale != 0.f ? std::fabs((double)scale)
                                        : 1.0 / std::sqrt((double)cache->head_dim));
    p.qscale = std::max((float)factor, kMinScale);
    p.qflip = scale < 0.f ? 0x80000000u : 0u;
    p.out = out;
    p.out_bf16 = out_dtype == ALSPEC_BF16;
    p.lse = lse;
    p.ctr = static_cast<unsigned*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + ticket_bytes(ctas));
    p.timeout_ns = (unsigned long long)(timeout_ms > 0 ? timeout_ms : 2000) * 1000000ull;
    return launch(kern.fn, (unsigned)ctas, (unsigned)kern.threads, kern.smem, stream, p);
}

}  // extern "C"
