// Kernels of the paged key-value cache: writing rows (quantised for e4m3
// pages), reading them back, and attention of one new token per sequence.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace alspec {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

// Element types of pages, sources and outputs (alspec_dtype).
enum : int { kF32 = 0, kBf16 = 1, kE4m3 = 2 };

// Where rows live in the pools.
struct PageLayout {
    long long page_stride, head_stride, token_stride;  // elements
    int n_pages, page_size, hkv;

    __device__ __forceinline__ long long row(int page, int head, int slot) const {
        return page * page_stride + head * head_stride + slot * token_stride;
    }
    __device__ __forceinline__ long long scale(int page, int head, int slot) const {
        return ((long long)page * hkv + head) * page_size + slot;
    }
};

// Eight values as they lie, fp32 or bf16 (16-byte aligned), and as fp32.
template <int T>
struct Raw8 {
    uint4 r[T == kF32 ? 2 : 1];

    __device__ __forceinline__ void load(const void* base, long long i) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) +
                                                        i * (T == kF32 ? 4 : 2));
        r[0] = __ldg(p);
        if constexpr (T == kF32) r[1] = __ldg(p + 1);
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
        const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (T == kF32) {
                x[j] = __uint_as_float(w[j]);
            } else {
                x[2 * j] = __uint_as_float(w[j] << 16);
                x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
        if constexpr (T == kF32) {
            x[4] = __uint_as_float(r[1].x), x[5] = __uint_as_float(r[1].y);
            x[6] = __uint_as_float(r[1].z), x[7] = __uint_as_float(r[1].w);
        }
    }
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight values to fp32, or rounded to bf16 (16-byte aligned).
template <int T>
__device__ __forceinline__ void store8(void* base, long long i, const float (&x)[8]) {
    if constexpr (T == kF32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                       pack_bf16(x[6], x[7]));
    }
}

// ---------------------------------------------------------------- append

struct AppendParams {
    PageLayout lay;
    void* pages[2];
    float* scales[2];
    const void* src[2];
    long long src_stride[2];
    const int* positions;
    const int* seq_ids;
    const int* table;
    int n, batch, max_pages;
    unsigned* err;
};

constexpr int kAppendThreads = 256;
// CTAs for each SM that a launch asks for, at most.  Registers let two (fp32 to
// e4m3) to four (bf16 to bf16) be resident; the others take over as those end.
// 16411 tokens of 8 heads of 128 elements, bf16 to e4m3, bf16 to bf16 and fp32
// to fp32: 20.3, 25.4 and 54.0 us with six; 19.6, 28.6 and 54.8 with three;
// 23.5, 26.4 and 53.3 with four.
constexpr int kAppendCtas = 6;

// Two quotients x / s correctly rounded, from r = 1 / s rounded: the remainder
// of the product is exact, and one more step with it rounds right (P.
// Markstein, Computation of elementary functions on the IBM RISC System/6000,
// 1990).  Holds where nothing underflows; append takes it for scales away
// from the ends of the range.
__device__ __forceinline__ float2 quotients(float2 x, float s, float r) {
    const float2 rr = make_float2(r, r);
    const float2 q = __fmul2_rn(x, rr);
    return __ffma2_rn(__ffma2_rn(make_float2(-q.x, -q.y), make_float2(s, s), x), rr, q);
}

// The larger of two pairs of unsigned 16-bit integers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// D / 16 lanes hold one (token, KV head)'s row of K and of V, sixteen values
// each, so every access is 16 bytes wide and amax is a few shuffles.  A
// thread goes from row to row with the next row's values and position on
// their way.  Bound by latency for a decode step; for a prompt by bytes and,
// quantising, by instructions: amax runs on pairs of bf16 magnitudes as
// integers, the division is a product and two fused steps on pairs (with
// eight values a lane and one division each, 16411 tokens of 8 heads took
// 29.1 us).
constexpr int kAppendLane = 16;  // values of a lane

template <int SRC>
struct AppendRow {
    Raw8<SRC> x[2][2];
    int t, h, pos, seq;

    template <int D>
    __device__ __forceinline__ void load(const AppendParams& p, unsigned row, unsigned rows,
                                         int col) {
        pos = -1;
        if (row >= rows) return;
        t = (int)(row / (unsigned)p.lay.hkv);
        h = (int)(row - (unsigned)t * (unsigned)p.lay.hkv);
        pos = __ldg(p.positions + t);
        seq = p.seq_ids ? __ldg(p.seq_ids + t) : t;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                x[w][i].load(p.src[w], t * p.src_stride[w] + (long long)h * D + col + 8 * i);
    }

    // Largest magnitude of this lane's values as the bits of an fp32: NaN is
    // above infinity, so either one makes the scale, and with it the row, not
    // finite.
    __device__ __forceinline__ uint32_t largest(int w) const {
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < (SRC == kF32 ? 2 : 1); ++j) {
                const uint4& r = x[w][i].r[j];
                if constexpr (SRC == kF32) {
                    a = max(a, max(max(r.x & 0x7fffffffu, r.y & 0x7fffffffu),
                                   max(r.z & 0x7fffffffu, r.w & 0x7fffffffu)));
                } else {
                    a = max_u16x2(a, max_u16x2(max_u16x2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu),
                                               max_u16x2(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu)));
                }
            }
        return SRC == kF32 ? a : max(a & 0xffff0000u, a << 16);
    }
};

template <int SRC, int DST, int D>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(
    const __grid_constant__ AppendParams p) {
    constexpr int LPR = D / kAppendLane;  // lanes per row
    pdl_wait_prerequisite();
    pdl_launch_dependents();
    const unsigned rows = (unsigned)p.n * (unsigned)p.lay.hkv;
    const unsigned step = gridDim.x * (kAppendThreads / LPR);
    const int col = (int)(threadIdx.x % LPR) * kAppendLane;
    AppendRow<SRC> next;
    unsigned row = blockIdx.x * (kAppendThreads / LPR) + threadIdx.x / LPR;
    next.template load<D>(p, row, rows, col);
    // A whole CTA makes the same number of rounds.
    for (unsigned base = blockIdx.x * (kAppendThreads / LPR); base < rows;
         base += step, row += step) {
        const AppendRow<SRC> cur = next;
        int page = -1, slot = 0;
        if (cur.pos >= 0) {
            const unsigned entry = (unsigned)cur.pos / (unsigned)p.lay.page_size;
            slot = cur.pos - (int)entry * p.lay.page_size;
            if (cur.seq >= 0 && cur.seq < p.batch && entry < (unsigned)p.max_pages)
                page = __ldg(p.table + (long long)cur.seq * p.max_pages + entry);
            if (page < 0 || page >= p.lay.n_pages) {
                page = -1;
                if (p.err && col == 0) atomicOr(p.err, kErrPage);
            }
        }
        if (base + step < rows) next.template load<D>(p, row + step, rows, col);
        const long long at = p.lay.row(page, cur.h, slot) + col;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float x[2][8];
            cur.x[w][0].unpack(x[0]);
            cur.x[w][1].unpack(x[1]);
            if constexpr (DST == kE4m3) {
                uint32_t a = cur.largest(w);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1)
                    a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
                float s = __fdiv_rn(__uint_as_float(a), kE4m3Max);
                s = s < kMinScale ? kMinScale : s;
                uint32_t c[4];
                if (s > 1e-30f && s < 1e36f) {
                    const float r = __frcp_rn(s);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 q = quotients(
                            make_float2(x[j / 4][2 * j % 8], x[j / 4][2 * j % 8 + 1]), s, r);
                        const uint32_t two = f32x2_to_e4m3x2(q.x, q.y);
                        c[j / 2] = j % 2 ? c[j / 2] | two << 16 : two;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t two =
                            f32x2_to_e4m3x2(__fdiv_rn(x[j / 4][2 * j % 8], s),
                                            __fdiv_rn(x[j / 4][2 * j % 8 + 1], s));
                        c[j / 2] = j % 2 ? c[j / 2] | two << 16 : two;
                    }
                }
                __syncwarp();
                if (page >= 0) {
                    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.pages[w]) + at) =
                        make_uint4(c[0], c[1], c[2], c[3]);
                    if (col == 0) p.scales[w][p.lay.scale(page, cur.h, slot)] = s;
                }
            } else if (page >= 0) {
                store8<DST>(p.pages[w], at, x[0]);
                store8<DST>(p.pages[w], at + 8, x[1]);
            }
        }
    }
}

// ---------------------------------------------------------------- gather

struct GatherParams {
    PageLayout lay;
    const void* pages[2];
    const float* scales[2];
    const int* table;
    const int* lens;
    void* out[2];
    int max_pages, max_len, blocks_per_seq;
    unsigned* err;
};

constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 64;  // tokens per CTA

// A CTA reads back 64 tokens of one sequence, K and V, of every gridDim.y'th
// KV head; D / 8 lanes hold a row.  Bound by bytes.  (One CTA for all heads,
// where that leaves CTAs enough: 64 tokens behind the end of a sequence cost
// one CTA that finds nothing to do, not one a head.)
template <int SRC, int DST, int D>
__global__ void __launch_bounds__(kGatherThreads) paged_gather_kernel(
    const __grid_constant__ GatherParams p) {
    constexpr int LPR = D / 8;
    constexpr int RPI = kGatherThreads / LPR;  // rows per iteration
    pdl_wait_prerequisite();
    pdl_launch_dependents();
    const int col = (int)(threadIdx.x % LPR) * 8;
    const int cap = (int)min((long long)p.max_len, (long long)p.max_pages * p.lay.page_size);
    const int b = (int)(blockIdx.x / (unsigned)p.blocks_per_seq);
    const int t0 = (int)(blockIdx.x - (unsigned)b * (unsigned)p.blocks_per_seq) * kGatherRows;
    int len = __ldg(p.lens + b);
    if (len < 0 || len > cap) {
        if (p.err && threadIdx.x == 0 && t0 == 0 && blockIdx.y == 0) atomicOr(p.err, kErrSeqLen);
        len = len < 0 ? 0 : cap;
    }
    if (t0 >= len) return;
    for (int h = blockIdx.y; h < p.lay.hkv; h += gridDim.y) {
        const long long bh = (long long)b * p.lay.hkv + h;
#pragma unroll
        for (int i = 0; i < kGatherRows / RPI; ++i) {
            const int t = t0 + i * RPI + (int)threadIdx.x / LPR;
            if (t >= len) continue;
            const int page = __ldg(p.table + (long long)b * p.max_pages + t / p.lay.page_size);
            if (page < 0 || page >= p.lay.n_pages) {
                if (p.err && col == 0) atomicOr(p.err, kErrPage);
                continue;
            }
            const int slot = t % p.lay.page_size;
            const long long src = p.lay.row(page, h, slot) + col;
            const long long dst = (bh * p.max_len + t) * D + col;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float x[8];
                if constexpr (SRC == kE4m3) {
                    const uint2 c = __ldg(reinterpret_cast<const uint2*>(
                        static_cast<const uint8_t*>(p.pages[w]) + src));
                    const float s = __ldg(p.scales[w] + p.lay.scale(page, h, slot));
                    const uint32_t r[2] = {c.x, c.y};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t f[2];
                        e4m3x4_to_f16x4(r[j], f[0], f[1]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[k]));
                            x[4 * j + 2 * k] = v.x * s;
                            x[4 * j + 2 * k + 1] = v.y * s;
                        }
                    }
                } else {
                    Raw8<SRC> raw;
                    raw.load(p.pages[w], src);
                    raw.unpack(x);
                }
                store8<DST>(p.out[w], dst, x);
            }
        }
    }
}

// ---------------------------------------------------------------- decode
//
// Every warp of a persistent grid (one CTA per SM) owns an equal share of
// the batch's tiles of 32 tokens (16 where rows are long), in the order
// (sequence, KV head, tile): the share is found from seq_lens alone, so ragged
// batches are balanced to a tile or so without a queue.  A warp streams its
// tiles through a ring of its own (TMA boxes of up to 32 rows x 128 bytes,
// swizzled; it refills a stage as soon as it has read it, so no other warp is
// waited for) and keeps the running maximum, sum and weighted values of flash
// decoding.  A (sequence,
// head) that ends inside one warp's share is written by that warp; one that
// spans warps is joined by its CTA, one that spans CTAs by the last of its
// CTAs to arrive (a ticket), in the order of the tiles, so the bits do not
// depend on who joins.
//
// Products run on m16n8 MMAs with the (up to 8) query heads of a KV group as
// rows 0-7 of A.  Rows 8-15 carry what the operand type rounds away, so that
// P V (and Q K) keep more bits than one operand has:
//   bf16 pages  Q is exact; P = hi + lo (16 bits), for fp32 outputs a third
//               bf16 term in a second MMA (24 bits);
//   e4m3 pages  codes widen exactly to f16; Q, scaled by a power of two per
//               head, is f16 (its bf16 fit).  The K scale multiplies a score,
//               the V scale a probability; the product, a weight, is f16
//               hi + lo over a power of two that follows the largest weight
//               so far (wexp): 22 bits, or 2^-36 of that largest;
//   fp32 pages  tf32 with hi + lo of both operands (2^-21.4).
// Bound by HBM bytes over bf16 pages (128K tokens of 8 KV heads: 84 us, 6.4
// TB/s), by instructions over e4m3 pages (8 x 16K-64K tokens: 148-153 us,
// 5.1-5.3 TB/s; a tile of 8 KB takes 128 conversions and 64 MMAs) and fp32 pages (4 x 20000
// tokens of 128 elements: 122-124 us, 5.3 TB/s), by the reads before the first
// tile and the joins after the last where the sequences are short (123 of
// 1-900 tokens: 30 us for 17.6 us of bytes).

// Query heads per work unit.  A KV head's further eights are units of their
// own, each of which streams its keys and values again (4 x 30000 bf16 tokens of
// 4 KV heads of 128 elements: 46.9 us with 8 query heads each, 82.2 with 16).
constexpr int kHeadRows = 8;

// Page types of the decode kernel.  Wide: for fp32 outputs (bf16 pages: P with
// a third term; both: a tile's products summed apart).
enum : int {
    kPagesF32 = 0,
    kPagesBf16 = 1,
    kPagesE4m3 = 2,
    kPagesBf16Wide = 3,
    kPagesE4m3Wide = 4
};
__host__ __device__ constexpr bool pages_e4m3(int t) {
    return t == kPagesE4m3 || t == kPagesE4m3Wide;
}

struct PagedParams {
    CUtensorMap tk, tv;  // 5-D: (element, slot, 128-byte segment, KV head, page)
    const void* q;
    long long q_stride;
    const float* ks;
    const float* vs;
    const int* table;
    const int* lens;
    int batch, hq, hkv, group, blocks;  // blocks: work units of 8 heads per KV head
    int max_pages, page_size, n_pages, box;
    unsigned page_mul, page_shift;      // t / page_size = umulhi(t, page_mul) >> page_shift
    int cap;        // max_pages * page_size, below 2^31
    int S, W;
    float qscale;   // |scale| * log2(e)
    unsigned qflip; // sign bit where scale is negative
    void* out;
    int out_bf16;
    float* lse;
    unsigned* ctr;  // error word and the tickets of the joins
    float* part;    // [CTA][2] partials for other CTAs
    unsigned long long timeout_ns;
};

constexpr int kPagedTickets = kCtrFixed;  // one ticket per CTA follows

// BOX: rows of a TMA box, as far as the layout in shared memory depends on it
// (rows of more than 128 bytes: a box holds its rows segment by segment).
template <int T, int D, int BOX>
struct PagedCfg {
    static constexpr int ES = T == kPagesF32 ? 4 : pages_e4m3(T) ? 1 : 2;
    static constexpr int RB = D * ES;                     // bytes of a row
    static constexpr int SEGB = RB < 128 ? RB : 128;      // bytes of a box row
    static constexpr int SEGS = RB / SEGB;                // boxes side by side
    static constexpr int SEG = BOX * SEGB;                // one segment of a box
    // Tokens of a tile; rows of 512 bytes 16, so that six warps have room
    // instead of three (4 x 20000 tokens of 128 fp32 elements 159 -> 128 us).
    static constexpr int TT = RB > 256 ? 16 : 32;
    static constexpr int TILEB = TT * RB;                 // K or V of a tile
    static constexpr unsigned kAll = 0xffffffffu >> (32 - TT);  // a full tile's mask
    static constexpr int STAGEB = 2 * TILEB;
    // Warps, and two stages each.  128 KB on their way keep HBM busy; 192 KB
    // made the SMs unequal (128K tokens of bf16: some CTAs done after 60 us,
    // some after 85; 87.6 us a call against 84.2, 30000 x 8 of 64 bf16
    // elements 87.2 against 81.0), 96 KB took 90.4 us.  fp32 pages cost more
    // instructions a byte: six warps, as many as fit.
    static constexpr int NW = STAGEB >= 16384 ? (T == kPagesF32 ? 6 : 4) : STAGEB >= 8192 ? 8 : 16;
    static constexpr int ST = 2;
    static constexpr int kThreads = NW * 32;
    // Offset of a row (a multiple of 8, or its row within 8 added later).
    __host__ __device__ static constexpr int row(int r) {
        return r / BOX * (SEGS * SEG) + r % BOX * SEGB;
    }
    static constexpr int PART = 2 * kHeadRows + kHeadRows * D;  // floats: m, l, o
    static constexpr int kOffHead = NW * ST * STAGEB;  // partials of the warps' first runs
    static constexpr int kOffScale = kOffHead + NW * PART * 4;
    // A stage's queries (rows 16 bytes apart, so that their reads meet no
    // bank twice), for bf16 pages: 123 sequences of 450 tokens 31.2 -> 30.6
    // us.  The ring of fp32 pages leaves no room, e4m3 pages lost more in
    // registers (8 x 16K-64K tokens 147 -> 150 us).
    static constexpr bool kCopyQ = T == kPagesBf16 || T == kPagesBf16Wide;
    static constexpr int QROW = 2 * D + 16;
    static constexpr int kOffQ = kOffScale + (pages_e4m3(T) ? NW * ST * 2 * TT * 4 : 0);
    static constexpr int kOffMeta = kOffQ + (kCopyQ ? NW * ST * kHeadRows * QROW : 0);
    static constexpr int kOffBar = kOffMeta + NW * ST * 16;
    static constexpr int kOffPiece = kOffBar + NW * ST * 8;
    static constexpr int kOffMisc = kOffPiece + 2 * NW * 32;
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kSmemBytes <= kSmemLimit, "shared memory budget");
    static_assert(BOX <= TT, "a box of one tile");
    static_assert(ST >= 2 && PART * 4 <= ST * STAGEB, "ring");
    static_assert(kOffMeta % 16 == 0 && kOffPiece % 16 == 0, "alignment");
};

// Tiles of one sequence: tile i covers tokens [TT i, TT i + TT) for i < a and
// [TT (i + f - a), ...) from there on; every tile holds a token of the set.
struct PagedSeq {
    int len, n, a, f;
};

template <int TT>
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int len) {
    PagedSeq s;
    s.len = min(max(len, 0), p.cap);
    const int all = (s.len + TT - 1) / TT;
    if ((p.S | p.W) == 0) {
        s.a = s.n = all;
        s.f = 0;
    } else {
        s.a = (min(p.S, s.len) + TT - 1) / TT;
        const int w0 = max(0, s.len - p.W);
        s.f = max(s.a, w0 / TT);
        s.n = s.a + (w0 < s.len ? all - s.f : 0);
    }
    return s;
}

// A tile's place: sequence, work unit (KV head and block of 8 query heads),
// tile of the run, as its tiles of one (sequence, unit) are called.
struct PagedPos {
    int b, u, i;
    PagedSeq s;
};

// What the shares are measured in: two a tile, and one more a run, because
// starting and ending a run takes a warp about half a tile's time (shares of
// tiles alone left warps with ten runs of one tile 8 us behind the others; 123
// sequences of 1-900 tokens 35.2 -> 30.8 us).
// Tile i of a run is at place 2 i + 1 of the run's 2 n + 1.
__device__ __forceinline__ int paged_cost(int n) { return n > 0 ? 2 * n + 1 : 0; }

// The batch's costs: lane i of a warp holds sequences [i * chunk, (i + 1) *
// chunk), their cost for one unit and the running sum up to their end.
struct PagedBatch {
    int chunk, cost, incl;
    int len;          // of the lane's sequence, with chunk 1
    int units;
    long long total;  // of all sequences and units
};

__device__ __forceinline__ int warp_inclusive(int x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

template <int TT>
__device__ __forceinline__ PagedBatch paged_batch(const PagedParams& p) {
    const int lane = threadIdx.x & 31;
    PagedBatch s;
    s.chunk = (p.batch + 31) / 32;
    s.units = p.hkv * p.blocks;
    s.cost = s.len = 0;
#pragma unroll 4
    for (int b = lane * s.chunk; b < min(p.batch, (lane + 1) * s.chunk); ++b) {
        s.len = __ldg(p.lens + b);
        s.cost += paged_cost(paged_seq<TT>(p, s.len).n);
    }
    s.incl = warp_inclusive(s.cost);
    s.total = (long long)__shfl_sync(0xffffffffu, s.incl, 31) * s.units;
    return s;
}

// Where x (0 <= x < total) lies among the costs in the order (sequence, unit,
// tile); `i` is the place in the run.  Called by a whole warp.
template <int TT>
__device__ __forceinline__ PagedPos paged_find(const PagedParams& p, const PagedBatch& t,
                                               long long x) {
    const int lane = threadIdx.x & 31;
    PagedPos r;
    const int w = __ffs(__ballot_sync(0xffffffffu, (long long)t.incl * t.units > x)) - 1;
    long long before =
        __shfl_sync(0xffffffffu, t.incl, w) - __shfl_sync(0xffffffffu, t.cost, w);
    r.b = w;
    if (t.chunk == 1) {
        r.s = paged_seq<TT>(p, __shfl_sync(0xffffffffu, t.len, w));
    } else {
        // The same among the sequences of that lane.
        for (int b0 = w * t.chunk;; b0 += 32) {
            const int b = b0 + lane;
            const bool in = b < min(p.batch, (w + 1) * t.chunk);
            const int m = in ? paged_cost(paged_seq<TT>(p, __ldg(p.lens + b)).n) : 0;
            const int incl = warp_inclusive(m);
            const unsigned past =
                __ballot_sync(0xffffffffu, (before + incl) * t.units > x);
            if (past || b0 + 32 >= (w + 1) * t.chunk) {
                const int v = past ? __ffs(past) - 1 : 0;
                before += __shfl_sync(0xffffffffu, incl, v) - __shfl_sync(0xffffffffu, m, v);
                r.b = b0 + v;
                break;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        r.s = paged_seq<TT>(p, __ldg(p.lens + r.b));
    }
    const unsigned off = (unsigned)(x - before * t.units);
    const unsigned cost = (unsigned)paged_cost(r.s.n);
    r.u = (int)(off / cost);
    r.i = (int)(off % cost);
    return r;
}

// Shares: the cost is spread over `workers` warps, warp w owning the tiles
// whose places lie in [w * total / workers, (w + 1) * total / workers).  With
// two or more each, no share inside a run is without a tile.
__device__ __forceinline__ long long share_begin(long long total, long long workers, long long w) {
    return w * total / workers;
}
__device__ __forceinline__ long long share_of(long long total, long long workers, long long x) {
    return ((x + 1) * workers - 1) / total;
}

// A warp's part of a run that is not the whole run.
struct PagedPiece {
    int b, u, lo, hi;  // tiles [lo, hi) of n; hi == 0: none
    int n, c0, c1;     // the CTAs that share the (sequence, unit)
    int pad;
};

// Two neighbouring elements of the output.
__device__ __forceinline__ void paged_store2(const PagedParams& p, long long i, float x, float y) {
    if (p.out_bf16)
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + i) = pack_bf16(x, y);
    else
        *reinterpret_cast<float2*>(static_cast<float*>(p.out) + i) = make_float2(x, y);
}

// 1 / l, 0 where nothing was attended to.
__device__ __forceinline__ float paged_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

__device__ __forceinline__ float paged_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// 2^x to 2 ulp (0 below the normal range).
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x for a power of two in [2^-126, 2^126].
__device__ __forceinline__ float pow2_inverse(float x) {
    return __uint_as_float(0x7f000000u - __float_as_uint(x));
}

// Partials of one head joined: running maximum, sum, four weighted values.
struct PagedSum {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);

    // N more partials at once: their weights do not wait for one another.
    template <int N>
    __device__ __forceinline__ void add(const float (&pm)[N], const float (&pl)[N],
                                        const float4 (&v)[N]) {
        float M = m;
#pragma unroll
        for (int k = 0; k < N; ++k) M = fmaxf(M, pm[k]);
        const float f = m == M ? 1.f : fast_exp2(m - M);
        m = M;
        l *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float g = pm[k] == M ? 1.f : fast_exp2(pm[k] - M);
            l = fmaf(pl[k], g, l);
            o.x = fmaf(v[k].x, g, o.x);
            o.y = fmaf(v[k].y, g, o.y);
            o.z = fmaf(v[k].z, g, o.z);
            o.w = fmaf(v[k].w, g, o.w);
        }
    }
    // Elements e .. e + 3 of the rows of D elements from head `head0` on.
    template <int D>
    __device__ __forceinline__ void write(const PagedParams& p, long long head0, int e) const {
        const float inv = paged_inverse(l);
        paged_store2(p, head0 * D + e, o.x * inv, o.y * inv);
        paged_store2(p, head0 * D + e + 2, o.z * inv, o.w * inv);
        if (p.lse && e % D == 0) p.lse[head0 + e / D] = paged_lse(m, l);
    }
};

template <int T, int D, int BOX>
struct PagedWarp {
    using C = PagedCfg<T, D, BOX>;
    static constexpr bool kB16 = T == kPagesBf16 || T == kPagesBf16Wide;
    static constexpr int KS = T == kPagesF32 ? D / 8 : D / 16;  // k steps of Q K
    static constexpr int NT = D / 8;                            // output n tiles
    static constexpr int CH = C::RB / 16;                       // 16-byte chunks of a row
    static constexpr int NG = C::TT / 8;                        // groups of 8 tokens
    static_assert(NG == 4 || T == kPagesF32, "tiles of 16-bit MMAs");
    static constexpr bool kSplitQ = T == kPagesF32;
    static constexpr bool kApart = T == kPagesF32 || T == kPagesBf16Wide || T == kPagesE4m3Wide;

    uint32_t qa[KS][2];                    // A rows 0-7
    uint32_t qb[kSplitQ ? KS : 1][2];      // A rows 8-15: what qa's type rounds away
    float acc[NT][4];                      // rows 0-7 and 8-15
    float m, l;                            // this lane's head: maximum, share of the sum
    float rowscale;                        // log2-domain factor of a score
    float wexp;                            // e4m3: acc holds sums times 1 / wexp
    uint32_t k_off, v_off;                 // this lane's part of a fragment's address

    __device__ __forceinline__ void init(int lane) {
        const int row8 = lane & 7, mat = lane >> 3, j = lane & 3;
        const int sw = C::SEGB == 128 ? row8 : (row8 >> 1) & 3;
        k_off = (uint32_t)(row8 * C::SEGB + ((mat ^ sw) << 4));
        if constexpr (T == kPagesF32)
            v_off = (uint32_t)(2 * j * 128 + (((lane >> 4) ^ (2 * j)) << 4) + ((lane >> 2) & 3) * 4);
        else
            v_off = (uint32_t)((mat & 1) * C::row(8) + row8 * C::SEGB + (((mat >> 1) ^ sw) << 4));
    }

    __device__ __forceinline__ void reset() {
        m = -INFINITY;
        l = 0.f;
        wexp = kMinScale;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    }

    // Queries of unit u of sequence b, of which `rows` copies a stage's rows if
    // C::kCopyQ; lanes of absent heads hold zeros.
    __device__ __forceinline__ void load_q(const PagedParams& p, int b, int u,
                                           const unsigned char* rows, int lane) {
        const int r = lane >> 2, j = lane & 3;
        const int blk = (u % p.blocks) * kHeadRows;
        const bool live = blk + r < p.group;
        const long long at = b * p.q_stride +
                             (long long)((u / p.blocks) * p.group + (live ? blk + r : 0)) * D;
        rowscale = p.qscale;
        if constexpr (kB16) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(rows + r * C::QROW);
            const uint32_t flip = p.qflip | p.qflip >> 16;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qa[k][0] = live ? q[8 * k + j] ^ flip : 0u;
                qa[k][1] = live ? q[8 * k + j + 4] ^ flip : 0u;
            }
        } else if constexpr (pages_e4m3(T)) {
            // Lane j of a quad holds elements 16 k + 4 j .. + 3 of k step k:
            // the order in which the codes of K come out of ldmatrix.
            const uint2* q = reinterpret_cast<const uint2*>(
                static_cast<const __nv_bfloat16*>(p.q) + at);
            uint2 raw[KS];
            uint32_t a = 0;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                raw[k] = live ? __ldg(q + 4 * k + j) : make_uint2(0u, 0u);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t x = w ? raw[k].y : raw[k].x;
                    a = max(a, max((x << 16) & 0x7fff0000u, x & 0x7fff0000u));
                }
            }
            a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
            // 2^e >= the row's largest magnitude, e in [-125, 127].
            const int e = min(max((int)(a >> 23) - 126, -125), 127);
            const float inv = __uint_as_float((uint32_t)(127 - min(e, 126)) << 23 | p.qflip) *
                              (e == 127 ? 0.5f : 1.f);
            rowscale = p.qscale * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t x = w ? raw[k].y : raw[k].x;
                    // (Elements below 2^-14 of the largest lose what is below
                    // 2^-25 of it.)
                    qa[k][w] = pack_f16(__uint_as_float(x << 16) * inv,
                                        __uint_as_float(x & 0xffff0000u) * inv);
                }
        } else {
            const float* q = static_cast<const float*>(p.q) + at;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const float x = live ? __ldg(q + 8 * k + j + 4 * w) : 0.f;
                    split_tf32(__uint_as_float(__float_as_uint(x) ^ p.qflip), qa[k][w], qb[k][w]);
                }
        }
    }

    __device__ __forceinline__ static void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = pack_f16(x - f.x, y - f.y);
    }
    // x and y become what hi and the residual leave.
    __device__ __forceinline__ static uint32_t take_bf16(float& x, float& y) {
        const uint32_t hi = pack_bf16(x, y);
        x -= __uint_as_float(hi << 16);
        y -= __uint_as_float(hi & 0xffff0000u);
        return hi;
    }
    // hi + lo = x to 2^-21.4: hi is x cut off, lo the rest, of which the MMA
    // ignores the low 13 bits; the factor raises lo by 0.36 .. 0.72 of what
    // they stand for, half a step on the average.  No integer addition: it
    // would carry a NaN's payload into the sign (the NaN of fp32 arithmetic is
    // 0x7fffffff) and the largest finite values into infinity.  A NaN whose
    // payload is in the low bits alone leaves hi infinite, but lo NaN.
    __device__ __forceinline__ static void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
        hi = __float_as_uint(x) & 0xffffe000u;
        lo = __float_as_uint((x - __uint_as_float(hi)) * (1.f + 0x1.7p-12f));
    }

    __device__ __forceinline__ static float lds(uint32_t addr) {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
        return v;
    }

    // One tile: bit t of `mask` says whether token t counts (the rows of V of
    // the others are zero); ks and vs are the tile's scales.
    __device__ __forceinline__ void tile(uint32_t stage, unsigned mask, const float* ks,
                                         const float* vs, int lane) {
        const int j = lane & 3;
        // Scores of groups of 8 tokens; over fp32 pages the groups' MMAs in
        // turn.
        float s[NG][4];
        const uint32_t ka[2] = {stage + k_off, (stage + k_off) ^ 64u};
        // For fp32 outputs the sums run in two halves, those of the low parts
        // of fp32 keys apart: an MMA's sum may lose 2^-23 of its running value
        // at every step.
        constexpr bool kHalves = T == kPagesF32 || T == kPagesBf16Wide;
        float odd[kHalves ? NG : 1][4], low[T == kPagesF32 ? NG : 1][4];
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[n][i] = 0.f;
                if constexpr (kHalves) odd[n][i] = 0.f;
                if constexpr (T == kPagesF32) low[n][i] = 0.f;
            }
#pragma unroll
        for (int c = 0; c < CH; c += 4) {
            uint32_t f[NG][4];
#pragma unroll
            for (int n = 0; n < NG; ++n)
                ldsm_x4(ka[(c >> 2) & 1] + (uint32_t)(C::row(8 * n) + (c >> 3) * C::SEG), f[n][0],
                        f[n][1], f[n][2], f[n][3]);
            if constexpr (kB16) {
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    mma_bf16_16816(s[n], qa[c / 2][0], 0u, qa[c / 2][1], 0u, f[n][0], f[n][1]);
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    mma_bf16_16816(kHalves ? odd[kHalves ? n : 0] : s[n], qa[c / 2 + 1][0], 0u,
                                   qa[c / 2 + 1][1], 0u, f[n][2], f[n][3]);
            } else if constexpr (pages_e4m3(T)) {
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16x4(f[n][i], b0, b1);
                        mma_f16_16816(s[n], qa[c + i][0], 0u, qa[c + i][1], 0u, b0, b1);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        const int k = c / 2 + i;
                        uint32_t h0, l0, h1, l1;
                        split_tf32(__uint_as_float(f[n][2 * i]), h0, l0);
                        split_tf32(__uint_as_float(f[n][2 * i + 1]), h1, l1);
                        mma_tf32_1688(i ? odd[kHalves ? n : 0] : s[n], qa[k][0], qb[kSplitQ ? k : 0][0],
                                      qa[k][1], qb[kSplitQ ? k : 0][1], h0, h1);
                        mma_tf32_1688(low[T == kPagesF32 ? n : 0], qa[k][0], qb[kSplitQ ? k : 0][0],
                                      qa[k][1], qb[kSplitQ ? k : 0][1], l0, l1);
                    }
            }
        }
        if constexpr (kHalves) {
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[n][i] += odd[n][i];
                    if constexpr (T == kPagesF32) s[n][i] += low[n][i];
                }
        }
        // Lane (r, j) holds head r, tokens 8 n + 2 j and + 1.  x: scores, up
        // to the factor `f` that makes them logarithms to base 2.
        float x[NG][2], vsc[NG][2], f = rowscale;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                x[n][i] = kSplitQ ? s[n][i] + s[n][i + 2] : s[n][i];
            if constexpr (pages_e4m3(T)) {
                const float2 kk = *reinterpret_cast<const float2*>(ks + 8 * n + 2 * j);
                const float2 vv = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * j);
                x[n][0] *= kk.x * rowscale;
                x[n][1] *= kk.y * rowscale;
                vsc[n][0] = vv.x;
                vsc[n][1] = vv.y;
            }
        }
        if constexpr (pages_e4m3(T)) f = 1.f;
        if (mask != C::kAll) {
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (!((mask >> (8 * n + 2 * j + i)) & 1u)) x[n][i] = -INFINITY, vsc[n][i] = 0.f;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < NG; ++n) mx = fmaxf(mx, fmaxf(x[n][0], x[n][1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * f;
        // The reference of the exponentials follows the maximum only when it
        // is 2^8 behind: until then weights of up to 2^8 do no harm, and the
        // sums need no rescaling.
        const float m_new = mx > m + 8.f ? mx : m;
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = m == m_new ? 1.f : fast_exp2(m - base);
        // e4m3: the V scales over the weights' power of two.
        float sv[pages_e4m3(T) ? NG : 1][2], over = 0.f;
        if constexpr (pages_e4m3(T)) {
            const float winv = pow2_inverse(wexp);
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    sv[n][i] = vsc[n][i] * winv;
                    over = fmaxf(over, fabsf(sv[n][i]));
                }
        }
        const bool again = alpha != 1.f || over == INFINITY;
        float sum = 0.f, wmax = 0.f;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[n][i] = fast_exp2(fmaf(x[n][i], f, -base));
                sum += x[n][i];
                if constexpr (pages_e4m3(T)) {
                    sv[n][i] *= x[n][i];
                    wmax = fmaxf(wmax, fabsf(sv[n][i]));
                }
            }
        float rescale = alpha;
        // f16 ends at 2^-24, and neither the largest probability nor the
        // largest V scale says how large the largest weight is (an attention
        // sink has a small value, an outlier hardly any probability), so the
        // weights' own maximum sets their power of two: to 2^11 .. 2^12 of it
        // when the probabilities' reference moves up past what came before,
        // and when a weight passes 2^15.
        const bool moved = (!kApart || pages_e4m3(T)) &&
                           __any_sync(0xffffffffu, again || wmax > 32768.f);
        if constexpr (pages_e4m3(T)) {
            if (moved) {
                wmax = 0.f;
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        sv[n][i] = x[n][i] * vsc[n][i];
                        wmax = fmaxf(wmax, fabsf(sv[n][i]));
                    }
                wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, 1));
                wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, 2));
                const float now = wexp * alpha;
                const float to = wmax > now * 32768.f ? wmax * (1.f / 2048.f) : now;
                // (In [2^-126, 2^126], so that 1 / wexp is a normal number.)
                wexp = __uint_as_float(
                    min(max(__float_as_uint(to) & 0x7f800000u, 0x00800000u), 0x7e800000u));
                const float winv = pow2_inverse(wexp);
                rescale = now * winv;
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) sv[n][i] *= winv;
            }
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) x[n][i] = sv[n][i];
        }
        m = m_new;
        l = l * alpha + sum;
        // For fp32 outputs a tile's products are summed apart and then added,
        // because the MMAs' sums lose towards zero (one chain over all of a
        // warp's tiles: 1.8e-5 of the result at 2 x 16 x 55854 fp32 tokens).
        if (!kApart && moved) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][k] *= rescale;
        }
        // O += P V.
        const uint32_t v0 = stage + C::TILEB + v_off;
        if constexpr (T == kPagesF32) {
            // Rows 2 j and 2 j + 1 of a k step: the second is 128 bytes on,
            // its chunks exchanged by the swizzle.
            const uint32_t v1 = (v0 + 128u) ^ 16u;
            uint32_t hi[NG][2], lo[NG][2];
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) split_tf32(x[n][i], hi[n][i], lo[n][i]);
#pragma unroll
            for (int i0 = 0; i0 < NT; i0 += 2) {
                float sum[2][4] = {};
#pragma unroll
                for (int n = 0; n < NG; ++n)  // tokens 8 n ..: k step n
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int i = i0 + w;
                        const uint32_t add = (uint32_t)(C::row(8 * n) + (i >> 2) * C::SEG);
                        const uint32_t flip = (uint32_t)((2 * i & 7) << 4);
                        uint32_t a0, a1, b0, b1;
                        split_tf32(lds((v0 ^ flip) + add), a0, a1);
                        split_tf32(lds((v1 ^ flip) + add), b0, b1);
                        mma_tf32_1688(sum[w], hi[n][0], lo[n][0], hi[n][1], lo[n][1], a0, b0);
                        mma_tf32_1688(sum[w], hi[n][0], lo[n][0], hi[n][1], lo[n][1], a1, b1);
                    }
                add_sums(i0, rescale, sum);
            }
        } else {
            uint32_t a[2][4], third[2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // tokens 16 k ..
                if constexpr (pages_e4m3(T)) {
                    split_f16(x[2 * k][0], x[2 * k][1], a[k][0], a[k][1]);
                    split_f16(x[2 * k + 1][0], x[2 * k + 1][1], a[k][2], a[k][3]);
                } else {
                    a[k][0] = take_bf16(x[2 * k][0], x[2 * k][1]);
                    a[k][1] = take_bf16(x[2 * k][0], x[2 * k][1]);
                    a[k][2] = take_bf16(x[2 * k + 1][0], x[2 * k + 1][1]);
                    a[k][3] = take_bf16(x[2 * k + 1][0], x[2 * k + 1][1]);
                    if constexpr (T == kPagesBf16Wide) {
                        third[k][0] = take_bf16(x[2 * k][0], x[2 * k][1]);
                        third[k][1] = take_bf16(x[2 * k + 1][0], x[2 * k + 1][1]);
                    }
                }
            }
            // Matrices of one ldmatrix: tokens 0-7 and 8-15 of a step, chunks
            // c and c + 1.
            auto load = [&](int k, int c, uint32_t (&f)[4]) {
                ldsm_x4_t((v0 ^ (uint32_t)((c & 7) << 4)) +
                              (uint32_t)(C::row(16 * k) + (c >> 3) * C::SEG),
                          f[0], f[1], f[2], f[3]);
            };
            if constexpr (T == kPagesBf16Wide) {
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    float sum[2][4] = {};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t f[4];
                        load(k, c, f);
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            mma_bf16_16816(sum[w], a[k][0], a[k][1], a[k][2], a[k][3], f[2 * w],
                                           f[2 * w + 1]);
                            mma_bf16_16816(sum[w], third[k][0], 0u, third[k][1], 0u, f[2 * w],
                                           f[2 * w + 1]);
                        }
                    }
                    add_sums(c, rescale, sum);
                }
            } else if constexpr (T == kPagesE4m3Wide) {
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    float sum[2][2][4] = {};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t f[4];
                        load(k, c, f);
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            uint32_t b0[2], b1[2];
                            codes_of(f[2 * w], f[2 * w + 1], b0, b1);
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                mma_f16_16816(sum[w][e], a[k][0], a[k][1], a[k][2], a[k][3], b0[e],
                                              b1[e]);
                        }
                    }
                    add_sums(2 * c, rescale, sum[0]);
                    add_sums(2 * c + 2, rescale, sum[1]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int c = 0; c < CH; c += 2) {
                        uint32_t f[4];
                        load(k, c, f);
                        if constexpr (pages_e4m3(T)) {
#pragma unroll
                            for (int w = 0; w < 2; ++w) {
                                uint32_t b0[2], b1[2];
                                codes_of(f[2 * w], f[2 * w + 1], b0, b1);
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    mma_f16_16816(acc[2 * (c + w) + e], a[k][0], a[k][1], a[k][2],
                                                  a[k][3], b0[e], b1[e]);
                            }
                        } else {
                            mma_bf16_16816(acc[c], a[k][0], a[k][1], a[k][2], a[k][3], f[0], f[1]);
                            mma_bf16_16816(acc[c + 1], a[k][0], a[k][1], a[k][2], a[k][3], f[2],
                                           f[3]);
                        }
                    }
            }
        }
    }

    // V codes of tokens 0-7 and 8-15 as ldmatrix leaves them (a pair of columns
    // of one token per half word) to the operands of the even and the odd
    // column.
    __device__ __forceinline__ static void codes_of(uint32_t low, uint32_t high, uint32_t (&b0)[2],
                                                    uint32_t (&b1)[2]) {
        e4m3x4_to_f16x4(__byte_perm(low, 0u, 0x3120), b0[0], b0[1]);
        e4m3x4_to_f16x4(__byte_perm(high, 0u, 0x3120), b1[0], b1[1]);
    }

    // A tile's sums of output tiles i and i + 1 onto the running ones.
    __device__ __forceinline__ void add_sums(int i, float rescale, const float (&sum)[2][4]) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i + w][k] = fmaf(acc[i + w][k], rescale, sum[w][k]);
    }

    // Calls f(column, value, value of column + 1) for this lane's elements of
    // its head's row.
    template <typename F>
    __device__ __forceinline__ void each2(int lane, F f) const {
        const int j = lane & 3;
#pragma unroll
        for (int i = 0; i < NT; i += 2)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if constexpr (pages_e4m3(T)) {
                    // Tiles i and i + 1 hold the even and odd columns of 16.
                    f(8 * i + 4 * j + 2 * k, (acc[i][k] + acc[i][k + 2]) * wexp,
                      (acc[i + 1][k] + acc[i + 1][k + 2]) * wexp);
                } else {
                    f(8 * (i + k) + 2 * j, acc[i + k][0] + acc[i + k][2],
                      acc[i + k][1] + acc[i + k][3]);
                }
            }
    }

    // The row sum of the exponentials over the quad's lanes.
    __device__ __forceinline__ float row_sum() const {
        float s = l + __shfl_xor_sync(0xffffffffu, l, 1);
        return s + __shfl_xor_sync(0xffffffffu, s, 2);
    }

    // Partial of this warp: m[8], l[8], o[8][D].
    __device__ __forceinline__ void deposit(float* dst, int lane) const {
        const float s = row_sum();
        const int r = lane >> 2;
        if ((lane & 3) == 0) {
            dst[r] = m;
            dst[kHeadRows + r] = s;
        }
        float* o = dst + 2 * kHeadRows + r * D;
        each2(lane, [&](int col, float x, float y) {
            *reinterpret_cast<float2*>(o + col) = make_float2(x, y);
        });
    }

    __device__ __forceinline__ void write_out(const PagedParams& p, int b, int u, int lane) const {
        const float s = row_sum();
        const int row = (u % p.blocks) * kHeadRows + (lane >> 2);
        if (row < p.group) {
            const long long at = (long long)b * p.hq + (u / p.blocks) * p.group + row;
            const float inv = paged_inverse(s);
            if (p.lse && (lane & 3) == 0) p.lse[at] = paged_lse(m, s);
            each2(lane, [&](int col, float x, float y) {
                paged_store2(p, at * D + col, x * inv, y * inv);
            });
        }
        __syncwarp();
    }
};

template <int T, int D, int BOX>
__global__ void __launch_bounds__(PagedCfg<T, D, BOX>::kThreads, 1) paged_decode_kernel(
    const __grid_constant__ PagedParams p) {
    using C = PagedCfg<T, D, BOX>;
    extern __shared__ unsigned char pd_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(pd_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    PagedPiece* pieces = reinterpret_cast<PagedPiece*>(smem + C::kOffPiece);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
    unsigned char* ring = smem + warp * C::ST * C::STAGEB;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * C::ST;
    int4* meta = reinterpret_cast<int4*>(smem + C::kOffMeta) + warp * C::ST;
    unsigned char* queries = smem + C::kOffQ + warp * (C::ST * kHeadRows * C::QROW);
    float* scales = reinterpret_cast<float*>(smem + C::kOffScale) + warp * C::ST * 2 * C::TT;
    float* deposit0 = reinterpret_cast<float*>(smem + C::kOffHead) + warp * C::PART;
    const int units = p.hkv * p.blocks;
    // A warp's barriers are its own: no other warp has to see them.
    if (lane == 0) {
        for (int s = 0; s < C::ST; ++s) mbar_init(full + s, pages_e4m3(T) ? 33 : 1);
        fence_barrier_init();
        prefetch_tmap(&p.tk);
        prefetch_tmap(&p.tv);
    }
    __syncwarp();
    // Launched while the kernel ahead on the stream may still run: nothing is
    // read or written before it has completed, and only then may the next
    // one be launched (so whatever it reads early is older than that).
    pdl_wait_prerequisite();
    pdl_launch_dependents();

    const PagedBatch batch = paged_batch<C::TT>(p);
    const long long total = batch.total;
    const long long workers = min((long long)gridDim.x * C::NW, total / 2);
    const long long w = (long long)blockIdx.x * C::NW + warp;
    const long long x0 = w < workers ? share_begin(total, workers, w) : 0;
    const long long x1 = w < workers ? share_begin(total, workers, w + 1) : 0;
    // The next tile to be issued, and what is left of the share from there on.
    PagedPos pos{};
    long long left = 0;
    auto next_run = [&]() {
        pos.i = 0;
        if (++pos.u == units) {
            pos.u = 0;
            do {
                ++pos.b;
                pos.s = paged_seq<C::TT>(p, pos.b < p.batch ? __ldg(p.lens + pos.b) : 0);
            } while (pos.b < p.batch && pos.s.n == 0);
        }
    };
    if (w < workers) {
        // The first tile at or behind x0.
        pos = paged_find<C::TT>(p, batch, x0);
        const int place = pos.i;
        pos.i = place / 2;
        left = x1 - x0 + place - (2 * pos.i + 1);
        if (pos.i == pos.s.n) {
            --left;
            next_run();
        }
    }
    PagedPiece head{}, tail{};

    // Padded rows of the batch, and lengths out of range.
    auto empty_rows = [&]() {
        for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
            const int len = __ldg(p.lens + b);
            if ((len < 0 || len > p.cap) && threadIdx.x == 0)
                atomicOr(p.ctr + kCtrError, kErrSeqLen);
            if (len > 0) continue;
            for (int i = 2 * threadIdx.x; i < p.hq * D; i += 2 * C::kThreads)
                paged_store2(p, (long long)b * p.hq * D + i, 0.f, 0.f);
            for (int i = threadIdx.x; p.lse && i < p.hq; i += C::kThreads)
                p.lse[(long long)b * p.hq + i] = -INFINITY;
        }
    };

    if (left > 0) {
        const PagedPos start = pos;
        const long long base = x1 - left - (2 * pos.i + 1);  // of its run
        const uint64_t pol = p.blocks == 1 ? l2_evict_first_policy() : l2_evict_normal_policy();
        // A tile comes in boxes of `box` rows, K's and V's; lane i keeps the
        // page of box i.
        const int box = C::SEGS > 1 ? BOX : p.box;
        const int down = C::TT / box;
        const int sub = lane & (down - 1);
        const int from = lane / box, rem = lane % box;
        int page = 0;    // of this lane's box in the next tile to be issued
        int in_page = 0;
        int t0 = 0;      // that tile's first token
        bool need = false;  // a token of that box counts
        auto fetch_page = [&]() {
            t0 = (pos.i < pos.s.a ? pos.i : pos.i + pos.s.f - pos.s.a) * C::TT;
            const int t = t0 + sub * box;
            const int entry = (int)(__umulhi((unsigned)t, p.page_mul) >> p.page_shift);
            in_page = t - entry * p.page_size;
            need = t < pos.s.len &&
                   ((p.S | p.W) == 0 || t < p.S || min(t + box, pos.s.len) > pos.s.len - p.W);
            if (need) page = __ldg(p.table + (long long)pos.b * p.max_pages + entry);
        };
        bool first = true;
        auto issue = [&](int slot) {
            const int tokens = pos.s.len - t0;  // from here on
            const int h = p.blocks == 1 ? pos.u : pos.u / p.blocks;
            unsigned char* stage = ring + slot * C::STAGEB;
            // Boxes outside the set are left out, their pages not looked at: a
            // cache may have given them back.
            const unsigned boxes = __ballot_sync(0xffffffffu, need) & ((1u << down) - 1u);
            if (need && (unsigned)page >= (unsigned)p.n_pages) {
                atomicOr(p.ctr + kCtrError, kErrPage);
                page = 0;
            }
            // The run's queries come with its first tile.
            const int blk = (pos.u - h * p.blocks) * kHeadRows;
            const int rows = C::kCopyQ && (first || pos.i == 0) ? min(kHeadRows, p.group - blk) : 0;
            first = false;
            __syncwarp();
            if (elect_one()) {
                meta[slot] = make_int4(pos.b, pos.u, pos.i, t0);
                mbar_arrive_expect_tx(full + slot,
                                      (uint32_t)(__popc(boxes) * box * 2 * C::RB + rows * 2 * D));
            }
            if constexpr (C::kCopyQ) {
                __syncwarp();
                if (lane < rows)
                    bulk_load(queries + (slot * kHeadRows + lane) * C::QROW,
                              static_cast<const __nv_bfloat16*>(p.q) + pos.b * p.q_stride +
                                  (long long)(h * p.group + blk + lane) * D,
                              2 * D, full + slot, pol);
            }
            for (unsigned some = boxes; some; some &= some - 1u) {
                const int i = __ffs(some) - 1;
                const int pg = __shfl_sync(0xffffffffu, page, i);
                const int in = __shfl_sync(0xffffffffu, in_page, i);
                unsigned char* dst = stage + i * (box * C::RB);
                if (elect_one()) {
                    tma_load_5d(dst, &p.tk, in, h, pg, full + slot, pol);
                    tma_load_5d(dst + C::TILEB, &p.tv, in, h, pg, full + slot, pol);
                }
            }
            if constexpr (pages_e4m3(T)) {
                // Lane = token: its scales, and its arrival once they landed.
                const int pg = __shfl_sync(0xffffffffu, page, from);
                const int in = __shfl_sync(0xffffffffu, in_page, from) + rem;
                if (lane < tokens && (boxes >> from & 1u)) {
                    const long long at = ((long long)pg * p.hkv + h) * p.page_size + in;
                    cp_async_4(scales + slot * 2 * C::TT + lane, p.ks + at);
                    cp_async_4(scales + slot * 2 * C::TT + C::TT + lane, p.vs + at);
                }
                cp_async_arrive(full + slot);
            }
            // On to the next tile; its page numbers are on their way while
            // this one streams.
            left -= 2;
            if (++pos.i == pos.s.n) {
                --left;
                next_run();
            }
            fetch_page();
        };
        fetch_page();
        int issued = 0;
        for (; issued < C::ST && left > 0; ++issued) issue(issued);
        __syncwarp();

        PagedWarp<T, D, BOX> state;
        state.init(lane);
        state.reset();
        if constexpr (!C::kCopyQ) state.load_q(p, start.b, start.u, nullptr, lane);
        PagedSeq s = start.s;
        {
            // What this warp leaves to be joined, and with which CTAs.
            long long y = x1 - 1;
            PagedPos end = paged_find<C::TT>(p, batch, y);
            if (end.i == 0) end = paged_find<C::TT>(p, batch, --y);
            const long long end_base = y - end.i;
            end.i = (end.i - 1) / 2;
            auto piece = [&](PagedPiece& q, const PagedPos& at, long long run, int lo, int hi) {
                q.b = at.b, q.u = at.u, q.n = at.s.n, q.lo = lo, q.hi = hi;
                q.c0 = (int)(share_of(total, workers, run + 1) / C::NW);
                q.c1 = (int)(share_of(total, workers, run + 2 * q.n - 1) / C::NW);
            };
            const bool one = end.b == start.b && end.u == start.u;
            const int lo = one ? start.i : 0;
            if (!one && start.i > 0) piece(head, start, base, start.i, start.s.n);
            if (lo > 0 || end.i + 1 < end.s.n) piece(tail, end, end_base, lo, end.i + 1);
        }
        empty_rows();
        int done = 0, slot = 0;
        uint32_t parity = 0;
        bool lost = false, have0 = false, have1 = false;
        for (; done < issued; ++done) {
            // Bounded wait for the fill.
            if (!__all_sync(0xffffffffu, mbar_try_wait(full + slot, parity))) {
                const uint64_t since = global_ns();
                for (uint32_t it = 1;
                     !__all_sync(0xffffffffu, mbar_try_wait(full + slot, parity)); ++it) {
                    if ((it & 31) == 0 &&
                        __any_sync(0xffffffffu, global_ns() - since > p.timeout_ns)) {
                        lost = true;
                        break;
                    }
                }
                if (lost) break;
            }
            const int4 at = meta[slot];
            if (at.z == 0 && done > 0) {
                s = paged_seq<C::TT>(p, __ldg(p.lens + at.x));
                state.reset();
            }
            if (at.z == 0 ? C::kCopyQ || done > 0 : C::kCopyQ && done == 0)
                state.load_q(p, at.x, at.y, queries + slot * (kHeadRows * C::QROW), lane);
            // Tokens of the set: bit t of the mask.
            const int t = at.w + lane;
            const bool on = t < s.len && ((p.S | p.W) == 0 || t < p.S || t >= s.len - p.W);
            const unsigned mask = __ballot_sync(0xffffffffu, on) & C::kAll;
            unsigned char* stage = ring + slot * C::STAGEB;
            if (mask != C::kAll) {
                // Rows of V that do not count may hold anything: zeros, so
                // that 0 * NaN does not reach the sums.
                if (!on && lane < C::TT) {
                    for (int g = 0; g < C::SEGS; ++g)
                        for (int c = 0; c < C::SEGB; c += 16)
                            *reinterpret_cast<uint4*>(stage + C::TILEB + C::row(lane) +
                                                      g * C::SEG + c) =
                                make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            const float* sc = scales + slot * 2 * C::TT;
            state.tile(smem_addr(stage), mask, sc, sc + C::TT, lane);
            __syncwarp();
            const bool last = left <= 0 && done + 1 == issued;
            if (left > 0) {
                issue(slot);
                ++issued;
            }
            if (++slot == C::ST) {
                slot = 0;
                parity ^= 1u;
            }
            if (last || at.z + 1 == s.n) {
                const bool whole = done >= at.z && at.z + 1 == s.n;
                if (whole) {
                    state.write_out(p, at.x, at.y, lane);
                } else if (last) {
                    state.deposit(reinterpret_cast<float*>(ring), lane);
                    have1 = true;
                } else {
                    state.deposit(deposit0, lane);
                    have0 = true;
                }
            }
        }
        if (lost) {
            // Nothing more is asked for; let what was asked for land (bounded).
            if (lane == 0) atomicOr(p.ctr + kCtrError, kErrTimeout);
            const uint64_t since = global_ns();
            for (int n = done; n < issued; ++n)
                while (!mbar_try_wait(full + n % C::ST, (uint32_t)(n / C::ST) & 1u))
                    if (global_ns() - since > p.timeout_ns) break;
            __syncwarp();
            // Empty partials, so that the joins stay complete.
            state.reset();
            if (!have0) state.deposit(deposit0, lane);
            if (!have1) state.deposit(reinterpret_cast<float*>(ring), lane);
        }
    } else {
        empty_rows();
    }
    if ((long long)blockIdx.x * C::NW >= workers) return;
    if (lane == 0) {
        pieces[2 * warp] = head;
        pieces[2 * warp + 1] = tail;
    }
    __syncthreads();

    // Join what spans warps: runs of pieces of one (sequence, unit).  Piece 2 i
    // is warp i's first run, piece 2 i + 1 its last; every lane holds one.
    auto partial = [&](int i) {
        return reinterpret_cast<const float*>(
            smem + ((i & 1) ? (i >> 1) * (C::ST * C::STAGEB)
                            : C::kOffHead + (i >> 1) * (C::PART * 4)));
    };
    static_assert(2 * C::NW <= 32, "a lane per piece");
    PagedPiece a{};
    if (lane < 2 * C::NW) a = pieces[lane];
    const unsigned there = __ballot_sync(0xffffffffu, a.hi > 0);
    const unsigned before = there & ((1u << lane) - 1u);
    const int prev = before ? 31 - __clz(before) : lane;
    const int pb = __shfl_sync(0xffffffffu, a.b, prev), pu = __shfl_sync(0xffffffffu, a.u, prev);
    const unsigned starts = __ballot_sync(
        0xffffffffu, a.hi > 0 && (before == 0 || pb != a.b || pu != a.u));
    auto rows_of = [&](int u) { return min(kHeadRows, p.group - (u % p.blocks) * kHeadRows); };
    auto head_of = [&](int b, int u) {
        return (long long)b * p.hq + (u / p.blocks) * p.group + (u % p.blocks) * kHeadRows;
    };
    // Lane i holds the run that begins with piece i.  One that began in an
    // earlier CTA is this CTA's first partial, one that goes on in the next
    // its second.  The runs' parts of 128 elements go round the warps.
    const bool begins = (starts >> lane) & 1u;
    const unsigned after = starts & ~((2u << lane) - 1u);
    const unsigned pieces_of =
        there & ~((1u << lane) - 1u) & (after ? (after & -after) - 1u : ~0u);
    const int hi = __shfl_sync(0xffffffffu, a.hi, begins ? 31 - __clz(pieces_of) : lane);
    const bool whole = a.lo == 0 && hi == a.n;
    const int part = a.lo == 0 ? 1 : 0;
    const int open[2] = {__ffs(__ballot_sync(0xffffffffu, begins && !whole && part == 0)) - 1,
                         __ffs(__ballot_sync(0xffffffffu, begins && !whole && part == 1)) - 1};
    const int size = begins ? rows_of(a.u) * D : 0;
    const int parts = (size + 127) / 128;
    const int incl = warp_inclusive(parts);
    const int all = __shfl_sync(0xffffffffu, incl, 31);
    for (int t = warp; t < all; t += C::NW) {
        const int i = __ffs(__ballot_sync(0xffffffffu, incl > t)) - 1;
        const int e = (t - __shfl_sync(0xffffffffu, incl - parts, i)) * 128 + 4 * lane;
        const int b = __shfl_sync(0xffffffffu, a.b, i), u = __shfl_sync(0xffffffffu, a.u, i);
        const int end = __shfl_sync(0xffffffffu, size, i);
        const unsigned run = __shfl_sync(0xffffffffu, pieces_of, i);
        const int dest = __shfl_sync(0xffffffffu, whole ? -1 : part, i);
        if (e >= end) continue;
        const int r = e / D;
        PagedSum sum;
        constexpr int kAhead = 4;  // partials on their way together
        for (unsigned k = run; k;) {
            float m[kAhead], l[kAhead];
            float4 o[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {
                const float* q = partial(k ? __ffs(k) - 1 : i);
                m[n] = k ? q[r] : -INFINITY;
                l[n] = k ? q[kHeadRows + r] : 0.f;
                o[n] = k ? *reinterpret_cast<const float4*>(q + 2 * kHeadRows + e)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
                k &= k - 1;
            }
            sum.add(m, l, o);
        }
        if (dest < 0) {
            sum.write<D>(p, head_of(b, u), e);
        } else {
            float* mine = p.part + ((long long)blockIdx.x * 2 + dest) * C::PART;
            __stcg(reinterpret_cast<float4*>(mine + 2 * kHeadRows + e), sum.o);
            if (e % D == 0) {
                __stcg(mine + r, sum.m);
                __stcg(mine + kHeadRows + r, sum.l);
            }
        }
    }
    if (open[0] < 0 && open[1] < 0) return;
    // The last CTA of a (sequence, unit) to arrive joins it.
    __syncthreads();
    if (threadIdx.x < 2) {
        const int i = threadIdx.x == 0 ? open[0] : open[1];
        int last = 0;
        if (i >= 0) {
            // Releases what the CTA wrote before the barrier, and takes what
            // the others released.
            const int c0 = pieces[i].c0, more = pieces[i].c1 - c0;
            unsigned* ticket = p.ctr + kPagedTickets + c0;
            last = atom_add_acq_rel_gpu(ticket, 1u) == (unsigned)more;
            if (last) *ticket = 0u;
        }
        misc[threadIdx.x] = last;
    }
    __syncthreads();
    // Four elements of a run a thread at a time, of more where a run has more
    // than the CTA has threads: what they read comes from L2, so it is asked
    // for together.
    constexpr int kItems = (kHeadRows * D / 4 + C::kThreads - 1) / C::kThreads;
    constexpr int kAhead = 8;  // partials on their way together
    const int first = misc[0] ? rows_of(pieces[open[0]].u) * D : 0;
    const int both = first + (misc[1] ? rows_of(pieces[open[1]].u) * D : 0);
    for (int x0 = 4 * threadIdx.x; x0 < both; x0 += 4 * kItems * C::kThreads) {
        int e[kItems], c0[kItems], c1[kItems], longest = 0;
        long long head0[kItems];
        PagedSum sum[kItems];
#pragma unroll
        for (int n = 0; n < kItems; ++n) {
            const int x = x0 + 4 * n * C::kThreads;
            const PagedPiece& q = pieces[x < both ? open[x < first ? 0 : 1] : 0];
            e[n] = x < first ? x : x - first;
            c0[n] = q.c0;
            c1[n] = x < both ? q.c1 : -1;
            head0[n] = x < both ? head_of(q.b, q.u) : 0;
            longest = max(longest, c1[n] - c0[n] + 1);
        }
        for (int c = 0; c < longest; c += kAhead) {
            float m[kItems][kAhead], l[kItems][kAhead];
            float4 o[kItems][kAhead];
#pragma unroll
            for (int n = 0; n < kItems; ++n)
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    m[n][k] = -INFINITY, l[n][k] = 0.f, o[n][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    const int cta = c0[n] + c + k;
                    if (cta <= c1[n]) {
                        const float* at = p.part + ((long long)cta * 2 + (c + k == 0)) * C::PART;
                        m[n][k] = __ldcg(at + e[n] / D);
                        l[n][k] = __ldcg(at + kHeadRows + e[n] / D);
                        o[n][k] =
                            __ldcg(reinterpret_cast<const float4*>(at + 2 * kHeadRows + e[n]));
                    }
                }
#pragma unroll
            for (int n = 0; n < kItems; ++n) sum[n].add(m[n], l[n], o[n]);
        }
#pragma unroll
        for (int n = 0; n < kItems; ++n)
            if (c1[n] >= 0) sum[n].template write<D>(p, head0[n], e[n]);
    }
}

}  // namespace alspec
