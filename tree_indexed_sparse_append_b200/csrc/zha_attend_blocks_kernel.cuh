// Gathered attention over an 8-bit cache, and of drafted tokens over any cache: blocks
// of up to 16 walks of one tree share every row they read.
//   out = sum_i softmax_i(beta <q, k_i>) v_i,   lse = logsumexp_i(beta <q, k_i>)
// over a walk's chosen chunks, the tail, and the drafted tokens of its mask row.
//
// The GQA heads of a token, and the tokens of a draft, choose much the same chunks,
// and reading a row for one walk at a time costs its bytes and its decoding again
// for each of them. So a CTA takes (tree, 8 NW walks, part of their keys), an item of a
// plan made from the lists' lengths, by every CTA or by plan_kernel:
//   1. union   the walks' chunk lists set bits of a bitmap over the tree's chunks in
//              shared memory; a scan of its words ranks the chunks, and the CTA's
//              part is a run of ranks (then the tail). Each of its chunks gets a
//              mask of the walks that chose it.
//   2. tiles   each warp takes every WARPS-th tile of 16 keys: K and V rows come as
//              they are stored (cp.async, 16 bytes a lane, two tiles in flight), and go
//              through mma.sync as S^T = K Q^T (m = keys, n = walks) and
//              O^T += V^T P^T (m = columns), with the online softmax in between. The
//              walk's mask takes S to -inf where it did not choose the key.
//   3. merge   the warps' (m, l, O) are merged through shared memory, a warp a walk;
//              a walk whose block has one part is finished here, else the part's row
//              goes to scratch and combine_kernel merges the parts in order (the CTA
//              that ends last doing it, by a ticket, took 2 to 5 us longer).
//              The drafted tokens are more tiles, of the block's last part.
// No atomics on results: every call gives the same bits. mma.sync and not tcgen05: a
// decode step has 4 to 16 walks a tree, an eighth of a tcgen05 tile's 128 rows at most,
// and accumulators that never leave the warp's registers between two tiles. Trees of more
// walks are cut into blocks of 16 all the same, each with its own union: where their
// selections overlap, a row is decoded once a block, and a wider block for tcgen05 would
// decode it once. Keys are the m side, so that 8 walks (the heads of a group) fill an instruction.
//
// Operands. E4M3 codes are exact in fp16, so an 8-bit cache is decoded to fp16 pairs
// in registers; exponents stay outside: 2^e of a key scales its row of S, 2^e of
// a value its weight. A query is scaled by a power of two to below 2^11 and taken as
// one fp16 term when it is bf16 (8 bits: exact down to 2^-24, which is 2^-35 of the
// query's largest element), as two (22 bits) when it is fp32. Weights, scaled by
// 2^7, are one fp16 term (off by at most 2^-11 of themselves, an eighth of the
// rounding of the bf16 result) for a bf16 result and two for an fp32 one. A bf16 or fp32
// cache, and drafted tokens, take bf16 terms: one of a bf16 operand and three of an
// fp32 one (24 bits; of the nine products the six that are not below 2^-24), two
// (2^-17) or three of the weights. All sums, maxima and lse are fp32.
//
// The dot product may take its columns in any order, so a lane reads its K columns
// 16 bytes at a time, and the queries are laid out to match; the columns of V are
// permuted likewise. The 16-byte pieces of a tile's rows are swizzled so that both
// reads are free of bank conflicts.
//
// A value that is not finite reaches every walk of the block through a weight of
// zero (0 * NaN). So a walk with a NaN among its sums is computed again by itself,
// over its own keys (slow_walk): only those that attend to a NaN give NaN. So is a walk
// whose sums are small beside the block's largest values (VSUM_ONE).
//
// Measured, 8-bit cache, d = 128, bf16, 4 heads a KV head: 256 walks of 96 chunks of 8
// over 262,144 keys 19.5 us a call (the item kernel, a walk at a time: 39), 1,024 walks of
// 48 chunks of 16 over 65,536 keys 26.3 us (98), 64 walks of 1,024 chunks of 16 over
// 1,048,573 keys 47.5 us (145). The bytes take 3.7, 0.6 and 19.4 us at the copy rate. What
// bounds it is latency: a CTA of the second spends 11 us on the plan, the lists, the union
// and the merge, chains of dependent steps with barriers, and 6 on tiles; one of the third 14
// on tiles. A tile is some 450 instructions (decoding, 32 mma.sync, the softmax, the copies)
// at 0.5 a cycle and scheduler: four warps a scheduler do not hide all of their chains.
#pragma once

#include <cmath>
#include <type_traits>

#include "zha_attend_blocks.cuh"
#include "zha_internal.cuh"

namespace zha {
namespace {

constexpr int KEYS_MIN = 512;      // keys per item, at least
constexpr int KEYS_LONG = 4096;    // the same in calls of many blocks
constexpr int WINDOW = 1024;       // chunks whose ids and masks are held at a time
// weights are below e^NEAR < 2^8, and are scaled by 2^PSHIFT before they are rounded to fp16
constexpr float NEAR = 5.5f;
constexpr int PSHIFT = 7;
constexpr float LOG2E = 1.4426950408889634f;
// An 8-bit cache's weights are scaled by 2^(PSHIFT + e - vref) before they are rounded: e the
// value's power of two, vref the largest that the warp has met, any walk's. fp16 ends at 2^-24,
// so a small one is rounded to a multiple of that, and not to its own 11 bits (22 of two terms).
// Where no value of a part is more than 2^VFAR below the largest, that is an error of at most
// 2^-20 (2^-24) of the walk's heaviest weight, which is 1 or more. Where some are, what a walk
// has lost shows in its sums: a code is at most 448, so a key adds an error of at most 448 * 2^-25
// to a sum, 2^-18 (2^-22) of the walk's largest if that is 2^VSUM or more. A walk whose sums are
// all smaller is computed by itself.
constexpr int VFAR_ONE = 12, VFAR_TWO = 8;
constexpr int VSUM_ONE = 2, VSUM_TWO = 6;

// NW: groups of 8 walks a block. FAST: bf16 queries and results (an 8-bit or bf16 cache):
// one term of the query, one (8-bit) or two of a weight, summed in the accumulators. DRAFT:
// there may be drafted tokens. One kernel for all of it spilled registers at d = 128.
template <typename KT, int D, int NW, bool FAST, bool DRAFT>
struct Cfg {
    static constexpr bool F8 = sizeof(KT) == 1;
    static constexpr int BW = 8 * NW;                 // walks per block
    static constexpr int ROWB = D * (int)sizeof(KT);  // bytes per row
    static constexpr int PPR = ROWB / 16;             // 16-byte pieces per row
    static constexpr int PC = 16 / (int)sizeof(KT);   // columns of a piece
    static constexpr int WARPS = ROWB <= 256 ? 8 : ROWB <= 512 ? 4 : 2;
    static constexpr int STAGES = 2;
    static constexpr int TILE = 2 * 16 * ROWB;        // K and V of 16 keys
    static constexpr int RING = WARPS * STAGES * TILE;
    static constexpr int MT = D / 16;                 // accumulator tiles of 16 columns
    static constexpr int MS = D + 4;                  // floats of a merged row (2 MS = 8 mod 32 banks)
    static constexpr int MERGE = WARPS * BW * MS * 4; // the warps' sums
    static constexpr int BODY = RING > MERGE ? RING : MERGE;
    static constexpr int QBYTES = NW * (D / 16) * 256;  // one term of the block's queries
    static constexpr int QTERMS = FAST ? 1 : F8 ? 2 : 3;
    static constexpr int DTERMS = F8 && DRAFT ? (FAST ? 1 : 3) : 0;  // bf16 terms kept beside the fp16 ones, for the drafted tokens
    static constexpr int FIXED = BODY + QTERMS * QBYTES + 8 * WINDOW;  // but for the bitmap, its ranks and the DTERMS
    static_assert(FIXED + DTERMS * QBYTES + BLOCK_CHUNKS_MAX / 32 * 8 + 9 * 1024 <= 227 * 1024, "shared memory of an SM");
    static_assert(WARPS * 4 >= BW, "every walk has one of the first runs of list entries");
    static_assert(BODY / WARPS >= 16 * D * 4, "a warp stages 16 drafted rows: bf16 K and V, or fp32 K or V");
    static constexpr int MIN_CTAS = MT * 4 * NW <= 64 && BODY <= 80 * 1024 ? 2 : 1;
    // columns of a lane's run in V: row r < 8 of accumulator tile j is column
    // (j / (RUN / 2)) * 8 RUN + r RUN + 2 (j % (RUN / 2)), row r + 8 the one after it
    static constexpr int RUN = F8 && D > 64 ? 16 : sizeof(KT) == 4 ? 4 : 8;
    static constexpr int KTERMS = sizeof(KT) == 4 ? 3 : 1;  // operand terms of a cached value
};

__device__ __forceinline__ uint32_t s_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// A tile's rows follow each other, their 16-byte pieces swizzled: piece q of row r lies at
// q ^ twist(r) of the row (of the 128-byte line of two rows, when a row has 4 pieces).
// twist() is linear over the bits of r, so an access's place is one lane constant, an
// XOR and a sum with constants of the unrolled loops.
template <int PPR>
__host__ __device__ constexpr int twist(int r) {
    return PPR == 4 ? (((r >> 1) & 3) << 1) ^ ((r & 1) << 2) : ((r & 1) << 2) ^ (r & 2) ^ (r & 4);
}
// Bytes from the tile's start to piece q of row r (r, q of the lane), without the
// twists of constant rows.
template <int PPR>
__device__ __forceinline__ int place_of(int r, int q) {
    return (PPR == 4 ? (r >> 1) * 128 : r * PPR * 16) + ((q ^ twist<PPR>(r)) << 4);
}

// the codes of a word as two fp16 pairs
__device__ __forceinline__ void codes_half2(unsigned w, unsigned &lo, unsigned &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

template <bool F8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint4 &a, unsigned b0, unsigned b1) {
    if constexpr (F8)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// 8 x 8 b16 blocks across the warp, transposed
__device__ __forceinline__ unsigned transpose8(unsigned x) {
    unsigned y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// x, y rounded to the operand type as a pair, and what the rounding left of them.
template <bool F8>
__device__ __forceinline__ unsigned take_term(float &x, float &y) {
    if constexpr (F8) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        x -= f.x;
        y -= f.y;
        return *reinterpret_cast<const unsigned *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        x -= __bfloat162float(h.x);
        y -= __bfloat162float(h.y);
        return *reinterpret_cast<const unsigned *>(&h);
    }
}

__device__ __forceinline__ unsigned half2_pair(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const unsigned *>(&h);
}

// e^x for x <= NEAR (relative error 2^-22 + |x| 2^-23; 0 at -inf, NaN at NaN). Scores stay
// in natural units until the reference is taken from them: in units of log 2 the
// conversion's own factor would round a large score once more.
__device__ __forceinline__ float exp_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * LOG2E));
    return y;
}

__device__ __forceinline__ float load_q(const BlockArgs &a, long long at) {
    return a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.Q)[at]) : static_cast<const float *>(a.Q)[at];
}

// N columns of a drafted row
template <int N>
__device__ __forceinline__ void load_cols(const void *base, int bf16, long long at, float (&x)[N]) {
    constexpr int B = N < 8 ? N : 8;
    if (bf16) {
#pragma unroll
        for (int i = 0; i < N; i += B) {
            float y[B];
            load_cached<B>(static_cast<const __nv_bfloat16 *>(base) + at + i, y);
#pragma unroll
            for (int c = 0; c < B; ++c) x[i + c] = y[c];
        }
    } else if constexpr (N == 2) {
        const float2 v = __ldg(reinterpret_cast<const float2 *>(static_cast<const float *>(base) + at));
        x[0] = v.x;
        x[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at + i));
            x[i] = v.x;
            x[i + 1] = v.y;
            x[i + 2] = v.z;
            x[i + 3] = v.w;
        }
    }
}

// A warp ends a walk: m, l and o (this lane's D / 32 columns, from
// column lane * D / 32).
template <int D>
__device__ __forceinline__ void finish_walk(const BlockArgs &a, long long walk, int lane, float m, float l,
                                            const float (&o)[D / 32]) {
    constexpr int N = D / 32;
    const bool empty = l == 0.f;
    const float inv = empty ? 0.f : 1.f / l;
    float r[N];
#pragma unroll
    for (int c = 0; c < N; ++c) r[c] = empty ? 0.f : o[c] * inv;
    if (!a.o_vec) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
            if (a.out_bf16) from_float(r[c], static_cast<__nv_bfloat16 *>(a.out) + walk * D + lane * N + c);
            else static_cast<float *>(a.out)[walk * D + lane * N + c] = r[c];
        }
    } else if (a.out_bf16) {
        unsigned *p = reinterpret_cast<unsigned *>(static_cast<__nv_bfloat16 *>(a.out) + walk * D + lane * N);
#pragma unroll
        for (int c = 0; c < N; c += 2) p[c / 2] = bf16_pair(r[c], r[c + 1]);
    } else {
        float2 *p = reinterpret_cast<float2 *>(static_cast<float *>(a.out) + walk * D + lane * N);
#pragma unroll
        for (int c = 0; c < N; c += 2) p[c / 2] = make_float2(r[c], r[c + 1]);
    }
    if (lane == 0 && a.lse) a.lse[walk] = empty ? -INFINITY : m + logf(l);
}

// Shared memory of a CTA, in order: the body (ring of tiles, then the warps' sums),
// the queries, the bitmap, its words' ranks, the window's chunk ids
// and walk masks.
template <typename C>
struct Smem {
    unsigned char *body;
    uint2 *q, *qd;
    unsigned *bits, *pre, *mask;
    int *ids;
    __device__ Smem(unsigned char *base, const BlockArgs &a) {
        body = base;
        q = reinterpret_cast<uint2 *>(base + C::BODY);
        qd = q + C::QTERMS * (C::QBYTES / 8);
        bits = reinterpret_cast<unsigned *>(qd + C::DTERMS * (C::QBYTES / 8));
        pre = bits + a.words;
        ids = reinterpret_cast<int *>(pre + a.words);
        mask = reinterpret_cast<unsigned *>(ids + WINDOW);
    }
};

// A chunk's rank in the block's union.
__device__ __forceinline__ int rank_of(const unsigned *bits, const unsigned *pre, int c) {
    return (int)(pre[c >> 5] + __popc(bits[c >> 5] & ((1u << (c & 31)) - 1u)));
}

// Place of the n-th set bit (n from 0, below the number of them).
__device__ __forceinline__ int nth_bit(unsigned x, int n) {
    for (; n > 0; --n) x &= x - 1;
    return __ffs(x) - 1;
}

// Block-wide exclusive scan; returns the total. sh: one int a warp.
__device__ __forceinline__ int scan_block(int &x, int *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sh[warp] = inc;
    __syncthreads();
    int sums = lane < nwarps ? sh[lane] : 0;  // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, sums, o);
        if (lane >= o) sums += y;
    }
    x = inc - x + (warp ? __shfl_sync(FULL, sums, warp - 1) : 0);
    __syncthreads();
    return __shfl_sync(FULL, sums, 31);
}

// Keys of a block, before its union is known. Its walks' lists together, if no two share a
// chunk, which is what few blocks are planned by (an item too many is an idle SM's); of
// many blocks the longest list, or a quarter of all.
__device__ __forceinline__ int block_keys(const BlockArgs &a, int blk) {
    const int tree = blk / a.nb, g0 = (blk - tree * a.nb) * a.bw, nw = min(a.bw, a.G - g0);
    const int *cnt = a.sel_count + (long long)tree * a.G + g0;
    long long sum = 0;
    int top = 0;
#pragma unroll 8
    for (int w = 0; w < nw; ++w) {
        const int n = min(max(__ldg(cnt + w), 0), a.max_sel);
        sum += n;
        top = max(top, n);
    }
    if (a.many) sum = max((long long)top, sum / 4);
    return (int)(min(sum, (long long)a.n1) * a.C + a.tail);
}

// Cuts blocks into items of about `len` keys, so that a few long lists do not keep the
// GPU waiting: len is the call's keys over the items aimed at. Thread t plans blocks
// t * per .. ; item offsets go to off [NB + 1]. Returns the number of items. The whole CTA.
__device__ __forceinline__ int plan_blocks(const BlockArgs &a, int *off, int *sh, long long *sh_sum) {
    const int tid = threadIdx.x, nt = blockDim.x, per = (a.NB + nt - 1) / nt;
    const int b0 = min(a.NB, tid * per), b1 = min(a.NB, b0 + per);
    long long keys = 0;
    for (int b = b0; b < b1; ++b) {
        const int k = block_keys(a, b);
        off[b] = k;
        keys += k;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) keys += __shfl_xor_sync(FULL, keys, o);
    if ((tid & 31) == 0) sh_sum[tid >> 5] = keys;
    __syncthreads();
    keys = (tid & 31) < nt >> 5 ? sh_sum[tid & 31] : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) keys += __shfl_xor_sync(FULL, keys, o);
    const int len = (int)max((long long)(a.many ? KEYS_LONG : KEYS_MIN), (keys + a.target - 1) / a.target);
    int items = 0;
    for (int b = b0; b < b1; ++b) items += max(1, (off[b] + len - 1) / len);
    const int total = scan_block(items, sh);
    for (int b = b0; b < b1; ++b) {
        const int n = max(1, (off[b] + len - 1) / len);
        off[b] = items;
        items += n;
    }
    if (tid == 0) off[a.NB] = total;
    __syncthreads();
    return total;
}

// The block's lists as runs of 32 entries. The first LIST_U runs a warp takes are loaded
// before the counts are known (entries behind a count are unspecified, not out of
// range), `per` runs a walk, and stay in registers. The runs behind those are cut into one
// stretch a warp, LIST_U loaded before any is used; as many as the body has room for
// (it has no tiles yet) are left there for the first window, chunk and walk in a word.
// Long lists make this the setup's cost: a decode step over 262,144 keys, its longest list
// 7,237 chunks, takes 39 us, and took 48 with the runs dealt to the warps in turn (a
// search for the walk a run) and loaded again for the window.
constexpr int LIST_U = 4;
constexpr int WALK_SHIFT = 18, CHUNK_MASK = (1 << WALK_SHIFT) - 1;
static_assert(BLOCK_CHUNKS_MAX < CHUNK_MASK, "a word holds a chunk and a walk, and CHUNK_MASK is no chunk");
template <int BW>
struct Lists {
    int per;                   // first runs of a walk
    int w[LIST_U], c[LIST_U];  // this lane's first entries: walk (-1: none) and chunk
    int have, upto, total;     // count of walk `lane`; runs behind the first, of walks 0 .. lane and of all
    __device__ __forceinline__ void load(const BlockArgs &a, const int *row0, int nw) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, runs = (blockDim.x >> 5) * LIST_U;
        per = max(1, runs >> (32 - __clz(nw - 1)));  // runs over the next power of two from nw
#pragma unroll
        for (int u = 0; u < LIST_U; ++u) {
            const int run = warp * LIST_U + u, wk = run / per, at = (run - wk * per) * 32 + lane;
            w[u] = wk < nw && at < a.max_sel ? wk : -1;
            c[u] = w[u] >= 0 ? __ldg(row0 + (long long)wk * a.max_sel + at) : 0;
        }
    }
    // once the counts are known
    __device__ __forceinline__ void bound(const int *cnt) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int u = 0; u < LIST_U; ++u) {
            const int run = warp * LIST_U + u;
            if (w[u] >= 0 && (run - w[u] * per) * 32 + lane >= cnt[w[u]]) w[u] = -1;
        }
        have = lane < BW ? cnt[lane] : 0;
        upto = max(have - per * 32 + 31, 0) >> 5;
#pragma unroll
        for (int o = 1; o < BW; o <<= 1) {
            const int y = __shfl_up_sync(FULL, upto, o);
            if (lane >= o) upto += y;
        }
        total = __shfl_sync(FULL, upto, BW - 1);
    }
    // f(run, walk, chunk) for the first entries; walk < 0: none
    template <typename F>
    __device__ __forceinline__ void first(F f) const {
#pragma unroll
        for (int u = 0; u < LIST_U; ++u) f((int)(threadIdx.x >> 5) * LIST_U + u, w[u], c[u]);
    }
    // f(run, walk, chunk) for this warp's stretch of the runs from `from`; walk < 0: no entry
    template <typename F>
    __device__ __forceinline__ void rest(const BlockArgs &a, const int *row0, int from, F f) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5, n = total - from;
        if (n <= 0) return;
        const int r0 = from + (int)((long long)n * warp / nwarps), r1 = from + (int)((long long)n * (warp + 1) / nwarps);
        if (r0 >= r1) return;
        int wk = __popc(__ballot_sync(FULL, lane < BW && upto <= r0));  // r0 < total: below BW
        int end = __shfl_sync(FULL, upto, wk), count = __shfl_sync(FULL, have, wk);
        int start = wk ? __shfl_sync(FULL, upto, wk - 1) : 0;
        const int *row = row0 + (long long)wk * a.max_sel;
#pragma unroll 1
        for (int run = r0; run < r1; run += LIST_U) {
            int x[LIST_U], y[LIST_U];
#pragma unroll
            for (int u = 0; u < LIST_U; ++u) {
                if (run + u < r1) {
                    while (run + u >= end) {  // end < total here: there is a next walk
                        ++wk;
                        start = end;
                        end = __shfl_sync(FULL, upto, wk);
                        count = __shfl_sync(FULL, have, wk);
                        row += a.max_sel;
                    }
                    const int at = (per + run + u - start) * 32 + lane;
                    x[u] = at < count ? wk : -1;
                    y[u] = at < count ? __ldg(row + at) : 0;
                }
            }
#pragma unroll
            for (int u = 0; u < LIST_U; ++u)
                if (run + u < r1) f(run + u, x[u], y[u]);
        }
    }
};

// What a tile's key is: its row in the tree's cache (-1: none) and the walks that chose it.
struct KeyInfo {
    int row;
    unsigned walks;
};
struct Part {
    int tree, nw;               // nw: walks of the block
    long long walk0;
    int U, KT;                  // chunks in the union, U * C + tail keys
    int k0, k1;                 // the part's keys
    int r0, r1;                 // ranks in the window
};
__device__ __forceinline__ KeyInfo key_info(const BlockArgs &a, const Part &p, const int *ids, const unsigned *mask,
                                            int kp, int end) {
    KeyInfo k{-1, 0u};
    if (kp >= end) return k;
    const int chunked = p.U * a.C;
    if (kp < chunked) {
        const int ci = a.c_shift >= 0 ? kp >> a.c_shift : kp / a.C;
        k.row = ids[ci - p.r0] * a.C + (kp - ci * a.C);
        k.walks = mask[ci - p.r0];
    } else {
        k.row = a.n1 * a.C + (kp - chunked);
        k.walks = FULL;
    }
    return k;
}

// The ids and walks of the window's ranks r0 .. r1 - 1; every list writes its chunks' ids. held:
// runs that the union left in the ring (left), 0 when tiles have been there since. ends: the
// part's first and last chunk. Not inlined: what it needs is not held over the tiles, whose loop
// has no register to spare.
template <int BW, int FIRST, int ROOM>
__device__ __noinline__ void fill_window(const BlockArgs &a, const unsigned *left, const unsigned *bits, const unsigned *pre,
                                         int *ids, unsigned *mask, int r0, int r1, const int *row0, int nw,
                                         const int *cnt, const int *ends, int held) {
    const int lo = ends[0], hi = ends[1];
    auto take = [&](int, int w, int c) {
        if (w < 0 || c < lo || c > hi) return;
        const int r = rank_of(bits, pre, c);
        if (r >= r0 && r < r1) {
            ids[r - r0] = c;
            atomicOr(mask + (r - r0), 1u << w);
        }
    };
#pragma unroll 4
    for (int i = threadIdx.x; i < held * 32; i += blockDim.x) take(0, (int)(left[i] >> WALK_SHIFT), (int)(left[i] & CHUNK_MASK));
    if (held > 0 && held < ROOM) return;  // all of them
    Lists<BW> lists;
    lists.load(a, row0, nw);
    lists.bound(cnt);
    if (held == 0) lists.first(take);
    lists.rest(a, row0, held == 0 ? 0 : ROOM - FIRST, take);
}

// The mask row of walk w of the block.
__device__ __forceinline__ const unsigned char *mask_row(const BlockArgs &a, const Part &p, int w) {
    const int nd = a.n_draft;
    return a.mask + ((long long)(p.tree / a.H_kv) * nd + (int)((p.walk0 + w) % nd)) * nd;
}

// One walk over the part's keys that it chose, by a warp on the CUDA cores with fp32 weights:
// the way of a walk whose sums hold a NaN, which may be another walk's, or have lost too much.
template <typename KT, int D, typename S>
__device__ __noinline__ void slow_walk(const BlockArgs &a, const Part &p, const S &s, int w, int cnt, bool drafted,
                                       float &m, float &l, float (&o)[D / 32]) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const KT *K = static_cast<const KT *>(a.K) + p.tree * a.cap * D + lane * N;
    const KT *V = static_cast<const KT *>(a.V) + p.tree * a.cap * D + lane * N;
    float q[N];
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        q[c] = load_q(a, (p.walk0 + w) * D + lane * N + c);
        o[c] = 0.f;
    }
    auto add = [&](const float (&kx)[N], const float (&vx)[N]) {
        float d = 0.f;
#pragma unroll
        for (int c = 0; c < N; ++c) d = fmaf(kx[c], q[c], d);
        const float sc = warp_sum(d) * a.beta;
        const float mx = fmaxf(m, sc), ref = mx == -INFINITY ? 0.f : mx;
        const float scale = exp_of(m - ref), pw = exp_of(sc - ref);
        l = l * scale + pw;
#pragma unroll
        for (int c = 0; c < N; ++c) o[c] = fmaf(pw, vx[c], o[c] * scale);
        m = mx;
    };
    auto key = [&](long long row) {
        float kx[N], vx[N];
        const unsigned char *ke = nullptr, *ve = nullptr;
        if constexpr (sizeof(KT) == 1) {
            ke = a.Ks + p.tree * a.cap + row;
            ve = a.Vs + p.tree * a.cap + row;
        }
        load_row<N>(K + row * D, ke, kx);
        load_row<N>(V + row * D, ve, vx);
        add(kx, vx);
    };
    const int *list = a.sel + (p.walk0 + w) * a.max_sel;
    for (int i = 0; i < cnt; ++i) {
        const int c = __ldg(list + i);
        if (c < 0 || c >= a.n1) continue;
        const int kp = rank_of(s.bits, s.pre, c) * a.C;
        for (int j = max(0, p.k0 - kp); j < min(a.C, p.k1 - kp); ++j) key((long long)c * a.C + j);
    }
    for (int kp = max(p.k0, p.U * a.C); kp < p.k1; ++kp) key((long long)a.n1 * a.C + (kp - p.U * a.C));
    if (!drafted) return;
    const unsigned char *mrow = mask_row(a, p, w);
    for (int j = 0; j < a.n_draft; ++j) {
        if (!__ldg(mrow + j)) continue;
        float kx[N], vx[N];
        load_cols<N>(a.kd, a.d_bf16, ((long long)p.tree * a.n_draft + j) * D + lane * N, kx);
        load_cols<N>(a.vd, a.d_bf16, ((long long)p.tree * a.n_draft + j) * D + lane * N, vx);
        add(kx, vx);
    }
}

template <typename KT, int D, int NW, bool FAST, bool DRAFT>
__global__ void __launch_bounds__(Cfg<KT, D, NW, FAST, DRAFT>::WARPS * 32, Cfg<KT, D, NW, FAST, DRAFT>::MIN_CTAS)
    attend_block_kernel(const __grid_constant__ BlockArgs a) {
    chain_start();
    using C = Cfg<KT, D, NW, FAST, DRAFT>;
    constexpr bool F8 = C::F8;
    constexpr int BW = C::BW, MT = C::MT, PPR = C::PPR, WARPS = C::WARPS, STAGES = C::STAGES, THREADS = WARPS * 32;
    constexpr int KP = C::ROWB / 64;     // K pieces of a lane per key
    constexpr int KSP = C::PC / 4;       // k-steps of 16 columns per piece
    constexpr int KS = D / 16;
    constexpr int KTERMS = C::KTERMS, PT = F8 ? (FAST ? 1 : 2) : FAST ? 2 : 3;  // terms of a value, and of a weight at most
    constexpr int N = D / 32, HR = C::RUN / 2;
    extern __shared__ __align__(128) unsigned char smem_blocks[];
    __shared__ int s_cnt[BW];
    __shared__ int s_scan[WARPS];
    __shared__ int s_ends[2];            // the part's first and last chunk
    __shared__ float s_up[BW];           // the power of two that a walk's query is scaled by
    __shared__ float s_m[WARPS][BW], s_l[WARPS][BW];
    __shared__ int s_vmax[WARPS], s_vmin[WARPS];
    __shared__ uint2 s_meta[WARPS][STAGES][16];
    const Smem<C> s(smem_blocks, a);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    // the item: a block and a part of it
    const int item = (int)blockIdx.x;
    int blk = item, part = 0, parts = 1;
    if (a.target) {
        int first;
        if (a.item_blk) {
            blk = __ldcg(a.item_blk + item);
            if (blk < 0) {
                chain_done();
                return;
            }
            first = __ldcg(a.first + blk);
            parts = __ldcg(a.first + blk + 1) - first;
        } else {
            __shared__ int s_off[PLAN_LOCAL + 1];
            __shared__ long long s_sum[WARPS];
            const int items = plan_blocks(a, s_off, s_scan, s_sum);
            if (item >= items) {
                chain_done();
                return;
            }
            int lo = 0, hi = a.NB;  // s_off[lo] <= item < s_off[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_off[mid] <= item) lo = mid;
                else hi = mid;
            }
            blk = lo;
            first = s_off[blk];
            parts = s_off[blk + 1] - first;
            if (item == first && tid == 0) a.first[blk] = first;
        }
        part = item - first;
    }
    Part p;
    p.tree = blk / a.nb;
    const int g0 = (blk - p.tree * a.nb) * BW;
    p.walk0 = (long long)p.tree * a.G + g0;
    p.nw = min(BW, a.G - g0);

    // the first list entries and the counts
    const int *row0 = a.sel + p.walk0 * a.max_sel;
    Lists<BW> lists;
    lists.load(a, row0, p.nw);
    int my_cnt = 0;
    if (lane < p.nw) my_cnt = min(max(__ldg(a.sel_count + p.walk0 + lane), 0), a.max_sel);
    // the queries, 16 lanes a walk, on their way beside the lists
    constexpr int QC = D / 16, QW = 2 * WARPS, QP = (BW + QW - 1) / QW;
    float qx[QP][QC];
#pragma unroll
    for (int pass = 0; pass < QP; ++pass) {
        const int w = pass * QW + 2 * warp + (lane >> 4);
        const long long at = (p.walk0 + w) * D + (lane & 15) * QC;
        if (w >= p.nw) {
#pragma unroll
            for (int c = 0; c < QC; ++c) qx[pass][c] = 0.f;
        } else if (a.q_vec) {
            load_cols<QC>(a.Q, a.q_bf16, at, qx[pass]);
        } else {
#pragma unroll
            for (int c = 0; c < QC; ++c) qx[pass][c] = load_q(a, at + c);
        }
    }
    if (tid < BW) s_cnt[tid] = my_cnt;
    for (int i = tid; i < a.words; i += THREADS) s.bits[i] = 0u;
    __syncthreads();

    // 1. union of the walks' chunks
    lists.bound(s_cnt);
    constexpr int FIRST = WARPS * LIST_U, ROOM = C::BODY / 128;  // runs
    auto enter = [&](int run, int w, int c) {
        const bool good = w >= 0 && c >= 0 && c < a.n1;
        if (good) atomicOr(s.bits + (c >> 5), 1u << (c & 31));
        else if (w >= 0) report(a.status, DEV_BAD_INDEX);
        if (run < ROOM) reinterpret_cast<unsigned *>(s.body)[run * 32 + lane] = good ? (unsigned)(c | w << WALK_SHIFT) : (unsigned)CHUNK_MASK;
    };
    lists.first(enter);
    lists.rest(a, row0, 0, [&](int run, int w, int c) { enter(FIRST + run, w, c); });
    const int held = min(FIRST + lists.total, ROOM);
    // the queries in fragment order
    const int q_terms = FAST || a.q_bf16 ? 1 : C::QTERMS;
#pragma unroll
    for (int pass = 0; pass < QP; ++pass) {
        const int w = pass * QW + 2 * warp + (lane >> 4), ql = lane & 15;
        if (w >= BW) continue;  // the same for both halves of a warp
        float (&x)[QC] = qx[pass];
        float up = 1.f;
        if constexpr (F8) {
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < QC; ++c) top = fmaxf(top, fabsf(x[c]));
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
            // max|q| * 2^e in [2^10, 2^11)
            const int e = 10 - ((int)(__float_as_uint(top) >> 23) - 127);
            if (top > 0.f && top < INFINITY) up = __uint_as_float((unsigned)(127 + (e > 100 ? 100 : e < -118 ? -118 : e)) << 23);
        }
        if (ql == 0) s_up[w] = up;
        // 4 columns at a time
#pragma unroll
        for (int c = 0; c < QC; c += 4) {
            const int col = ql * QC + c, piece = col / C::PC;
            const int ks = (piece >> 2) * KSP + (col % C::PC) / 4;
            const int at2 = ((w >> 3) * KS + ks) * 32 + (w & 7) * 4 + (piece & 3);
            float y[4] = {x[c] * up, x[c + 1] * up, x[c + 2] * up, x[c + 3] * up};
            if constexpr (F8 && DRAFT) {
                float z[4] = {y[0], y[1], y[2], y[3]};
                for (int term = 0; term < (FAST || a.q_bf16 ? 1 : 3); ++term) {
                    const unsigned lo = take_term<false>(z[0], z[1]), hi = take_term<false>(z[2], z[3]);
                    s.qd[term * NW * KS * 32 + at2] = make_uint2(lo, hi);
                }
            }
            for (int term = 0; term < q_terms; ++term) {
                const unsigned lo = take_term<F8>(y[0], y[1]), hi = take_term<F8>(y[2], y[3]);
                s.q[term * NW * KS * 32 + at2] = make_uint2(lo, hi);
            }
        }
    }
    __syncthreads();
    // ranks: the words' popcounts, scanned
    const int wper = (a.words + THREADS - 1) / THREADS, wb = min(a.words, tid * wper), we = min(a.words, wb + wper);
    int before = 0;
    for (int w = wb; w < we; ++w) before += __popc(s.bits[w]);
    p.U = scan_block(before, s_scan);
    p.KT = p.U * a.C + a.tail;
    // the union may be shorter than the lists: fewer parts then, of KEYS_MIN keys at least
    int len = parts == 1 ? p.KT : (int)(((unsigned)p.KT + parts - 1) / (unsigned)parts);
    len = len < KEYS_MIN ? KEYS_MIN : (len + 16 * WARPS - 1) & ~(16 * WARPS - 1);
    const int np = p.KT > len ? (int)(((unsigned)p.KT + len - 1) / (unsigned)len) : 1;
    if (part >= np) {
        chain_done();
        return;
    }
    if (part == 0 && tid == 0 && a.target) a.np[blk] = np;
    p.k0 = part * len;  // part < np: below KT
    p.k1 = p.KT - p.k0 < len ? p.KT : p.k0 + len;
    const int rA = min(p.U, a.c_shift >= 0 ? p.k0 >> a.c_shift : p.k0 / a.C);
    int rB = a.c_shift >= 0 ? p.k1 >> a.c_shift : p.k1 / a.C;
    rB = min(p.U, rB + (rB * a.C < p.k1));
    for (int w = wb; w < we; ++w) {
        s.pre[w] = (unsigned)before;
        const unsigned bits = s.bits[w];
        const int n = __popc(bits);
        // the part's first and last chunk
        if (rA < rB && rA >= before && rA < before + n) s_ends[0] = 32 * w + nth_bit(bits, rA - before);
        if (rA < rB && rB > before && rB <= before + n) s_ends[1] = 32 * w + nth_bit(bits, rB - 1 - before);
        before += n;
    }

    // 2. tiles of 16 keys
    const int p_terms = FAST ? PT : a.out_bf16 ? (F8 ? 1 : 2) : (F8 ? 2 : 3);
    unsigned char *ring = s.body + warp * (STAGES * C::TILE);
    const uint32_t ring_s = s_addr(ring);
    // this lane's piece of each copy, and its places in a tile: pieces it copies (put0), K
    // (get_k: row g, piece t4) and V (get_v: row 2 t4, its run; the next row's run is at
    // 64 bytes' XOR, in the next row)
    const char *Kt = static_cast<const char *>(a.K) + p.tree * a.cap * C::ROWB + lane % PPR * 16;
    const char *Vt = static_cast<const char *>(a.V) + p.tree * a.cap * C::ROWB + lane % PPR * 16;
    const int put0 = place_of<PPR>(lane / PPR, lane % PPR);
    const int get_k = place_of<PPR>(g, t4);
    const int get_v = PPR == 4 ? place_of<PPR>(2 * t4, g >> 1) + (g & 1) * 8 : place_of<PPR>(2 * t4, g);
    constexpr int ROW8 = 8 * C::ROWB;                // rows r and r + 8 have one twist
    constexpr int ROW1 = PPR == 4 ? 0 : C::ROWB;
    const unsigned char *Kst = F8 ? a.Ks + p.tree * a.cap : nullptr, *Vst = F8 ? a.Vs + p.tree * a.cap : nullptr;
    float acc[MT][NW][4];  // rows g, g + 8 of the tile's columns; walks 2 t4, 2 t4 + 1 of group n
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[j][n][c] = 0.f;
    float m[NW][2], ref[NW][2], l[NW][2], rs[NW][2];  // ref: m, or 0 before there is one
#pragma unroll
    for (int n = 0; n < NW; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            m[n][c] = -INFINITY;
            ref[n][c] = l[n][c] = 0.f;
            rs[n][c] = a.beta / s_up[n * 8 + 2 * t4 + c];
        }
    int vref = 1;  // exponent byte that the sums of values are scaled by
    int vlow = 255;  // the least of this lane's rows

    // Online softmax of a tile: sc (keys g, g + 8) becomes the weights, scaled
    // as V is. walks: of the two keys, shifted down by 2 t4; kf: their powers of two; ve:
    // their V exponent bytes; vtop: the largest of the tile's. The reference m of a walk's weights
    // follows its maximum only when that is NEAR above it, so most tiles take no maximum
    // across lanes and rescale nothing (weights are at most e^NEAR).
    auto soften = [&](float (&sc)[NW][4], const unsigned (&walks)[2], const float (&kf)[2], const int (&ve)[2], int vtop) {
        const bool upv = F8 && vtop > vref;
        bool up = upv;
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float x = sc[n][c] * (F8 ? kf[c >> 1] * rs[n][c & 1] : rs[n][c & 1]);
                sc[n][c] = walks[c >> 1] & (1u << (8 * n + (c & 1))) ? x : -INFINITY;
                up |= sc[n][c] > m[n][c & 1] + NEAR;
            }
        if (__any_sync(FULL, up)) {
            float fv = 1.f;
            if (upv) {
                fv = exp_byte((unsigned)max(127 - (vtop - vref), 0));
                vref = vtop;
            }
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                float f[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = fmaxf(sc[n][c], sc[n][c + 2]);
#pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
                    const bool on = mx > m[n][c] + NEAR;
                    f[c] = on ? exp_of(m[n][c] - mx) : 1.f;
                    if (on) m[n][c] = ref[n][c] = mx;
                    l[n][c] *= f[c];
                    f[c] *= fv;
                }
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[j][n][c] *= f[c & 1];
            }
        }
        float pf[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)  // 2^(e of the value - vref + PSHIFT)
            pf[h] = F8 ? exp_byte((unsigned)max(127 + PSHIFT + ve[h] - vref, 0)) : 1.f;
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sc[n][c] = exp_of(sc[n][c] - ref[n][c & 1]);
                l[n][c & 1] += sc[n][c];
                if constexpr (F8) sc[n][c] *= pf[c >> 1];
            }
    };

    if (rA >= rB && tid == 0) s_ends[0] = 0, s_ends[1] = -1;
    p.r1 = min(rB, rA + WINDOW);
    for (int i = tid; i < p.r1 - rA; i += THREADS) s.mask[i] = 0u;
    __syncthreads();
    p.r0 = rA;
    fill_window<BW, FIRST, ROOM>(a, reinterpret_cast<unsigned *>(s.body), s.bits, s.pre, s.ids, s.mask, p.r0, p.r1, row0, p.nw, s_cnt, s_ends, held);
    __syncthreads();
    for (;;) {
        const int kw0 = p.r0 == rA ? p.k0 : p.r0 * a.C;
        const int kw1 = p.r1 == rB ? p.k1 : p.r1 * a.C;
        const int tiles = (kw1 - kw0 + 15) >> 4;
        const int mine = tiles > warp ? (tiles - warp + WARPS - 1) / WARPS : 0;

        int vtop = 1;
        struct Key {
            unsigned walks, ke, ve;
        };
        // starts tile i's copies; returns this lane's key of it (its exponents on their way)
        auto fetch = [&](int i) {
            Key key{0u, 1u, 1u};
            if (i < mine) {
                const KeyInfo k = key_info(a, p, s.ids, s.mask, kw0 + 16 * (warp + WARPS * i) + (lane & 15), kw1);
                key.walks = k.walks;
                if constexpr (F8) {
                    if (k.row >= 0) {
                        key.ke = __ldg(Kst + k.row);
                        key.ve = __ldg(Vst + k.row);
                    }
                }
                const uint32_t st = ring_s + (i % STAGES) * C::TILE;
#pragma unroll
                for (int x = 0; x < 16 * PPR / 32; ++x) {
                    // piece x * 32 + lane of the tile: constant rows rx and pieces qx beside the lane's
                    constexpr int LR = PPR < 32 ? 32 / PPR : 1;  // rows the lanes span
                    const int rx = PPR <= 32 ? x * LR : x / (PPR / 32), qx = PPR <= 32 ? 0 : x % (PPR / 32) * 32;
                    const int row = __shfl_sync(FULL, k.row, rx + lane / PPR);
                    const long long off = (long long)max(row, 0) * C::ROWB;
                    const uint32_t n = row < 0 ? 0u : 16u;
                    const uint32_t dst = st + (put0 ^ (twist<PPR>(rx) << 4)) + (PPR == 4 ? (rx >> 1) * 128 : rx * C::ROWB) + qx * 16;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(Kt + off + qx * 16), "r"(n)
                                 : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * C::ROWB), "l"(Vt + off + qx * 16),
                                 "r"(n)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            return key;
        };
        auto put_meta = [&](int i, const Key &k) {
            if (lane < 16) s_meta[warp][i % STAGES][lane] = make_uint2(k.walks, (k.ke << 23) | k.ve);
            if constexpr (F8) {
                vtop = __reduce_max_sync(FULL, (int)k.ve);
                vlow = min(vlow, k.walks ? (int)k.ve : 255);
            }
        };
        const Key first = fetch(0);
        Key ahead = fetch(1);  // of the tile fetched last
        put_meta(0, first);
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            const uint2 ma = s_meta[warp][i % STAGES][g], mb = s_meta[warp][i % STAGES][g + 8];
            const unsigned char *st = ring + (i % STAGES) * C::TILE;
            // S^T = K Q^T
            float sc[NW][4], odd[NW][4];  // two chains of sums; of several terms, the large products and the others
#pragma unroll
            for (int n = 0; n < NW; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) sc[n][c] = odd[n][c] = 0.f;
#pragma unroll
            for (int pc = 0; pc < KP; ++pc) {
                const unsigned char *kp = st + (get_k ^ (pc << 6));
                const uint4 k0 = *reinterpret_cast<const uint4 *>(kp), k1 = *reinterpret_cast<const uint4 *>(kp + ROW8);
                const unsigned w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int j = 0; j < KSP; ++j) {
                    const int ks = pc * KSP + j;
                    uint4 ka[KTERMS];
                    if constexpr (F8) {
                        codes_half2(w0[j], ka[0].x, ka[0].z);
                        codes_half2(w1[j], ka[0].y, ka[0].w);
                    } else if constexpr (KTERMS == 1) {
                        ka[0] = make_uint4(w0[2 * j], w1[2 * j], w0[2 * j + 1], w1[2 * j + 1]);
                    } else {
                        float x[8];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            x[c] = __uint_as_float(w0[c]);
                            x[c + 4] = __uint_as_float(w1[c]);
                        }
#pragma unroll
                        for (int kt = 0; kt < KTERMS; ++kt) {
                            ka[kt].x = take_term<false>(x[0], x[1]);
                            ka[kt].z = take_term<false>(x[2], x[3]);
                            ka[kt].y = take_term<false>(x[4], x[5]);
                            ka[kt].w = take_term<false>(x[6], x[7]);
                        }
                    }
#pragma unroll
                    for (int term = 0; term < C::QTERMS; ++term) {
                        if (term >= q_terms) break;
#pragma unroll
                        for (int n = 0; n < NW; ++n) {
                            const uint2 f = s.q[((term * NW + n) * KS + ks) * 32 + lane];
#pragma unroll
                            for (int kt = 0; kt < KTERMS; ++kt)
                                if (kt + term < 3)
                                    mma16816<F8>((KTERMS > 1 ? kt + term > 0 : term > 0 || ((FAST || a.q_bf16) && (ks & 1))) ? odd[n] : sc[n],
                                                 ka[kt], f.x, f.y);
                        }
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NW; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) sc[n][c] += odd[n][c];
            const unsigned walks[2] = {ma.x >> (2 * t4), mb.x >> (2 * t4)};
            const float kf[2] = {__uint_as_float(ma.y & 0x7f800000u), __uint_as_float(mb.y & 0x7f800000u)};
            const int ve[2] = {(int)(ma.y & 0xffu), (int)(mb.y & 0xffu)};
            soften(sc, walks, kf, ve, vtop);
            // O^T += V^T P^T. Of several terms, a tile's products are summed from the smallest and
            // then added: the instruction cuts its sums short, here by a tile's, not by all tiles'
            // (fp32 results over 2,000 keys 3.0e-7 off, 7.8e-7 with the sums in the accumulators).
            unsigned pb[PT][NW][2];
            const bool one = F8 && (FAST || p_terms == 1);
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                if (one) {
                    pb[0][n][0] = transpose8(half2_pair(sc[n][0], sc[n][1]));
                    pb[0][n][1] = transpose8(half2_pair(sc[n][2], sc[n][3]));
                } else {
#pragma unroll
                    for (int term = 0; term < PT; ++term) {
                        pb[term][n][0] = transpose8(take_term<F8>(sc[n][0], sc[n][1]));
                        pb[term][n][1] = transpose8(take_term<F8>(sc[n][2], sc[n][3]));
                    }
                }
            }
            const unsigned char *sv = st + 16 * C::ROWB;
            constexpr bool HALF = F8 && D == 64;  // a run is half a piece
            constexpr int VP = HALF ? 1 : PPR / 8;
            // accumulator tile j takes the operand's terms va
            auto add_tile = [&](int j, const uint4 (&va)[KTERMS]) {
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    if constexpr (FAST) {
#pragma unroll
                        for (int term = PT - 1; term >= 0; --term) mma16816<F8>(acc[j][n], va[0], pb[term][n][0], pb[term][n][1]);
                        continue;
                    }
                    if (one) {
                        mma16816<F8>(acc[j][n], va[0], pb[0][n][0], pb[0][n][1]);
                        continue;
                    }
                    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int sum = PT - 1; sum >= 0; --sum) {
                        if (sum >= p_terms) continue;
#pragma unroll
                        for (int vt = 0; vt < KTERMS; ++vt)
                            if (vt <= sum) mma16816<F8>(part, va[vt], pb[sum - vt][n][0], pb[sum - vt][n][1]);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[j][n][c] += part[c];
                }
            };
#pragma unroll
            for (int vp = 0; vp < VP; ++vp) {
                unsigned w[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // rows 2 t4, 2 t4 + 1, and those + 8
                    const unsigned char *vr = sv + (get_v ^ ((r & 1) << 6)) + (r & 1) * ROW1 + (r >> 1) * ROW8 + vp * 128;
                    if constexpr (HALF) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(vr);
                        w[r][0] = x.x;
                        w[r][1] = x.y;
                    } else {
                        const uint4 x = *reinterpret_cast<const uint4 *>(vr);
                        w[r][0] = x.x;
                        w[r][1] = x.y;
                        w[r][2] = x.z;
                        w[r][3] = x.w;
                    }
                }
                uint4 va[KTERMS];
                if constexpr (F8) {
#pragma unroll
                    for (int x = 0; x < (HALF ? 2 : 4); ++x)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const unsigned sel = h ? 0x7362u : 0x5140u;
                            codes_half2(__byte_perm(w[0][x], w[1][x], sel), va[0].x, va[0].y);
                            codes_half2(__byte_perm(w[2][x], w[3][x], sel), va[0].z, va[0].w);
                            add_tile(vp * HR + 2 * x + h, va);
                        }
                } else if constexpr (KTERMS == 1) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        va[0] = make_uint4(__byte_perm(w[0][x], w[1][x], 0x5410), __byte_perm(w[0][x], w[1][x], 0x7632),
                                           __byte_perm(w[2][x], w[3][x], 0x5410), __byte_perm(w[2][x], w[3][x], 0x7632));
                        add_tile(vp * HR + x, va);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 4; x += 2) {
                        float y[8];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            y[r] = __uint_as_float(w[r][x]);
                            y[r + 4] = __uint_as_float(w[r][x + 1]);
                        }
#pragma unroll
                        for (int vt = 0; vt < KTERMS; ++vt) {
                            va[vt].x = take_term<false>(y[0], y[1]);
                            va[vt].z = take_term<false>(y[2], y[3]);
                            va[vt].y = take_term<false>(y[4], y[5]);
                            va[vt].w = take_term<false>(y[6], y[7]);
                        }
                        add_tile(vp * HR + x / 2, va);
                    }
                }
            }
            __syncwarp();  // the tile and its meta are read
            put_meta(i + 1, ahead);
            ahead = fetch(i + 2);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (p.r1 >= rB) break;
        __syncthreads();  // the window's ids and masks are read
        p.r0 = p.r1;
        p.r1 = min(rB, p.r0 + WINDOW);
        for (int i = tid; i < p.r1 - p.r0; i += THREADS) s.mask[i] = 0u;
        __syncthreads();
        fill_window<BW, FIRST, ROOM>(a, reinterpret_cast<unsigned *>(s.body), s.bits, s.pre, s.ids, s.mask, p.r0, p.r1, a.sel + p.walk0 * a.max_sel, p.nw, s_cnt, s_ends, 0);
        __syncthreads();
    }

    if constexpr (F8) {
        vlow = __reduce_min_sync(FULL, vlow);
        if (lane == 0) {
            s_vmax[warp] = vref;
            s_vmin[warp] = vlow;
        }
    }

    // drafted tokens: tiles of 16, staged in the ring's space (an fp32 tile's K, then its
    // V) and taken in bf16 terms, in the column order of the cache
    const bool drafted = DRAFT && part == np - 1;
    if constexpr (DRAFT) if (drafted) {
        __syncthreads();  // every warp has left its ring
        const uint2 *qd = F8 ? s.qd : s.q;
        const int qdt = FAST || a.q_bf16 ? 1 : 3, pt = FAST || a.out_bf16 ? 2 : 3, nd = a.n_draft;
        const int eb = a.d_bf16 ? 2 : 4, row_b = D * eb, ppr = row_b / 16;
        const long long base_d = (long long)p.tree * nd * row_b;
        unsigned char *slot = s.body + warp * (C::BODY / WARPS / 16 * 16);
        // rows j0 .. j0 + 15 of k or v (zeros behind the last) to `to`
        auto stage = [&](const void *src, int j0, unsigned char *to) {
            for (int idx = lane; idx < 16 * ppr; idx += 32) {
                const int r = idx / ppr, q = idx - r * ppr, j = j0 + r;
                const char *from = static_cast<const char *>(src) + base_d + (long long)min(j, nd - 1) * row_b + q * 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s_addr(to) + r * row_b + ((q ^ (r & 7)) << 4)),
                             "l"(from), "r"(j < nd ? 16u : 0u)
                             : "memory");
            }
        };
        auto staged = [&]() {
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
        };
        // 4 columns of a staged row: as they are (bf16), and as fp32
        auto raw = [&](const unsigned char *at, int r, int col) {
            const int byte = col * 2;
            return *reinterpret_cast<const uint2 *>(at + r * row_b + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15));
        };
        auto cols = [&](const unsigned char *at, int r, int col, float (&x)[4]) {
            const int byte = col * eb;
            const unsigned char *p16 = at + r * row_b + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
            const float4 u = *reinterpret_cast<const float4 *>(p16);
            x[0] = u.x;
            x[1] = u.y;
            x[2] = u.z;
            x[3] = u.w;
        };
#pragma unroll 1
        for (int j0 = warp * 16; j0 < nd; j0 += WARPS * 16) {
            unsigned char *sk = slot, *sv = a.d_bf16 ? slot + 16 * row_b : slot;
            stage(a.kd, j0, sk);
            if (a.d_bf16) stage(a.vd, j0, sv);
            unsigned walks[2] = {0u, 0u};
#pragma unroll
            for (int n = 0; n < NW; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int w = n * 8 + 2 * t4 + c;
                    if (w >= p.nw) continue;
                    const unsigned char *mrow = mask_row(a, p, w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int j = j0 + g + 8 * h;
                        if (j < nd && __ldg(mrow + j)) walks[h] |= 1u << (8 * n + c);
                    }
                }
            staged();
            if (!__any_sync(FULL, walks[0] | walks[1])) continue;
            float sc[NW][4];
#pragma unroll
            for (int n = 0; n < NW; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) sc[n][c] = 0.f;
            if (a.d_bf16) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const int col = ((ks / KSP) * 4 + t4) * C::PC + (ks % KSP) * 4;
                    const uint2 x = raw(sk, g, col), y = raw(sk, g + 8, col);
#pragma unroll
                    for (int term = 0; term < 3; ++term) {
                        if (term >= qdt) break;
#pragma unroll
                        for (int n = 0; n < NW; ++n) {
                            const uint2 f = qd[((term * NW + n) * KS + ks) * 32 + lane];
                            mma16816<false>(sc[n], make_uint4(x.x, y.x, x.y, y.y), f.x, f.y);
                        }
                    }
                }
            } else {
#pragma unroll 2
                for (int ks = 0; ks < KS; ++ks) {
                    const int col = ((ks / KSP) * 4 + t4) * C::PC + (ks % KSP) * 4;
                    float x[2][4];
                    cols(sk, g, col, x[0]);
                    cols(sk, g + 8, col, x[1]);
#pragma unroll
                    for (int kt = 0; kt < 3; ++kt) {
                        uint4 ka;
                        ka.x = take_term<false>(x[0][0], x[0][1]);
                        ka.z = take_term<false>(x[0][2], x[0][3]);
                        ka.y = take_term<false>(x[1][0], x[1][1]);
                        ka.w = take_term<false>(x[1][2], x[1][3]);
                        for (int term = 0; term < qdt && term + kt < 3; ++term) {
#pragma unroll
                            for (int n = 0; n < NW; ++n) {
                                const uint2 f = qd[((term * NW + n) * KS + ks) * 32 + lane];
                                mma16816<false>(sc[n], ka, f.x, f.y);
                            }
                        }
                    }
                }
            }
            const float one[2] = {1.f, 1.f};
            const int byte[2] = {127, 127};
            soften(sc, walks, one, byte, 127);
            if (!a.d_bf16) {
                __syncwarp();
                stage(a.vd, j0, sv);
                staged();
            }
            unsigned pb[3][NW][2];
#pragma unroll
            for (int term = 0; term < 3; ++term)
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    pb[term][n][0] = transpose8(take_term<false>(sc[n][0], sc[n][1]));
                    pb[term][n][1] = transpose8(take_term<false>(sc[n][2], sc[n][3]));
                }
            // as a cached tile's: the products of va's terms from the smallest, then added
            auto add_draft = [&](int j, const uint4 *va, int vterms) {
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int sum = FAST ? 1 : 2; sum >= 0; --sum) {
                        if (sum >= pt) continue;
#pragma unroll
                        for (int vt = 0; vt < 3; ++vt)
                            if (vt <= sum && vt < vterms) mma16816<false>(part, va[vt], pb[sum - vt][n][0], pb[sum - vt][n][1]);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[j][n][c] += part[c];
                }
            };
#pragma unroll
            for (int j = 0; j < MT; j += 2) {
                const int col = j / HR * (8 * C::RUN) + g * C::RUN + 2 * (j % HR);
                if (a.d_bf16) {
                    uint2 v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = raw(sv, 2 * t4 + (r & 1) + (r >> 1) * 8, col);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        unsigned e[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) e[r] = x ? v[r].y : v[r].x;
                        const uint4 va[1] = {make_uint4(__byte_perm(e[0], e[1], 0x5410), __byte_perm(e[0], e[1], 0x7632),
                                                        __byte_perm(e[2], e[3], 0x5410), __byte_perm(e[2], e[3], 0x7632))};
                        add_draft(j + x, va, 1);
                    }
                } else {
                    float v[4][4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) cols(sv, 2 * t4 + (r & 1) + (r >> 1) * 8, col, v[r]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint4 va[3];
#pragma unroll
                        for (int vt = 0; vt < 3; ++vt) {
                            va[vt].x = take_term<false>(v[0][2 * x], v[1][2 * x]);
                            va[vt].z = take_term<false>(v[2][2 * x], v[3][2 * x]);
                            va[vt].y = take_term<false>(v[0][2 * x + 1], v[1][2 * x + 1]);
                            va[vt].w = take_term<false>(v[2][2 * x + 1], v[3][2 * x + 1]);
                        }
                        add_draft(j + x, va, 3);
                    }
                }
            }
            __syncwarp();  // the slot is staged again
        }
    }

    // 3. merge: every warp's sums to shared memory, then a warp per walk
#pragma unroll
    for (int n = 0; n < NW; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) l[n][c] += __shfl_xor_sync(FULL, l[n][c], o);
            if (g == 0) {
                s_m[warp][n * 8 + 2 * t4 + c] = m[n][c];
                s_l[warp][n * 8 + 2 * t4 + c] = l[n][c];
            }
        }
    const float back = F8 ? exp_byte((unsigned)vref) : 1.f, down = F8 ? 1.f / (1 << PSHIFT) : 1.f;
    {
        __syncthreads();  // the ring becomes the merge buffer
        float *sum = reinterpret_cast<float *>(s.body) + warp * BW * C::MS;
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int w = n * 8 + 2 * t4 + (c & 1);
                if (w >= p.nw) continue;
#pragma unroll
                for (int j = 0; j < MT; ++j) sum[w * C::MS + j * 16 + (c >> 1) * 8 + g] = acc[j][n][c] * down * back;
            }
        __syncthreads();
        float vsum = 0.f;  // sums below this have lost too much to the largest values
        if constexpr (F8) {
            int vmax = 0, vmin = 255;
#pragma unroll
            for (int x = 0; x < WARPS; ++x) {
                vmax = max(vmax, s_vmax[x]);
                vmin = min(vmin, s_vmin[x]);
            }
            const bool one = FAST || p_terms == 1;
            if (vmin < vmax - (one ? VFAR_ONE : VFAR_TWO))
                vsum = exp_byte((unsigned)vmax) * exp_byte((unsigned)(127 - PSHIFT + (one ? VSUM_ONE : VSUM_TWO)));
        }
        for (int w = warp; w < p.nw; w += WARPS) {
            float mm = -INFINITY, ll = 0.f, o[N];
#pragma unroll
            for (int x = 0; x < WARPS; ++x) mm = fmaxf(mm, s_m[x][w]);
            const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
            for (int c = 0; c < N; ++c) o[c] = 0.f;
#pragma unroll
            for (int x = 0; x < WARPS; ++x) {
                const float f = exp_of(s_m[x][w] - ref);
                ll += s_l[x][w] * f;
                const float *from = reinterpret_cast<const float *>(s.body) + (x * BW + w) * C::MS;
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    const int col = lane * N + c, in = col % (8 * C::RUN), e = in % C::RUN;
                    o[c] = fmaf(from[(col / (8 * C::RUN) * HR + e / 2) * 16 + (e & 1) * 8 + in / C::RUN], f, o[c]);
                }
            }
            bool bad = false;
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < N; ++c) {
                bad |= o[c] != o[c];
                top = fmaxf(top, fabsf(o[c]));
            }
            if (F8 && vsum > 0.f) bad |= ll > 0.f && warp_max(top) < vsum;
            bad = __any_sync(FULL, bad);
            if (bad) {
                // copies: what is passed by its address lies in local memory, in the tiles' loop too (1.1 to
                // 1.25 times the call's time)
                const Part pp = p;
                const Smem<C> ss(smem_blocks, a);
                float m2, l2, o2[N];
                slow_walk<KT, D>(a, pp, ss, w, s_cnt[w], drafted, m2, l2, o2);
                mm = m2;
                ll = l2;
#pragma unroll
                for (int c = 0; c < N; ++c) o[c] = o2[c];
            }
            if (np == 1) {
                finish_walk<D>(a, p.walk0 + w, lane, mm, ll, o);
            } else {
                float *dst = a.partial + ((long long)item * BW + w) * (D + 4);
#pragma unroll
                for (int c = 0; c < N; c += 2) *reinterpret_cast<float2 *>(dst + lane * N + c) = make_float2(o[c], o[c + 1]);
                if (lane == 0) {
                    dst[D] = mm;
                    dst[D + 1] = ll;
                }
            }
        }
    }
    chain_done();
}

template <typename KT, int D, int NW, bool FAST, bool DRAFT>
cudaError_t launch_blocks(const zha_tree *t, BlockArgs a, cudaStream_t st) {
    using C = Cfg<KT, D, NW, FAST, DRAFT>;
    const size_t smem = C::FIXED + C::DTERMS * C::QBYTES + 8 * (size_t)a.words;
    static OncePerDevice limit;
    cudaError_t e = limit(t->device, [] {
        return cudaFuncSetAttribute(attend_block_kernel<KT, D, NW, FAST, DRAFT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::FIXED + C::DTERMS * C::QBYTES + (int)(BLOCK_CHUNKS_MAX / 32) * 8);
    });
    if (e != cudaSuccess) return e;
    if (a.target) {
        // Few blocks: as many items as CTAs fit on the GPU, less one a block for the
        // rounding of each block's keys. More blocks: long ones are cut so that the last
        // CTAs end together, and items are longer, as each takes its block's lists anew.
        const int slots = num_sms() * C::MIN_CTAS;
        const bool few = a.NB <= slots / 2;
        a.target = few ? slots - a.NB : 2 * slots;
        a.many = !few;
        e = launch_plan(t, a, st);
        if (e != cudaSuccess) return e;
    }
    Probe pr(t, ZHA_K_ATTEND_PARTIAL, st);
    return launch_chained(attend_block_kernel<KT, D, NW, FAST, DRAFT>, dim3((unsigned)(a.NB + a.target)), dim3(C::WARPS * 32), smem, st, a);
}

template <typename KT, int D, bool FAST, bool DRAFT>
cudaError_t launch_blocks_n(const zha_tree *t, const BlockArgs &a, cudaStream_t st) {
    if constexpr (block_walks_max<KT>(D) >= 16) {
        if (a.bw == 16) return launch_blocks<KT, D, 2, FAST, DRAFT>(t, a, st);
    }
    return launch_blocks<KT, D, 1, FAST, DRAFT>(t, a, st);
}

template <typename KT, bool FAST, bool DRAFT>
cudaError_t launch_blocks_d(const zha_tree *t, const BlockArgs &a, cudaStream_t st) {
    switch (t->cfg.d) {
        case 64: return launch_blocks_n<KT, 64, FAST, DRAFT>(t, a, st);
        case 128: return launch_blocks_n<KT, 128, FAST, DRAFT>(t, a, st);
        default: return launch_blocks_n<KT, 256, FAST, DRAFT>(t, a, st);
    }
}

}  // namespace
}  // namespace zha
