// tree_attn.cuh -- what the attention kernels share: the requests as clamped
// into the buffers, the cut of the work into equal runs, the keys a token sees.
#pragma once

#include "sgq_device.cuh"
#include "sgq_launch.h"

namespace sgq {

namespace {

constexpr int kBN = 64;        // keys per unit
constexpr int kItemCost = 5;   // what an item costs beside its units, in units (measured with 1, 2, 4, 5 and 8:
                               // 24 ragged requests take 76, 69, 62, 61 and 60 us, 11 of 8-bit keys 92, 87,
                               // 80, 79 and 80, 300 of up to 400 keys 102, 102, 105, 105 and 107)
constexpr int kMaxGrid = 160;  // one CTA per SM
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Requests, as clamped into the ranges the pointers are known to cover.
struct Request {
    int tok, n;    // first row of q, new tokens
    int len, keys; // cached tokens, len + n
    int row_tiles;
    int tiles;     // units per (key head, row tile)
};

__device__ __forceinline__ Request request_of(const AttnProblem &p, int r, int G, int MT, int &bits)
{
    Request q;
    const int c0 = p.cu_new[r], c1 = p.cu_new[r + 1];
    q.tok = min(max(c0, 0), p.T);
    q.n = min(max(c1, q.tok), p.T) - q.tok;
    int len = p.lens[r];
    const long long cap = (long long)p.table_ld * p.cache.page;
    if (c0 != q.tok || c1 != q.tok + q.n || len < 0 || (long long)len + q.n > cap)
        bits |= SGQ_STATUS_BAD_COUNT;
    len = (int)min((long long)max(len, 0), max(0ll, cap - q.n));
    q.len = len;
    q.keys = (int)min((long long)len + q.n, cap);
    q.row_tiles = (int)(((long long)q.n * G + MT - 1) / MT);
    q.tiles = q.n ? (q.keys + kBN - 1) / kBN : 0;
    return q;
}

// What request q costs; an item is one (key head, row tile) of it.
__device__ __forceinline__ long long cost_of(const Request &q, int Hkv)
{
    return q.tiles ? (long long)Hkv * q.row_tiles * (q.tiles + kItemCost) : 0;
}

// Start of CTA c's run of C equal ones (1 <= C <= U), and the CTA whose run
// holds position u.
__device__ __forceinline__ long long run_start(long long U, int c, int C) { return U * c / C; }
__device__ __forceinline__ int cta_of(long long U, long long u, int C)
{
    return (int)(((u + 1) * C - 1) / U);
}

// A CTA's share of an item that several CTAs work on, c0 to c0 + parts - 1
// (parts = 0: none): the one it goes on with ([0]) and the one it starts ([1]).
// 16 bytes are what a workspace is aligned to.
struct __align__(16) Split {
    int parts, c0, tok, n, h, rt, pad[2];
};

// The part that CTA c leaves of either: D sums of MT rows, four of a row side by
// side and the rows next to each other ([D / 4][MT][4]), then the rows'
// references, then their sums.
__device__ __forceinline__ float *part_of(const AttnProblem &p, int c, int which, int MT, int D)
{
    return reinterpret_cast<float *>(static_cast<char *>(p.workspace) + 2 * kMaxGrid * sizeof(Split)) +
           (size_t)(2 * c + which) * (MT * (D + 2));
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two e4m3 values (bits 0..15) as two fp16 in order; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v)
{
    uint32_t d;
    asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(d) : "r"(v));
    return d;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// The first 64 bits of token i's tree words.
__device__ __forceinline__ uint64_t tree_bits(const AttnProblem &p, const Request &q, int i)
{
    if (!p.tree)
        return 0;
    const uint32_t *w = p.tree + (long long)(q.tok + i) * p.tree_words;
    return w[0] | (p.tree_words > 1 ? (uint64_t)w[1] << 32 : 0);
}

// The 64 keys from kb0 on, and before `end`, that token i sees, bit by key: all
// of the context, and of the drafted tokens those its tree words name (`first`:
// tree_bits; no tree: itself and the ones before it).
__device__ __forceinline__ uint64_t visible(const AttnProblem &p, const Request &q, int i,
                                            uint64_t first, int kb0, int end)
{
    const int start = kb0 - q.len;
    const int s = max(start, 0);
    uint64_t d = 0;
    if (!p.tree) {
        const int ones = i + 1 - s;
        d = ones >= 64 ? ~0ull : ones > 0 ? (1ull << ones) - 1 : 0ull;
    } else if (s == 0 || p.tree_words <= 2) {
        d = s < 64 ? first >> s : 0ull;
    } else {
        const uint32_t *w = p.tree + (long long)(q.tok + i) * p.tree_words;
        const int k = s >> 5, sh = s & 31;
        const uint64_t w0 = k < p.tree_words ? w[k] : 0u;
        const uint64_t w1 = k + 1 < p.tree_words ? w[k + 1] : 0u;
        const uint64_t w2 = k + 2 < p.tree_words ? w[k + 2] : 0u;
        d = (w0 | (w1 << 32)) >> sh;
        if (sh)
            d |= w2 << (64 - sh);
    }
    if (start < 0) {
        const int sh = -start;
        d = sh >= 64 ? ~0ull : (d << sh) | ((1ull << sh) - 1);
    }
    const int left = end - kb0;
    return left >= 64 ? d : left > 0 ? d & ((1ull << left) - 1) : 0ull;
}

// The segments of one CTA's run, in order: each is `nu` units, from unit j0 on,
// of one item.
struct Walk {
    int r = 0, h = 0, rt = 0; // request, key head, row tile
    int j0 = 0, nu = 0;
    Request rq{};
    long long base = 0, u = 0, u_end = 0; // cost before request r, the run
    long long item0 = 0;                  // cost before the item

    __device__ __forceinline__ int key_end() const { return min(rq.keys, (j0 + nu) * kBN); }
    __device__ __forceinline__ bool whole() const { return nu == rq.tiles; }

    __device__ __forceinline__ bool next(const AttnProblem &p, int G, int MT)
    {
        int bits = 0;
        while (u < u_end) {
            while (u >= base + cost_of(rq, p.cache.heads)) {
                base += cost_of(rq, p.cache.heads);
                rq = request_of(p, ++r, G, MT, bits);
            }
            const long long in_r = u - base;
            const int cost = rq.tiles + kItemCost;
            // (a 32-bit division where it will do: 64-bit ones take a call)
            const long long item = in_r >> 31 ? in_r / cost : (long long)((uint32_t)in_r / (uint32_t)cost);
            const int p0 = (int)(in_r - item * cost);
            const int p1 = (int)min((long long)(rq.tiles + kItemCost), p0 + (u_end - u));
            u += p1 - p0;
            if (p0 >= rq.tiles)
                continue;
            item0 = base + item * cost;
            j0 = p0;
            nu = min(p1, rq.tiles) - p0;
            h = item >> 31 ? (int)(item / rq.row_tiles) : (int)((uint32_t)item / (uint32_t)rq.row_tiles);
            rt = (int)(item - (long long)h * rq.row_tiles);
            return true;
        }
        return false;
    }
};

} // namespace

} // namespace sgq
