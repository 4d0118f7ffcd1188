// tree_attn.cu -- sgq_tree_attn: attention of each request's new tokens (a
// tree of drafted tokens, a chain, or one token) over its pages of the cache.
//
//   s_j = scale k_scale q.k_j over the keys j the token sees,
//   o   = v_scale sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  m = max s_j
//
// One pass over the keys with the running maximum and sum of the softmax, in
// base 2. The G = Hq / Hkv query heads that share a key head, times the
// request's new tokens, are the rows of one matrix product: a tile of MT rows
// reads each key and value once for all of them.
//
// Work is cut into units of (request, key head, row tile, 64 keys) in that
// order, and every CTA takes an equal run of them, whatever the requests'
// lengths are (they are known on the device only). A run that starts or ends
// inside a (request, key head, row tile) leaves its unnormalised sums with
// their maximum and sum in the workspace, and combine_kernel joins them in
// order; a whole one is written out directly.
#include "sgq_device.cuh"
#include "sgq_launch.h"
#include "step_launch.cuh"

#include <algorithm>
#include <cuda_fp8.h>

namespace sgq {

namespace {

constexpr int kBN = 64;        // keys per unit
constexpr int kThreads = 128;
constexpr int kMaxGrid = 296;  // two CTAs on each of 148 SMs
constexpr int kMaxMT = 64;
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

__device__ __forceinline__ long long units_of(const Request &q, int Hkv)
{
    return (long long)Hkv * q.row_tiles * q.tiles;
}

// First unit of CTA c of C, and the CTA that holds unit u.
__device__ __forceinline__ long long first_unit(long long U, int c, int C) { return U * c / C; }
__device__ __forceinline__ int cta_of(long long U, long long u, int C)
{
    return (int)(((u + 1) * C - 1) / U);
}

__host__ __device__ inline size_t units_bytes(int R) { return ((size_t)(R + 1) * 8 + 255) / 256 * 256; }

// ---- instructions ----

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool take)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(take ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// D += A B on 16 x 8 x 16 with fp32 sums; 8-bit keys and values are exact in
// fp16, so they and q (scaled, see load_q) and the weights are fp16 there.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <int D_, int KV, int MT_>
struct Cfg {
    static constexpr int D = D_, MT = MT_;
    static constexpr bool F8 = KV == SGQ_TYPE_E4M3;
    static constexpr int ES = F8 ? 1 : 2;
    static constexpr int ROWB = D * ES;               // bytes of one key
    static constexpr int CPR = ROWB / 16;             // 16-byte chunks of one key
    static constexpr int HALF = kBN * ROWB;           // keys (or values) of a stage
    static constexpr int STAGE = 2 * HALF;
    static constexpr int NST = STAGE >= 32768 ? 3 : STAGE >= 16384 ? 5 : 8;
    static constexpr int NR = NST + 1;                // ring of row offsets
    static constexpr int WM = MT / 16, WN = 4 / WM;   // warps along rows and along keys
    static constexpr int KW = kBN / WN;               // keys per warp and unit
    static constexpr int NT = KW / 8;                 // score tiles of 8 keys
    static constexpr int KS = D / 16;                 // products' steps along the head
    static constexpr int DT = D / 8;                  // output tiles of 8 columns
    static constexpr int SMEM = NST * STAGE + NR * kBN * 8 + NR * 8;
    static_assert(WN * MT * D * 4 <= NST * STAGE, "the warps' sums fit the stages");
};

// Byte offset of 16-byte chunk c of key row r within a half stage. Eight
// consecutive rows at one chunk fall into eight different 16-byte bank groups
// (ldmatrix); with 8-bit keys so do two rows' aligned runs of four chunks.
template <class C>
__device__ __forceinline__ uint32_t chunk_off(int r, int c)
{
    int x;
    if constexpr (C::ROWB == 64)
        x = (r >> 1) & 3;
    else if constexpr (C::F8)
        x = ((r & 1) << 2) | ((r >> 1) & 3);
    else
        x = r & 7;
    return (uint32_t)(r * C::ROWB + ((c ^ x) << 4));
}

// The 64 keys from kb0 on that a token sees, bit by key: all of the context,
// and of the drafted tokens those its tree words name (no tree: itself and the
// ones before it).
__device__ __forceinline__ uint64_t visible(const AttnProblem &p, const Request &q, int i, int kb0)
{
    const int start = kb0 - q.len;
    const int s = max(start, 0);
    uint64_t d = 0;
    if (p.tree) {
        const uint32_t *w = p.tree + (long long)(q.tok + i) * p.tree_words;
        const int k = s >> 5, sh = s & 31;
        const uint64_t w0 = k < p.tree_words ? w[k] : 0u;
        const uint64_t w1 = k + 1 < p.tree_words ? w[k + 1] : 0u;
        const uint64_t w2 = k + 2 < p.tree_words ? w[k + 2] : 0u;
        d = (w0 | (w1 << 32)) >> sh;
        if (sh)
            d |= w2 << (64 - sh);
    } else {
        const int ones = i + 1 - s;
        d = ones >= 64 ? ~0ull : ones > 0 ? (1ull << ones) - 1 : 0ull;
    }
    if (start < 0) {
        const int sh = -start;
        d = sh >= 64 ? ~0ull : (d << sh) | ((1ull << sh) - 1);
    }
    const int left = q.keys - kb0;
    return left >= 64 ? d : left > 0 ? d & ((1ull << left) - 1) : 0ull;
}

template <int D, int KV, int MT>
__global__ void __launch_bounds__(kThreads, 2) attn_kernel(const AttnProblem p)
{
    using C = Cfg<D, KV, MT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long s_scan[4];
    __shared__ int s_r;
    __shared__ long long s_first;
    __shared__ float s_m[4][MT], s_l[4][MT];
    long long *ring = reinterpret_cast<long long *>(smem + C::NST * C::STAGE); // [NR][64], -1: no key
    uint32_t *bad = reinterpret_cast<uint32_t *>(ring + C::NR * kBN);          // [NR][2]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp / C::WN, wn = warp % C::WN;
    const int qd = lane & 3, gr = lane >> 2;
    const int Hkv = p.cache.heads, G = p.Hq / Hkv;
    const uint32_t sm0 = smem_u32(smem);
    int bits = 0;
    grid_launch_dependents();
    grid_dependency_wait();

    // Units before each request; this CTA's run [u, u_end).
    long long *ws_units = static_cast<long long *>(p.workspace);
    float *ws_part = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + units_bytes(p.R));
    const int per = (p.R + kThreads - 1) / kThreads;
    const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    long long mine = 0;
    for (int r = r0; r < r1; ++r)
        mine += units_of(request_of(p, r, G, MT, bits), Hkv);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(~0u, inc, o);
        if (lane >= o)
            inc += t;
    }
    if (lane == 31)
        s_scan[warp] = inc;
    if (tid == 0)
        s_r = p.R;
    __syncthreads();
    long long U = 0, at = inc - mine;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        at += w < warp ? s_scan[w] : 0;
        U += s_scan[w];
    }
    long long u = first_unit(U, blockIdx.x, gridDim.x);
    const long long u_end = first_unit(U, blockIdx.x + 1, gridDim.x);
    if (blockIdx.x == 0 || (u >= at && u < at + mine)) {
        long long s = at;
        for (int r = r0; r < r1; ++r) {
            const long long n = units_of(request_of(p, r, G, MT, bits), Hkv);
            if (u >= s && u < s + n) {
                s_r = r;
                s_first = s;
            }
            if (blockIdx.x == 0)
                ws_units[r] = s;
            s += n;
        }
        if (blockIdx.x == 0 && r1 == p.R)
            ws_units[p.R] = U;
    }
    if (bits && blockIdx.x == 0)
        set_status(p.status, bits);
    __syncthreads();
    int r = s_r;
    if (u >= u_end || r >= p.R)
        return;
    long long base = s_first;
    Request rq = request_of(p, r, G, MT, bits);
    bits = 0;

    while (u < u_end) {
        while (u >= base + units_of(rq, Hkv)) {
            base += units_of(rq, Hkv);
            rq = request_of(p, ++r, G, MT, bits);
        }
        const long long in_r = u - base;
        const long long item = in_r / rq.tiles;
        const int j0 = (int)(in_r - item * rq.tiles);
        const int nt = (int)min((long long)(rq.tiles - j0), u_end - u);
        const int h = (int)(item / rq.row_tiles), rt = (int)(item - (long long)h * rq.row_tiles);
        const int32_t *table = p.table + (long long)r * p.table_ld;

        // Element offset of key `key`'s row for this head, or -1.
        auto page_id = [&](int key) -> int {
            return key < rq.keys ? table[key / p.cache.page] : -1;
        };
        auto put_row = [&](int tile, int row, int id) { // whole warps, 32 consecutive rows
            const int key = (j0 + tile) * kBN + row;
            const bool want = key < rq.keys, ok = want && id >= 0 && id < p.cache.num_pages;
            ring[(tile % C::NR) * kBN + row] =
                ok ? id * p.cache.page_stride + (key % p.cache.page) * p.cache.slot_stride : -1;
            const uint32_t b = __ballot_sync(~0u, want && !ok);
            if ((row & 31) == 0)
                bad[(tile % C::NR) * 2 + (row >> 5)] = b;
            if (b && (row & 31) == 0)
                set_status(p.status, SGQ_STATUS_BAD_INDEX);
        };
        auto issue = [&](int tile) {
            const uint32_t st = sm0 + (uint32_t)(tile % C::NST) * C::STAGE;
            const long long *off = ring + (tile % C::NR) * kBN;
            const uint8_t *kh = static_cast<const uint8_t *>(p.cache.k) + h * p.cache.head_stride * C::ES;
            const uint8_t *vh = static_cast<const uint8_t *>(p.cache.v) + h * p.cache.head_stride * C::ES;
#pragma unroll
            for (int i = 0; i < kBN * C::CPR / kThreads; ++i) {
                const int idx = tid + i * kThreads, row = idx / C::CPR, c = idx % C::CPR;
                const long long o = off[row];
                const bool take = o >= 0;
                const long long e = take ? o * C::ES + c * 16 : 0;
                const uint32_t d = st + chunk_off<C>(row, c);
                cp_async16_zfill(d, kh + e, take);
                cp_async16_zfill(d + C::HALF, vh + e, take);
            }
        };

        // Fill: offsets of the first NST units, loads of the first NST - 1.
        for (int i = tid; i < C::NST * kBN; i += kThreads) {
            const int tile = i / kBN, row = i % kBN;
            put_row(tile, row, page_id((j0 + tile) * kBN + row));
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < C::NST - 1; ++s) {
            if (s < nt)
                issue(s);
            cp_async_commit();
        }
        int next_id = -1;
        if (tid < kBN)
            next_id = page_id((j0 + C::NST) * kBN + tid);

        // This thread's two rows: row g of the tile is (token g / G, head g % G).
        int tok_i[2];
        bool live[2];
        const uint16_t *qrow[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int g = rt * MT + wm * 16 + gr + 8 * e;
            tok_i[e] = g / G;
            live[e] = tok_i[e] < rq.n;
            if (!live[e])
                tok_i[e] = 0;
            qrow[e] = p.q + (rq.tok + tok_i[e]) * p.ld_q + (long long)(h * G + (live[e] ? g % G : 0)) * D;
        }
        // q in the products' A layout. With 8-bit keys a thread's 16 bytes of
        // a key are four steps' worth, so the head's order inside the steps is
        // permuted, the same way for q and k; and q becomes fp16, each row by
        // the power of two that brings its largest value into [2^7, 2^8): exact
        // for values down to 2^-21 of that, below it off by at most 2^-33 of it.
        uint32_t qf[C::KS][4];
        float factor[2] = {p.scale * p.cache.k_scale * kLog2e, p.scale * p.cache.k_scale * kLog2e};
        if constexpr (!C::F8) {
#pragma unroll
            for (int s = 0; s < C::KS; ++s)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    qf[s][e] = live[e] ? *reinterpret_cast<const uint32_t *>(qrow[e] + s * 16 + 2 * qd) : 0u;
                    qf[s][e + 2] = live[e] ? *reinterpret_cast<const uint32_t *>(qrow[e] + s * 16 + 8 + 2 * qd) : 0u;
                }
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint2 raw[C::KS];
                float mx = 0.0f;
#pragma unroll
                for (int s = 0; s < C::KS; ++s) {
                    raw[s] = live[e] ? *reinterpret_cast<const uint2 *>(qrow[e] + (s >> 2) * 64 + qd * 16 + (s & 3) * 4)
                                     : make_uint2(0u, 0u);
                    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(raw[s].x << 16)), fabsf(__uint_as_float(raw[s].x & 0xffff0000u))));
                    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(raw[s].y << 16)), fabsf(__uint_as_float(raw[s].y & 0xffff0000u))));
                }
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
                // exponent of the power of two, kept where both it and its
                // inverse are normal fp32 numbers
                const int ex = (int)(__float_as_uint(mx) >> 23) - 127;
                const int up = min(max(7 - ex, -126), 126);
                const float mul = pow2f(up);
                factor[e] *= pow2f(-up);
#pragma unroll
                for (int s = 0; s < C::KS; ++s) {
                    qf[s][e] = pack2<true>(__uint_as_float(raw[s].x << 16) * mul,
                                           __uint_as_float(raw[s].x & 0xffff0000u) * mul);
                    qf[s][e + 2] = pack2<true>(__uint_as_float(raw[s].y << 16) * mul,
                                               __uint_as_float(raw[s].y & 0xffff0000u) * mul);
                }
            }
        }

        float acc[C::DT][4];
#pragma unroll
        for (int d = 0; d < C::DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[d][e] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        for (int t = 0; t < nt; ++t) {
            cp_async_wait<C::NST - 2>();
            __syncthreads();
            if (t + C::NST - 1 < nt)
                issue(t + C::NST - 1);
            cp_async_commit();
            if (tid < kBN) {
                put_row(t + C::NST, tid, next_id);
                next_id = page_id((j0 + t + C::NST + 1) * kBN + tid);
            }
            const uint32_t ks = sm0 + (uint32_t)(t % C::NST) * C::STAGE, vs = ks + C::HALF;
            const int kb0 = (j0 + t) * kBN, kw = wn * C::KW;

            float s[C::NT][4];
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[n][e] = 0.0f;
            if constexpr (!C::F8) {
#pragma unroll
                for (int n2 = 0; n2 < C::NT / 2; ++n2)
#pragma unroll
                    for (int st = 0; st < C::KS; ++st) {
                        uint32_t b[4];
                        ldmatrix4(b, ks + chunk_off<C>(kw + n2 * 16 + ((lane >> 4) << 3) + (lane & 7),
                                                       st * 2 + ((lane >> 3) & 1)));
                        mma16816<false>(s[2 * n2], qf[st], b[0], b[1]);
                        mma16816<false>(s[2 * n2 + 1], qf[st], b[2], b[3]);
                    }
            } else {
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int sg = 0; sg < C::KS / 4; ++sg) {
                        const uint4 b = *reinterpret_cast<const uint4 *>(
                            smem + (ks - sm0) + chunk_off<C>(kw + n * 8 + gr, sg * 4 + qd));
                        const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int st = 0; st < 4; ++st)
                            mma16816<true>(s[n], qf[sg * 4 + st], e4m3x2_to_f16x2(w[st] & 0xffffu),
                                           e4m3x2_to_f16x2(w[st] >> 16));
                    }
            }
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[n][e] *= factor[e >> 1];

            // Units that reach the drafted tokens, or hold a key without a page.
            const uint32_t bad0 = bad[(t % C::NR) * 2], bad1 = bad[(t % C::NR) * 2 + 1];
            const bool masked = kb0 + kBN > rq.len || (bad0 | bad1);
            uint64_t vis[2] = {~0ull, ~0ull};
            bool odd_v = false;
            if (masked) {
                const uint64_t good = ~((uint64_t)bad0 | ((uint64_t)bad1 << 32));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    vis[e] = (visible(p, rq, tok_i[e], kb0) & good) >> kw;
#pragma unroll
                    for (int n = 0; n < C::NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (!((vis[e] >> (n * 8 + 2 * qd + c)) & 1))
                                s[n][2 * e + c] = -INFINITY;
                }
                // a value that is not finite must not reach, times zero, the
                // rows that do not see its key
                for (int i = tid; i < kBN * C::CPR; i += kThreads) {
                    const int row = i / C::CPR;
                    if (kb0 + row >= rq.len) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            smem + (vs - sm0) + chunk_off<C>(row, i % C::CPR));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if constexpr (C::F8)
                                odd_v |= __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
                            else
                                odd_v |= __vcmpeq2(w[k] & 0x7f807f80u, 0x7f807f80u) != 0;
                        }
                    }
                }
                odd_v = __syncthreads_or(odd_v);
            }

            float corr[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = m[e];
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
                    mx = fmaxf(mx, fmaxf(s[n][2 * e], s[n][2 * e + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
                const float ref = mx == -INFINITY ? 0.0f : mx; // nothing seen yet
                corr[e] = exp2_fast(m[e] - ref);
                m[e] = mx;
                float sum = 0.0f;
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        s[n][2 * e + c] = exp2_fast(s[n][2 * e + c] - ref);
                        sum += s[n][2 * e + c];
                    }
                l[e] = l[e] * corr[e] + sum;
            }
#pragma unroll
            for (int d = 0; d < C::DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[d][e] *= corr[e >> 1];

            if (!odd_v) {
                // The weights are rounded to the values' type for the product
                // (bf16: off by at most 2^-8 of each, fp16: 2^-11 or, the small ones, 2^-25);
                // their sum l is of the unrounded ones.
#pragma unroll
                for (int k2 = 0; k2 < C::NT / 2; ++k2) {
                    const uint32_t a[4] = {pack2<C::F8>(s[2 * k2][0], s[2 * k2][1]),
                                           pack2<C::F8>(s[2 * k2][2], s[2 * k2][3]),
                                           pack2<C::F8>(s[2 * k2 + 1][0], s[2 * k2 + 1][1]),
                                           pack2<C::F8>(s[2 * k2 + 1][2], s[2 * k2 + 1][3])};
#pragma unroll
                    for (int d2 = 0; d2 < C::CPR / 2; ++d2) {
                        uint32_t b[4];
                        ldmatrix4_trans(b, vs + chunk_off<C>(kw + k2 * 16 + (((lane >> 3) & 1) << 3) + (lane & 7),
                                                             d2 * 2 + (lane >> 4)));
                        if constexpr (!C::F8) {
                            mma16816<false>(acc[2 * d2], a, b[0], b[1]);
                            mma16816<false>(acc[2 * d2 + 1], a, b[2], b[3]);
                        } else {
                            // a transposed 16-bit element is two columns of one
                            // key: even columns make one product, odd the next
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t x = b[2 * c], y = b[2 * c + 1];
                                mma16816<true>(acc[4 * d2 + 2 * c], a,
                                               e4m3x2_to_f16x2(__byte_perm(x, 0, 0x4420)),
                                               e4m3x2_to_f16x2(__byte_perm(y, 0, 0x4420)));
                                mma16816<true>(acc[4 * d2 + 2 * c + 1], a,
                                               e4m3x2_to_f16x2(__byte_perm(x, 0, 0x4431)),
                                               e4m3x2_to_f16x2(__byte_perm(y, 0, 0x4431)));
                            }
                        }
                    }
                }
            } else {
                // Rare: key by key in fp32, each row adding the keys it sees.
                float w[C::NT][4];
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[n][e] = s[n][e];
#pragma unroll 1
                for (int k = 0; k < C::KW; ++k) {
                    const int from = (lane & ~3) | ((k & 7) >> 1);
                    float pk[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        pk[e] = __shfl_sync(~0u, w[k >> 3][2 * e + (k & 1)], from);
                    const uint8_t *row = smem + (vs - sm0);
#pragma unroll
                    for (int d = 0; d < C::DT; ++d)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float v;
                            if constexpr (C::F8) {
                                const int col = 16 * (d >> 1) + 4 * qd + 2 * c + (d & 1);
                                const uint8_t b = row[chunk_off<C>(kw + k, col >> 4) + (col & 15)];
                                const uint32_t hv = e4m3x2_to_f16x2(b);
                                v = __half2float(__ushort_as_half((unsigned short)(hv & 0xffffu)));
                            } else {
                                const int col = 8 * d + 2 * qd + c;
                                v = bf16_bits_to_float(*reinterpret_cast<const uint16_t *>(
                                    row + chunk_off<C>(kw + k, col >> 3) + 2 * (col & 7)));
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if ((vis[e] >> k) & 1)
                                    acc[d][2 * e + c] = fmaf(pk[e], v, acc[d][2 * e + c]);
                        }
                }
            }
        }
        cp_async_wait_all();
        __syncthreads(); // the stages are free: the warps' sums go there

        // Join the warps that shared the rows, and write.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(~0u, l[e], 1);
            l[e] += __shfl_xor_sync(~0u, l[e], 2);
            if (qd == 0) {
                s_m[wn][wm * 16 + gr + 8 * e] = m[e];
                s_l[wn][wm * 16 + gr + 8 * e] = l[e];
            }
        }
        __syncthreads();
        float *buf = reinterpret_cast<float *>(smem); // [WN][MT][D]
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = wm * 16 + gr + 8 * e;
            float top = s_m[0][row];
#pragma unroll
            for (int w = 1; w < C::WN; ++w)
                top = fmaxf(top, s_m[w][row]);
            const float f = C::WN == 1 || m[e] == -INFINITY ? 1.0f : exp2_fast(m[e] - top);
            float *o = buf + ((size_t)wn * MT + row) * D;
#pragma unroll
            for (int d = 0; d < C::DT; ++d)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = C::F8 ? 16 * (d >> 1) + 4 * qd + 2 * c + (d & 1) : 8 * d + 2 * qd + c;
                    o[col] = acc[d][2 * e + c] * f;
                }
        }
        __syncthreads();
        const bool whole = nt == rq.tiles;
        float *part = ws_part + (size_t)(2 * blockIdx.x + (j0 == 0 ? 1 : 0)) * (MT * (D + 2));
        for (int i = tid; i < MT * (D / 4); i += kThreads) {
            const int row = i / (D / 4), c = (i % (D / 4)) * 4;
            const int g = rt * MT + row, ti = g / G;
            if (ti >= rq.n)
                continue;
            float top = s_m[0][row];
#pragma unroll
            for (int w = 1; w < C::WN; ++w)
                top = fmaxf(top, s_m[w][row]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < C::WN; ++w) {
                const float4 x = *reinterpret_cast<const float4 *>(buf + ((size_t)w * MT + row) * D + c);
                o.x += x.x;
                o.y += x.y;
                o.z += x.z;
                o.w += x.w;
                sum += s_m[w][row] == -INFINITY ? s_l[w][row] : s_l[w][row] * exp2_fast(s_m[w][row] - top);
            }
            if (whole) {
                const float inv = sum == 0.0f ? 0.0f : p.cache.v_scale / sum;
                const long long t = rq.tok + ti;
                const int hq = h * G + g % G;
                const uint2 b = make_uint2(pack2<false>(o.x * inv, o.y * inv), pack2<false>(o.z * inv, o.w * inv));
                *reinterpret_cast<uint2 *>(p.out + t * p.ld_out + (long long)hq * D + c) = b;
                if (p.lse && c == 0)
                    p.lse[t * p.Hq + hq] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(part + (size_t)row * D + c) = o;
                if (c == 0) {
                    part[MT * D + row] = top;
                    part[MT * D + MT + row] = sum;
                }
            }
        }
        __syncthreads();
        u += nt;
    }
}

// One CTA per (token, query head): joins the parts of its row in key order.
template <int D>
__global__ void __launch_bounds__(kThreads) combine_kernel(const AttnProblem p, int MT, int C)
{
    constexpr int LPR = D / 4;              // threads per row of a part
    constexpr int NG = kThreads / LPR;      // parts read side by side
    __shared__ float4 s_o[NG][LPR];
    __shared__ float s_m[NG], s_l[NG];
    const int hq = blockIdx.x % p.Hq;
    const int t = blockIdx.x / p.Hq;
    const int Hkv = p.cache.heads, G = p.Hq / Hkv, h = hq / G;
    grid_launch_dependents();
    grid_dependency_wait();
    int lo = 0, hi = p.R; // the request of row t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_new[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    int bits = 0;
    const Request q = request_of(p, lo, G, MT, bits);
    if (t < q.tok || t >= q.tok + q.n || q.tiles == 0)
        return;
    const long long *ws_units = static_cast<const long long *>(p.workspace);
    const float *ws_part = reinterpret_cast<const float *>(static_cast<const char *>(p.workspace) + units_bytes(p.R));
    const long long U = ws_units[p.R];
    const int g = (t - q.tok) * G + hq % G, rt = g / MT, row = g % MT;
    const long long u0 = ws_units[lo] + ((long long)h * q.row_tiles + rt) * q.tiles;
    if (u0 + q.tiles > U)
        return;
    const int c0 = cta_of(U, u0, C), c1 = cta_of(U, u0 + q.tiles - 1, C);
    if (c0 == c1)
        return; // written whole
    const int parts = U >= C ? c1 - c0 + 1 : q.tiles; // fewer units than CTAs: one each
    const int grp = threadIdx.x / LPR, x = threadIdx.x % LPR;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.0f;
    for (int k = grp; k < parts; k += NG) {
        const int c = U >= C ? c0 + k : cta_of(U, u0 + k, C);
        const float *part = ws_part + (size_t)(2 * c + (k == 0 ? 1 : 0)) * (MT * (D + 2));
        const float pm = part[MT * D + row], pl = part[MT * D + MT + row];
        const float4 v = *reinterpret_cast<const float4 *>(part + (size_t)row * D + 4 * x);
        const float top = fmaxf(m, pm), ref = top == -INFINITY ? 0.0f : top;
        const float a = exp2_fast(m - ref), b = exp2_fast(pm - ref);
        o = make_float4(o.x * a + v.x * b, o.y * a + v.y * b, o.z * a + v.z * b, o.w * a + v.w * b);
        l = l * a + pl * b;
        m = top;
    }
    s_o[grp][x] = o;
    if (x == 0) {
        s_m[grp] = m;
        s_l[grp] = l;
    }
    __syncthreads();
    if (grp)
        return;
    float top = s_m[0];
#pragma unroll
    for (int k = 1; k < NG; ++k)
        top = fmaxf(top, s_m[k]);
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        const float a = s_m[k] == -INFINITY ? 1.0f : exp2_fast(s_m[k] - top); // then all zero, or NaN
        const float4 v = s_o[k][x];
        o = make_float4(o.x + v.x * a, o.y + v.y * a, o.z + v.z * a, o.w + v.w * a);
        l += s_l[k] * a;
    }
    const float inv = l == 0.0f ? 0.0f : p.cache.v_scale / l;
    *reinterpret_cast<uint2 *>(p.out + t * p.ld_out + (long long)hq * D + 4 * x) =
        make_uint2(pack2<false>(o.x * inv, o.y * inv), pack2<false>(o.z * inv, o.w * inv));
    if (p.lse && x == 0)
        p.lse[(long long)t * p.Hq + hq] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
}

template <int D, int KV, int MT>
cudaError_t launch_t(const AttnProblem &p, int grid, cudaStream_t stream)
{
    return launch_step(attn_kernel<D, KV, MT>, grid, kThreads, Cfg<D, KV, MT>::SMEM, 1, stream, p);
}

template <int D, int KV>
cudaError_t launch_d(const AttnProblem &p, int num_sms, cudaStream_t stream)
{
    const int grid = std::min(2 * num_sms, kMaxGrid);
    const int G = p.Hq / p.cache.heads;
    const long long rows = (long long)((p.T + p.R - 1) / p.R) * G;
    const int MT = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    cudaError_t e = MT == 16   ? launch_t<D, KV, 16>(p, grid, stream)
                    : MT == 32 ? launch_t<D, KV, 32>(p, grid, stream)
                               : launch_t<D, KV, 64>(p, grid, stream);
    if (e != cudaSuccess)
        return e;
    return launch_step(combine_kernel<D>, (unsigned)(p.T * p.Hq), kThreads, 0, 1, stream, p, MT, grid);
}

} // namespace

size_t attn_workspace_bytes(int T, int R, int Hq, int Hkv, int D)
{
    (void)T;
    (void)Hq;
    (void)Hkv;
    return units_bytes(R) + (size_t)2 * kMaxGrid * kMaxMT * (D + 2) * sizeof(float);
}

cudaError_t launch_attn(const AttnProblem &p, int num_sms, cudaStream_t stream)
{
    const bool f8 = p.cache.type == SGQ_TYPE_E4M3;
    if (p.cache.dim == 64)
        return f8 ? launch_d<64, SGQ_TYPE_E4M3>(p, num_sms, stream)
                  : launch_d<64, SGQ_TYPE_BF16>(p, num_sms, stream);
    return f8 ? launch_d<128, SGQ_TYPE_E4M3>(p, num_sms, stream)
              : launch_d<128, SGQ_TYPE_BF16>(p, num_sms, stream);
}

} // namespace sgq
