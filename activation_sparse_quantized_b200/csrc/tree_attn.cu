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
// Work is cut into units of 64 keys of one item = (request, key head, row
// tile), and every CTA (one per SM) takes an equal run of them, whatever the
// requests' lengths are (they are known on the device only). An item also
// costs kItemCost units of its own, so that a run of many short requests is
// no longer than one of a few long ones. A run that starts or ends inside an
// item leaves its unnormalised sums with their reference and sum in the
// workspace, and combine_kernel joins them in order; a whole item is written
// out directly.
//
// Both products are tcgen05.mma of 128 rows and 128 keys:
//  * one warp looks up the pages and copies keys and values by the box
//    (cp.async.bulk.tensor, 128-byte swizzle), two ring slots per 128 keys;
//    what lies behind a segment's keys, and bad pages, is filled with zeros by
//    a box outside the map;
//  * one thread issues S = Q K^T (both from shared memory) into one of two
//    accumulators, and O += P V with P read from tensor memory, where it takes
//    S's place;
//  * four warps, one accumulator row per thread, turn S into P. Their reference
//    for the exponent moves only when a row's maximum outgrows it by 2^8, so
//    O is rescaled rarely;
//  * a tile of 32 or 64 rows (MT) is laid into the 128 several times, and copy
//    c takes part c of the keys, its P zero elsewhere: the copies' O are
//    partial sums over the keys, joined at the segment's end. All four warps
//    then share the exponentials of a few rows;
//  * 8-bit keys and values are made fp16 (exact) by four more warps on their
//    way to the slots the products read.
//
// Every wait on a barrier is bounded by 0.2 s; one that runs out sets
// SGQ_STATUS_TIMEOUT, the thread waits on nothing more and the kernel runs to
// its end.
#include "step_launch.cuh"
#include "tc_device.cuh"
#include "tree_attn.cuh"

#include <algorithm>

namespace sgq {

namespace {

constexpr int kTile = 128; // keys per product
constexpr int kSoftWarps = 4, kSoftThreads = 32 * kSoftWarps;
constexpr int kProducer = 4, kIssuer = 5, kConvert = 6; // warps
constexpr uint32_t kColO = 256;                         // tensor-memory columns: S0, S1, O
constexpr float kGrowth = 8.0f;                         // binary orders a row's maximum may outgrow its reference

template <int D_, int KV, int MT_>
struct Cfg {
    static constexpr int D = D_, MT = MT_;
    static constexpr bool F8 = KV == SGQ_TYPE_E4M3;
    static constexpr int THREADS = F8 ? 320 : 192;
    static constexpr int COPIES = 128 / MT, KW = kTile / COPIES; // copies of the rows, keys of each
    static constexpr int SUB = kTile * 128;                      // 128 rows x 64 elements, swizzled
    static constexpr int NSUB = D / 64;
    static constexpr int SLOT = NSUB * SUB;                      // 128 keys (or values), 16 bits
    static constexpr int RAW = kTile * 128;                      // the same, 8 bits (see TcArgs::pitch)
    static constexpr int NS = F8 ? 4 : D == 128 ? 6 : 12;
    static constexpr int RS = F8 ? (D == 128 ? 4 : 6) : 0;
    static constexpr int Q = SLOT;
    static constexpr int BARS = 2 * NS + 2 * RS + 8;
    static constexpr int SMEM = 1024 + Q + NS * SLOT + RS * RAW + BARS * 8;
    static constexpr int LOADS = F8 ? RS : NS; // slots the copies go to
    static_assert(SMEM <= 227 * 1024 - 1800, "room for the static arrays");
};

struct TcArgs {
    AttnProblem p;
    int box;   // rows of a copy's box: the largest power of two up to 64 that divides the page
    int pitch; // bytes from row to row of an 8-bit slot: a box starts on 128 bytes, so a box
               // of one 64-byte row leaves the other 64 empty
};

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory"); }

// Byte offset of 16-byte chunk c (8 elements) of row r of an operand.
__device__ __forceinline__ uint32_t op_off(int r, int c)
{
    return (uint32_t)((c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <int D, int KV, int MT>
__global__ void __launch_bounds__(Cfg<D, KV, MT>::THREADS, 1)
    attn_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap)
{
    using C = Cfg<D, KV, MT>;
    const AttnProblem &p = a.p;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ long long s_scan[4], s_first;
    __shared__ int s_r;
    __shared__ float s_m[C::COPIES][MT], s_l[C::COPIES][MT], s_f[MT];
    __shared__ uint32_t s_bad[8][4]; // keys without a page of the last tiles, bit by key
    __shared__ uint32_t s_odd[4];    // values that are not finite, bit by key
    __shared__ int s_acc[2];         // the first product of a segment adds to O
    uint8_t *smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    const uint32_t sQ = smem_u32(smem), sKV = sQ + C::Q, sRaw = sKV + C::NS * C::SLOT;
    const uint32_t bars = sRaw + C::RS * C::RAW;
    const uint32_t bFull = bars, bEmpty = bFull + 8 * C::NS, bRFull = bEmpty + 8 * C::NS, bREmpty = bRFull + 8 * C::RS;
    const uint32_t bS = bREmpty + 8 * C::RS, bP = bS + 16, bO = bP + 16, bQ = bO + 16, bDone = bQ + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.cache.heads, G = p.Hq / Hkv;

    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "n"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < C::NS; ++s) {
            bar_init(bFull + 8 * s, C::F8 ? 4 : 1);
            bar_init(bEmpty + 8 * s, 1);
        }
        for (int s = 0; s < C::RS; ++s) {
            bar_init(bRFull + 8 * s, 1);
            bar_init(bREmpty + 8 * s, 4);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(bS + 8 * b, 1);
            bar_init(bP + 8 * b, kSoftWarps);
            bar_init(bO + 8 * b, 1);
            s_acc[b] = 0;
        }
        bar_init(bQ, 1);
        bar_init(bDone, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_r = p.R;
    }
    grid_launch_dependents();
    grid_dependency_wait();

    // Cost before each request; this CTA's run.
    long long *ws_units = static_cast<long long *>(p.workspace);
    float *ws_part = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + units_bytes(p.R));
    int bits = 0;
    bool ok = true;
    const int per = (p.R + kSoftThreads - 1) / kSoftThreads;
    const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    long long mine = 0, at = 0;
    if (warp < kSoftWarps) {
        for (int r = r0; r < r1; ++r)
            mine += cost_of(request_of(p, r, G, MT, bits), Hkv);
        long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(~0u, inc, o);
            if (lane >= o)
                inc += t;
        }
        if (lane == 31)
            s_scan[warp] = inc;
        at = inc - mine;
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    const long long U = s_scan[0] + s_scan[1] + s_scan[2] + s_scan[3];
    Walk walk;
    walk.u = run_start(U, blockIdx.x, gridDim.x);
    walk.u_end = run_start(U, blockIdx.x + 1, gridDim.x);
    if (warp < kSoftWarps) {
        for (int w = 0; w < warp; ++w)
            at += s_scan[w];
        if (blockIdx.x == 0 || (walk.u >= at && walk.u < at + mine)) {
            long long s = at;
            int none = 0;
            for (int r = r0; r < r1; ++r) {
                const long long n = cost_of(request_of(p, r, G, MT, none), Hkv);
                if (walk.u >= s && walk.u < s + n) {
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
    }
    __syncthreads();
    walk.r = s_r;
    walk.base = s_first;
    if (walk.r >= p.R)
        walk.u_end = walk.u; // nothing to do
    else {
        int none = 0;
        walk.rq = request_of(p, walk.r, G, MT, none);
    }

    if (warp == kProducer) {
        // ---- pages -> slots ----------------------------------------------
        const uint32_t full = C::F8 ? bRFull : bFull, empty = C::F8 ? bREmpty : bEmpty;
        const uint32_t dst0 = C::F8 ? sRaw : sKV;
        const uint32_t bytes = C::F8 ? kTile * D : C::SLOT; // of one slot's boxes
        constexpr uint32_t STEP = C::F8 ? C::RAW : C::SLOT;
        const int row_bytes = C::F8 ? a.pitch : 128;
        constexpr int PARTS = C::F8 ? 1 : C::NSUB; // boxes side by side in a row
        const int boxes = kTile / a.box;
        const int page = p.cache.page;
        int i = 0, issued = 0; // tiles, slots so far
        while (walk.next(p, G, MT)) {
            const int32_t *table = p.table + (long long)walk.r * p.table_ld;
            const int key0 = walk.j0 * kBN, end = walk.key_end();
            const int nt = (walk.nu + 1) / 2;
            // the pages of a tile's boxes: box lane + 32 j of the tile in id[j]
            int id[4];
            auto look = [&](int t) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + t * kTile + (lane + 32 * j) * a.box;
                    id[j] = lane + 32 * j < boxes && key < end ? table[key / page] : -1;
                }
            };
            look(0);
            for (int t = 0; t < nt; ++t, ++i) {
                int pid[4], slot[4];
                bool any = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + t * kTile + (lane + 32 * j) * a.box;
                    const bool want = lane + 32 * j < boxes && key < end;
                    const bool good = want && id[j] >= 0 && id[j] < p.cache.num_pages;
                    pid[j] = good ? id[j] : p.cache.num_pages; // outside the map: zeros
                    slot[j] = good ? key % page : 0;
                    any |= want && !good;
                }
                any = __any_sync(~0u, any);
                if (lane < 4)
                    s_bad[i & 7][lane] = 0;
                __syncwarp();
                if (any) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int b = lane + 32 * j, key = key0 + t * kTile + b * a.box;
                        if (b < boxes && key < end && pid[j] == p.cache.num_pages)
                            for (int k = 0; k < a.box; ++k)
                                atomicOr(&s_bad[i & 7][(b * a.box + k) >> 5], 1u << ((b * a.box + k) & 31));
                    }
                    if (lane == 0)
                        set_status(p.status, SGQ_STATUS_BAD_INDEX);
                    __syncwarp();
                }
                if (t + 1 < nt)
                    look(t + 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int n = 2 * i + kv, s = n % C::LOADS;
                    if (n >= C::LOADS)
                        bar_wait(empty + 8 * s, (n / C::LOADS - 1) & 1, ok);
                    if (!__all_sync(~0u, ok)) {
                        ok = false;
                        break;
                    }
                    issued = n + 1;
                    if (lane == 0)
                        bar_expect(full + 8 * s, bytes);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int b = lane + 32 * j;
                        if (b < boxes)
#pragma unroll
                            for (int c = 0; c < PARTS; ++c)
                                tma_load_4d(dst0 + s * STEP + c * C::SUB + b * a.box * row_bytes, kv ? &vmap : &kmap,
                                            c * 64, slot[j], walk.h, pid[j], full + 8 * s);
                    }
                }
            }
        }
        // every copy has landed before the CTA ends, whatever went wrong
        bool landed = true;
        for (int n = max(0, issued - C::LOADS); n < issued; ++n)
            bar_wait(full + 8 * (n % C::LOADS), (n / C::LOADS) & 1, landed);
        ok = ok && landed;
    } else if (warp == kIssuer) {
        // ---- the products ------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t idS = idesc_f16(!C::F8, false, kTile), idO = idesc_f16(!C::F8, true, D);
            const uint64_t dq = desc_sw128(sQ, 16, 1024);
            auto scores = [&](int i) {
                const int n = 2 * i, s = n % C::NS;
                bar_wait(bFull + 8 * s, (n / C::NS) & 1, ok);
                tc_after();
                const uint64_t dk = desc_sw128(sKV + s * C::SLOT, 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t step = (uint64_t)(((k >> 2) * C::SUB + (k & 3) * 32) >> 4);
                    mma_ss(tmem + (i & 1) * kTile, dq + step, dk + step, idS, k > 0);
                }
                tc_commit(bEmpty + 8 * s);
                tc_commit(bS + 8 * (i & 1));
            };
            int i = 0, seg = 0;
            while (walk.next(p, G, MT)) {
                const int nt = (walk.nu + 1) / 2;
                bar_wait(bQ, seg & 1, ok);
                ++seg;
                scores(i);
                for (int t = 0; t < nt; ++t, ++i) {
                    if (t + 1 < nt)
                        scores(i + 1);
                    const int n = 2 * i + 1, s = n % C::NS;
                    bar_wait(bFull + 8 * s, (n / C::NS) & 1, ok);
                    bar_wait(bP + 8 * (i & 1), (i >> 1) & 1, ok);
                    tc_after();
                    const uint32_t add = t > 0 || *(volatile int *)&s_acc[i & 1];
                    const uint64_t dv = desc_sw128(sKV + s * C::SLOT, C::SUB, 1024);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_ts(tmem + kColO, tmem + (i & 1) * kTile + 8 * k, dv + (uint64_t)((k * 2048) >> 4), idO, add | (k > 0));
                    tc_commit(bEmpty + 8 * s);
                    tc_commit(bO + 8 * (i & 1));
                }
            }
            tc_commit(bDone);
            bool done = true;
            bar_wait(bDone, 0, done);
            ok = ok && done;
        }
        __syncwarp();
    } else if (C::F8 && warp >= kConvert) {
        // ---- 8-bit slots -> fp16 slots -----------------------------------
        const int ct = tid - 32 * kConvert;
        int n = 0;
        while (walk.next(p, G, MT)) {
            const int last = n + 2 * ((walk.nu + 1) / 2);
            for (; n < last; ++n) {
                const int rs = n % max(C::RS, 1), s = n % C::NS;
                bar_wait(bRFull + 8 * rs, (n / max(C::RS, 1)) & 1, ok);
                if (n >= C::NS)
                    bar_wait(bEmpty + 8 * s, (n / C::NS - 1) & 1, ok);
                __syncwarp();
                const uint8_t *src = smem + (sRaw - sQ) + rs * C::RAW;
                uint8_t *dst = smem + (sKV - sQ) + s * C::SLOT;
#pragma unroll 4
                for (int k = 0; k < kTile * D / 16 / 128; ++k) {
                    const int idx = ct + k * 128, row = idx / (D / 16), c = idx % (D / 16);
                    const int x = c ^ (((row * a.pitch) >> 7) & (D / 16 - 1)); // the copies' swizzle
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + row * a.pitch + 16 * x);
                    *reinterpret_cast<uint4 *>(dst + op_off(row, 2 * c)) =
                        make_uint4(e4m3x2_to_f16x2(v.x & 0xffffu), e4m3x2_to_f16x2(v.x >> 16),
                                   e4m3x2_to_f16x2(v.y & 0xffffu), e4m3x2_to_f16x2(v.y >> 16));
                    *reinterpret_cast<uint4 *>(dst + op_off(row, 2 * c + 1)) =
                        make_uint4(e4m3x2_to_f16x2(v.z & 0xffffu), e4m3x2_to_f16x2(v.z >> 16),
                                   e4m3x2_to_f16x2(v.w & 0xffffu), e4m3x2_to_f16x2(v.w >> 16));
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(bFull + 8 * s);
                    bar_arrive(bREmpty + 8 * rs);
                }
            }
        }
    } else {
        // ---- the softmax -------------------------------------------------
        const int quad = warp / (MT / 32), row = (warp % (MT / 32)) * 32 + lane; // copy, row of the tile
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;
        const uint32_t tO = tmem + kColO + lanes;
        int i = 0;
        while (walk.next(p, G, MT)) {
            const Request &rq = walk.rq;
            const int nt = (walk.nu + 1) / 2, end = walk.key_end(), key0 = walk.j0 * kBN;

            // Q, once per copy of the rows. With 8-bit keys q becomes fp16, each
            // row by the power of two that brings its largest value into
            // [2^7, 2^8): exact for values down to 2^-21 of that, below it off
            // by at most 2^-33 of it. A negative scale's sign goes to q, so that
            // the largest score is the largest exponent.
            {
                constexpr int CH = D / 8, N = MT * CH / kSoftThreads;
                uint4 v[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int idx = tid + k * kSoftThreads, g = walk.rt * MT + idx / CH, ti = g / G;
                    v[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (ti < rq.n)
                        v[k] = *reinterpret_cast<const uint4 *>(
                            p.q + (rq.tok + ti) * p.ld_q + (long long)(walk.h * G + g % G) * D + 8 * (idx % CH));
                }
                const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int idx = tid + k * kSoftThreads, qr = idx / CH, c = idx % CH;
                    uint32_t w[4] = {v[k].x ^ flip, v[k].y ^ flip, v[k].z ^ flip, v[k].w ^ flip};
                    if constexpr (C::F8) {
                        float mx = 0.0f;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
#pragma unroll
                        for (int o = CH / 2; o; o >>= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
                        // both the power and its inverse are normal fp32 numbers
                        const int up = min(max(7 - ((int)(__float_as_uint(mx) >> 23) - 127), -126), 126);
                        const float mul = pow2f(up);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack2<true>(__uint_as_float(w[e] << 16) * mul, __uint_as_float(w[e] & 0xffff0000u) * mul);
                        if (c == 0)
                            s_f[qr] = pow2f(-up);
                    }
#pragma unroll
                    for (int cp = 0; cp < C::COPIES; ++cp)
                        *reinterpret_cast<uint4 *>(smem + op_off(qr + cp * MT, c)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_async_smem();
                soft_sync();
                if (tid == 0)
                    bar_arrive(bQ);
            }
            const int g = walk.rt * MT + row;
            const bool live = g / G < rq.n;
            const int tok_i = live ? g / G : 0;
            const bool warp_live = __any_sync(~0u, live);
            float factor = fabsf(p.scale) * p.cache.k_scale * kLog2e;
            if constexpr (C::F8)
                factor *= s_f[row];
            factor = fmaxf(factor, 1e-37f); // a scale of zero: all scores alike
            float m = -INFINITY, l = 0.0f; // reference (base 2), sum

            for (int t = 0; t < nt; ++t, ++i) {
                const uint32_t tS = tmem + (i & 1) * kTile + lanes;
                const int kt = key0 + t * kTile, kq = kt + quad * C::KW; // first key of the tile, of this copy
                bar_wait(bS + 8 * (i & 1), (i >> 1) & 1, ok);
                if (i >= 2)
                    bar_wait(bO + 8 * (i & 1), ((i - 2) >> 1) & 1, ok);
                __syncwarp();
                tc_after();
                if (tid == 0)
                    s_acc[i & 1] = 0;
                uint32_t s[C::KW];
                if (warp_live) {
#pragma unroll
                    for (int c = 0; c < C::KW; c += 32)
                        tmem_ld32(tS + quad * C::KW + c, s + c);
#pragma unroll
                    for (int c = 0; c < C::KW; c += 32)
                        tmem_ld_wait(s + c);
                }
                // Tiles that reach the drafted tokens or the end, or hold a key
                // without a page.
                const uint32_t *bad = s_bad[i & 7];
                if (kt + kTile > min(rq.len, end) || (bad[0] | bad[1] | bad[2] | bad[3])) {
                    uint64_t vis[(C::KW + 63) / 64];
#pragma unroll
                    for (int c = 0; c < C::KW; c += 64) {
                        const int w = (quad * C::KW + c) >> 5;
                        const uint64_t b = C::KW >= 64 ? bad[w] | ((uint64_t)bad[w + 1] << 32) : bad[w];
                        vis[c / 64] = visible(p, rq, tok_i, kq + c, end) & ~b;
                    }
#pragma unroll
                    for (int c = 0; c < C::KW; ++c)
                        if (!((vis[c / 64] >> (c & 63)) & 1))
                            s[c] = 0xff800000u;
                    // Values behind the end become zero; one that is not finite
                    // must not reach, times zero, the rows that do not see it.
                    const int n = 2 * i + 1, sl = n % C::NS;
                    bar_wait(bFull + 8 * sl, (n / C::NS) & 1, ok);
                    uint8_t *vs = smem + (sKV - sQ) + sl * C::SLOT;
                    bool odd = false;
                    if (kt + tid >= end) {
#pragma unroll
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4 *>(vs + op_off(tid, c)) = make_uint4(0u, 0u, 0u, 0u);
                    } else if (kt + tid >= rq.len) {
                        constexpr uint32_t EXP = C::F8 ? 0x7c007c00u : 0x7f807f80u;
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(vs + op_off(tid, c));
                            odd |= (__vcmpeq2(v.x & EXP, EXP) | __vcmpeq2(v.y & EXP, EXP) | __vcmpeq2(v.z & EXP, EXP) |
                                    __vcmpeq2(v.w & EXP, EXP)) != 0;
                        }
                    }
                    __syncwarp();
                    const uint32_t ob = __ballot_sync(~0u, odd);
                    if (lane == 0)
                        s_odd[warp] = ob;
                    soft_sync();
                    if (s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3]) {
                        // Rare: what is not finite is added to O here, for the
                        // rows that see it, and taken out of the slot.
                        if (t > 0)
                            bar_wait(bO + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, ok);
                        __syncwarp();
                        tc_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + c, o);
                            tmem_ld_wait(o);
                            if (t == 0)
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = 0u;
#pragma unroll 1
                            for (int k = 0; k < C::KW; ++k) {
                                const int kr = quad * C::KW + k; // row of the slot
                                if (!((s_odd[kr >> 5] >> (kr & 31)) & 1) || !((vis[k >> 6] >> (k & 63)) & 1))
                                    continue;
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const uint16_t b = *reinterpret_cast<const uint16_t *>(vs + op_off(kr, (c + e) >> 3) + 2 * (e & 7));
                                    const float v = C::F8 ? __half2float(__ushort_as_half(b)) : bf16_bits_to_float(b);
                                    if (!isfinite(v))
                                        o[e] = __float_as_uint(__uint_as_float(o[e]) + v);
                                }
                            }
                            __syncwarp();
                            tmem_st32(tO + c, o);
                        }
                        tmem_st_wait();
                        soft_sync();
                        if (odd) {
                            constexpr uint16_t EXP = C::F8 ? 0x7c00 : 0x7f80;
                            for (int e = 0; e < D; ++e) {
                                uint16_t *b = reinterpret_cast<uint16_t *>(vs + op_off(tid, e >> 3) + 2 * (e & 7));
                                if ((*b & EXP) == EXP)
                                    *b = 0;
                            }
                        }
                        if (tid == 0)
                            s_acc[i & 1] = t == 0;
                    }
                    fence_async_smem();
                    soft_sync();
                }
                if (warp_live) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int c = 0; c < C::KW; ++c)
                        mx = fmaxf(mx, __uint_as_float(s[c]));
                    mx *= factor;
                    // the reference moves for the first keys seen, and when outgrown
                    const bool grow = mx > m + kGrowth || (m == -INFINITY && mx > m);
                    if (__any_sync(~0u, grow)) {
                        const float to = grow ? mx : m;
                        const float corr = grow ? exp2_fast(m - to) : 1.0f;
                        m = to;
                        l *= corr;
                        if (t > 0) {
                            bar_wait(bO + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, ok);
                            __syncwarp();
                            tc_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(tO + c, o);
                                tmem_ld_wait(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                                tmem_st32(tO + c, o);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.0f : m; // nothing seen yet
                    // The weights are rounded to the values' type for the product
                    // (bf16: off by at most 2^-8 of each, fp16: 2^-11 or, the
                    // small ones, 2^-25); their sum l is of the unrounded ones.
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    uint32_t w[C::KW / 2];
#pragma unroll
                    for (int c = 0; c < C::KW; c += 2) {
                        const float x = exp2_fast(fmaf(__uint_as_float(s[c]), factor, -ref));
                        const float y = exp2_fast(fmaf(__uint_as_float(s[c + 1]), factor, -ref));
                        sum[c & 2] += x;
                        sum[(c & 2) + 1] += y;
                        w[c / 2] = pack2<C::F8>(x, y);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    if constexpr (C::COPIES == 1) {
                        tmem_st32(tS, w);
                        tmem_st32(tS + 32, w + 32);
                    } else {
                        const uint32_t z[32] = {};
#pragma unroll
                        for (int b = 0; b < C::COPIES; ++b) {
                            if constexpr (MT == 64)
                                tmem_st32(tS + 32 * b, b == quad ? w : z);
                            else
                                tmem_st16(tS + 16 * b, b == quad ? w : z);
                        }
                    }
                    tmem_st_wait();
                }
                tc_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(bP + 8 * (i & 1));
            }

            // ---- the segment's end: O is complete ----
            const int last = i - 1;
            if (last >= 1)
                bar_wait(bO + 8 * ((last - 1) & 1), ((last - 1) >> 1) & 1, ok);
            bar_wait(bO + 8 * (last & 1), (last >> 1) & 1, ok);
            __syncwarp();
            tc_after();
            const bool whole = walk.whole();
            float *part = ws_part + (size_t)(2 * blockIdx.x + (walk.j0 == 0 ? 1 : 0)) * (MT * (D + 2));
            if constexpr (C::COPIES == 1) {
                const long long tk = rq.tok + tok_i;
                const int hq = walk.h * G + g % G;
                const float inv = l == 0.0f ? 0.0f : p.cache.v_scale / l;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + c, o);
                    tmem_ld_wait(o);
                    if (live && whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(p.out + tk * p.ld_out + (long long)hq * D + c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t b[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                b[x] = pack2<false>(__uint_as_float(o[8 * e + 2 * x]) * inv, __uint_as_float(o[8 * e + 2 * x + 1]) * inv);
                            dst[e] = make_uint4(b[0], b[1], b[2], b[3]);
                        }
                    } else if (live) {
                        uint4 *dst = reinterpret_cast<uint4 *>(part + (size_t)row * D + c);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                    __syncwarp();
                }
                if (live && whole && p.lse)
                    p.lse[tk * p.Hq + hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
                if (live && !whole) {
                    part[MT * D + row] = m;
                    part[MT * D + MT + row] = l;
                }
                tc_before();
                soft_sync(); // s_f and the operand are free for the next segment
            } else {
                // join the copies, in the operand's place (its products are done)
                s_m[quad][row] = m;
                s_l[quad][row] = l;
                soft_sync();
                float top = s_m[0][row];
#pragma unroll
                for (int c = 1; c < C::COPIES; ++c)
                    top = fmaxf(top, s_m[c][row]);
                const float f = m == -INFINITY ? 1.0f : exp2_fast(m - top); // then all zero, or NaN
                constexpr int HALF = C::COPIES / 2;
                float4 *buf = reinterpret_cast<float4 *>(smem) + ((quad % HALF) * MT + row) * (D / 4);
#pragma unroll
                for (int pass = 0; pass < 2; ++pass) {
                    if ((quad >= HALF) == (pass == 0) && warp_live)
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + c, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float4 x = make_float4(__uint_as_float(o[4 * e]) * f, __uint_as_float(o[4 * e + 1]) * f,
                                                       __uint_as_float(o[4 * e + 2]) * f, __uint_as_float(o[4 * e + 3]) * f);
                                float4 &b = buf[(c / 4 + e) ^ (row & 7)];
                                if (pass)
                                    x = make_float4(x.x + b.x, x.y + b.y, x.z + b.z, x.w + b.w);
                                b = x;
                            }
                        }
                    tc_before();
                    soft_sync();
                }
                for (int k = tid; k < MT * (D / 4); k += kSoftThreads) {
                    const int rr = k / (D / 4), c4 = k % (D / 4), gg = walk.rt * MT + rr, ti = gg / G;
                    if (ti >= rq.n)
                        break;
                    const float4 *b = reinterpret_cast<const float4 *>(smem) + rr * (D / 4) + (c4 ^ (rr & 7));
                    float4 o = b[0];
                    if constexpr (HALF == 2) {
                        const float4 x = b[MT * (D / 4)];
                        o = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
                    }
                    float mt = s_m[0][rr], sum = 0.0f;
#pragma unroll
                    for (int c = 1; c < C::COPIES; ++c)
                        mt = fmaxf(mt, s_m[c][rr]);
#pragma unroll
                    for (int c = 0; c < C::COPIES; ++c)
                        sum += s_m[c][rr] == -INFINITY ? s_l[c][rr] : s_l[c][rr] * exp2_fast(s_m[c][rr] - mt);
                    if (whole) {
                        const float inv = sum == 0.0f ? 0.0f : p.cache.v_scale / sum;
                        const long long tk = rq.tok + ti;
                        const int hq = walk.h * G + gg % G;
                        *reinterpret_cast<uint2 *>(p.out + tk * p.ld_out + (long long)hq * D + 4 * c4) =
                            make_uint2(pack2<false>(o.x * inv, o.y * inv), pack2<false>(o.z * inv, o.w * inv));
                        if (p.lse && c4 == 0)
                            p.lse[tk * p.Hq + hq] = sum == 0.0f ? -INFINITY : (mt + log2f(sum)) * kLn2;
                    } else {
                        *reinterpret_cast<float4 *>(part + (size_t)rr * D + 4 * c4) = o;
                        if (c4 == 0) {
                            part[MT * D + rr] = mt;
                            part[MT * D + MT + rr] = sum;
                        }
                    }
                }
                soft_sync(); // the operand's place is free for the next segment
            }
        }
    }
    if (!ok)
        set_status(p.status, SGQ_STATUS_TIMEOUT);
    tc_before();
    __syncthreads();
    if (warp == kIssuer)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

// One CTA per (token, query head): joins the parts of its row in key order.
constexpr int kJoinThreads = 128;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const AttnProblem p, int MT, int C)
{
    constexpr int LPR = D / 4;              // threads per row of a part
    constexpr int NG = kJoinThreads / LPR;      // parts read side by side
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
    const long long u0 = ws_units[lo] + ((long long)h * q.row_tiles + rt) * (q.tiles + kItemCost);
    if (u0 + q.tiles + kItemCost > U)
        return;
    const int c0 = cta_of(U, u0, C), c1 = cta_of(U, u0 + q.tiles - 1, C);
    if (c0 == c1)
        return; // written whole
    const int parts = U >= C ? c1 - c0 + 1 : q.tiles; // fewer positions than CTAs: one each
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

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps, looked up once.
EncodeTiled encoder()
{
    static const EncodeTiled f = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<EncodeTiled>(fn);
    }();
    return f;
}

// (element, slot, head, page) of the cache; a box is 128 bytes of a row (64
// where the row has no more) times `box` slots of one page and head. A
// dimension of one entry has no stride of its own: any valid one will do.
bool encode(CUtensorMap *map, const sgq_cache &c, void *base, int box)
{
    const bool f8 = c.type == SGQ_TYPE_E4M3;
    const int es = f8 ? 1 : 2, inner = std::min(c.dim, 128 / es);
    const cuuint64_t row = (cuuint64_t)c.dim * es;
    const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page, (cuuint64_t)c.heads, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {c.page > 1 ? (cuuint64_t)c.slot_stride * es : row,
                                   c.heads > 1 ? (cuuint64_t)c.head_stride * es : row,
                                   c.num_pages > 1 ? (cuuint64_t)c.page_stride * es : row};
    const cuuint32_t boxes[4] = {(cuuint32_t)inner, (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
    return encoder()(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, boxes,
                     ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     inner * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int KV, int MT>
cudaError_t launch_t(const AttnProblem &p, int grid, cudaStream_t stream)
{
    using C = Cfg<D, KV, MT>;
    TcArgs a;
    a.p = p;
    a.box = 1;
    while (a.box < 64 && p.cache.page % (2 * a.box) == 0)
        a.box *= 2;
    a.pitch = a.box == 1 ? 128 : D;
    CUtensorMap kmap, vmap;
    if (!encoder())
        return cudaErrorNotSupported;
    if (!encode(&kmap, p.cache, p.cache.k, a.box) || !encode(&vmap, p.cache, p.cache.v, a.box))
        return cudaErrorInvalidValue;
    cudaError_t e = launch_step(attn_kernel<D, KV, MT>, grid, C::THREADS, C::SMEM, 1, stream, a, kmap, vmap);
    if (e != cudaSuccess)
        return e;
    return launch_step(combine_kernel<D>, (unsigned)(p.T * p.Hq), kJoinThreads, 0, 1, stream, p, MT, grid);
}

template <int D, int KV>
cudaError_t launch_d(const AttnProblem &p, int num_sms, cudaStream_t stream)
{
    const int grid = std::min(num_sms, kMaxGrid);
    const int G = p.Hq / p.cache.heads;
    const long long rows = (long long)((p.T + p.R - 1) / p.R) * G;
    return rows <= 32   ? launch_t<D, KV, 32>(p, grid, stream)
           : rows <= 64 ? launch_t<D, KV, 64>(p, grid, stream)
                        : launch_t<D, KV, 128>(p, grid, stream);
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
