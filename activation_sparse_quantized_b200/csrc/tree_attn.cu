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
// workspace, and join_kernel joins them in order; a whole item is written out
// directly.
//
// Both products are tcgen05.mma of 128 rows and 128 keys. Eight warps:
//  * one looks up the pages and copies keys and values by the box
//    (cp.async.bulk.tensor, 128-byte swizzle), two ring slots per 128 keys;
//    what lies behind a segment's keys, and bad pages, is filled with zeros by
//    a box outside the map;
//  * one thread of another issues S = Q K^T (both from shared memory) into one
//    of two accumulators, one tile ahead and across segments, and O += P V
//    with P read from tensor memory, where it takes S's place;
//  * four, one accumulator row per thread, turn S into P. Their reference for
//    the exponent moves only when a row's maximum outgrows it by 2^8, so O is
//    rescaled rarely;
//  * two fetch the next segment's Q, look through the values next to the end,
//    and make 8-bit keys and values fp16 (exact) on their way to the slots the
//    products read.
// A tile of 32 or 64 rows (MT) is laid into the 128 several times, and copy c
// takes part c of the keys, its P zero elsewhere: the copies' O are partial
// sums over the keys, joined at the segment's end. All four softmax warps then
// share the exponentials of a few rows.
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
constexpr int kSoftThreads = 128, kAuxThreads = 64, kThreads = 256;
constexpr int kSoftWarps = 4, kProducer = 4, kIssuer = 5, kAux = 6; // warps
constexpr uint32_t kColO = 256; // tensor-memory columns: S0, S1, O
constexpr float kGrowth = 8.0f; // binary orders a row's maximum may outgrow its reference

template <int D_, int KV, int MT_>
struct Cfg {
    static constexpr int D = D_, MT = MT_;
    static constexpr bool F8 = KV == SGQ_TYPE_E4M3;
    static constexpr int COPIES = 128 / MT, KW = kTile / COPIES; // copies of the rows, keys of each
    static constexpr int SUB = kTile * 128;                      // 128 rows x 64 elements, swizzled
    static constexpr int NSUB = D / 64;
    static constexpr int SLOT = NSUB * SUB;                      // 128 keys (or values), 16 bits
    static constexpr int RAW = kTile * 128;                      // the same, 8 bits (see TcArgs::pitch)
    static constexpr int NS = F8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
    static constexpr int RS = F8 ? 4 : 0;
    static constexpr int Q = SLOT, JOIN = MT == 128 ? 0 : 128 * 32 * 4;
    static constexpr int BARS = 2 * NS + 2 * RS + 12;
    static constexpr int SMEM = 1024 + Q + JOIN + NS * SLOT + RS * RAW + BARS * 8;
    static constexpr int LOADS = F8 ? RS : NS; // slots the copies go to
    static_assert(SMEM <= 227 * 1024 - 4096, "room for the static arrays");
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
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap)
{
    using C = Cfg<D, KV, MT>;
    const AttnProblem &p = a.p;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ long long s_scan[4], s_first;
    __shared__ int s_r;
    __shared__ Request s_rq;
    __shared__ float s_m[C::COPIES][MT], s_l[C::COPIES][MT];
    __shared__ float s_f[C::F8 ? 4 : 1][C::F8 ? MT : 1]; // q's powers of two, by segment
    __shared__ uint32_t s_bad[8][4];                     // keys without a page of the last tiles, bit by key
    __shared__ uint32_t s_odd[4][4];                     // values that are not finite of the last tail tiles
    __shared__ int s_acc[2];                             // the first product of a segment adds to O
    uint8_t *smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    const uint32_t sQ = smem_u32(smem), sKV = sQ + C::Q, sRaw = sKV + C::NS * C::SLOT;
    const uint32_t sJoin = sRaw + C::RS * C::RAW, bars = sJoin + C::JOIN;
    const uint32_t bFull = bars, bEmpty = bFull + 8 * C::NS, bRFull = bEmpty + 8 * C::NS, bREmpty = bRFull + 8 * C::RS;
    const uint32_t bS = bREmpty + 8 * C::RS, bP = bS + 16, bO = bP + 16, bTail = bO + 16;
    const uint32_t bQ = bTail + 32, bQFree = bQ + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.cache.heads, G = p.Hq / Hkv;

    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "n"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (warp == kProducer && lane == 0) {
        for (int s = 0; s < C::NS; ++s) {
            bar_init(bFull + 8 * s, C::F8 ? 2 : 1);
            bar_init(bEmpty + 8 * s, 1);
        }
        for (int s = 0; s < C::RS; ++s) {
            bar_init(bRFull + 8 * s, 1);
            bar_init(bREmpty + 8 * s, 2);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(bS + 8 * b, 1);
            bar_init(bP + 8 * b, kSoftWarps);
            bar_init(bO + 8 * b, 1);
            s_acc[b] = 0;
        }
        for (int b = 0; b < 4; ++b)
            bar_init(bTail + 8 * b, 2);
        bar_init(bQ, 2);
        bar_init(bQFree, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_r = p.R;
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    }
    grid_launch_dependents();
    grid_dependency_wait();

    // The requests' costs, their sum U, and this CTA's run of [0, U).
    int bits = 0;
    bool ok = true;
    const int per = (p.R + kSoftThreads - 1) / kSoftThreads;
    const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    long long mine = 0, at = 0;
    Request rq0{};
    if (warp < kSoftWarps) {
        for (int r = r0; r < r1; ++r) {
            rq0 = request_of(p, r, G, MT, bits);
            mine += cost_of(rq0, Hkv);
        }
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
        if (bits && blockIdx.x == 0)
            set_status(p.status, bits);
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    const long long U = s_scan[0] + s_scan[1] + s_scan[2] + s_scan[3];
    const int ctas = (int)min((long long)gridDim.x, U); // those with work
    Walk walk;
    if ((int)blockIdx.x < ctas) {
        walk.u = run_start(U, blockIdx.x, ctas);
        walk.u_end = run_start(U, blockIdx.x + 1, ctas);
    }
    if (warp < kSoftWarps && walk.u < walk.u_end) {
        for (int w = 0; w < warp; ++w)
            at += s_scan[w];
        if (walk.u >= at && walk.u < at + mine) {
            int r = r0, none = 0;
            if (per > 1)
                for (; r < r1; ++r) {
                    rq0 = request_of(p, r, G, MT, none);
                    const long long n = cost_of(rq0, Hkv);
                    if (walk.u < at + n)
                        break;
                    at += n;
                }
            s_r = r;
            s_first = at;
            s_rq = rq0;
        }
    }
    __syncthreads();
    walk.r = s_r;
    walk.base = s_first;
    walk.rq = s_rq;

    if (warp == kProducer) {
        // ---- pages -> slots ----------------------------------------------
        // Lane x of round j copies piece x + 32 j of a slot: a box of `box` rows
        // and 128 bytes (one round for pages of at least 8 slots). The pages of
        // the next two tiles are looked up ahead.
        const uint32_t full = C::F8 ? bRFull : bFull, empty = C::F8 ? bREmpty : bEmpty;
        const uint32_t dst0 = C::F8 ? sRaw : sKV;
        const uint32_t bytes = C::F8 ? kTile * D : C::SLOT; // of one slot's boxes
        constexpr uint32_t STEP = C::F8 ? C::RAW : C::SLOT;
        constexpr int PARTS = C::F8 ? 1 : C::NSUB; // boxes side by side in a row
        const int row_bytes = C::F8 ? a.pitch : 128;
        const int pieces = kTile / a.box * PARTS, rounds = (pieces + 31) / 32;
        const int page = p.cache.page, page_up = kTile / page, slot_up = kTile % page;
        int i = 0, issued = 0; // tiles, slots so far
        while (walk.next(p, G, MT)) {
            const int32_t *table = p.table + (long long)walk.r * p.table_ld;
            const int key0 = walk.j0 * kBN, end = walk.key_end();
            const int nt = (walk.nu + 1) / 2;
            // this lane's box of round 0: page index, slot in it, ids of the next tiles
            const int first = key0 + lane / PARTS * a.box;
            int pg = first / page, sl = first - pg * page;
            auto look = [&](int t, int at_page) {
                return lane < pieces && t < nt && first + t * kTile < end ? table[at_page] : -1;
            };
            int pg_next = pg, sl_next = sl; // one tile on
            auto step = [&](int &g, int &s) {
                g += page_up;
                s += slot_up;
                if (s >= page) {
                    s -= page;
                    ++g;
                }
            };
            int id0 = look(0, pg);
            step(pg_next, sl_next);
            int id1 = look(1, pg_next);
            for (int t = 0; t < nt; ++t, ++i) {
                int pg2 = pg_next, sl2 = sl_next;
                step(pg2, sl2);
                const int id2 = look(t + 2, pg2);
                if (lane < 4)
                    s_bad[i & 7][lane] = 0;
                // round 0's box; its page is waited for here
                const int key = first + t * kTile;
                const bool want = lane < pieces && key < end;
                const bool good = want && id0 >= 0 && id0 < p.cache.num_pages;
                const int pid = good ? id0 : p.cache.num_pages; // outside the map: zeros
                const int slot = good ? sl : 0;
                bool any = __any_sync(~0u, want && !good);
                __syncwarp();
                if (any && want && !good && lane % PARTS == 0)
                    for (int k = 0; k < a.box; ++k) {
                        const int b = lane / PARTS * a.box + k;
                        atomicOr(&s_bad[i & 7][b >> 5], 1u << (b & 31));
                    }
                for (int j = 1; j < rounds; ++j) { // boxes of fewer than 8 rows: their keys without a page
                    const int b = (lane + 32 * j) / PARTS, kb = key0 + t * kTile + b * a.box;
                    if (kb < end) {
                        const int id = table[kb / page];
                        if (id < 0 || id >= p.cache.num_pages) {
                            any = true;
                            for (int k = 0; k < a.box; ++k)
                                atomicOr(&s_bad[i & 7][(b * a.box + k) >> 5], 1u << ((b * a.box + k) & 31));
                        }
                    }
                }
                if (any)
                    set_status(p.status, SGQ_STATUS_BAD_INDEX);
                __syncwarp();
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
                    const CUtensorMap *map = kv ? &vmap : &kmap;
                    const uint32_t dst = dst0 + s * STEP;
                    if (lane < pieces)
                        tma_load_4d(dst + (lane % PARTS) * C::SUB + lane / PARTS * a.box * row_bytes, map, lane % PARTS * 64, slot,
                                    walk.h, pid, full + 8 * s);
                    for (int j = 1; j < rounds; ++j) {
                        const int x = lane + 32 * j, b = x / PARTS, kb = key0 + t * kTile + b * a.box;
                        int id = kb < end ? table[kb / page] : -1;
                        if (id < 0 || id >= p.cache.num_pages)
                            id = p.cache.num_pages;
                        tma_load_4d(dst + (x % PARTS) * C::SUB + b * a.box * row_bytes, map, x % PARTS * 64, kb % page, walk.h, id,
                                    full + 8 * s);
                    }
                }
                pg = pg_next;
                sl = sl_next;
                pg_next = pg2;
                sl_next = sl2;
                id0 = id1;
                id1 = id2;
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
            int seg = 0, left = 0, i = 0; // segments begun, their tiles without scores, tiles
            // The scores of tile n, the next one; false when there is none.
            auto scores = [&](int n) -> bool {
                if (left == 0) {
                    if (!walk.next(p, G, MT))
                        return false;
                    left = (walk.nu + 1) / 2;
                    bar_wait(bQ, seg & 1, ok);
                    ++seg;
                }
                --left;
                const int s = 2 * n % C::NS;
                bar_wait(bFull + 8 * s, (2 * n / C::NS) & 1, ok);
                tc_after();
                const uint64_t dk = desc_sw128(sKV + s * C::SLOT, 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t step = (uint64_t)(((k >> 2) * C::SUB + (k & 3) * 32) >> 4);
                    mma_ss(tmem + (n & 1) * kTile, dq + step, dk + step, idS, k > 0);
                }
                tc_commit(bEmpty + 8 * s);
                tc_commit(bS + 8 * (n & 1));
                if (left == 0)
                    tc_commit(bQFree);
                return true;
            };
            bool first = true, more = scores(0);
            while (more) {
                const bool last = left == 0; // of its segment
                more = scores(i + 1);
                const int n = 2 * i + 1, s = n % C::NS;
                bar_wait(bFull + 8 * s, (n / C::NS) & 1, ok);
                bar_wait(bP + 8 * (i & 1), (i >> 1) & 1, ok);
                tc_after();
                const uint32_t add = !first || *(volatile int *)&s_acc[i & 1];
                const uint64_t dv = desc_sw128(sKV + s * C::SLOT, C::SUB, 1024);
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_ts(tmem + kColO, tmem + (i & 1) * kTile + 8 * k, dv + (uint64_t)((k * 2048) >> 4), idO, add | (k > 0));
                tc_commit(bEmpty + 8 * s);
                tc_commit(bO + 8 * (i & 1));
                first = last;
                ++i;
            }
            // every product is complete before the tensor memory is freed
            bool done = true;
            if (i >= 2)
                bar_wait(bO + 8 * (i & 1), ((i - 2) >> 1) & 1, done);
            if (i >= 1)
                bar_wait(bO + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, done);
            ok = ok && done;
        }
        __syncwarp();
    } else if (warp >= kAux) {
        // ---- Q, the values next to the end, 8-bit slots -> fp16 slots --------
        const int ct = tid - 32 * kAux;
        int i = 0, seg = 0, tail = 0;
        while (walk.next(p, G, MT)) {
            const Request &rq = walk.rq;
            // Q, once per copy of the rows. With 8-bit keys q becomes fp16, each
            // row by the power of two that brings its largest value into
            // [2^7, 2^8): exact for values down to 2^-21 of that, below it off
            // by at most 2^-33 of it. A negative scale's sign goes to q, so that
            // the largest score is the largest exponent.
            constexpr int CH = D / 8, N = 8;
            const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;
            bool waited = false;
#pragma unroll 1
            for (int k0 = 0; k0 < MT * CH / kAuxThreads; k0 += N) {
                uint4 v[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int idx = ct + (k0 + k) * kAuxThreads, g = walk.rt * MT + idx / CH, ti = g / G;
                    v[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (k0 + k < MT * CH / kAuxThreads && ti < rq.n)
                        v[k] = *reinterpret_cast<const uint4 *>(
                            p.q + (rq.tok + ti) * p.ld_q + (long long)(walk.h * G + g - ti * G) * D + 8 * (idx % CH));
                }
                if (!waited && seg > 0)
                    bar_wait(bQFree, (seg - 1) & 1, ok); // the last segment's scores are done
                waited = true;
                __syncwarp();
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int idx = ct + (k0 + k) * kAuxThreads, qr = idx / CH, c = idx % CH;
                    if (k0 + k >= MT * CH / kAuxThreads)
                        break;
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
                            s_f[seg & 3][qr] = pow2f(-up);
                    }
#pragma unroll
                    for (int cp = 0; cp < C::COPIES; ++cp)
                        *reinterpret_cast<uint4 *>(smem + op_off(qr + cp * MT, c)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                bar_arrive(bQ);
            ++seg;

            const int nt = (walk.nu + 1) / 2, end = walk.key_end(), key0 = walk.j0 * kBN;
            for (int t = 0; t < nt; ++t, ++i) {
                const int kt = key0 + t * kTile;
                if constexpr (C::F8) {
#pragma unroll 1
                    for (int n = 2 * i; n < 2 * i + 2; ++n) {
                        const int rs = n % max(C::RS, 1), s = n % C::NS;
                        bar_wait(bRFull + 8 * rs, (n / max(C::RS, 1)) & 1, ok);
                        if (n >= C::NS)
                            bar_wait(bEmpty + 8 * s, (n / C::NS - 1) & 1, ok);
                        __syncwarp();
                        const uint8_t *src = smem + (sRaw - sQ) + rs * C::RAW;
                        uint8_t *dst = smem + (sKV - sQ) + s * C::SLOT;
#pragma unroll 4
                        for (int k = 0; k < kTile * D / 16 / kAuxThreads; ++k) {
                            const int idx = ct + k * kAuxThreads, row = idx / (D / 16), c = idx % (D / 16);
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
                if (kt + kTile <= min(rq.len, end))
                    continue;
                // A tail tile: values behind the end become zero, and of the
                // drafted tokens' those that are not finite are marked.
                const int n = 2 * i + 1, sl = n % C::NS;
                bar_wait(bFull + 8 * sl, (n / C::NS) & 1, ok);
                __syncwarp();
                uint8_t *vs = smem + (sKV - sQ) + sl * C::SLOT;
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {
                    const int vr = ct + 64 * b;
                    bool odd = false;
                    if (kt + vr >= end) {
#pragma unroll
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4 *>(vs + op_off(vr, c)) = make_uint4(0u, 0u, 0u, 0u);
                    } else if (kt + vr >= rq.len) {
                        constexpr uint32_t EXP = C::F8 ? 0x7c007c00u : 0x7f807f80u;
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(vs + op_off(vr, c));
                            odd |= (__vcmpeq2(v.x & EXP, EXP) | __vcmpeq2(v.y & EXP, EXP) | __vcmpeq2(v.z & EXP, EXP) |
                                    __vcmpeq2(v.w & EXP, EXP)) != 0;
                        }
                    }
                    __syncwarp();
                    const uint32_t ob = __ballot_sync(~0u, odd);
                    if (lane == 0)
                        s_odd[tail & 3][vr >> 5] = ob;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(bTail + 8 * (tail & 3));
                ++tail;
            }
        }
    } else {
        // ---- the softmax -------------------------------------------------
        const int quad = warp / (MT / 32), row = (warp % (MT / 32)) * 32 + lane; // copy, row of the tile
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;
        const uint32_t tO = tmem + kColO + lanes;
        Split split{};
        int i = 0, seg = 0, tail = 0;
        while (walk.next(p, G, MT)) {
            const Request &rq = walk.rq;
            const int nt = (walk.nu + 1) / 2, end = walk.key_end(), key0 = walk.j0 * kBN;
            const int g = walk.rt * MT + row, ti = g / G;
            const bool live = ti < rq.n;
            const int tok_i = live ? ti : 0;
            const bool warp_live = __any_sync(~0u, live);
            const uint64_t first = key0 + nt * kTile > rq.len ? tree_bits(p, rq, tok_i) : 0;
            const float base_factor = fabsf(p.scale) * p.cache.k_scale * kLog2e;
            float factor = fmaxf(base_factor, 1e-37f); // a scale of zero: all scores alike
            float m = -INFINITY, l = 0.0f;             // reference (base 2), sum

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
                if constexpr (C::F8)
                    if (t == 0)
                        factor = fmaxf(base_factor * s_f[seg & 3][row], 1e-37f);
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
                const bool is_tail = kt + kTile > min(rq.len, end);
                uint64_t vis[(C::KW + 63) / 64];
                if (is_tail || (bad[0] | bad[1] | bad[2] | bad[3])) {
#pragma unroll
                    for (int c = 0; c < C::KW; c += 64) {
                        const int w = (quad * C::KW + c) >> 5;
                        const uint64_t b = C::KW >= 64 ? bad[w] | ((uint64_t)bad[w + 1] << 32) : bad[w];
                        vis[c / 64] = visible(p, rq, tok_i, first, kq + c, end) & ~b;
                    }
#pragma unroll
                    for (int c = 0; c < C::KW; ++c)
                        if (!((vis[c / 64] >> (c & 63)) & 1))
                            s[c] = 0xff800000u;
                }
                if (warp_live) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int c = 0; c < C::KW; ++c)
                        mx = fmaxf(mx, __uint_as_float(s[c]));
                    mx *= factor;
                    // the reference moves for the first keys seen, and when outgrown
                    const bool grow = mx > m + kGrowth;
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
                if (is_tail) {
                    bar_wait(bTail + 8 * (tail & 3), (tail >> 2) & 1, ok);
                    const uint32_t *odd = s_odd[tail & 3];
                    ++tail;
                    if (odd[0] | odd[1] | odd[2] | odd[3]) {
                        // Rare: what is not finite must not reach, times zero, the
                        // rows that do not see its key. It is added to O here, for
                        // the rows that do, and taken out of the slot.
                        const int n = 2 * i + 1, sl = n % C::NS;
                        uint8_t *vs = smem + (sKV - sQ) + sl * C::SLOT;
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
                                if (!((odd[kr >> 5] >> (kr & 31)) & 1) || !((vis[k >> 6] >> (k & 63)) & 1))
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
                        if ((odd[warp] >> lane) & 1) {
                            constexpr uint16_t EXP = C::F8 ? 0x7c00 : 0x7f80;
                            for (int e = 0; e < D; ++e) {
                                uint16_t *b = reinterpret_cast<uint16_t *>(vs + op_off(tid, e >> 3) + 2 * (e & 7));
                                if ((*b & EXP) == EXP)
                                    *b = 0;
                            }
                        }
                        if (tid == 0)
                            s_acc[i & 1] = t == 0;
                        fence_async_smem();
                        soft_sync();
                    }
                }
                tc_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(bP + 8 * (i & 1));
            }
            ++seg;

            // ---- the segment's end: O is complete ----
            const int last = i - 1;
            const bool whole = walk.whole();
            const int which = walk.j0 == 0 ? 1 : 0;
            float *part = part_of(p, blockIdx.x, which, MT, D);
            if (which && !whole) {
                split.parts = cta_of(U, walk.item0 + rq.tiles - 1, ctas) - (int)blockIdx.x + 1;
                split.tok = rq.tok;
                split.n = rq.n;
                split.h = walk.h;
                split.rt = walk.rt;
            }
            const long long tk = rq.tok + tok_i;
            const int hq = walk.h * G + g - ti * G;
            if (last >= 1)
                bar_wait(bO + 8 * ((last - 1) & 1), ((last - 1) >> 1) & 1, ok);
            bar_wait(bO + 8 * (last & 1), (last >> 1) & 1, ok);
            __syncwarp();
            tc_after();
            float f = 1.0f, top = m, sum = l;
            if constexpr (C::COPIES > 1) {
                s_m[quad][row] = m;
                s_l[quad][row] = l;
                soft_sync();
                top = s_m[0][row];
#pragma unroll
                for (int c = 1; c < C::COPIES; ++c)
                    top = fmaxf(top, s_m[c][row]);
                sum = 0.0f; // a copy that saw nothing has l = 0 (or NaN)
#pragma unroll
                for (int c = 0; c < C::COPIES; ++c)
                    sum += s_m[c][row] == -INFINITY ? s_l[c][row] : s_l[c][row] * exp2_fast(s_m[c][row] - top);
                f = m == -INFINITY ? 1.0f : exp2_fast(m - top);
            }
            const float inv = sum == 0.0f ? 0.0f : p.cache.v_scale / sum;
            if (live && quad == 0) {
                if (!whole) {
                    part[MT * D + row] = top;
                    part[MT * D + MT + row] = sum;
                } else if (p.lse) {
                    p.lse[tk * p.Hq + hq] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
                }
            }
            uint16_t *orow = p.out + tk * p.ld_out + (long long)hq * D;
            float *prow = part + (size_t)row * D;
            constexpr int CW = 32 / C::COPIES; // columns of each 32 that this thread writes
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                float o[CW];
                if (warp_live) {
                    uint32_t raw[32];
                    tmem_ld32(tO + c0, raw);
                    tmem_ld_wait(raw);
                    if constexpr (C::COPIES == 1) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __uint_as_float(raw[e]);
                    } else {
                        float4 *buf = reinterpret_cast<float4 *>(smem + (sJoin - sQ)) + (quad * MT + row) * 8;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            buf[e ^ (row & 7)] = make_float4(__uint_as_float(raw[4 * e]) * f, __uint_as_float(raw[4 * e + 1]) * f,
                                                             __uint_as_float(raw[4 * e + 2]) * f, __uint_as_float(raw[4 * e + 3]) * f);
                    }
                }
                if constexpr (C::COPIES > 1) {
                    soft_sync();
                    const float4 *buf = reinterpret_cast<const float4 *>(smem + (sJoin - sQ)) + row * 8;
#pragma unroll
                    for (int e = 0; e < CW / 4; ++e) {
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int c = 0; c < C::COPIES; ++c) {
                            const float4 y = buf[c * MT * 8 + ((quad * (CW / 4) + e) ^ (row & 7))];
                            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                        }
                        o[4 * e] = x.x;
                        o[4 * e + 1] = x.y;
                        o[4 * e + 2] = x.z;
                        o[4 * e + 3] = x.w;
                    }
                    soft_sync();
                }
                if (live) {
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < CW; e += 8)
                            *reinterpret_cast<uint4 *>(orow + c0 + quad * CW + e) =
                                make_uint4(pack2<false>(o[e] * inv, o[e + 1] * inv), pack2<false>(o[e + 2] * inv, o[e + 3] * inv),
                                           pack2<false>(o[e + 4] * inv, o[e + 5] * inv), pack2<false>(o[e + 6] * inv, o[e + 7] * inv));
                    } else {
#pragma unroll
                        for (int e = 0; e < CW; e += 4)
                            *reinterpret_cast<float4 *>(prow + c0 + quad * CW + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                __syncwarp();
            }
            tc_before();
        }
        if (tid == 0)
            static_cast<Split *>(p.workspace)[blockIdx.x] = split;
    }
    if (!ok)
        set_status(p.status, SGQ_STATUS_TIMEOUT);
    tc_before();
    __syncthreads();
    if (warp == kIssuer)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

// Joins the parts of the item that CTA blockIdx.x of the attention started and
// did not finish, in key order: one warp per row, kJoinRows rows a CTA.
constexpr int kJoinRows = 8;

template <int D>
__global__ void __launch_bounds__(32 * kJoinRows) join_kernel(const AttnProblem p, int MT)
{
    constexpr int LPR = D / 4; // lanes per row: with D = 64 two parts are read side by side
    constexpr int SIDE = 32 / LPR;
    const int lane = threadIdx.x & 31, row = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
    grid_launch_dependents();
    grid_dependency_wait();
    const Split sp = static_cast<const Split *>(p.workspace)[blockIdx.x];
    const int G = p.Hq / p.cache.heads, g = sp.rt * MT + row, ti = g / G;
    if (sp.parts == 0 || ti >= sp.n)
        return;
    const int x = lane % LPR;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.0f;
#pragma unroll 4
    for (int k = lane / LPR; k < sp.parts; k += SIDE) {
        const float *part = part_of(p, blockIdx.x + k, k == 0, MT, D);
        const float pm = part[MT * D + row], pl = part[MT * D + MT + row];
        const float4 v = *reinterpret_cast<const float4 *>(part + (size_t)row * D + 4 * x);
        const float top = fmaxf(m, pm), ref = top == -INFINITY ? 0.0f : top;
        const float a = exp2_fast(m - ref), b = exp2_fast(pm - ref);
        o = make_float4(o.x * a + v.x * b, o.y * a + v.y * b, o.z * a + v.z * b, o.w * a + v.w * b);
        l = l * a + pl * b;
        m = top;
    }
    if constexpr (SIDE == 2) {
        const float m2 = __shfl_xor_sync(~0u, m, 16), l2 = __shfl_xor_sync(~0u, l, 16);
        const float4 v = make_float4(__shfl_xor_sync(~0u, o.x, 16), __shfl_xor_sync(~0u, o.y, 16),
                                     __shfl_xor_sync(~0u, o.z, 16), __shfl_xor_sync(~0u, o.w, 16));
        const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top;
        const float a = exp2_fast(m - ref), b = exp2_fast(m2 - ref);
        o = make_float4(o.x * a + v.x * b, o.y * a + v.y * b, o.z * a + v.z * b, o.w * a + v.w * b);
        l = l * a + l2 * b;
        m = top;
    }
    if (lane >= LPR)
        return;
    const long long t = sp.tok + ti;
    const int hq = sp.h * G + g - ti * G;
    const float inv = l == 0.0f ? 0.0f : p.cache.v_scale / l;
    *reinterpret_cast<uint2 *>(p.out + t * p.ld_out + (long long)hq * D + 4 * x) =
        make_uint2(pack2<false>(o.x * inv, o.y * inv), pack2<false>(o.z * inv, o.w * inv));
    if (p.lse && x == 0)
        p.lse[t * p.Hq + hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
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
    cudaError_t e = launch_step(attn_kernel<D, KV, MT>, dim3(grid), kThreads, C::SMEM, 1, stream, a, kmap, vmap);
    if (e != cudaSuccess)
        return e;
    return launch_step(join_kernel<D>, dim3(grid, MT / kJoinRows), 32 * kJoinRows, 0, 1, stream, p, MT);
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
    (void)R;
    (void)Hq;
    (void)Hkv;
    return kMaxGrid * sizeof(Split) + (size_t)2 * kMaxGrid * kMaxMT * (D + 2) * sizeof(float);
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
