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
// Both products are tcgen05.mma of 128 rows and 128 keys. The warps:
//  * one walks the run and copies keys, one copies values, into a ring of 128-key
//    slots in the products' swizzled layout; what lies behind a segment's keys,
//    and bad pages, is filled with zeros. The copies are bulk tensor copies, a
//    box per 128 bytes of so many slots of a page, where a box has 512 bytes at
//    least, else cp.async of 16 bytes a lane. A box takes its warp some 40 ns
//    (11 requests of 8-bit keys in pages of 24, 16 boxes of 512 bytes a slot: 79 us,
//    in pages of 128 75);
//  * one thread issues S = Q K^T (both from shared memory) into one of two
//    accumulators, one tile ahead and across segments, and O += P V with P
//    read from tensor memory, where it takes S's place;
//  * two groups of four turn S into P, one accumulator row per thread, and
//    have an O of their own, so that one group's exponentials overlap the
//    other's. The reference for the exponent moves only when a row's maximum
//    outgrows it by 2^8, so O is rescaled rarely;
//  * one or two fetch the next segment's Q, the rest look through the values
//    next to the end. With 8-bit keys and values q is split into two 8-bit
//    parts, so that S is a product of 8-bit operands as they lie, and the
//    values are made fp16 (exact): weights of 8 bits would lose a long row's
//    tail.
// Row tiles (MT): with 256 rows each group has 128 of them and both see every
// key. With 128 the groups take the tiles of keys in turn (a segment of one
// tile is one group's alone), and their O are joined at the segment's end. With
// 32 they do too, and the rows are laid into Q's 128 four times, so that each
// warp finds the scores of all of them in its lanes and takes a quarter of the
// keys: the warps agree on the rows' maxima and put their quarters of P side by
// side in shared memory, where the product reads it (its rows from 32 on are
// whatever lies there, and so are those of O).
//
// What bounds it: with few rows and 16-bit keys memory (24 requests of 16000 keys
// and more, 32 query and 8 key heads of 128: 255 us at full clock, 285 to 295 under the
// power limit, 6.2 and 5.4 TB/s), with 8-bit ones a tile's copies, conversion, scores,
// weights and products one after the other (11 requests of up to 60000 keys, 32 / 8
// heads of 64: 78 us, 0.85 us a tile); with 512 rows a request the chain of scores,
// exponentials, products (12 requests of up to 16384 keys, 64 / 8 heads of 128: 163 us at
// full clock, 186 under the power limit, 622 and 545 TFLOP/s). Slower there: scores in
// halves of 64 keys, one with the softmax while the next are computed (by 4%); 64 scores
// in registers at a time (8%), and the other warps' registers for them (14%). Slower with
// few rows: scores two tiles ahead (by 38% on 24 requests of up to 16111 keys), for which
// the ring holds too little.
//
// The copies' ring tells a slot's phases by their parity alone. That holds as long
// as scores are one tile ahead of the products with the values: in a ring of an odd
// number of slots the values two turns back are then used up before the keys between.
//
// Every wait for another warp's work is bounded, by 0.2 s for data and by 90 s for the
// next segment and for the end of one's scores, which may take 10 s; one that runs out
// sets SGQ_STATUS_TIMEOUT, its warp waits for no data any more and the kernel comes to its
// end, which is passed on as the last segment. The warps of a group also meet at barriers
// of their own, which have no limit: they come to the same ones as long as they work on
// the same segments, and they do whatever runs out, since the warp that passes segments on
// stops for good kPassClocks after the last one, before any other has waited for 90 s (at
// 250 MHz and more). A segment's slot may then be written before every warp has read it,
// so what they read there is kept in bounds field by field.
#include "step_launch.cuh"
#include "tc_device.cuh"
#include "tree_attn.cuh"

#include <algorithm>
#include <cuda_fp8.h>

namespace sgq {

namespace {

constexpr int kTile = 128; // keys per product
constexpr int kGroup = 128; // threads of a softmax group
constexpr int kSoftWarps = 8, kKeys = 8, kValues = 9, kIssuer = 10, kQ = 11; // warps
constexpr uint32_t kColO = 256; // tensor-memory columns: S0, S1, the groups' O
constexpr float kGrowth = 8.0f; // binary orders a row's maximum may outgrow its reference
// fp16 weights (8-bit caches) are 2^7 times the bf16 ones: up to 2^15 of fp16's 2^16, and so
// with all the room below that there is (the sums l carry the same factor).
constexpr float kLift16 = 7.0f;
constexpr float kLeast = 1e-45f; // the smallest positive fp32 number
constexpr int kRing = 8;        // segments, and tail tiles, that are known to more than one warp
constexpr int kBoxBytes = 512;  // smallest box of a bulk copy
constexpr int kTiles = 16;      // tiles that are
// Limits, see the top. A segment has up to 2^23 tiles, which take up to 2200 clocks each.
constexpr long long kPassClocks = 20000000000; // from one segment passed on to the next
constexpr unsigned long long kSegWaitNs = 90000000000ull, kSlotWaitNs = 2000000000ull, kDrainNs = 400000000ull;

template <int D_, int KV, int MT_>
struct Cfg {
    static constexpr int D = D_, MT = MT_;
    static constexpr bool F8 = KV == SGQ_TYPE_E4M3, TWO = MT == 256, FEW = MT == 32;
    static constexpr int QW = F8 && !TWO ? 1 : 2, VW = !F8 ? 1 : TWO ? 2 : 4; // warps for Q, for the values read
    static constexpr int kV = kQ + QW, THREADS = 32 * (kV + VW);
    // Whether what takes the softmax's warps to the barriers of the rare path is voted on at
    // one. (With 16-bit keys and rows for both groups, whom that would bring together at
    // every tail tile, they meet by waits like the others instead, which one that ran out
    // may bring them to differently: 12 wide trees 184 us against 189; with 8-bit keys the
    // vote is better, 257 against 268.)
    static constexpr bool VOTE = !TWO || F8;
    static constexpr int MEET = TWO ? 2 * kGroup : kGroup;    // threads that meet there
    static constexpr int ROWS = FEW ? 32 : 128;               // of a group
    static constexpr int COPIES = 128 / ROWS;                 // of the rows, in Q
    static constexpr int SUB = kTile * 128;                   // 128 rows x 128 bytes, swizzled
    static constexpr int NSUB = D / 64;
    static constexpr float LIFT = F8 ? kLift16 : 0.0f;
    static constexpr int SLOT = NSUB * SUB;                   // 128 keys (or values), 16 bits
    static constexpr int Q1 = F8 ? 2 * SUB : SLOT, Q = TWO ? 2 * Q1 : Q1; // 128 rows of q; all of them
    static constexpr int P1 = FEW ? ROWS * 256 : 0, P = 2 * P1; // P of a group in shared memory
    static constexpr int KV_BYTES = F8 ? (TWO ? 64 : 96) * 1024 : (TWO ? 4 : 5) * (D == 128 ? 1 : 2) * SLOT; // the ring of copies
    static constexpr int SLOTS = F8 ? KV_BYTES / (kTile * D) : KV_BYTES / SLOT;
    static constexpr int NV = F8 ? 2 : 0;                     // fp16 values
    static constexpr int ROWB = F8 ? D : 2 * D, CPR = ROWB / 16; // bytes, 16-byte chunks of a key
    static constexpr int OUT1 = 32 * 64, OUT = MT == 128 ? 8 * OUT1 : 0; // 16 columns of a warp's rows, for the other group
    static constexpr int BARS = 2 * SLOTS + 2 * NV + 6 + 3 * kRing + 4;
    static constexpr int SMEM = 1024 + Q + P + KV_BYTES + NV * SLOT + OUT + BARS * 8;
    static_assert(SMEM <= 227 * 1024 - 8192, "room for the static arrays");
    // copies run ahead of the softmax by the ring's tiles, 8-bit ones by NV more and the
    // one in between: its entries live that long, those of tail tiles without the ring
    static_assert(SLOTS / 2 + NV + 2 <= kTiles && (F8 ? NV + 1 : SLOTS / 2 + 1) <= kRing, "ring entries");
};

// What a CTA's warps need of a segment (nt = 0: the run has ended). The softmax's warps
// keep its slot; the others have read it by then, or a wait has run out.
struct Seg {
    int nt, r;                  // tiles, request
    int tok, n, len;            // the request's first row, new tokens, cached ones
    int key0, end;              // its keys
    int h, rt;                  // key head, row tile
    int first_tail, tail_index; // tiles from here on reach the drafted tokens or the end; the
                                // first one's number among the run's
    int whole, which;           // the whole item; else which part it is
};

// A place in a ring of n slots that every warp walks in steps of one or two.
struct Ring {
    int s;
    uint32_t ph;
    __device__ __forceinline__ void step(int by, int n)
    {
        s += by;
        if (s >= n) {
            s -= n;
            ph ^= 1;
        }
    }
};

template <int N>
__device__ __forceinline__ void named_sync(int bar)
{
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(N) : "memory");
}

// named_sync, and whether any of its threads has v != 0.
template <int N>
__device__ __forceinline__ bool named_or(int bar, uint32_t v)
{
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                 "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"(v), "r"(bar), "n"(N)
                 : "memory");
    return any;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Byte offset of 16-byte chunk c of row r of an operand of 16-bit elements.
__device__ __forceinline__ uint32_t op_off(int r, int c)
{
    return (uint32_t)((c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <int D, int KV, int MT>
__global__ void __launch_bounds__(Cfg<D, KV, MT>::THREADS, 1)
    attn_kernel(const __grid_constant__ AttnProblem p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const int box)
{
    using C = Cfg<D, KV, MT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ long long s_scan[4], s_first;
    __shared__ int s_r;
    __shared__ Request s_rq;
    __shared__ Seg s_seg[kRing];
    __shared__ float s_m[2][C::COPIES][C::ROWS], s_l[2][C::COPIES][C::ROWS]; // by group and copy
    __shared__ float s_mx[C::FEW ? 4 : 1][C::COPIES][C::FEW ? 32 : 1];       // a tile's maxima, by group and turn
    __shared__ long long s_out[C::FEW ? 2 : 1][C::FEW ? 32 : 1];             // where rows are written
    __shared__ float s_f[C::F8 ? 4 : 1][C::F8 ? MT : 1]; // q's powers of two, by segment
    __shared__ uint32_t s_bad[kTiles][4];                // keys without a page, bit by key, by tile
    __shared__ uint32_t s_odd[kRing][4];                 // values that are not finite, by tail tile
    __shared__ int s_late;                               // a wait ran out
    __shared__ int s_acc[2];                             // a group's first product of a segment adds to O
    uint8_t *smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    const uint32_t sQ = smem_u32(smem), sP = sQ + C::Q, sKV = sP + C::P, sV = sKV + C::KV_BYTES, sOut = sV + C::NV * C::SLOT;
    const uint32_t bFull = sOut + C::OUT, bEmpty = bFull + 8 * C::SLOTS;
    const uint32_t bVFull = bEmpty + 8 * C::SLOTS, bVEmpty = bVFull + 8 * C::NV;
    const uint32_t bS = bVEmpty + 8 * C::NV, bP = bS + 16, bO = bP + 16;
    const uint32_t bTail = bO + 16, bSeg = bTail + 8 * kRing, bSegFree = bSeg + 8 * kRing, bQ = bSegFree + 8 * kRing, bQFree = bQ + 8, bDone = bQFree + 8, bMeet = bDone + 8;
    // the ring of copies: keys in one slot, values in the next
    constexpr uint32_t slot_bytes = kTile * C::ROWB;
    constexpr int slots = C::SLOTS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = p.cache.heads, G = p.Hq / Hkv;

    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "n"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        // The next kernel may start: not before this CTA has its tensor memory, which a
        // CTA of that kernel would hold while it waits for this one.
        grid_launch_dependents();
    } else if (warp == kKeys && lane == 0) {
        for (int s = 0; s < C::SLOTS; ++s) {
            bar_init(bFull + 8 * s, box ? 1 : 32); // one bulk copy's thread, or the lanes of a warp
            // read by the products and followed by the value warps; 8-bit keys by the
            // products alone, 8-bit values by the value warps alone
            bar_init(bEmpty + 8 * s, !C::F8 ? 1 + C::VW : s & 1 ? C::VW : 1);
        }
        for (int s = 0; s < C::NV; ++s) {
            bar_init(bVFull + 8 * s, C::VW);
            bar_init(bVEmpty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(bS + 8 * b, 1);
            bar_init(bP + 8 * b, 4);
            bar_init(bO + 8 * b, 1);
            s_acc[b] = 0;
        }
        for (int b = 0; b < kRing; ++b) {
            bar_init(bTail + 8 * b, C::VW);
            bar_init(bSeg + 8 * b, 1);
            bar_init(bSegFree + 8 * b, kSoftWarps);
        }
        bar_init(bQ, C::F8 || C::FEW ? C::QW : 32 * C::QW);
        bar_init(bQFree, 1);
        bar_init(bDone, 1);
        s_late = 0;
        bar_init(bMeet, kSoftWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    grid_dependency_wait();

    // The requests' costs, their sum U, and this CTA's run of [0, U).
    int bits = 0;
    bool ok = true, led = true; // no wait for data, for a segment ran out
    const int per = (p.R + kGroup - 1) / kGroup;
    const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    long long mine = 0, at = 0;
    Request rq0{};
    if (warp < 4) {
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
    long long u = 0, u_end = 0;
    if ((int)blockIdx.x < ctas) {
        u = run_start(U, blockIdx.x, ctas);
        u_end = run_start(U, blockIdx.x + 1, ctas);
    }
    if (warp < 4 && u < u_end) {
        for (int w = 0; w < warp; ++w)
            at += s_scan[w];
        if (u >= at && u < at + mine) {
            int r = r0, none = 0;
            if (per > 1)
                for (; r < r1; ++r) {
                    rq0 = request_of(p, r, G, MT, none);
                    const long long n = cost_of(rq0, Hkv);
                    if (u < at + n)
                        break;
                    at += n;
                }
            s_r = r;
            s_first = at;
            s_rq = rq0;
        }
    }
    __syncthreads();

    if (warp == kKeys || warp == kValues) {
        // ---- the run's segments; pages -> slots ------------------------------
        // Lane x knows rows x, x + 32, x + 64, x + 96 of a slot; the pages of the
        // next tile are looked up ahead. Lane x then copies chunk x % CPR of row
        // x / CPR of each group of 32 / CPR rows.
        const bool keys = warp == kKeys;
        Walk walk;
        if (keys && u < u_end) {
            walk.u = u;
            walk.u_end = u_end;
            walk.r = s_r;
            walk.base = s_first;
            walk.rq = s_rq;
        }
        constexpr int ES = C::F8 ? 1 : 2, RPI = 32 / C::CPR; // rows of one copy instruction
        const int page = p.cache.page, page_up = kTile / page, slot_up = kTile % page;
        constexpr int PARTS = C::F8 ? 1 : C::NSUB; // boxes side by side in a row
        const int pieces = box ? kTile / box * PARTS : 0;
        const CUtensorMap *map = keys ? &kmap : &vmap;
        const uint32_t lead = elect_lane();
        const uint8_t *cache = static_cast<const uint8_t *>(keys ? p.cache.k : p.cache.v) + 16 * (lane % C::CPR);
        Ring ring{keys ? 0 : 1, 0}, seg{0, 0};
        Split split0{}, split1{};
        long long passed = clock64(); // when the last segment was
        int i = 0, tails = 0; // tiles, tail tiles so far
        for (;;) {
            int nt, r, key0, end, h;
            if (keys) {
                const bool more = __all_sync(~0u, ok) && walk.next(p, G, MT);
                nt = more ? (walk.nu + 1) / 2 : 0;
                r = walk.r;
                key0 = walk.j0 * kBN;
                end = walk.key_end();
                h = walk.h;
                const int first_tail = max(0, (min(walk.rq.len, end) - key0) / kTile);
                bar_wait(bSegFree + 8 * seg.s, seg.ph ^ 1, led, kSlotWaitNs);
                const long long now = clock64();
                led = __all_sync(~0u, led && now - passed < kPassClocks);
                passed = now;
                if (!led) // too late, or the slot is in use: nothing more is passed on
                    break;
                if (lane == 0) {
                    Seg &sg = s_seg[seg.s];
                    sg.nt = nt;
                    sg.r = r;
                    sg.tok = walk.rq.tok;
                    sg.n = walk.rq.n;
                    sg.len = walk.rq.len;
                    sg.key0 = key0;
                    sg.end = end;
                    sg.h = h;
                    sg.rt = walk.rt;
                    sg.first_tail = first_tail;
                    sg.tail_index = tails;
                    sg.whole = walk.whole();
                    sg.which = walk.j0 == 0;
                    bar_arrive(bSeg + 8 * seg.s);
                }
                tails += max(0, nt - first_tail);
            } else {
                bar_wait(bSeg + 8 * seg.s, seg.ph, led, kSegWaitNs);
                led = __all_sync(~0u, led);
                nt = led ? s_seg[seg.s].nt : 0;
                r = s_seg[seg.s].r;
                key0 = s_seg[seg.s].key0;
                end = s_seg[seg.s].end;
                h = s_seg[seg.s].h;
            }
            seg.step(1, kRing);
            if (nt == 0)
                break;
            const int32_t *table = p.table + (long long)r * p.table_ld;
            if (keys && !walk.whole()) { // a part for join_kernel
                Split sp;
                sp.c0 = cta_of(U, walk.item0, ctas);
                sp.parts = cta_of(U, walk.item0 + walk.rq.tiles - 1, ctas) - sp.c0 + 1;
                sp.tok = walk.rq.tok;
                sp.n = walk.rq.n;
                sp.h = h;
                sp.rt = walk.rt;
                if (walk.j0 == 0)
                    split1 = sp;
                else
                    split0 = sp;
            }
            if (box) {
                // Lane x looks up piece x of a slot: rows of one page, 128 bytes.
                // The next two tiles' pages are looked up ahead.
                const int first = key0 + lane / PARTS * box;
                int pg = first / page, sl = first - pg * page;
                auto look = [&](int t, int at_page) {
                    return lane < pieces && t < nt && first + t * kTile < end ? table[at_page] : -1;
                };
                auto step = [&](int &g, int &s) { // one tile on
                    g += page_up;
                    s += slot_up;
                    if (s >= page) {
                        s -= page;
                        ++g;
                    }
                };
                int pg_next = pg, sl_next = sl;
                int id0 = look(0, pg);
                step(pg_next, sl_next);
                int id1 = look(1, pg_next);
#pragma unroll 1
                for (int t = 0; t < nt; ++t, ++i) {
                    int pg2 = pg_next, sl2 = sl_next;
                    step(pg2, sl2);
                    const int id2 = look(t + 2, pg2);
                    const bool want = lane < pieces && first + t * kTile < end;
                    const bool good = want && id0 >= 0 && id0 < p.cache.num_pages;
                    const int pid = good ? id0 : p.cache.num_pages; // outside the map: zeros
                    const int slot = good ? sl : 0;
                    const uint32_t lost = __ballot_sync(~0u, want && !good);
                    if (keys && lane < 4) { // the keys without a page, 32 a lane
                        uint32_t b = 0;
                        if (lost) {
                            for (int k = 0; k < 32; ++k)
                                b |= ((lost >> ((32 * lane + k) / box * PARTS)) & 1) << k;
                            set_status(p.status, SGQ_STATUS_BAD_INDEX);
                        }
                        s_bad[i % kTiles][lane] = b;
                    }
                    bar_wait(bEmpty + 8 * ring.s, ring.ph ^ 1, ok);
                    __syncwarp();
                    const uint32_t full = bFull + 8 * ring.s, dst = sKV + ring.s * slot_bytes;
                    if (!__all_sync(~0u, ok)) // the slot may be in use
                        break;
                    if (lane == 0)
                        bar_expect(full, kTile * C::ROWB);
                    __syncwarp();
#pragma unroll 8
                    for (int x = 0; x < pieces; ++x) {
                        const int at = __shfl_sync(~0u, pid, x), s = __shfl_sync(~0u, slot, x);
                        tma_load_4d(dst + x % PARTS * C::SUB + x / PARTS * box * min(C::ROWB, 128), map, x % PARTS * 64, s, h, at,
                                    full, lead);
                    }
                    ring.step(2, slots);
                    sl = sl_next;
                    pg_next = pg2;
                    sl_next = sl2;
                    id0 = id1;
                    id1 = id2;
                }
                continue;
            }
            const uint8_t *head = cache + h * p.cache.head_stride * ES;
            // this lane's rows: page index, slot in it, the next tile's page ids
            int pg[4], sl[4], id[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = key0 + lane + 32 * j;
                pg[j] = key / page;
                sl[j] = key - pg[j] * page;
                id[j] = key < end ? table[pg[j]] : -1;
            }
#pragma unroll 1
            for (int t = 0; t < nt; ++t, ++i) {
                // these rows' offsets, -1 where there is none; the next ones' pages
                long long off[4];
                uint32_t bad[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + t * kTile + lane + 32 * j;
                    const bool want = key < end, good = want && id[j] >= 0 && id[j] < p.cache.num_pages;
                    off[j] = good ? (id[j] * p.cache.page_stride + sl[j] * p.cache.slot_stride) * ES : -1;
                    bad[j] = __ballot_sync(~0u, want && !good);
                    pg[j] += page_up;
                    sl[j] += slot_up;
                    if (sl[j] >= page) {
                        sl[j] -= page;
                        ++pg[j];
                    }
                    id[j] = key + kTile < end ? table[pg[j]] : -1;
                }
                if (keys && lane < 4) {
                    const uint32_t b = lane < 2 ? (lane ? bad[1] : bad[0]) : lane == 2 ? bad[2] : bad[3];
                    s_bad[i % kTiles][lane] = b;
                    if (b)
                        set_status(p.status, SGQ_STATUS_BAD_INDEX);
                }
                bar_wait(bEmpty + 8 * ring.s, ring.ph ^ 1, ok);
                __syncwarp();
                const uint32_t dst = sKV + ring.s * slot_bytes;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll 8
                    for (int k = 0; k < 32 / RPI; ++k) {
                        const int row = 32 * j + k * RPI + lane / C::CPR;
                        const long long o = __shfl_sync(~0u, off[j], k * RPI + lane / C::CPR);
                        const int c = lane % C::CPR;
                        uint32_t at; // the swizzle: of 128 bytes, or of 64 with rows of 64
                        if constexpr (!C::F8)
                            at = op_off(row, c);
                        else if constexpr (D == 128)
                            at = row * 128 + ((c ^ (row & 7)) << 4);
                        else
                            at = row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
                        cp_async16_zfill(dst + at, head + max(o, 0ll), o >= 0);
                    }
                cp_async_arrive(bFull + 8 * ring.s);
                ring.step(2, slots);
            }
        }
        if (keys && lane < 2)
            static_cast<Split *>(p.workspace)[2 * blockIdx.x + lane] = lane ? split1 : split0;
        cp_async_wait_all();
    } else if (warp == kIssuer) {
        // ---- the products ------------------------------------------------
        constexpr uint32_t idS = idesc_f16(!C::F8, false, kTile), idO = idesc_f16(!C::F8, true, D);
        const uint32_t lead = elect_lane(); // it issues, see mma_ss
        Ring kr{0, 0}, vr{1, 0}, seg{0, 0};
        uint32_t q_ph = 0;
        int left = 0, nt = 0; // tiles of the segment without scores, all of them
        bool ended = false;
        // Whether there is a next tile; its segment is looked up.
        auto next = [&]() -> bool {
            if (left == 0 && !ended) {
                bar_wait(bSeg + 8 * seg.s, seg.ph, led, kSegWaitNs);
                __syncwarp();
                left = (int)__reduce_max_sync(~0u, __all_sync(~0u, led) ? (unsigned)s_seg[seg.s].nt : 0u);
                seg.step(1, kRing);
                ended = left == 0;
                nt = -left; // its Q has not been waited for
            }
            return !ended;
        };
        // The scores of the next tile for group g's rows, into S number buf.
        auto scores = [&](int g, int buf) {
            if (nt < 0) {
                bar_wait(bQ, q_ph, ok);
                q_ph ^= 1;
                nt = -nt;
            }
            bar_wait(bFull + 8 * kr.s, kr.ph, ok);
            if (!box)
                fence_async_smem(); // the copies' writes, for the product's reads
            __syncwarp();
            tc_after();
            const uint32_t d = tmem + buf * kTile, ka = sKV + kr.s * slot_bytes;
            const Desc dq(op_desc(sQ + g * C::Q1, 16, 1024));
            if constexpr (C::F8) {
                // q's two parts one after the other
                const Desc dk(op_desc(ka, 16, 8 * D, D == 128 ? 2 : 4));
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    mma_ss_f8(d, dq, 2 * k, dk, 2 * k, idS, k > 0, lead);
                    mma_ss_f8(d, dq, (C::SUB >> 4) + 2 * k, dk, 2 * k, idS, 1, lead);
                }
            } else {
                const Desc dk(op_desc(ka, 16, 1024));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t st = ((k >> 2) * C::SUB + (k & 3) * 32) >> 4;
                    mma_ss(d, dq, st, dk, st, idS, k > 0, lead);
                }
            }
            tc_commit(bS + 8 * buf, p.debug_withhold_scores ? 0u : lead);
            if (!C::TWO || g == 1) {
                tc_commit(bEmpty + 8 * kr.s, lead);
                if (--left == 0)
                    tc_commit(bQFree, lead);
                kr.step(2, slots);
            }
        };
        // Tile i's product with the values into O number buf.
        auto values = [&](int i, int buf, uint32_t p_ph, bool begun) {
            const uint32_t vfull = C::F8 ? bVFull + 8 * (i & 1) : bFull + 8 * vr.s;
            bar_wait(vfull, C::F8 ? (i >> 1) & 1 : vr.ph, ok);
            bar_wait(bP + 8 * buf, p_ph, ok);
            if (!C::F8 && !box)
                fence_async_smem();
            __syncwarp();
            tc_after();
            const uint32_t add = begun || *(volatile int *)&s_acc[buf];
            const Desc dv(op_desc(C::F8 ? sV + (i & 1) * C::SLOT : sKV + vr.s * slot_bytes, C::SUB, 1024));
            const uint32_t o = tmem + kColO + buf * 128;
            if constexpr (C::FEW) {
                const Desc dp(op_desc(sP + buf * C::P1, 16, 1024));
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_ss(o, dp, ((k >> 2) * C::ROWS * 128 + (k & 3) * 32) >> 4, dv, (k * 2048) >> 4, idO, add | (k > 0), lead);
            } else {
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_ts(o, tmem + buf * kTile + 8 * k, dv, (k * 2048) >> 4, idO, add | (k > 0), lead);
            }
            tc_commit(bO + 8 * buf, lead);
            if (!C::TWO || buf == 1) {
                tc_commit(C::F8 ? bVEmpty + 8 * (i & 1) : bEmpty + 8 * vr.s, lead);
                vr.step(2, slots);
            }
        };
        int i = 0, t = 0; // tile, its number in its segment
        bool more = next();
        int nt_i = abs(nt); // its segment's tiles
        // The tiles' products, scores one tile ahead. Into the next segment only
        // if its Q is there (with rows for both groups: never), else after the
        // values. The first tile has no values before it.
        for (int step = -1; step < 0 || more; ++step) {
            if (step < 0) {
                if (!more)
                    break;
                scores(0, 0);
                if constexpr (C::TWO)
                    scores(1, 1);
                continue;
            }
            more = next();
            const bool crosses = more && nt < 0;
            const bool ahead = more && (!crosses || (!C::TWO && __all_sync(~0u, bar_test(bQ, q_ph))));
            if constexpr (C::TWO) {
                values(i, 0, i & 1, t > 0);
                if (ahead)
                    scores(0, 0);
                values(i, 1, i & 1, t > 0);
                if (more && !ahead)
                    scores(0, 0);
                if (more)
                    scores(1, 1);
            } else {
                if (ahead)
                    scores(0, (i + 1) & 1);
                values(i, i & 1, (i >> 1) & 1, t >= 2);
                if (more && !ahead)
                    scores(0, (i + 1) & 1);
            }
            ++i;
            if (++t == nt_i) {
                t = 0;
                nt_i = abs(nt);
            }
        }
        // every product and every arrival is complete before the CTA ends
        bool done = true;
        tc_commit(bDone, lead);
        bar_wait(bDone, 0, done);
        ok = ok && done;
        __syncwarp();
    } else if (warp >= kQ && warp < C::kV) {
        // ---- Q -----------------------------------------------------------
        // The rows in the operand's layout, once per copy. With 8-bit keys each
        // row is scaled by the power of two that brings its largest value into
        // [2^7, 2^8) and split in two 8-bit parts, 4 bits each of its 8: exact
        // for values down to 2^-2, below it off by at most 2^-10, i.e. 2^-17 of
        // the largest.
        constexpr int QT = 32 * C::QW, CH = D / 8;           // 16-byte chunks of a row
        constexpr int ALL = (C::TWO ? 256 : MT) * CH / QT, N = ALL < 16 ? ALL : 16;
        const int ct = tid - 32 * kQ;
        const uint32_t inv_g = 0xffffffffu / (uint32_t)G + 1; // x / G = (x inv_g) >> 32 for x G < 2^32
        Ring seg{0, 0};
        uint32_t free_ph = 1; // the operand is free at first
        int segs = 0;
        for (;;) {
            bar_wait(bSeg + 8 * seg.s, seg.ph, led, kSegWaitNs);
            led = __all_sync(~0u, led);
            if (!led || s_seg[seg.s].nt == 0)
                break;
            const int tok = s_seg[seg.s].tok, n = s_seg[seg.s].n, h = s_seg[seg.s].h, g0 = s_seg[seg.s].rt * MT;
            seg.step(1, kRing);
            const int t0 = g0 / G, rem0 = g0 - t0 * G;
            if constexpr (!C::F8 && !C::FEW) {
                // many rows: straight into their places
                bar_wait(bQFree, free_ph, ok, kSegWaitNs);
                __syncwarp();
#pragma unroll 4
                for (int k = 0; k < ALL; ++k) {
                    const int idx = ct + k * QT, qr = idx / CH, x = rem0 + qr;
                    const int dt = G == 1 ? x : (int)__umulhi((uint32_t)x, inv_g), ti = t0 + dt;
                    const uint16_t *src = p.q + min(tok + ti, p.T - 1) * p.ld_q + (long long)(h * G + x - dt * G) * D + 8 * (idx % CH);
                    cp_async16_zfill(sQ + (qr >> 7) * C::Q1 + op_off(qr & 127, idx % CH), ti < n ? src : p.q, ti < n);
                }
                cp_async_arrive(bQ);
                free_ph ^= 1;
            } else {
                // rows behind the tile's own are left as they lie: nothing of theirs is written
                const int used = n * G - g0;
#pragma unroll 1
                for (int k0 = 0; k0 < ALL && k0 * QT / CH < used; k0 += N) {
                    uint4 v[N];
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const int idx = ct + (k0 + k) * QT, x = rem0 + idx / CH;
                        const int dt = G == 1 ? x : (int)__umulhi((uint32_t)x, inv_g), ti = t0 + dt;
                        v[k] = make_uint4(0u, 0u, 0u, 0u);
                        if (ti < n)
                            v[k] = *reinterpret_cast<const uint4 *>(p.q + min(tok + ti, p.T - 1) * p.ld_q + (long long)(h * G + x - dt * G) * D +
                                                                    8 * (idx % CH));
                    }
                    if (k0 == 0)
                        bar_wait(bQFree, free_ph, ok, kSegWaitNs); // the last segment's scores are done
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        if ((k0 + k) * QT / CH >= used)
                            break;
                        const int idx = ct + (k0 + k) * QT, qr = idx / CH, c = idx % CH;
                        uint8_t *dst = smem + (C::TWO ? (qr >> 7) * C::Q1 : 0);
                        const int r = C::TWO ? qr & 127 : qr;
                        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                        if constexpr (C::F8) {
                            float f[8], mx = 0.0f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                f[2 * e] = __uint_as_float(w[e] << 16);
                                f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                                mx = fmaxf(mx, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
                            }
#pragma unroll
                            for (int o = CH / 2; o; o >>= 1)
                                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
                            // both the power and its inverse are normal fp32 numbers
                            const int up = min(max(7 - ((int)(__float_as_uint(mx) >> 23) - 127), -126), 126);
                            // (an infinity would be saturated: such a row is made NaN)
                            const float mul = mx < INFINITY ? pow2f(up) : NAN;
                            uint32_t part[2][2];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 x = make_float2(f[2 * e] * mul, f[2 * e + 1] * mul);
                                const uint32_t hi = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
                                const uint32_t h2 = e4m3x2_to_f16x2(hi);
                                const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
                                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x - hf.x, x.y - hf.y), __NV_SATFINITE, __NV_E4M3);
                                part[0][e >> 1] = e & 1 ? part[0][e >> 1] | hi << 16 : hi;
                                part[1][e >> 1] = e & 1 ? part[1][e >> 1] | lo << 16 : lo;
                            }
                            if (c == 0)
                                s_f[segs & 3][qr] = pow2f(-up);
#pragma unroll
                            for (int cp = 0; cp < C::COPIES; ++cp)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    *reinterpret_cast<uint2 *>(dst + e * C::SUB + op_off(r + cp * MT, c >> 1) + 8 * (c & 1)) =
                                        make_uint2(part[e][0], part[e][1]);
                        } else {
#pragma unroll
                            for (int cp = 0; cp < C::COPIES; ++cp)
                                *reinterpret_cast<uint4 *>(dst + op_off(r + cp * MT, c)) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                free_ph ^= 1;
                ++segs;
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(bQ);
            }
        }
    } else if (warp >= C::kV) {
        // ---- the values next to the end, 8-bit values -> fp16 -------------------
        constexpr int VT = 32 * C::VW;
        const int ct = tid - 32 * C::kV;
        Ring seg{0, 0}, vr{C::F8 ? 1 : 0, 0};
        int i = 0;
        for (;;) {
            bar_wait(bSeg + 8 * seg.s, seg.ph, led, kSegWaitNs);
            led = __all_sync(~0u, led);
            const int nt = s_seg[seg.s].nt, first_tail = s_seg[seg.s].first_tail, tail_index = s_seg[seg.s].tail_index;
            const int key0 = s_seg[seg.s].key0, end = s_seg[seg.s].end, len = s_seg[seg.s].len;
            if (!led || nt == 0)
                break;
            seg.step(1, kRing);
            for (int t = 0; t < nt; ++t) {
                const bool is_tail = t >= first_tail;
                uint8_t *vs; // the tile's values, 16 bits
                if constexpr (C::F8) {
                    bar_wait(bFull + 8 * vr.s, vr.ph, ok);
                    bar_wait(bVEmpty + 8 * (i & 1), ((i >> 1) & 1) ^ 1, ok);
                    __syncwarp();
                    const uint8_t *src = smem + (sKV - sQ) + vr.s * slot_bytes;
                    vs = smem + (sV - sQ) + (i & 1) * C::SLOT;
                    constexpr int M = kTile * D / 16 / VT;
                    uint4 v[M];
#pragma unroll
                    for (int k = 0; k < M; ++k) {
                        const int idx = ct + k * VT, row = idx / (D / 16), c = idx % (D / 16);
                        // the copies' swizzle: of 128 bytes, or of 64 with rows of 64
                        const int x = c ^ (D == 128 ? row & 7 : (row >> 1) & 3);
                        v[k] = *reinterpret_cast<const uint4 *>(src + row * D + 16 * x);
                    }
#pragma unroll
                    for (int k = 0; k < M; ++k) {
                        const int idx = ct + k * VT, row = idx / (D / 16), c = idx % (D / 16);
                        *reinterpret_cast<uint4 *>(vs + op_off(row, 2 * c)) =
                            make_uint4(e4m3x2_to_f16x2(v[k].x & 0xffffu), e4m3x2_to_f16x2(v[k].x >> 16),
                                       e4m3x2_to_f16x2(v[k].y & 0xffffu), e4m3x2_to_f16x2(v[k].y >> 16));
                        *reinterpret_cast<uint4 *>(vs + op_off(row, 2 * c + 1)) =
                            make_uint4(e4m3x2_to_f16x2(v[k].z & 0xffffu), e4m3x2_to_f16x2(v[k].z >> 16),
                                       e4m3x2_to_f16x2(v[k].w & 0xffffu), e4m3x2_to_f16x2(v[k].w >> 16));
                    }
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(bEmpty + 8 * vr.s);
                    vr.step(2, slots);
                    if (is_tail)
                        named_sync<VT>(4); // the rows below are other warps' too
                } else {
                    bar_wait(bFull + 8 * vr.s, vr.ph, ok); // the keys, passed on
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(bEmpty + 8 * vr.s);
                    vr.step(1, slots);
                    bar_wait(bFull + 8 * vr.s, vr.ph, ok);
                    __syncwarp();
                    vs = smem + (sKV - sQ) + vr.s * slot_bytes;
                }
                const uint32_t tail = (uint32_t)(tail_index + t - first_tail) % kRing;
                if (is_tail) {
                    // A tail tile: values behind the end become zero, and of the
                    // drafted tokens' those that are not finite are marked.
                    const int kt = key0 + t * kTile;
#pragma unroll 1
                    for (int vrow = ct; vrow < kTile; vrow += VT) {
                        bool odd = false;
                        if (kt + vrow >= end) {
#pragma unroll
                            for (int c = 0; c < D / 8; ++c)
                                *reinterpret_cast<uint4 *>(vs + op_off(vrow, c)) = make_uint4(0u, 0u, 0u, 0u);
                        } else if (kt + vrow >= len) {
                            constexpr uint32_t EXP = C::F8 ? 0x7c007c00u : 0x7f807f80u;
#pragma unroll
                            for (int c = 0; c < D / 8; ++c) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(vs + op_off(vrow, c));
                                odd |= (__vcmpeq2(v.x & EXP, EXP) | __vcmpeq2(v.y & EXP, EXP) | __vcmpeq2(v.z & EXP, EXP) |
                                        __vcmpeq2(v.w & EXP, EXP)) != 0;
                            }
                        }
                        __syncwarp();
                        const uint32_t ob = __ballot_sync(~0u, odd);
                        if (lane == 0)
                            s_odd[tail][vrow >> 5] = ob;
                    }
                }
                if (C::F8 || is_tail)
                    fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(C::F8 ? bVFull + 8 * (i & 1) : bEmpty + 8 * vr.s);
                    if (is_tail)
                        bar_arrive(bTail + 8 * tail);
                }
                if (!C::F8)
                    vr.step(1, slots);
                ++i;
            }
        }
    } else {
        // ---- the softmax -------------------------------------------------
        const int grp = warp >> 2, wq = warp & 3;
        const int quad = C::FEW ? wq : 0, row = C::FEW ? lane : wq * 32 + lane; // copy, row of the group's
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint32_t tS = tmem + grp * kTile + lanes, tO = tmem + kColO + grp * 128 + lanes;
        const int gtid = tid & (kGroup - 1);
        const float base_factor = fabsf(p.scale) * p.cache.k_scale * kLog2e;
        Ring seg{0, 0};
        // The warps of a group, or with rows for both of both, meet.
        uint32_t meet_ph = 0;
        auto meet = [&] {
            if constexpr (C::VOTE) {
                named_sync<C::MEET>(C::TWO ? 1 : 2 + grp);
            } else {
                __syncwarp();
                if (lane == 0)
                    bar_arrive(bMeet);
                bar_wait(bMeet, meet_ph, ok);
                meet_ph ^= 1;
                __syncwarp();
            }
        };
        uint32_t s_ph = 0; // of this group's next tile: S, P, O take the same turns
        int i0 = 0, segs = 0;
        for (;;) {
            bar_wait(bSeg + 8 * seg.s, seg.ph, led, kSegWaitNs);
            led = __all_sync(~0u, led);
            const Seg sg = s_seg[seg.s];
            if (!led || sg.nt == 0)
                break;
            const bool both = !C::TWO && sg.nt > 1; // groups that have tiles of it
            const bool takes = C::TWO || both || (i0 & 1) == grp;
            const int t0 = C::TWO ? 0 : (grp ^ i0) & 1, dt = C::TWO ? 1 : 2;
            const int trow = C::TWO ? grp * 128 + row : row; // row of the tile
            const int g = sg.rt * MT + trow, ti = g / G;
            const bool live = ti < sg.n;
            const int tok_i = live ? ti : 0;
            const bool warp_live = __any_sync(~0u, live);
            Request rq;
            rq.tok = sg.tok;
            rq.n = sg.n;
            rq.len = sg.len;
            const uint64_t first = takes && sg.first_tail < sg.nt ? tree_bits(p, rq, tok_i) : 0;
            // a scale of zero makes all scores alike: the least number there is, since zero
            // times an unseen key's -infinity would be none
            float factor = fmaxf(base_factor, kLeast);
            // the reference, as a score and in base 2, and the sum
            float ms = -INFINITY, m = -INFINITY, l = 0.0f;

#pragma unroll 1
            for (int t = t0; t < sg.nt; t += dt) {
                const int kt = sg.key0 + t * kTile;
                bar_wait(bS + 8 * grp, s_ph, ok);
                __syncwarp();
                tc_after();
                if (gtid == 0)
                    s_acc[grp] = 0;
                if constexpr (C::F8)
                    if (t == t0)
                        factor = fmaxf(base_factor * s_f[segs & 3][trow], kLeast);
                // Tiles that reach the drafted tokens or the end, or hold a key
                // without a page.
                const uint32_t *bad = s_bad[(i0 + t) % kTiles];
                const bool is_tail = t >= sg.first_tail;
                const bool masked = is_tail || (bad[0] | bad[1] | bad[2] | bad[3]);
                // the keys of the tile's chunk c that the row sees
                auto seen = [&](int c) {
                    return (uint32_t)visible(p, rq, tok_i, first, kt + 32 * c, sg.end) & ~bad[c];
                };
                auto mask = [&](uint32_t *s, int c) { // unseen keys' scores to -infinity
                    const uint32_t vis = seen(c);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        s[e] = (vis >> e) & 1 ? s[e] : 0xff800000u;
                };
                // A negative scale's sign goes to the scores, so that the largest
                // one is the largest exponent.
                auto turn = [&](uint32_t *s) {
                    if (p.scale < 0.0f)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            s[e] ^= 0x80000000u;
                };
                auto highest = [](const uint32_t *s, float *mx) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
                };
                // The reference moves for the first keys seen, and when outgrown;
                // O (by the warp that has its lanes) and l with it.
                auto refer = [&](float top) {
                    const bool grow = (top - ms) * factor > kGrowth;
                    if (__any_sync(~0u, grow)) {
                        const float corr = grow ? exp2_fast((ms - top) * factor) : 1.0f;
                        ms = grow ? top : ms;
                        // (a score that leaves fp32 there is no reference: what follows is NaN)
                        m = grow ? top * factor == -INFINITY ? NAN : top * factor : m;
                        l *= corr;
                        if (t >= dt && quad == 0) { // this group's last product is done: S was issued after it
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(tO + c, o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                                tmem_st16(tO + c, o);
                            }
                            tmem_st_wait(); // the product that bP lets in adds to what is stored here
                        }
                    }
                    return m == -INFINITY ? 0.0f : m; // nothing seen yet
                };
                // The weights are rounded to the values' type for the product
                // (bf16: off by at most 2^-8 of each, fp16: 2^-11 or, those below
                // 2^-14, 2^-25, which is 2^-32 of the row's largest at most); their
                // sum l is of the unrounded ones.
                // (A third of the exponentials by polynomial on the FMA pipe did
                // not change 12 wide trees' time, half of them made it 5% longer.)
                // The reference is taken off as a score, before the factor: in base 2 it is
                // rounded, and from 2^28 on by more than the weights' type can take. (That is an
                // addition per pair of scores: 191.5 us against 188.6 on 12 wide trees, 77.1
                // against 76.0 on 11 requests of 8-bit keys; a branch to it for large references
                // costs those 188.8 and 81.) A row whose reference leaves fp32 in base 2 is NaN.
                auto weigh = [&](const uint32_t *s, float ref, uint32_t *w, float2 *sum) {
                    const float score = ms == -INFINITY ? 0.0f : ms, lift = ref * 0.0f + C::LIFT;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 x = add2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(-score, -score));
                        x = ffma2(x, make_float2(factor, factor), make_float2(lift, lift));
                        x = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                        sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], x);
                        w[e / 2] = pack2<C::F8>(x.x, x.y);
                    }
                };
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                float2 sum[2] = {};
                if constexpr (C::FEW) {
                    uint32_t s[32], w[16];
                    tmem_ld32(tS + 32 * quad, s);
                    tmem_ld_wait(s);
                    turn(s);
                    if (masked)
                        mask(s, quad);
                    highest(s, mx);
                    s_mx[2 * grp + s_ph][quad][lane] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    named_sync<kGroup>(2 + grp);
                    float top = s_mx[2 * grp + s_ph][0][lane];
#pragma unroll
                    for (int c = 1; c < 4; ++c)
                        top = fmaxf(top, s_mx[2 * grp + s_ph][c][lane]);
                    const float ref = refer(top);
                    weigh(s, ref, w, sum);
                    uint8_t *dst = smem + (sP - sQ) + grp * C::P1 + (quad >> 1) * C::ROWS * 128 + row * 128;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<uint4 *>(dst + ((((quad & 1) * 4 + c) ^ (row & 7)) << 4)) =
                            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                    fence_async_smem();
                } else if (warp_live) {
                    // twice over the scores; changed ones go back for the second time
                    uint32_t s[32];
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld32(tS + 32 * c, s);
                        tmem_ld_wait(s);
                        turn(s);
                        if (masked)
                            mask(s, c);
                        if (masked || p.scale < 0.0f)
                            tmem_st32(tS + 32 * c, s);
                        highest(s, mx);
                    }
                    tmem_st_wait();
                    const float ref = refer(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld32(tS + 32 * c, s);
                        tmem_ld_wait(s);
                        uint32_t w[16];
                        weigh(s, ref, w, sum);
                        tmem_st16(tS + 16 * c, w); // over scores already read
                    }
                    tmem_st_wait();
                }
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                if (is_tail) {
                    const int tail = sg.tail_index + t - sg.first_tail;
                    bar_wait(bTail + 8 * (tail % kRing), (tail / kRing) & 1, ok);
                    const uint32_t *odd = s_odd[tail % kRing];
                    // (One answer for all that meet below, also where the wait ran out: then
                    // odd may change under the reads.)
                    const uint32_t some = odd[0] | odd[1] | odd[2] | odd[3];
                    if (C::VOTE ? named_or<C::MEET>(C::TWO ? 1 : 2 + grp, some) : some != 0) {
                        // Rare: what is not finite must not reach, times zero, the
                        // rows that do not see its key. It is added to O here, for
                        // the rows that do, and taken out of the slot.
                        uint8_t *vs;
                        if constexpr (C::F8)
                            vs = smem + (sV - sQ) + ((i0 + t) & 1) * C::SLOT;
                        else
                            vs = smem + (sKV - sQ) + (2 * (i0 + t) + 1) % slots * slot_bytes;
                        __syncwarp();
                        if (quad == 0)
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(tO + c, o);
                                if (t < dt)
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        o[e] = 0u;
#pragma unroll 1
                                for (int k = 0; k < kTile; ++k) {
                                    if (!((odd[k >> 5] >> (k & 31)) & 1) || !((seen(k >> 5) >> (k & 31)) & 1))
                                        continue;
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const uint16_t b = *reinterpret_cast<const uint16_t *>(vs + op_off(k, (c + e) >> 3) + 2 * (e & 7));
                                        const float x = C::F8 ? __half2float(__ushort_as_half(b)) : bf16_bits_to_float(b);
                                        if (!isfinite(x))
                                            o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
                                    }
                                }
                                __syncwarp();
                                tmem_st16(tO + c, o);
                            }
                        tmem_st_wait();
                        meet(); // every group that reads the slot has read it
                        if ((odd[wq] >> lane) & 1) {
                            constexpr uint16_t EXP = C::F8 ? 0x7c00 : 0x7f80;
                            for (int e = 0; e < D; ++e) {
                                uint16_t *b = reinterpret_cast<uint16_t *>(vs + op_off(gtid, e >> 3) + 2 * (e & 7));
                                if ((*b & EXP) == EXP)
                                    *b = 0;
                            }
                        }
                        if (gtid == 0)
                            s_acc[grp] = t < dt;
                        fence_async_smem();
                        meet();
                    }
                }
                tc_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(bP + 8 * grp);
                s_ph ^= 1;
            }

            // ---- the segment's end -----------------------------------------------
            if (takes && warp_live) {
                float *part = part_of(p, blockIdx.x, sg.which, MT, D);
                const long long tk = sg.tok + tok_i;
                const int hq = sg.h * G + g - ti * G;
                const long long orow = tk * p.ld_out + (long long)hq * D;
                // A group's reference and sum (m, l), joined with the other's where
                // both have keys: l becomes the row's sum, the result the factor of
                // this group's O. One that saw nothing has l = 0 (or NaN) and O = 0.
                auto join = [&](float mo, float lo) {
                    const float top = both ? fmaxf(m, mo) : m;
                    float f = 1.0f;
                    if (both) {
                        f = m == -INFINITY ? 1.0f : exp2_fast(m - top);
                        const float fo = mo == -INFINITY ? 1.0f : exp2_fast(mo - top);
                        l = l * f + lo * fo;
                    }
                    if (live && quad == 0 && (!both || grp == 0)) {
                        if (!sg.whole) {
                            part[MT * D + trow] = top;
                            part[MT * D + MT + trow] = l;
                        } else if (p.lse) {
                            p.lse[tk * p.Hq + hq] = l == 0.0f ? -INFINITY : (top + (log2f(l) - C::LIFT)) * kLn2;
                        }
                    }
                    if (sg.whole) // the sum's inverse and the values' scale, on the way
                        f *= l == 0.0f ? 0.0f : p.cache.v_scale / l;
                    return f;
                };
                if constexpr (C::FEW) {
                    // The first warp of a group has all of its O. Half of the columns
                    // at a time go where P was, and all the warps write them out.
                    auto sync = [&] {
                        if (both)
                            named_sync<2 * kGroup>(1);
                        else
                            named_sync<kGroup>(2 + grp);
                    };
                    s_l[grp][quad][row] = l;
                    if (quad == 0) {
                        s_m[grp][0][row] = m;
                        s_out[grp][row] = orow;
                    }
                    bar_wait(bO + 8 * grp, s_ph ^ 1, ok); // this group's O is complete
                    __syncwarp();
                    tc_after();
                    sync();
                    l = (s_l[grp][0][row] + s_l[grp][1][row]) + (s_l[grp][2][row] + s_l[grp][3][row]);
                    const int og = grp ^ 1;
                    const float f = join(s_m[og][0][row], (s_l[og][0][row] + s_l[og][1][row]) + (s_l[og][2][row] + s_l[og][3][row]));
                    float4 *out = reinterpret_cast<float4 *>(smem + (sP - sQ));
                    const int wtid = both ? tid : gtid, wth = both ? 2 * kGroup : kGroup;
                    const int used = min(32, sg.n * G - sg.rt * MT);
                    const float4 *a = out + (both ? 0 : grp) * (C::P1 / 16);
                    // 2^lg float4 of a row at a time: all of up to 16 rows
                    const int lg = D == 128 && used <= 16 ? 5 : 4, rows_lg = lg == 5 ? 4 : 5;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 4 << lg) {
                        if (quad == 0)
#pragma unroll 1
                            for (int c = 0; c < 4 << lg; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(tO + c0 + c, o);
                                tmem_ld_wait(o);
                                if (row < used)
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        out[grp * (C::P1 / 16) + (row << lg) + ((c / 4 + e) ^ (row & 7))] =
                                            make_float4(__uint_as_float(o[4 * e]) * f, __uint_as_float(o[4 * e + 1]) * f,
                                                        __uint_as_float(o[4 * e + 2]) * f, __uint_as_float(o[4 * e + 3]) * f);
                                __syncwarp();
                            }
                        sync();
                        // rows next to each other in a part, columns in the output
#pragma unroll 2
                        for (int k = wtid; k < 512; k += wth) {
                            const int r = sg.whole ? k >> lg : k & ((1 << rows_lg) - 1), e = sg.whole ? k & ((1 << lg) - 1) : k >> rows_lg;
                            if (r >= used)
                                continue;
                            const int at = (r << lg) + (e ^ (r & 7));
                            float4 x = a[at];
                            if (both) {
                                const float4 y = a[C::P1 / 16 + at];
                                x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                            }
                            if (sg.whole)
                                *reinterpret_cast<uint2 *>(p.out + s_out[both ? 0 : grp][r] + c0 + 4 * e) = make_uint2(pack2<false>(x.x, x.y), pack2<false>(x.z, x.w));
                            else
                                reinterpret_cast<float4 *>(part)[(c0 / 4 + e) * MT + r] = x;
                        }
                        sync();
                    }
                } else {
                    bar_wait(bO + 8 * grp, s_ph ^ 1, ok);
                    __syncwarp();
                    tc_after();
                    const int pair = 5 + wq; // the barrier of the row's two warps
                    if (both) {
                        s_m[grp][0][row] = m;
                        s_l[grp][0][row] = l;
                        named_sync<64>(pair);
                    }
                    const float f = join(s_m[grp ^ 1][0][row], s_l[grp ^ 1][0][row]);
                    // Sixteen columns of a row: rows next to each other in a part,
                    // whole sectors of the output.
                    auto write = [&](const float4 *x, int col) {
                        if (live && sg.whole) {
                            uint4 *o = reinterpret_cast<uint4 *>(p.out + orow + col);
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                o[e] = make_uint4(pack2<false>(x[2 * e].x, x[2 * e].y), pack2<false>(x[2 * e].z, x[2 * e].w),
                                                  pack2<false>(x[2 * e + 1].x, x[2 * e + 1].y), pack2<false>(x[2 * e + 1].z, x[2 * e + 1].w));
                        } else if (live) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                reinterpret_cast<float4 *>(part)[(col / 4 + e) * MT + trow] = x[e];
                        }
                    };
                    // with both groups at it, either writes half of the columns, after
                    // an exchange of the other half between the row's two warps
                    float4 *mine = reinterpret_cast<float4 *>(smem + (sOut - sQ) + warp * C::OUT1);
                    const float4 *other = reinterpret_cast<const float4 *>(smem + (sOut - sQ) + (warp ^ 4) * C::OUT1);
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t raw[32];
                        tmem_ld32(tO + c, raw);
                        tmem_ld_wait(raw);
                        float4 x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x[e] = make_float4(__uint_as_float(raw[4 * e]) * f, __uint_as_float(raw[4 * e + 1]) * f,
                                               __uint_as_float(raw[4 * e + 2]) * f, __uint_as_float(raw[4 * e + 3]) * f);
                        if (both) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mine[lane * 4 + (e ^ ((lane >> 1) & 3))] = grp ? x[e] : x[4 + e];
                            named_sync<64>(pair);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 b = other[lane * 4 + (e ^ ((lane >> 1) & 3))];
                                if (grp)
                                    x[e] = x[4 + e];
                                x[e] = make_float4(x[e].x + b.x, x[e].y + b.y, x[e].z + b.z, x[e].w + b.w);
                            }
                            named_sync<64>(pair);
                            write(x, c + 16 * grp);
                        } else {
                            write(x, c);
                            write(x + 4, c + 16);
                        }
                        __syncwarp();
                    }
                }
                tc_before();
            }
            __syncwarp();
            if (lane == 0)
                bar_arrive(bSegFree + 8 * seg.s);
            seg.step(1, kRing);
            i0 += sg.nt;
            ++segs;
        }
    }
    tc_before();
    if (!ok || !led) {
        set_status(p.status, SGQ_STATUS_TIMEOUT);
        s_late = 1;
    }
    __syncthreads();
    if (warp == kIssuer) {
        if (s_late) {
            // bulk copies that nothing waited for may be on their way still, and take
            // microseconds
            unsigned long long t0, t;
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
            do
                asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
            while (t - t0 < kDrainNs);
        }
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
    }
}

// Joins the parts of the items that several CTAs worked on, in key order. A unit
// is 8 rows of 64 columns (a lane: one row, sixteen columns, four by four); the
// CTAs of an item share its units, CTA c0 + x taking units x, x + parts, ...,
// and a CTA's warps share the parts of each where there are fewer units than
// warps. Bound by the trips to L2: four parts' loads are on their way at once.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps, 2) join_kernel(const AttnProblem p, int MT)
{
    constexpr int BATCH = 4, VEC = 4;
    __shared__ float4 s_o[kJoinWarps][VEC][32];
    __shared__ float s_m[kJoinWarps][32], s_l[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_launch_dependents();
    grid_dependency_wait();
    const Split sp = static_cast<const Split *>(p.workspace)[blockIdx.x];
    if (sp.parts == 0)
        return;
    const int G = p.Hq / p.cache.heads, first = (int)(blockIdx.x >> 1) - sp.c0;
    const int rows = (int)min((long long)MT, (long long)sp.n * G - (long long)sp.rt * MT);
    const int units = (rows + 7) / 8 * (D / 64);
    const int mine = units > first ? (units - first + sp.parts - 1) / sp.parts : 0;
    int wpu = kJoinWarps; // warps per unit
    while (wpu > 1 && wpu * mine > kJoinWarps)
        wpu >>= 1;
    for (int k0 = 0; k0 < mine; k0 += kJoinWarps / wpu) {
        const int k = k0 + warp / wpu, u = first + k * sp.parts;
        const int row = u / (D / 64) * 8 + (lane & 7), c4 = u % (D / 64) * 16 + (lane >> 3);
        float4 o[VEC] = {};
        float m = -INFINITY, l = 0.0f;
        if (k < mine && row < rows) {
            for (int b = warp % wpu; b < sp.parts; b += BATCH * wpu) {
                float pm[BATCH], pl[BATCH];
                float4 v[BATCH][VEC];
#pragma unroll
                for (int e = 0; e < BATCH; ++e) {
                    const int c = b + e * wpu;
                    const bool in = c < sp.parts;
                    const float *part = part_of(p, sp.c0 + (in ? c : 0), !in || c == 0, MT, D);
                    pm[e] = in ? part[MT * D + row] : -INFINITY;
                    pl[e] = in ? part[MT * D + MT + row] : 0.0f;
#pragma unroll
                    for (int x = 0; x < VEC; ++x)
                        v[e][x] = in ? reinterpret_cast<const float4 *>(part)[(c4 + 4 * x) * MT + row] : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                float top = m;
#pragma unroll
                for (int e = 0; e < BATCH; ++e)
                    top = fmaxf(top, pm[e]);
                const float ref = top == -INFINITY ? 0.0f : top, f = exp2_fast(m - ref);
                m = top;
                l *= f;
#pragma unroll
                for (int x = 0; x < VEC; ++x)
                    o[x] = make_float4(o[x].x * f, o[x].y * f, o[x].z * f, o[x].w * f);
#pragma unroll
                for (int e = 0; e < BATCH; ++e) {
                    const float w = exp2_fast(pm[e] - ref);
                    l += pl[e] * w;
#pragma unroll
                    for (int x = 0; x < VEC; ++x)
                        o[x] = make_float4(o[x].x + v[e][x].x * w, o[x].y + v[e][x].y * w, o[x].z + v[e][x].z * w, o[x].w + v[e][x].w * w);
                }
            }
        }
        if (wpu > 1) {
#pragma unroll
            for (int x = 0; x < VEC; ++x)
                s_o[warp][x][lane] = o[x];
            s_m[warp][lane] = m;
            s_l[warp][lane] = l;
            __syncthreads();
            if (warp % wpu == 0) {
                float top = m;
                for (int w = 1; w < wpu; ++w)
                    top = fmaxf(top, s_m[warp + w][lane]);
                const float ref = top == -INFINITY ? 0.0f : top, f = exp2_fast(m - ref);
                m = top;
                l *= f;
#pragma unroll
                for (int x = 0; x < VEC; ++x)
                    o[x] = make_float4(o[x].x * f, o[x].y * f, o[x].z * f, o[x].w * f);
                for (int w = 1; w < wpu; ++w) {
                    const float e = exp2_fast(s_m[warp + w][lane] - ref);
                    l += s_l[warp + w][lane] * e;
#pragma unroll
                    for (int x = 0; x < VEC; ++x) {
                        const float4 v = s_o[warp + w][x][lane];
                        o[x] = make_float4(o[x].x + v.x * e, o[x].y + v.y * e, o[x].z + v.z * e, o[x].w + v.w * e);
                    }
                }
            }
            __syncthreads();
        }
        if (k < mine && row < rows && warp % wpu == 0) {
            const int g = sp.rt * MT + row, ti = g / G, hq = sp.h * G + g - ti * G;
            const long long t = sp.tok + ti;
            const float inv = l == 0.0f ? 0.0f : p.cache.v_scale / l, lift = p.cache.type == SGQ_TYPE_E4M3 ? kLift16 : 0.0f;
            uint16_t *out = p.out + t * p.ld_out + (long long)hq * D + 4 * c4;
#pragma unroll
            for (int x = 0; x < VEC; ++x)
                *reinterpret_cast<uint2 *>(out + 16 * x) =
                    make_uint2(pack2<false>(o[x].x * inv, o[x].y * inv), pack2<false>(o[x].z * inv, o[x].w * inv));
            if (p.lse && c4 == 0)
                p.lse[t * p.Hq + hq] = l == 0.0f ? -INFINITY : (m + (log2f(l) - lift)) * kLn2;
        }
    }
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
    // Bulk copies where a box, the largest power of two up to 64 slots that
    // divides the page, has kBoxBytes at least: 79 us against 88 by cp.async on 11
    // requests of up to 60000 8-bit keys in pages of 24 (boxes of 512 bytes), 61 against
    // 86 on 24 ragged ones in pages of 32 (boxes of 4 KB); with pages of 12 (boxes of
    // 256 bytes) 103 against 96.
    int box = 1;
    while (box < 64 && p.cache.page % (2 * box) == 0)
        box *= 2;
    CUtensorMap kmap{}, vmap{};
    if (box * std::min(C::ROWB, 128) < kBoxBytes || kTile / box * C::ROWB > 32 * 128) // a lane a piece
        box = 0;
    else if (!encoder())
        return cudaErrorNotSupported;
    else if (!encode(&kmap, p.cache, p.cache.k, box) || !encode(&vmap, p.cache, p.cache.v, box))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(attn_kernel<D, KV, MT>, C::SMEM, done);
    if (e != cudaSuccess)
        return e;
    e = launch_step(attn_kernel<D, KV, MT>, dim3(grid), C::THREADS, C::SMEM, 1, stream, p, kmap, vmap, box);
    if (e != cudaSuccess)
        return e;
    return launch_step(join_kernel<D>, dim3(2 * grid), 32 * kJoinWarps, 0, 1, stream, p, MT);
}

// Rows of a tile, for what a request has on average.
int row_tile(int T, int R, int Hq, int Hkv)
{
    const long long rows = (long long)((T + R - 1) / R) * (Hq / Hkv);
    return rows <= 32 ? 32 : rows <= 128 ? 128 : 256;
}

template <int D, int KV>
cudaError_t launch_d(const AttnProblem &p, int num_sms, cudaStream_t stream)
{
    const int grid = std::min(num_sms, kMaxGrid);
    switch (row_tile(p.T, p.R, p.Hq, p.cache.heads)) {
    case 32: return launch_t<D, KV, 32>(p, grid, stream);
    case 128: return launch_t<D, KV, 128>(p, grid, stream);
    default: return launch_t<D, KV, 256>(p, grid, stream);
    }
}

} // namespace

size_t attn_workspace_bytes(int T, int R, int Hq, int Hkv, int D)
{
    return 2 * kMaxGrid * sizeof(Split) +
           (size_t)2 * kMaxGrid * row_tile(T, R, Hq, Hkv) * (D + 2) * sizeof(float);
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
