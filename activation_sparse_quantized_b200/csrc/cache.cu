// cache.cu -- sgq_cache_plan and sgq_cache_write: the bookkeeping of a paged
// key/value cache on the GPU, and the store of a step's keys and values.
#include "sgq_device.cuh"
#include "sgq_launch.h"
#include "step_launch.cuh"

#include <algorithm>
#include <cuda_fp8.h>

namespace sgq {

namespace {

// ---------------------------------------------------------------------------
// The plan: whole-number prefix sums over the requests, then one output row
// per new token and one table entry per new page.
//
//   cu[r]   = min(max_tokens, sum over s < r of n_s)
//   want_r  = ceil((l_r + n_r) / page),  need_r = max(0, want_r - held_r)
//   base_r  = sum over s < r of need_s;  served: need_r = 0 or base_r + need_r <= free
//   page j of request r: table[r][j] for j < held_r, else the free list's entry
//   number base_r + (j - held_r) from its end
//
// One cluster of up to 8 CTAs: every CTA makes the sums for itself (the inputs
// are a few KB), then the CTAs share out the pages and the tokens, each found
// by bisection of its prefix sum, so that one long request is shared as well as
// many short ones. The cluster's barrier stands between the last read of held
// and free_count and the first write of held_out and free_count_out, which may
// be the same words. What bounds it is latency: a load, two scans, a load.
//
// More tokens than the cluster has threads go to a second kernel over all SMs,
// which reads the slots off the finished table: 16 requests with 136 tokens
// take 4.6 us on the one kernel, and 2000 requests with 301,000 tokens 16.8 us on
// two, 75 us on one.
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive sum of v over the CTA's threads; total receives the whole sum.
__device__ __forceinline__ long long block_scan(long long v, long long *part, long long &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(~0u, s, o);
        if (lane >= o)
            s += t;
    }
    if (lane == 31)
        part[warp] = s;
    __syncthreads();
    long long w = part[lane]; // kPlanThreads / 32 = 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(~0u, w, o);
        if (lane >= o)
            w += t;
    }
    total = __shfl_sync(~0u, w, 31);
    const long long before = __shfl_sync(~0u, w, warp ? warp - 1 : 0);
    __syncthreads();
    return s - v + (warp ? before : 0);
}

// The largest v of the CTA's threads, in each of them. Not before the threads
// are done with part.
__device__ __forceinline__ long long block_max(long long v, long long *part)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = max(v, __shfl_xor_sync(~0u, v, o));
    if (lane == 0)
        part[warp] = v;
    __syncthreads();
    v = part[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = max(v, __shfl_xor_sync(~0u, v, o));
    return v;
}

// The last r < R with sum[r] <= x; sum is non-decreasing from 0.
__device__ __forceinline__ int place_in(const int32_t *sum, int R, int x)
{
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Pages of len + n tokens (both at most 2^30).
__device__ __forceinline__ int pages_of(int len, int n, int page)
{
    return (int)(((uint32_t)len + n + page - 1) / (uint32_t)page);
}

// Row t of the outputs: new token i of request r, on page `id` (-1: none).
__device__ __forceinline__ int put_token(const PlanProblem &p, int t, int r, int i, int len, int id, int off, bool served)
{
    int bits = 0;
    long long slot = -1;
    if (served) {
        if (id >= 0 && id < p.num_pages)
            slot = (long long)id * p.page + off;
        else
            bits = SGQ_STATUS_BAD_INDEX;
    }
    p.slots[t] = slot;
    if (p.pos)
        p.pos[t] = len + (p.depth ? p.depth[t] : i);
    if (p.req)
        p.req[t] = r;
    return bits;
}

// rows: whether this kernel writes the tokens' rows (else token_kernel does).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanProblem p, const int rows)
{
    extern __shared__ int32_t sh[];
    __shared__ long long part[32];
    int32_t *cu = sh;               // [R + 1]
    int32_t *base = cu + p.R + 1;   // [R], sums of pages, up to INT_MAX
    int32_t *len = base + p.R;      // [R]
    int32_t *held = len + p.R;      // [R]
    const int tid = threadIdx.x;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int gtid = (int)rank * kPlanThreads + tid, gsize = (int)ctas * kPlanThreads;
    int bits = 0;
    grid_launch_dependents();
    grid_dependency_wait();

    const int count = *p.free_count;
    for (int r = tid; r < p.R; r += kPlanThreads) {
        int l = p.lens[r], n = p.news[r], h = p.held[r];
        // a request whose state cannot be is given no tokens
        if (l < 0 || n < 0 || h < 0 || h > p.table_ld || (long long)h * p.page < l) {
            bits |= SGQ_STATUS_BAD_COUNT;
            n = 0;
            l = max(l, 0);
            h = min(max(h, 0), p.table_ld);
        }
        len[r] = l;
        base[r] = n;
        held[r] = h;
    }
    const int avail = min(max(count, 0), p.num_pages);
    if (count != avail)
        bits |= SGQ_STATUS_BAD_COUNT;
    __syncthreads();
    if (ctas > 1)
        cluster_arrive(); // this CTA has read held and free_count

    // tokens
    const int per = (p.R + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    long long sum = 0, total;
    for (int r = r0; r < r1; ++r)
        sum += base[r];
    long long at = block_scan(sum, part, total);
    if (total > p.max_tokens)
        bits |= SGQ_STATUS_BAD_COUNT;
    for (int r = r0; r < r1; ++r) {
        cu[r] = (int32_t)min(at, (long long)p.max_tokens);
        at += base[r];
    }
    if (tid == 0)
        cu[p.R] = (int32_t)min(total, (long long)p.max_tokens);
    __syncthreads();

    // pages: needed ones, -1 for a request longer than a table row
    auto need_of = [&](int r) {
        const int n = cu[r + 1] - cu[r];
        const int want = n ? pages_of(len[r], n, p.page) : 0;
        return want > p.table_ld ? -1 : max(0, want - held[r]);
    };
    sum = 0;
    for (int r = r0; r < r1; ++r)
        sum += max(need_of(r), 0);
    at = block_scan(sum, part, total);
    // the pages of the requests before the first that does not fit
    long long used = total;
    for (int r = r0; r < r1; ++r) {
        const int need = need_of(r);
        if (need < 0)
            bits |= SGQ_STATUS_BAD_COUNT;
        base[r] = (int32_t)min(at, 0x7fffffffll);
        at += max(need, 0);
        if (need > 0 && at > avail) {
            bits |= SGQ_STATUS_NO_PAGES;
            used = min(used, at - need);
        }
    }
    if (total > avail) {
        __syncthreads();
        used = -block_max(-used, part);
    }
    __syncthreads();
    auto served = [&](int r, int need) { return need == 0 || (need > 0 && (long long)base[r] + need <= avail); };
    auto fresh = [&](int r, int j) { return p.free_pages[avail - 1 - (base[r] + (j - held[r]))]; };

    // new tokens
    const int T = rows ? cu[p.R] : 0;
    for (int t = gtid; t < T; t += gsize) {
        const int r = place_in(cu, p.R, t), i = t - cu[r];
        const uint32_t at_pos = (uint32_t)len[r] + i; // below 2^31
        const bool ok = served(r, need_of(r));
        const int j = at_pos / (uint32_t)p.page, off = at_pos - j * p.page;
        const int id = !ok ? -1 : j < held[r] ? p.table[(long long)r * p.table_ld + j] : fresh(r, j);
        bits |= put_token(p, t, r, i, len[r], id, off, ok);
    }

    if (ctas > 1)
        cluster_wait(); // every CTA has read held and free_count
    // new pages
    for (int q = gtid; q < (int)used; q += gsize) {
        const int r = place_in(base, p.R, q), j = held[r] + (q - base[r]);
        p.table[(long long)r * p.table_ld + j] = fresh(r, j);
    }
    for (int r = gtid; r < p.R; r += gsize) {
        const int need = need_of(r);
        p.held_out[r] = held[r] + (served(r, need) ? need : 0);
        p.cu_new[r] = cu[r];
    }
    if (gtid == 0) {
        p.cu_new[p.R] = cu[p.R];
        *p.free_count_out = avail - (int)used;
    }
    if (bits)
        set_status(p.status, bits);
}

// The tokens' rows off the finished table: a request that was not served has
// fewer pages than its last token needs, and none of its tokens gets a slot.
constexpr int kTokenThreads = 256;

__global__ void __launch_bounds__(kTokenThreads) token_kernel(const PlanProblem p)
{
    extern __shared__ int32_t cu[]; // [R + 1]
    grid_launch_dependents();
    grid_dependency_wait();
    for (int r = threadIdx.x; r <= p.R; r += kTokenThreads)
        cu[r] = p.cu_new[r];
    __syncthreads();
    const int T = cu[p.R];
    int bits = 0;
    for (int t = blockIdx.x * kTokenThreads + threadIdx.x; t < T; t += gridDim.x * kTokenThreads) {
        const int r = place_in(cu, p.R, t), i = t - cu[r], len = p.lens[r];
        const int j = ((uint32_t)len + i) / (uint32_t)p.page, off = len + i - j * p.page;
        const bool ok = pages_of(len, cu[r + 1] - cu[r], p.page) <= p.held_out[r];
        const int id = ok ? p.table[(long long)r * p.table_ld + j] : -1;
        bits |= put_token(p, t, r, i, len, id, off, ok);
    }
    if (bits)
        set_status(p.status, bits);
}

// ---------------------------------------------------------------------------
// The store: one CTA per token, D / 16 threads per head, each eight pairs of
// several heads, so that a position's cosines and sines are read once and the
// heads' loads are in flight together. The products and sums of the rotation
// are rounded one by one (no contraction), so that a stored value does not
// depend on how the compiler orders them. 4001 tokens of 64 query and 8 key heads
// of 128 are bound by memory: 35.7 us, 4.7 TB/s; a thread per (head, eight pairs)
// with its own cosines, two thirds of the loads, took 46. 16 tokens are bound by
// the chain of loads: 2.3 us.
// ---------------------------------------------------------------------------

__device__ __forceinline__ void unpack_bf16(const uint4 &u, float *f)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)float_to_bf16_bits(f[2 * i]) |
               ((uint32_t)float_to_bf16_bits(f[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 pack_e4m3(const float *f, float scale)
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(f[4 * i] / scale, f[4 * i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(f[4 * i + 2] / scale, f[4 * i + 3] / scale), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

constexpr int kWriteThreads = 512; // at most
constexpr int kWriteBatch = 4;     // heads of a thread at once, with many tokens

template <int D, int BATCH>
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const WriteProblem p)
{
    constexpr int CPR = D / 16;
    constexpr bool EARLY = BATCH == 1;
    const int STEP = blockDim.x / CPR; // heads side by side
    const int Hkv = p.cache.heads, heads = p.Hq + 2 * Hkv;
    grid_launch_dependents();
    grid_dependency_wait();
    // With one head a thread every load that needs no other's result is on its way
    // before the first wait (rows behind the last token are read, and not used). With
    // more the registers cost more than that brings: 38.2 us against 35.7.
    const long long t = blockIdx.x;
    const int c = threadIdx.x % CPR;
    uint4 raw[BATCH][2];
    auto load = [&](int h0) {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int h = h0 + b * STEP;
            const uint16_t *src = h < p.Hq ? p.q + t * p.ld_q + (long long)h * D
                                  : h < p.Hq + Hkv ? p.k + t * p.ld_k + (long long)(h - p.Hq) * D
                                                   : p.v + t * p.ld_v + (long long)(h - p.Hq - Hkv) * D;
            if (h < heads) {
                raw[b][0] = *reinterpret_cast<const uint4 *>(src + 8 * c);
                raw[b][1] = *reinterpret_cast<const uint4 *>(src + D / 2 + 8 * c);
            }
        }
    };
    const int n = p.n_tokens ? *p.n_tokens : p.T, pos = p.rope ? p.pos[t] : 0;
    const long long slot = p.slots[t];
    if (EARLY)
        load(threadIdx.x / CPR);
    if (t == 0 && threadIdx.x == 0 && (n < 0 || n > p.T))
        set_status(p.status, SGQ_STATUS_BAD_COUNT);
    if (t >= n)
        return;
    float cs[8], sn[8];
    if (p.rope) {
        if (pos < 0 || pos >= p.rope_len) {
            if (threadIdx.x == 0)
                set_status(p.status, SGQ_STATUS_BAD_INDEX);
            return;
        }
        const float4 *rc = reinterpret_cast<const float4 *>(p.rope + (long long)pos * D + 8 * c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 a = rc[i], b = rc[D / 8 + i];
            cs[4 * i] = a.x, cs[4 * i + 1] = a.y, cs[4 * i + 2] = a.z, cs[4 * i + 3] = a.w;
            sn[4 * i] = b.x, sn[4 * i + 1] = b.y, sn[4 * i + 2] = b.z, sn[4 * i + 3] = b.w;
        }
    }
    // where keys and values go
    const bool store = slot >= 0 && slot < (long long)p.cache.num_pages * p.cache.page;
    if (!store && slot != -1 && threadIdx.x == 0)
        set_status(p.status, SGQ_STATUS_BAD_INDEX);
    long long base = 0;
    if (store) {
        const long long pg = slot / p.cache.page;
        base = pg * p.cache.page_stride + (slot - pg * p.cache.page) * p.cache.slot_stride + 8 * c;
    }
    for (int h0 = threadIdx.x / CPR; h0 < heads; h0 += BATCH * STEP) {
        if (!EARLY || h0 >= STEP)
            load(h0);
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            int h = h0 + b * STEP;
            if (h >= heads)
                break;
            float lo[8], hi[8];
            unpack_bf16(raw[b][0], lo);
            unpack_bf16(raw[b][1], hi);
            if (p.rope && h < p.Hq + Hkv) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = __fsub_rn(__fmul_rn(lo[i], cs[i]), __fmul_rn(hi[i], sn[i]));
                    const float y = __fadd_rn(__fmul_rn(hi[i], cs[i]), __fmul_rn(lo[i], sn[i]));
                    lo[i] = x;
                    hi[i] = y;
                }
            }
            if (h < p.Hq) {
                uint16_t *dst = p.q_out + t * p.ld_qo + (long long)h * D + 8 * c;
                *reinterpret_cast<uint4 *>(dst) = pack_bf16(lo);
                *reinterpret_cast<uint4 *>(dst + D / 2) = pack_bf16(hi);
                continue;
            }
            if (!store)
                continue;
            const bool is_k = h < p.Hq + Hkv;
            h -= is_k ? p.Hq : p.Hq + Hkv;
            const long long e = base + h * p.cache.head_stride;
            void *dst = is_k ? p.cache.k : p.cache.v;
            if (p.cache.type == SGQ_TYPE_E4M3) {
                const float scale = is_k ? p.cache.k_scale : p.cache.v_scale;
                uint8_t *d8 = static_cast<uint8_t *>(dst) + e;
                *reinterpret_cast<uint2 *>(d8) = pack_e4m3(lo, scale);
                *reinterpret_cast<uint2 *>(d8 + D / 2) = pack_e4m3(hi, scale);
            } else {
                uint16_t *d16 = static_cast<uint16_t *>(dst) + e;
                *reinterpret_cast<uint4 *>(d16) = pack_bf16(lo);
                *reinterpret_cast<uint4 *>(d16 + D / 2) = pack_bf16(hi);
            }
        }
    }
}

} // namespace

cudaError_t launch_plan(const PlanProblem &p, int num_sms, cudaStream_t stream)
{
    const bool rows = p.max_tokens <= kPlanCtas * kPlanThreads;
    int ctas = 1;
    while (ctas < kPlanCtas && ctas * kPlanThreads < std::max(p.R, p.max_tokens))
        ctas *= 2;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(plan_kernel, (4 * SGQ_MAX_REQUESTS + 1) * 4, done);
    if (e == cudaSuccess)
        e = launch_step(plan_kernel, dim3(ctas), kPlanThreads, (size_t)(4 * p.R + 1) * 4, ctas, stream, p, (int)rows);
    if (rows || e != cudaSuccess)
        return e;
    const int grid = std::min(4 * num_sms, (p.max_tokens + kTokenThreads - 1) / kTokenThreads);
    return launch_step(token_kernel, dim3(grid), kTokenThreads, (size_t)(p.R + 1) * 4, 1, stream, p);
}

cudaError_t launch_write(const WriteProblem &p, int num_sms, cudaStream_t stream)
{
    // as many threads as take all the heads at once, in whole warps; with few
    // tokens, where latency counts, one head each
    const bool few = p.T < 2 * num_sms;
    const int heads = p.Hq + 2 * p.cache.heads, batch = few ? 1 : kWriteBatch;
    const int threads = (heads + batch - 1) / batch * (p.cache.dim / 16);
    const int block = std::min(kWriteThreads, (threads + 31) / 32 * 32);
    const auto kern = p.cache.dim == 64 ? (few ? write_kernel<64, 1> : write_kernel<64, kWriteBatch>)
                                        : (few ? write_kernel<128, 1> : write_kernel<128, kWriteBatch>);
    return launch_step(kern, dim3(p.T), block, 0, 1, stream, p);
}

} // namespace sgq
