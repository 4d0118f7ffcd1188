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
// per new token.
//
//   cu[r]   = min(max_tokens, sum over s < r of n_s)
//   want_r  = ceil((l_r + n_r) / page),  need_r = max(0, want_r - held_r)
//   base_r  = sum over s < r of need_s;  served: need_r = 0 or base_r + need_r <= free
//   page j of request r: table[r][j] for j < held_r, else the free list's entry
//   number base_r + (j - held_r) from its end
//
// One cluster of up to 8 CTAs: every CTA makes the sums for itself (the inputs
// are a few KB), then the CTAs share out the tokens and the table rows. The
// cluster's barrier stands between the last read of held and free_count and
// the first write of held_out and free_count_out, which may be the same words.
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;

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

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanProblem p)
{
    extern __shared__ int32_t sh[];
    __shared__ long long part[32];
    int32_t *cu = sh;            // [R + 1]
    int32_t *base = cu + p.R + 1; // [R] first free-list entry, or -1: not served
    int32_t *len = base + p.R;   // [R]
    int32_t *held = len + p.R;   // [R]
    const int tid = threadIdx.x;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    int bits = 0;
    grid_launch_dependents();
    grid_dependency_wait();

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
    const long long avail = min(max(*p.free_count, 0), p.num_pages);
    if (*p.free_count != avail)
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

    // pages
    sum = 0;
    for (int r = r0; r < r1; ++r) {
        const int n = cu[r + 1] - cu[r];
        const long long want = n ? ((long long)len[r] + n + p.page - 1) / p.page : 0;
        int need = (int)max(0ll, min(want, (long long)p.table_ld + 1) - held[r]);
        if (want > p.table_ld) { // longer than a table row
            bits |= SGQ_STATUS_BAD_COUNT;
            need = -1;
        }
        base[r] = need;
        sum += max(need, 0);
    }
    at = block_scan(sum, part, total);
    for (int r = r0; r < r1; ++r) {
        const int need = base[r];
        const bool served = need == 0 || (need > 0 && at + need <= avail);
        if (need > 0 && !served)
            bits |= SGQ_STATUS_NO_PAGES;
        base[r] = served ? (int32_t)min(at, avail) : -1;
        at += max(need, 0);
    }
    __syncthreads();

    // new tokens
    const int T = cu[p.R];
    for (int t = rank * kPlanThreads + tid; t < T; t += ctas * kPlanThreads) {
        int lo = 0, hi = p.R; // cu[lo] <= t < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        const int i = t - cu[lo];
        long long slot = -1;
        if (base[lo] >= 0) {
            const long long at_pos = (long long)len[lo] + i;
            const int j = (int)(at_pos / p.page), off = (int)(at_pos - (long long)j * p.page);
            const int id = j < held[lo]
                               ? p.table[(long long)lo * p.table_ld + j]
                               : p.free_pages[avail - 1 - (base[lo] + (j - held[lo]))];
            if (id >= 0 && id < p.num_pages)
                slot = (long long)id * p.page + off;
            else
                bits |= SGQ_STATUS_BAD_INDEX;
        }
        p.slots[t] = slot;
        if (p.pos)
            p.pos[t] = len[lo] + (p.depth ? p.depth[t] : i);
        if (p.req)
            p.req[t] = lo;
    }

    if (ctas > 1)
        cluster_wait(); // every CTA has read held and free_count
    // table rows: one warp per request
    const int lane = tid & 31;
    for (int r = rank * (kPlanThreads / 32) + (tid >> 5); r < p.R;
         r += ctas * (kPlanThreads / 32)) {
        const int n = cu[r + 1] - cu[r], h = held[r];
        int want = h;
        if (n && base[r] >= 0) {
            want = max(h, (int)(((long long)len[r] + n + p.page - 1) / p.page));
            for (int j = h + lane; j < want; j += 32)
                p.table[(long long)r * p.table_ld + j] =
                    p.free_pages[avail - 1 - (base[r] + (j - h))];
        }
        if (lane == 0)
            p.held_out[r] = want;
    }
    for (int r = rank * kPlanThreads + tid; r <= p.R; r += ctas * kPlanThreads)
        p.cu_new[r] = cu[r];
    // pages handed out: the served requests are those before the first that
    // did not fit, so the sum ends at the last served one
    int used = 0;
    if (rank == 0) {
        for (int r = tid; r < p.R; r += kPlanThreads) {
            const int n = cu[r + 1] - cu[r], h = held[r];
            if (n && base[r] >= 0)
                used = max(used, base[r] + max(0, (int)(((long long)len[r] + n + p.page - 1) /
                                                        p.page) - h));
        }
        used = __reduce_max_sync(~0u, used);
        if (lane == 0)
            part[tid >> 5] = used;
    }
    __syncthreads();
    if (rank == 0 && tid == 0) {
        for (int w = 0; w < kPlanThreads / 32; ++w)
            used = max(used, (int)part[w]);
        *p.free_count_out = (int32_t)(avail - used);
    }
    if (bits)
        set_status(p.status, bits);
}

// ---------------------------------------------------------------------------
// The store: one thread per (token, head, eight pairs). The products and sums
// of the rotation are rounded one by one (no contraction), so that a stored
// value does not depend on how the compiler orders them.
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

constexpr int kWriteThreads = 256;

__global__ void __launch_bounds__(kWriteThreads) write_kernel(const WriteProblem p)
{
    const int D = p.cache.dim, half = D / 2, Hkv = p.cache.heads;
    const int cpr = D / 16, heads = (p.q ? p.Hq : 0) + 2 * Hkv, per = heads * cpr;
    grid_launch_dependents();
    grid_dependency_wait();
    const int T = p.n_tokens ? min(max(*p.n_tokens, 0), p.T) : p.T;
    const long long g = (long long)blockIdx.x * kWriteThreads + threadIdx.x;
    const long long t = g / per;
    if (p.n_tokens && g == 0 && *p.n_tokens != T)
        set_status(p.status, SGQ_STATUS_BAD_COUNT);
    if (t >= T)
        return;
    const int rest = (int)(g - t * per), c = rest % cpr;
    int h = rest / cpr;
    if (!p.q)
        h += p.Hq;
    const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + Hkv;
    if (!is_q)
        h -= is_k ? p.Hq : p.Hq + Hkv;
    const uint16_t *src = is_q   ? p.q + t * p.ld_q
                          : is_k ? p.k + t * p.ld_k
                                 : p.v + t * p.ld_v;
    src += (long long)h * D + 8 * c;
    float lo[8], hi[8];
    unpack_bf16(*reinterpret_cast<const uint4 *>(src), lo);
    unpack_bf16(*reinterpret_cast<const uint4 *>(src + half), hi);
    if (p.rope) {
        const int pos = p.pos[t];
        if (pos < 0 || pos >= p.rope_len) {
            set_status(p.status, SGQ_STATUS_BAD_INDEX);
            return;
        }
        if (is_q || is_k) {
            const float4 *rc =
                reinterpret_cast<const float4 *>(p.rope + (long long)pos * D + 8 * c);
            const float4 *rs = reinterpret_cast<const float4 *>(
                p.rope + (long long)pos * D + half + 8 * c);
            const float4 c0 = rc[0], c1 = rc[1], s0 = rs[0], s1 = rs[1];
            const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = __fsub_rn(__fmul_rn(lo[i], cs[i]), __fmul_rn(hi[i], sn[i]));
                const float b = __fadd_rn(__fmul_rn(hi[i], cs[i]), __fmul_rn(lo[i], sn[i]));
                lo[i] = a;
                hi[i] = b;
            }
        }
    }
    if (is_q) {
        uint16_t *dst = p.q_out + t * p.ld_qo + (long long)h * D + 8 * c;
        *reinterpret_cast<uint4 *>(dst) = pack_bf16(lo);
        *reinterpret_cast<uint4 *>(dst + half) = pack_bf16(hi);
        return;
    }
    const long long slot = p.slots[t];
    if (slot < 0 || slot >= (long long)p.cache.num_pages * p.cache.page) {
        if (slot != -1)
            set_status(p.status, SGQ_STATUS_BAD_INDEX);
        return;
    }
    const long long pg = slot / p.cache.page, off = slot - pg * p.cache.page;
    const long long e = pg * p.cache.page_stride + off * p.cache.slot_stride +
                        h * p.cache.head_stride + 8 * c;
    void *dst = is_k ? p.cache.k : p.cache.v;
    if (p.cache.type == SGQ_TYPE_E4M3) {
        const float scale = is_k ? p.cache.k_scale : p.cache.v_scale;
        uint8_t *d8 = static_cast<uint8_t *>(dst) + e;
        *reinterpret_cast<uint2 *>(d8) = pack_e4m3(lo, scale);
        *reinterpret_cast<uint2 *>(d8 + half) = pack_e4m3(hi, scale);
    } else {
        uint16_t *d16 = static_cast<uint16_t *>(dst) + e;
        *reinterpret_cast<uint4 *>(d16) = pack_bf16(lo);
        *reinterpret_cast<uint4 *>(d16 + half) = pack_bf16(hi);
    }
}

} // namespace

cudaError_t launch_plan(const PlanProblem &p, int num_sms, cudaStream_t stream)
{
    (void)num_sms;
    int ctas = 1;
    while (ctas < 8 && ctas * kPlanThreads < p.max_tokens)
        ctas *= 2;
    return launch_step(plan_kernel, dim3(ctas), kPlanThreads, (size_t)(4 * p.R + 1) * 4, ctas, stream, p);
}

cudaError_t launch_write(const WriteProblem &p, int num_sms, cudaStream_t stream)
{
    (void)num_sms;
    const long long per =
        (long long)((p.q ? p.Hq : 0) + 2 * p.cache.heads) * (p.cache.dim / 16);
    const long long grid = (p.T * per + kWriteThreads - 1) / kWriteThreads;
    return launch_step(write_kernel, dim3((unsigned)grid), kWriteThreads, 0, 1, stream, p);
}

} // namespace sgq
