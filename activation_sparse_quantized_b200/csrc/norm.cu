// norm.cu -- sgq_residual_norm: the norms before and after a block, fused with
// its gate and its scaled addition to the residual.
//
//   u  = a                                             (no w_post)
//   u  = a * rsqrt(mean(a^2) + eps) * (w_offset + w_post)
//   r' = resid + scale * gate * u
//   x  = bf16(r' * rsqrt(mean(r'^2) + eps) * (w_offset + w_pre))
//
// One CTA per row; a row is read once, stays in registers as fp32 through both
// sums of squares, and r' and x are each rounded once. x is formed from the
// unrounded r', whatever resid's type.
#include "sgq_device.cuh"
#include "sgq_launch.h"
#include "step_launch.cuh"

namespace sgq {

namespace {

// Eight consecutive elements as loaded (16 or 32 bytes), and as fp32.
template <int TYPE>
struct Raw {
    static constexpr int kWords = TYPE == SGQ_TYPE_F32 ? 2 : 1;
    uint4 w[kWords];
};

template <int TYPE>
__device__ __forceinline__ Raw<TYPE> load8(const void *base, long long elem)
{
    Raw<TYPE> r;
    const uint4 *p = reinterpret_cast<const uint4 *>(
        static_cast<const char *>(base) + elem * (TYPE == SGQ_TYPE_F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < Raw<TYPE>::kWords; ++i)
        r.w[i] = p[i];
    return r;
}

template <int TYPE>
__device__ __forceinline__ void unpack8(const Raw<TYPE> &r, float *f)
{
    if constexpr (TYPE == SGQ_TYPE_F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i + 0] = __uint_as_float(r.w[i].x);
            f[4 * i + 1] = __uint_as_float(r.w[i].y);
            f[4 * i + 2] = __uint_as_float(r.w[i].z);
            f[4 * i + 3] = __uint_as_float(r.w[i].w);
        }
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)float_to_bf16_bits(f[2 * i]) |
               ((uint32_t)float_to_bf16_bits(f[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum of v over the CTA, the same in every thread. part: one float per warp,
// not used by any earlier sum of the row.
__device__ __forceinline__ float block_sum(float v, float *part)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (int)(threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    return v;
}

template <int AT, int RT, int WT, int K>
__global__ void __launch_bounds__(1024) norm_kernel(const NormProblem p)
{
    __shared__ float part[2][32];
    const int row = blockIdx.x, nt = blockDim.x;
    grid_launch_dependents();
    grid_dependency_wait(); // a and resid come from the previous kernels

    float v[K][8];
    Raw<RT> rr[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * (threadIdx.x + k * nt);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[k][i] = 0.0f;
        if (c < p.H) {
            rr[k] = load8<RT>(p.resid, row * p.ld_r + c);
            // the gate is read after the first sum only; its trip from memory
            // starts here (8191 rows of 5120: 75.7 us against 79.6)
            if (p.gate && p.w_post)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(
                    static_cast<const char *>(p.gate) +
                    (row * p.ld_gate + c) * (WT == SGQ_TYPE_F32 ? 4 : 2)));
            if (p.a)
                unpack8<AT>(load8<AT>(p.a, row * p.ld_a + c), v[k]);
        }
    }
    float mul = p.scale;
    if (p.w_post) {
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss = fmaf(v[k][i], v[k][i], ss);
        mul *= rsqrtf(block_sum(ss, part[0]) / p.H + p.eps);
    }
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * (threadIdx.x + k * nt);
        if (c < p.H) {
            float w[8], r[8];
            if (p.w_post) {
                unpack8<WT>(load8<WT>(p.w_post, c), w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[k][i] *= p.w_offset + w[i];
            }
            if (p.gate) {
                unpack8<WT>(load8<WT>(p.gate, row * p.ld_gate + c), w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[k][i] *= w[i];
            }
            unpack8<RT>(rr[k], r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[k][i] = p.a ? fmaf(mul, v[k][i], r[i]) : r[i];
            if (p.resid_out) {
                if constexpr (RT == SGQ_TYPE_F32) {
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.resid_out) +
                                                           row * p.ld_ro + c);
                    o[0] = make_float4(v[k][0], v[k][1], v[k][2], v[k][3]);
                    o[1] = make_float4(v[k][4], v[k][5], v[k][6], v[k][7]);
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.resid_out) +
                                               row * p.ld_ro + c) = pack_bf16x8(v[k]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss = fmaf(v[k][i], v[k][i], ss);
        }
    }
    if (!p.x)
        return;
    const float inv = rsqrtf(block_sum(ss, part[1]) / p.H + p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * (threadIdx.x + k * nt);
        if (c < p.H) {
            float w[8];
            unpack8<WT>(load8<WT>(p.w_pre, c), w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[k][i] *= inv * (p.w_offset + w[i]);
            *reinterpret_cast<uint4 *>(p.x + row * p.ld_x + c) = pack_bf16x8(v[k]);
        }
    }
}

template <int AT, int RT, int WT>
cudaError_t launch_t(const NormProblem &p, cudaStream_t stream)
{
    const int chunks = p.H / 8;
    const int k = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
    const int block = ((chunks + k - 1) / k + 31) / 32 * 32;
    switch (k) {
    case 1: return launch_step(norm_kernel<AT, RT, WT, 1>, dim3(p.B), block, 0, 1, stream, p);
    case 2: return launch_step(norm_kernel<AT, RT, WT, 2>, dim3(p.B), block, 0, 1, stream, p);
    default: return launch_step(norm_kernel<AT, RT, WT, 4>, dim3(p.B), block, 0, 1, stream, p);
    }
}

template <int AT, int RT>
cudaError_t launch_w(const NormProblem &p, cudaStream_t stream)
{
    return p.w_type == SGQ_TYPE_F32 ? launch_t<AT, RT, SGQ_TYPE_F32>(p, stream)
                                    : launch_t<AT, RT, SGQ_TYPE_BF16>(p, stream);
}

} // namespace

cudaError_t launch_norm(const NormProblem &p, int num_sms, cudaStream_t stream)
{
    (void)num_sms;
    const bool af = p.a_type == SGQ_TYPE_F32, rf = p.r_type == SGQ_TYPE_F32;
    if (af)
        return rf ? launch_w<SGQ_TYPE_F32, SGQ_TYPE_F32>(p, stream)
                  : launch_w<SGQ_TYPE_F32, SGQ_TYPE_BF16>(p, stream);
    return rf ? launch_w<SGQ_TYPE_BF16, SGQ_TYPE_F32>(p, stream)
              : launch_w<SGQ_TYPE_BF16, SGQ_TYPE_BF16>(p, stream);
}

} // namespace sgq
