// tc_device.cuh -- barriers, copies and tensor-core instructions (mbarrier,
// cp.async, tcgen05) of the attention kernel.
#pragma once

#include "sgq_device.cuh"

#include <cuda.h>

namespace sgq {

namespace {

constexpr unsigned long long kBarWaitNs = 200000000ull; // a barrier wait gives up after 0.2 s
constexpr unsigned kBarSuspendNs = 20000;

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// This thread's arrival, and `bytes` more to come from bulk copies.
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// Box (x, y, z, w) of a tensor map into shared memory, counted on bar; by one
// thread of the calling warp (lead != 0).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, uint32_t bar, uint32_t lead)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %7, 0;\n\t"
                 "@q cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "r"(lead)
                 : "memory");
}

// One lane of a warp that is together: 1 there, 0 in the others.
__device__ __forceinline__ uint32_t elect_lane()
{
    uint32_t lead;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(lead));
    return lead;
}

// 16 bytes into shared memory, or zeros.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool take)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(take ? 16 : 0)
                 : "memory");
}

// This thread's arrival, once its cp.async so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Waits for the phase of the given parity to complete, for at most `limit` of
// wall time. A thread whose wait gave up has ok = false and waits no more, so
// that a broken hand-off ends the kernel within a fraction of a second.
__device__ __forceinline__ void bar_wait(uint32_t bar, uint32_t parity, bool &ok,
                                         unsigned long long limit = kBarWaitNs)
{
    unsigned long long t0 = 0;
    while (ok) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done)
                     : "r"(bar), "r"(parity), "n"(kBarSuspendNs)
                     : "memory");
        if (done)
            return;
        unsigned long long t;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t0 == 0)
            t0 = t;
        else if (t - t0 > limit)
            ok = false;
    }
}

// Whether the phase of the given parity has completed.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done;
}

// This thread's shared-memory writes, (and those it has waited for) made visible
// to the tensor core's reads.
__device__ __forceinline__ void fence_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Descriptor of a swizzled operand in shared memory (sm_100 form); layout 2:
// 128-byte swizzle, 4: 64-byte. K-major: sbo = stride of 8-row groups. MN-major:
// lbo = stride of swizzle-wide blocks along M or N, sbo = of 8-row groups along K.
__device__ __forceinline__ uint64_t op_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout = 2)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)layout << 61);
}

// Instruction descriptor of tcgen05.mma kind::f16 with fp32 sums, M = 128
// (fp16 operands' code is also kind::f8f6f4's for e4m3).
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, bool b_mn_major, int n)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// A descriptor as its two halves: steps inside an operand change the low one
// alone, and stay 32-bit adds.
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ explicit Desc(uint64_t d) : lo((uint32_t)d), hi((uint32_t)(d >> 32)) {}
};

// The products of one thread of the calling warp (lead != 0), which is one
// predicate: the warp stays together and keeps the operands in its uniform
// registers. A branch around the instruction made each product cost some 50 ns.
__device__ __forceinline__ void mma_ss(uint32_t d, Desc a, uint32_t astep, Desc b, uint32_t bstep,
                                       uint32_t idesc, uint32_t acc, uint32_t lead)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                 "setp.ne.b32 q, %7, 0;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
                 "r"(a.lo + astep), "r"(a.hi), "r"(b.lo + bstep), "r"(b.hi), "r"(idesc), "r"(acc), "r"(lead)
                 : "memory");
}

// The same on 8-bit operands (32 along K).
__device__ __forceinline__ void mma_ss_f8(uint32_t d, Desc a, uint32_t astep, Desc b, uint32_t bstep,
                                          uint32_t idesc, uint32_t acc, uint32_t lead)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                 "setp.ne.b32 q, %7, 0;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n\t}" ::"r"(d),
                 "r"(a.lo + astep), "r"(a.hi), "r"(b.lo + bstep), "r"(b.hi), "r"(idesc), "r"(acc), "r"(lead)
                 : "memory");
}

// A read from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, Desc b, uint32_t bstep, uint32_t idesc,
                                       uint32_t acc, uint32_t lead)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "setp.ne.b32 q, %6, 0;\n\tmov.b64 y, {%2, %3};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b.lo + bstep), "r"(b.hi), "r"(idesc), "r"(acc), "r"(lead)
                 : "memory");
}

// Every MMA the leading thread issued so far, complete, arrives once on bar.
__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t lead)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
                 "r"(lead)
                 : "memory");
}

#define SGQ_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define SGQ_RW8(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7])
#define SGQ_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// 32 consecutive 32-bit columns of this thread's tensor-memory lane; the
// values may be used after tmem_ld_wait on them.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                 "%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : SGQ_R8(r, 0), SGQ_R8(r, 8), SGQ_R8(r, 16), SGQ_R8(r, 24)
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_ld_wait(uint32_t *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : SGQ_RW8(r, 0), SGQ_RW8(r, 8), SGQ_RW8(r, 16), SGQ_RW8(r, 24)::"memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                 "%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
                 SGQ_I8(r, 0), SGQ_I8(r, 8), SGQ_I8(r, 16), SGQ_I8(r, 24)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                 "%12,%13,%14,%15}, [%16];"
                 : SGQ_R8(r, 0), SGQ_R8(r, 8)
                 : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" : SGQ_RW8(r, 0), SGQ_RW8(r, 8)::"memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                 "%12,%13,%14,%15,%16};" ::"r"(addr),
                 SGQ_I8(r, 0), SGQ_I8(r, 8)
                 : "memory");
}

__device__ __forceinline__ void tmem_st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

} // namespace

} // namespace sgq
