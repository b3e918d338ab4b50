// What the gated delta rule's tcgen05 kernels share: warp-uniform issue, splitting of fp32 operands in bf16
// parts, set-up and tear-down of barriers and TMEM.
#pragma once

#include <type_traits>

#include "ssd_delta.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace tc {

constexpr int kC = kDeltaChunk;
constexpr int kPanel = kC * 128;  // bytes of 64 rows of 64 bf16

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// The products are issued by one elected thread, but from code that the whole warp runs: descriptors and
// TMEM addresses then stay in uniform registers. From inside `if (lane == 0)` each product took about 90
// cycles to issue, most of them moving its operands into uniform registers.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r;
}
template <bool kAcc>
__device__ __forceinline__ void mma_el(uint32_t leader, uint32_t d, uint32_t left, uint64_t right, uint32_t id) {
    if constexpr (kAcc)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 p, 0, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(left), "l"(right), "r"(id), "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.ne.b32 p, 0, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(left), "l"(right), "r"(id), "r"(leader)
            : "memory");
}
__device__ __forceinline__ void mma_ss_el(uint32_t leader, uint32_t d, uint64_t left, uint64_t right, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(left), "l"(right), "r"(id), "r"(leader), "r"(acc)
        : "memory");
}
// The same for one head of a pair: its 64 accumulator lanes (head 0: lanes 0-63) are written, the others stay as they
// are, so that nothing of one head's operands, not even 0 x inf, enters the other's rows.
template <bool kAcc>
__device__ __forceinline__ void mma_half_el(uint32_t leader, int head, uint32_t d, uint32_t left, uint64_t right, uint32_t id) {
    const uint32_t off0 = head ? 0xffffffffu : 0u;  // lanes 0-63 not written
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.ne.b32 p, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %6, %6}, p;\n\t}" ::"r"(d),
        "r"(left), "l"(right), "r"(id), "r"(leader), "r"(off0), "r"(~off0), "n"(kAcc ? 1 : 0)
        : "memory");
}
__device__ __forceinline__ void mma_ss_half_el(uint32_t leader, int head, uint32_t d, uint64_t left, uint64_t right, uint32_t id,
                                               uint32_t acc) {
    const uint32_t off0 = head ? 0xffffffffu : 0u;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%6, %6, %7, %7}, p;\n\t}" ::"r"(d),
        "l"(left), "l"(right), "r"(id), "r"(leader), "r"(acc), "r"(off0), "r"(~off0)
        : "memory");
}
__device__ __forceinline__ void commit_el(uint32_t leader, uint64_t *bar) {
    if (leader) mma_commit(bar);
    __syncwarp();
}

// hi + lo parts of a pair of fp32 values (lo: what hi leaves, rounded: 2^-18 of the value at worst)
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    asm("{\n\t.reg .b64 v, h, m;\n\t.reg .f32 a, b;\n\t"
        "mov.b64 v, {%1, %2};\n\tmov.b64 h, {%3, %4};\n\tmov.b64 m, {%5, %5};\n\t"
        "fma.rn.f32x2 v, h, m, v;\n\tmov.b64 {a, b}, v;\n\tcvt.rn.bf16x2.f32 %0, b, a;\n\t}"
        : "=r"(lo)
        : "f"(x), "f"(y), "f"(bf16_lo(hi)), "f"(bf16_hi(hi)), "f"(-1.f));
}
__device__ __forceinline__ float2 pair_of(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }

// What a kernel begins with: barriers (count of arrivals each), TMEM, the abort flag.
struct Setup {
    uint32_t tmem;
    volatile int *abort_flag;
};
template <int M>
__device__ __forceinline__ Setup set_up(uint64_t *bar, const int (&counts)[M], int wait_us, int warp) {
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + M);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bar + M + 1);
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < M; ++i) mbar_init(bar + i, counts[i]);
        abort_flag[0] = 0;
        abort_flag[1] = wait_us;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return Setup{*tmem_slot, abort_flag};
}
// And ends with: every issued product has completed (fin) before TMEM is released.
__device__ __forceinline__ void tear_down(uint32_t tmem, uint64_t *fin, int warp, int lane) {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if (lane == 0) {
            const unsigned long long t0 = now_ns();
            while (!mbar_try(fin, 0) && now_ns() - t0 < kWaitNs) {
            }
        }
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}
// Loads in flight land before the CTA exits: the last two uses of the stages' barriers.
__device__ __forceinline__ void drain_loads(uint64_t *full, int it) {
    for (int i = 1; i <= 2; ++i) {
        if (it - i < 0) continue;
        const unsigned long long w0 = now_ns();
        while (!mbar_try(&full[(it - i) & 1], (uint32_t)((it - i) >> 1) & 1u) && now_ns() - w0 < kWaitNs) {
        }
    }
}

// tcgen05.wait::ld with 16 registers of an earlier load as operands: no use of them moves above it.
#define SSD_W4(i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3])
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : SSD_W4(0), SSD_W4(4), SSD_W4(8), SSD_W4(12)::"memory");
}
#undef SSD_W4

}  // namespace tc
}  // namespace ssd
