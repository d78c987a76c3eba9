// k3_tmem.cuh -- accumulator reads, asynchronous copies, the barriers of CTA pairs, and tensor-map making,
// shared by the operand product and the grouped products.
#pragma once
#include "k3_tcgen05.cuh"

namespace k3 {

// 16 or 32 columns of the accumulator, one row per lane.  The wait names the
// registers, so that nothing made from them can move above it.
K3_DEV void tmem_ld_chunk(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
K3_DEV void tmem_ld_chunk(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// 16 bytes from global to shared memory, asynchronously.
K3_DEV void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

K3_DEV uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
K3_DEV void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
K3_DEV uint32_t addr_of_rank(uint32_t addr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
// A tile of this CTA, its bytes counted on barrier `bar`, a shared::cluster address (the
// even CTA's).
K3_DEV void pair_load_2d(uint32_t dst, const CUtensorMap *map, int x, int row, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"((uint64_t)map), "r"(x), "r"(row), "r"(bar)
                 : "memory");
}
// Arrival at a pair's barrier in the even CTA (bar: there; full0: its shared::cluster
// address) behind what this thread, and after a warp barrier its warp, has written to its
// own CTA's shared memory and shown to the tensor core by the proxy fence.  The thread that
// issues the MMAs is in the even CTA, so the odd one's release has cluster scope; its fence
// covers the CTA's shared memory alone, which is all that is handed over (65536 rows x 1536
// x 7168 with 64 experts, gathered and in group order: 533 and 451 us; 528 and 448 with the
// CTA's scope, which gives no order between two CTAs; 1150 and 1025 with the arrive's own
// release at cluster scope, which waits for all memory).
K3_DEV void pair_arrive(uint32_t bar, uint32_t full0, int rank)
{
    if (rank)
        asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n\t"
                     "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(full0)
                     : "memory");
    else
        mbar_arrive(bar);
}
// The other side: a relaxed wait or test of the even CTA's barrier, then the acquire of what
// both CTAs' shared memory holds.
K3_DEV uint32_t mbar_try_wait_pair(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(20000u)
                 : "memory");
    return ok;
}
K3_DEV bool mbar_test_pair(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
K3_DEV bool tc_wait_pair(uint32_t bar, uint32_t parity, int *err, volatile int *abort_flag)
{
    return tc_wait_tile<mbar_try_wait_pair>(bar, parity, 0, err, abort_flag);
}
K3_DEV void pair_acquire() { asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory"); }
// Arrival at the barrier of the same offset in the pair's CTA `rank`, for a
// hand-over of tensor memory alone: the accumulator's loads are ordered by their
// wait and the tcgen05 fence before this, and no ordinary memory is handed over, so
// the arrival is relaxed (a release at cluster scope took 1200 clocks, on the path
// of the next tile's first MMA).
K3_DEV void mbar_arrive_rank(uint32_t bar, uint32_t rank)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr_of_rank(bar, rank)) : "memory");
}
// The waits for barriers that the other CTA's threads, copies or commits arrive
// at: cluster scope, bounded as mbar_wait.
K3_DEV uint32_t mbar_try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(20000u)
                 : "memory");
    return ok;
}
static __device__ __noinline__ bool mbar_wait_cluster_slow(uint32_t bar, uint32_t parity, int *err)
{
    const uint64_t t0 = global_ns();
    for (uint32_t n = 1;; n++) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((n & 63u) == 0 && global_ns() - t0 > kWaitLimitNs) {
            set_device_error(err, K3MOE_ETIMEOUT);
            return false;
        }
    }
}
K3_DEV bool tc_wait_cluster(uint32_t bar, uint32_t parity, int *err, volatile int *abort_flag)
{
    if (*abort_flag) return false;
    if (mbar_try_wait_cluster(bar, parity) || mbar_wait_cluster_slow(bar, parity, err)) return true;
    *abort_flag = 1;
    return false;
}
// Non-blocking: has the phase completed?
K3_DEV bool mbar_test_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
// Arrival at the barrier of this offset in both CTAs once everything issued
// before has completed.
K3_DEV void pair_commit(uint32_t bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
                 "%1;\n\t}" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            fn = nullptr;
        }
        return (PFN_cuTensorMapEncodeTiled_v12000)fn;
    }();
    return encode;
}
inline int encode_map(CUtensorMap *map, CUtensorMapDataType type, int nd, const void *p, const cuuint64_t *dims,
             const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle)
{
    const auto encode = map_encoder();
    if (!encode) return K3MOE_ECUDA;
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode(map, type, (cuuint32_t)nd, (void *)p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? K3MOE_OK
               : K3MOE_EINVAL;
}

}  // namespace k3
