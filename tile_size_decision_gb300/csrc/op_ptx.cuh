// Inline-PTX building blocks of the norm and product operators, beyond those
// of the GEMM: cluster launch control, distributed shared memory, register
// budgets, the 8-bit MMA, further tensor-memory loads, and asynchronous copies
// in groups.
#pragma once

#include "sm103_ptx.cuh"

namespace tiles {
namespace ptx {

// A 32-bit value from the shared memory of a CTA of the cluster.
__device__ __forceinline__ float ld_shared_cluster(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// Barrier `id` (1 .. 15) among `threads` threads of the block.
__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Arrive on an mbarrier given by its shared::cluster address without making
// this thread's earlier writes visible to the cluster, for arrivals that only hand back a buffer (a cluster-scope release
// costs a memory barrier of several hundred clocks).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Arrive with an expected transaction count on an mbarrier of the cluster.
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t cluster_addr,
                                                              uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(
                     cluster_addr), "r"(bytes)
                 : "memory");
}

// ---- cluster launch control ----------------------------------------------------

// Ask for a cluster of this grid that has not started yet: if there is one it
// is cancelled and its work is the caller's.  The 16-byte answer is written
// at `dst`, and 16 bytes are completed on `bar`, in every CTA of the cluster.
// One thread of the cluster asks, and not again after an answer without one.
__device__ __forceinline__ void try_cancel_cluster(void* dst, uint64_t* bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(smem_addr(dst)), "r"(smem_addr(bar))
        : "memory");
}

// The x index of the first CTA of the cluster an answer gives, or -1.
__device__ __forceinline__ int cancelled_cta_x(const void* answer) {
    int x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b64 lo, hi;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.v2.b64 {lo, hi}, [%1];\n\t"
        "mov.b128 r, {lo, hi};\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "mov.b32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n\t}"
        : "=r"(x)
        : "r"(smem_addr(answer))
        : "memory");
    return x;
}

// ---- register budgets ---------------------------------------------------------

// Executed by every warp of a warpgroup: give registers back, or take some
// of those given back, down or up to N a thread.
template <int N>
__device__ __forceinline__ void registers_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void registers_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// The instruction descriptor with either operand's order given (0 = K-major,
// 1 = MN-major), and that of kind::f8f6f4 with e4m3 operands (format 0, both
// K-major): the fields sit at the same bits.
__host__ __device__ constexpr uint32_t idesc_f16_f32acc_majors(bool bf16, bool a_mn, bool b_mn,
                                                               int m, int n) {
    return idesc_f16_f32acc(bf16, b_mn, m, n) | ((a_mn ? 1u : 0u) << 15);
}

__host__ __device__ constexpr uint32_t idesc_e4m3_f32acc(int m, int n) {
    return idesc_f16_f32acc(false, false, m, n);
}

// D[tmem] (+)= A[smem] x B[smem] with 8-bit operands (kind::f8f6f4, K = 32
// elements an instruction; otherwise as mma_f16).
template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// Warp-collective load of 16 consecutive fp32 columns of the warp's 32 TMEM
// lanes into r[first .. first + 15] (lane i receives row lane base + i).
template <int N>
__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[N], int first) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[first]), "=r"(r[first + 1]), "=r"(r[first + 2]), "=r"(r[first + 3]),
          "=r"(r[first + 4]), "=r"(r[first + 5]), "=r"(r[first + 6]), "=r"(r[first + 7]),
          "=r"(r[first + 8]), "=r"(r[first + 9]), "=r"(r[first + 10]), "=r"(r[first + 11]),
          "=r"(r[first + 12]), "=r"(r[first + 13]), "=r"(r[first + 14]), "=r"(r[first + 15])
        : "r"(taddr));
}

// Warp-collective load of 32 fp32 columns of 16 TMEM lanes in the matrix
// fragment layout: lane t gets, for each group i of 8 columns, row t/4,
// columns 8i + 2(t%4) and the next in r[4i], r[4i+1], and row t/4 + 8 of the
// same columns in r[4i+2], r[4i+3].
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Store four 8 x 8 matrices of 16-bit values transposed: lane t holds row
// t/4, columns 2(t%4) and the next of matrix i in r_i, and gives in `saddr`
// the address of row t%8 (16 bytes) of matrix t/8's transpose.
__device__ __forceinline__ void st_matrix_x4_trans(uint32_t saddr, uint32_t r0, uint32_t r1,
                                                   uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     saddr), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

// {d.x, d.y} += {a.x * b.x, a.y * b.y}, fused, in one instruction.
__device__ __forceinline__ void fma_pair(uint64_t& d, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

__device__ __forceinline__ uint64_t pack_pair(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}

__device__ __forceinline__ void unpack_pair(uint64_t v, uint32_t& lo, uint32_t& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}

// tmem_ld_wait, and no use of r moves ahead of it: the compiler does not know
// that a load's registers are filled only then, and copies of them made
// early (to pair them for fma_pair, say) double the instructions.
template <int N>
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[N]) {
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Between the generic proxy's accesses so far, seen from any CTA of the cluster,
// and the async proxy's that follow.
__device__ __forceinline__ void fence_proxy_async() {
    asm volatile("fence.proxy.async;" ::: "memory");
}

// An asynchronous global -> shared copy of 4 bytes.
__device__ __forceinline__ void cp_async_4(void* smem_dst, const void* gmem_src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(smem_dst)),
                 "l"(gmem_src)
                 : "memory");
}

// Close this thread's copies since the last call into a group, and wait
// until at most N of its groups are in flight.
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait_groups() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace ptx
}  // namespace tiles
