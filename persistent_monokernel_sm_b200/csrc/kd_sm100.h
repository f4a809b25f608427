// kd_sm100.h -- inline-PTX helpers for the tcgen05 / TMA operators (kd_gemm.cu, kd_attention.cu):
// mbarriers with bounded waits, tensor-map loads, tensor-memory allocation and access, and the
// shared-memory and instruction descriptors of tcgen05.mma. Internal to libkd.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kd_layout.h"
#include "kd_ops.h"

namespace kd {

// Set by a wait that ran out of its limit, unless a handle's control words are (one word per source
// file that includes this); kd_op_sync reads and clears them.
static __device__ unsigned int g_op_status;

// What a CTA's waits go by: its give-up flag, their limit in SM clocks, and the control words of the
// handle that reports one which runs out (NULL: g_op_status does). The waits read the SM's own
// clock: a read of the global timer costs about as much as the wait it would guard.
struct Guard {
    volatile int* dead;
    OpWaits waits;
};
constexpr long long kSuspendClocks = 1 << 20;    // more than try_wait suspends a thread for
constexpr long long kDrainClocks = 200000000ll;  // of the wait for copies in flight: about 0.1 s

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
// One lane of a fully converged warp. The compiler knows of elect.sync that one lane runs what
// follows, and then feeds tcgen05 and TMA instructions from uniform registers directly.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xffffffff;\nselp.b32 %0, 1, 0, q;\n}" : "=r"(p));
    return p != 0;
}

// ---------------------------------------------------------------- mbarriers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// arrive on a barrier of any CTA of the cluster (address from map_rank)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.b32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// A look that does not wait (try_wait may suspend the thread for a while).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.b32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void raise_timeout(const Guard& w) {
    *w.dead = 1;
    if (!w.waits.ctl) atomicExch(&g_op_status, 1u);
    else if (atomicCAS(w.waits.ctl + kCtlStatus, 0ull, (unsigned long long)kStatusTimeout) == 0ull)
        atomicExch(w.waits.ctl + kCtlWhere, ((unsigned long long)kWhereOperator << 24) | (unsigned long long)((blockIdx.x & 0xffff) << 8));
}
// Waits until the phase of `parity` has completed. Gives up when the limit has passed or
// another wait of this CTA has given up (*dead), and then returns false: the caller unwinds.
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, const Guard& w) {
    const long long t0 = clock64();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try(bar, parity)) return true;
        if (*w.dead) return false;
        if (clock64() - t0 > w.waits.limit) {
            raise_timeout(w);
            return false;
        }
    }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const Guard& w) {
    if (mbar_try(bar, parity)) return true;
    return mbar_wait_long(bar, parity, w);
}
// Before a kernel's first wait: with a limit that is shorter than a thread may be suspended for, that wait
// without a suspension, so that the limit is kept.
__device__ __forceinline__ bool mbar_first(uint32_t bar, uint32_t parity, const Guard& w) {
    if (__builtin_expect(w.waits.limit >= kSuspendClocks, 1)) return true;
    const long long t0 = clock64();
    while (!mbar_test(bar, parity))
        if (clock64() - t0 > w.waits.limit) {
            raise_timeout(w);
            return false;
        }
    return true;
}
// The same by all lanes of a warp, with one answer.
__device__ __forceinline__ bool mbar_wait_all(uint32_t bar, uint32_t parity, const Guard& w) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, w)) != 0;
}
// Once a wait has given up and all threads have stopped: bounded waits that let what is under way land.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity))
        if (clock64() - t0 > kDrainClocks) return;
}
__device__ __forceinline__ void drain_pause() {
    const long long t0 = clock64();
    while (clock64() - t0 < kDrainClocks) {}
}

// Programmatic launches. grid_wait: until the kernels before this one on the stream have ended and
// their writes are visible; every CTA calls it before it touches global memory. grid_release: a
// following launch that waits likewise may be set up from now on.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Register shares of whole warpgroups (all four warps call one of them once).
template <int N>
__device__ __forceinline__ void set_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---------------------------------------------------------------- TMA loads
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
template <int CG = 1>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
            "[%4];" ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else  // the barrier may be the other CTA's of the pair
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
            "{%2, %3}], [%4];" ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// ---------------------------------------------------------------- tensor memory
template <int CG = 1>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {  // one whole warp (of either CTA of a pair)
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int CG = 1>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {  // the warp that allocated
    if constexpr (CG == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrives on `bar` when every tcgen05 operation this thread issued before has completed.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The same for a CTA pair: on the barrier at this offset in both CTAs.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// D (fp32, tensor memory) = A B^T (+ D): operands in shared memory.
template <int CG = 1>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((int)add)
            : "memory");
    else  // over the pair's shared memories: M 256, either CTA holds 128 rows of A and D and half of B
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((int)add)
            : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((int)add)
        : "memory");
}

// Instruction descriptor of kind::f16 with fp32 accumulators. bf16: operand type (else fp16);
// a_mn / b_mn: that operand is stored with its M or N dimension contiguous (else K).
__host__ __device__ inline uint32_t make_idesc(int m, int n, bool bf16, bool a_mn, bool b_mn) {
    uint32_t d = 1u << 4;
    if (bf16) d |= (1u << 7) | (1u << 10);
    if (a_mn) d |= 1u << 15;
    if (b_mn) d |= 1u << 16;
    d |= (uint32_t)(n >> 3) << 17;
    d |= (uint32_t)(m >> 4) << 24;
    return d;
}
// Shared-memory descriptor of an operand tile in the 128-byte swizzled layout that TMA writes:
// atoms of 8 rows of 128 bytes. K-contiguous: sbo is the distance of 8-row groups (1024 here).
// M/N-contiguous: a row is 64 elements of one k; sbo is the distance of groups of 8 k's, lbo
// that of the next 64 elements.
__device__ __forceinline__ uint64_t make_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)((lbo >> 4) & 0x3fff) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3fff) << 32) | (1ull << 46) | (2ull << 61);
}

#define KD_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define KD_I8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
// This warp's 32 lanes, 16 or 32 consecutive columns: register j = column j.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : KD_R8(r, 0), KD_R8(r, 8)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : KD_R8(r, 0), KD_R8(r, 8), KD_R8(r, 16), KD_R8(r, 24)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::KD_I8(r, 0),
        KD_I8(r, 8), KD_I8(r, 16), KD_I8(r, 24), "r"(addr)
        : "memory");
}

// ---------------------------------------------------------------- 16-bit types
template <typename T> struct Half2;
template <> struct Half2<__nv_bfloat16> {
    static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ void unpack(uint32_t v, float& lo, float& hi) {
        lo = __uint_as_float(v << 16);
        hi = __uint_as_float(v & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&p);
    }
};
template <> struct Half2<__half> {
    static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ void unpack(uint32_t v, float& lo, float& hi) {
        const float2 f = __half22float2(*reinterpret_cast<__half2*>(&v));
        lo = f.x, hi = f.y;
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        __half2 p = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&p);
    }
};

// ---------------------------------------------------------------- host side (kd_gemm.cu)
// Tensor map of a row-major 2-D (rows x cols, ld elements between rows) or 3-D array of 16-bit
// elements with 128-byte swizzled boxes. Returns a KD_* code; the text goes to kd_op_error.
int make_map_2d(CUtensorMap* m, int dtype, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_cols,
                int box_rows);
int make_map_3d(CUtensorMap* m, int dtype, const void* base, int64_t c0, int64_t c1, int64_t c2, int64_t ld1,
                int64_t ld2, int box0, int box1, int box2);
int op_fail(int code, const char* fmt, ...);
int op_sm_count(int* sms);  // of the current device; KD_ECUDA without one

}  // namespace kd
