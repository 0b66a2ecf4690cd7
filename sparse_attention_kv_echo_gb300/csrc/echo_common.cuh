// echo_common.cuh -- device helpers shared by the libecho kernels (sm_103a).
//
// Thin inline-PTX wrappers for mbarrier, TMA (cp.async.bulk.tensor), the 5th
// generation tensor core (tcgen05: TMEM allocation, MMA, commit, TMEM loads),
// bounded waits, order-preserving float keys and block-wide scans.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "echo.h"
#include "echo_internal.h"

namespace echo {

// Any wait inside a kernel gives up after this long and reports ECHO_ST_TIMEOUT.
constexpr uint64_t kWaitNs = kWaitLimitNs;

__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Request b's tokens [lo, hi): rows lo.. of every per-token array.  The
// request's region is [tok_off[b], tok_off[b+1]); tok_end (optional) holds its
// current end (a context that grows inside its region), else the region is
// full.  False, with an empty range at 0, when inconsistent with n_tokens.
__device__ __forceinline__ bool seg_bounds(const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens, int b,
                                           int64_t* lo, int64_t* hi) {
    const int64_t l = tok_off[b], r = tok_off[b + 1];
    const int64_t h = tok_end ? tok_end[b] : r;
    if (l < 0 || r < l || r > n_tokens || h < l || h > r) {
        *lo = 0;
        *hi = 0;
        return false;
    }
    *lo = l;
    *hi = h;
    return true;
}

__device__ __forceinline__ void set_status(int32_t* status, int bits) {
    if (status) atomicOr(reinterpret_cast<int*>(status), bits);
}

// ---------------------------------------------------------------- ordering
// Unsigned key with the order of the float; -0 first becomes +0.
__device__ __forceinline__ uint32_t order_key(float x) {
    x = __fadd_rn(x, 0.0f);  // -0 + +0 = +0 under round-to-nearest
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_to_float(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// 256-bin index of a score shifted by the predicted threshold.
__device__ __forceinline__ uint32_t shifted_bin(float score, float shift) {
    return order_key(__fsub_rn(__fadd_rn(score, 0.0f), shift)) >> 24;
}

// ---------------------------------------------------------------- mbarrier
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// try_wait that may suspend the thread for up to hint_ns (it wakes as soon as
// the phase completes), so waiting warps take neither issue slots nor
// mbarrier bandwidth from the warps that do the work.
__device__ __forceinline__ bool mbar_try_wait_sleep(uint32_t bar, uint32_t parity, uint32_t hint_ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(hint_ns)
        : "memory");
    return ok != 0;
}

// Wait for the phase of the given parity.  Returns false when *abort becomes
// non-zero (abort may be NULL) or after limit_ns (0: unless the phase is
// complete at the first look).
__device__ __forceinline__ bool mbar_wait_limit(uint32_t bar, uint32_t parity, const volatile int* abort,
                                                uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    if (limit_ns == 0) return false;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
        if (abort && *abort) return false;
        if (global_ns() - t0 > limit_ns) return false;
    }
}

// The same with the library's limit, kWaitNs.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const volatile int* abort) {
    return mbar_wait_limit(bar, parity, abort, kWaitNs);
}

// What the waits of a CTA watch whose work may go on for longer than any fixed limit: abort
// ends them, and the limit runs from the last move of beat, which the warps that do the work
// move (a warp that stores the result of a long piece, or loads what follows it, waits for
// as long as the piece takes).  In shared memory.
struct Watch {
    uint64_t limit_ns;
    int abort;
    uint32_t beat;
};

__device__ __forceinline__ void watch_init(Watch* w, uint64_t limit_ns) {
    w->limit_ns = limit_ns;
    w->abort = 0;
    w->beat = 0;
}

__device__ __forceinline__ void give_up(Watch* w) { static_cast<volatile Watch*>(w)->abort = 1; }
__device__ __forceinline__ bool gave_up(const Watch* w) { return static_cast<const volatile Watch*>(w)->abort != 0; }
__device__ __forceinline__ void watch_beat(Watch* w) { atomicAdd(&w->beat, 1u); }

// Whether a wait that began or last saw a beat at *t0, with *seen beats, goes on.
__device__ __forceinline__ bool watch_goes_on(const Watch* w, uint32_t* seen, uint64_t* t0) {
    const volatile Watch* const v = w;
    if (v->abort) return false;
    const uint32_t beat = v->beat;
    const uint64_t now = global_ns();
    if (beat != *seen) {
        *seen = beat;
        *t0 = now;
    }
    return now - *t0 <= v->limit_ns;
}

// mbar_wait under a watch.
__device__ __forceinline__ bool mbar_wait_watch(uint32_t bar, uint32_t parity, const Watch* w) {
    if (mbar_try_wait(bar, parity)) return true;
    uint32_t seen = static_cast<const volatile Watch*>(w)->beat;
    uint64_t t0 = global_ns();
    do {
        if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    } while (watch_goes_on(w, &seen, &t0));
    return false;
}

// ---------------------------------------------------------------- TMA
__device__ __forceinline__ void prefetch_tmap(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// 2-D tiled load of a box into shared memory; completion is signalled on bar
// as transaction bytes.  x is the innermost coordinate (elements).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t x,
                                            int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

// Same, with an L2 eviction-priority policy (createpolicy).
__device__ __forceinline__ void tma_load_2d_hint(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t x,
                                                 int32_t y, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

// 1-D tiled load of a box into shared memory (x: first element; x * element
// size must be a multiple of 16 bytes), with an L2 eviction-priority policy.
__device__ __forceinline__ void tma_load_1d_hint(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t x,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.1d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3}], [%2], %4;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "l"(policy)
        : "memory");
}

__device__ __forceinline__ uint64_t policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ uint64_t policy_evict_last() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// 4-byte asynchronous copy global -> shared; src_bytes 0 writes zeros without reading.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
                 "r"(src_bytes)
                 : "memory");
}

// The barrier's current phase also waits for this thread's cp.async copies
// (no change to its expected arrival count).
__device__ __forceinline__ void cp_async_mbar_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// ---------------------------------------------------------------- programmatic dependent launch
// Wait until the grid this one depends on has completed and its writes are
// visible (a no-op for a normal launch).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Let the next grid of the stream start its prologue now.
__device__ __forceinline__ void pdl_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A[smem desc] x B[smem desc]^T, kind::f8f6f4, one CTA.
__device__ __forceinline__ void mma_f8f6f4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive once on bar when every tcgen05 operation issued so far by this thread completes.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns; thread i of the warp gets lane (base lane + i).
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor for a K-major operand stored with the
// 128-byte swizzle (rows of 128 bytes, 8-row groups 1024 bytes apart), as
// written by TMA with CU_TENSOR_MAP_SWIZZLE_128B.  The tile must start on a
// 1024-byte boundary.  Fields: start address >> 4 [0,14), leading byte
// offset >> 4 [16,30) (unused for this layout), stride byte offset >> 4
// [32,46), descriptor version 1 [46,48), base offset 0 [49,52), swizzle mode
// 2 = 128B [61,64).
__device__ __forceinline__ uint64_t sw128_kmajor_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

// Instruction descriptor of kind::f8f6f4 with E4M3 A and B (both K-major),
// fp32 accumulator, shape M x N: D format [4,6) = 1 (f32), A/B format
// [7,10) [10,13) = 0 (E4M3), N >> 3 at [17,23), M >> 4 at [24,29).
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// ---------------------------------------------------------------- block scans
// Exclusive prefix sum over a block of NT threads (NT a multiple of 32, <= 1024).
// scratch: >= NT/32 + 1 uint32 in shared memory.  Returns the exclusive prefix
// and writes the block total to *total (every thread).
template <int NT>
__device__ __forceinline__ uint32_t block_exclusive_scan(uint32_t v, uint32_t* scratch, uint32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        uint32_t w = (lane < NT / 32) ? scratch[lane] : 0u;
        uint32_t s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane < NT / 32) scratch[lane] = s - w;
        if (lane == 31) scratch[NT / 32] = s;
    }
    __syncthreads();
    const uint32_t out = scratch[warp] + x - v;
    *total = scratch[NT / 32];
    __syncthreads();
    return out;
}

}  // namespace echo
