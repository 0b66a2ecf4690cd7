// echo_paged.cuh -- what the calls over a paged latent cache share: where a
// token's cache row is, and which tokens a row sees.
#pragma once

#include <cuda_bf16.h>

#include "echo_common.cuh"
#include "echo_internal.h"

namespace echo {

constexpr int kLatDqk = ECHO_MLA_DQK;            // 576
constexpr int kLatDv = ECHO_MLA_DV;              // 512
constexpr int64_t kLatRowBytes = kLatDqk * 2;    // 1152

constexpr int64_t kMaxLen = ECHO_CHUNK_MAX_TOKENS;  // tile ends stay below 2^31

// The arguments of a chunk call that the kernels read (device pointers).
struct ChunkArgs {
    int B;
    int heads;
    int64_t n_rows;
    const int64_t* row_off;
    const int64_t* tok_off;
    const int64_t* tok_end;
    int64_t n_tokens;
    const int32_t* page_tab;
    const uint8_t* kv;
    int64_t kv_rows;
    int64_t req_rows;
    uint32_t page;
    const int32_t* sel;
    int k;
    int64_t window;
    int64_t sinks;
    const uint32_t* mask;  // [n_rows, words] the tree nodes each row sees (echo_mla_tree), null: no trees
    int words;
    const uint16_t* q;
    float scale;
    uint64_t wait_ns;  // limit of the kernels' waits, from the last progress
    int32_t* status;
};

// Host checks of the arguments the chunk calls share.
inline int check_chunk(int B, const int64_t* row_off, int64_t n_rows, int heads, const uint16_t* q,
                       const int64_t* tok_off, int64_t n_tokens, const echo_pages* pg, int64_t window, int64_t sinks,
                       float scale, const int32_t* status) {
    if (B <= 0 || n_rows < 0 || heads <= 0 || n_tokens < 0 || window < 0 || sinks < 0) return ECHO_EINVAL;
    if (B > ECHO_MAX_REQUESTS || heads > ECHO_MLA_HEADS || n_rows > ECHO_CHUNK_MAX_ROWS) return ECHO_EUNSUPPORTED;
    if (!row_off || (n_rows > 0 && !q) || !tok_off || !pg || !status) return ECHO_EINVAL;
    if ((n_tokens > 0 && !pg->page_tab) || !pg->kv || pg->page < 1 || pg->kv_rows <= 0 || pg->req_rows < 0) return ECHO_EINVAL;
    if (pg->req_rows > pg->kv_rows / B) return ECHO_EINVAL;
    if (!(scale > 0.f) || scale > 3.4028234e38f) return ECHO_EINVAL;
    if (!is_aligned(q, 16) || !is_aligned(pg->kv, 16)) return ECHO_EINVAL;
    return ECHO_OK;
}

inline ChunkArgs chunk_args(int B, const int64_t* row_off, int64_t n_rows, int heads, const uint16_t* q,
                            const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens, const echo_pages* pg,
                            const int32_t* sel, int k, int64_t window, int64_t sinks, float scale, int32_t* status) {
    ChunkArgs a;
    a.B = B;
    a.heads = heads;
    a.n_rows = n_rows;
    a.row_off = row_off;
    a.tok_off = tok_off;
    a.tok_end = tok_end;
    a.n_tokens = n_tokens;
    a.page_tab = pg->page_tab;
    a.kv = static_cast<const uint8_t*>(pg->kv);
    a.kv_rows = pg->kv_rows;
    a.req_rows = pg->req_rows;
    a.page = static_cast<uint32_t>(pg->page);
    a.sel = sel;
    a.k = sel ? k : 0;
    a.window = window < kMaxLen ? window : kMaxLen;  // no context is longer: positions + window stay in 64 bits
    a.sinks = sinks;
    a.mask = nullptr;
    a.words = 0;
    a.q = q;
    a.scale = scale;
    a.wait_ns = wait_limit_ns();
    a.status = status;
    return a;
}

// Rows [r0, r0 + n) of request b, its token rows from off on and its length.
// False: the row bounds are inconsistent (n = 0).  Inconsistent token bounds,
// more rows than tokens or than the masks of trees have bits, or more than kMaxLen
// tokens leave len = 0.
__device__ __forceinline__ bool chunk_request(const ChunkArgs& a, int b, int64_t* r0, int64_t* n, int64_t* off,
                                              int64_t* len) {
    const int64_t lo = a.row_off[b], hi = a.row_off[b + 1];
    int64_t t0, t1;
    bool ok = seg_bounds(a.tok_off, a.tok_end, a.n_tokens, b, &t0, &t1);
    *off = t0;
    *len = t1 - t0;
    *r0 = lo;
    *n = hi - lo;
    if (lo < 0 || hi < lo || hi > a.n_rows) {
        *r0 = 0;
        *n = 0;
        set_status(a.status, ECHO_ST_BADDATA);
        return false;
    }
    if (hi > lo && (!ok || *len < *n || *len > kMaxLen || (a.mask && *n > 32ll * a.words))) {
        set_status(a.status, ECHO_ST_BADDATA);
        *len = 0;
    }
    return true;
}

// Where a request's tokens are: its pool's first row and the page position of its token 0.
struct PageView {
    const int32_t* tab;    // the table entry that holds token 0
    uint32_t shift;        // token 0's offset in its page
    int64_t base;          // first row of the request's pool
    int64_t rows;          // rows of the pool
};

__device__ __forceinline__ PageView page_view(const ChunkArgs& a, int b, int64_t off) {
    PageView v;
    const int64_t e = off < (1ll << 31) ? static_cast<uint32_t>(off) / a.page : off / a.page;
    v.tab = a.page_tab + e;
    v.shift = static_cast<uint32_t>(off - e * a.page);
    v.base = a.req_rows ? b * a.req_rows : 0;
    v.rows = a.req_rows ? a.req_rows : a.kv_rows;
    return v;
}

// Table entry (from v.tab on) that holds token t (t < 2^31), and the token's offset in its page.
__device__ __forceinline__ uint32_t page_of(const ChunkArgs& a, const PageView& v, uint32_t t, uint32_t* at) {
    uint32_t e;
    if (a.page == 1) {
        e = t;
        *at = 0;
        return e;
    }
    const uint64_t x = static_cast<uint64_t>(v.shift) + t;  // below 2^32: both are below 2^31
    e = static_cast<uint32_t>(x) / a.page;
    *at = static_cast<uint32_t>(x) - e * a.page;
    return e;
}

// Cache row `at` of the page a table entry p >= 0 names, -1 (and *bad) when that leaves the pool.
__device__ __forceinline__ int64_t page_row(const ChunkArgs& a, const PageView& v, int32_t p, uint32_t at, bool* bad) {
    const int64_t row = static_cast<int64_t>(p) * a.page + at;
    if (row >= v.rows) {
        *bad = true;
        return -1;
    }
    return v.base + row;
}

// Cache row of token t, -1 when it has none.
__device__ __forceinline__ int64_t token_row(const ChunkArgs& a, const PageView& v, uint32_t t, bool* bad) {
    uint32_t at;
    const int32_t p = v.tab[page_of(a, v, t, &at)];
    return p < 0 ? -1 : page_row(a, v, p, at, bad);
}

// ---------------------------------------------------------------- shares of a row of units
// `parts` shares of `total` units (total >= parts): share i is units
// [share_start(i), share_start(i + 1)).
__device__ __forceinline__ int64_t share_start(int64_t total, int parts, int i) {
    if (total < (1 << 24))  // parts is at most 128: a 32-bit division does
        return static_cast<uint32_t>(total) * static_cast<uint32_t>(i) / static_cast<uint32_t>(parts);
    return total * i / parts;
}

// The share that holds unit u.
__device__ __forceinline__ int share_of(int64_t total, int parts, int64_t u) {
    int i = static_cast<int>(min(static_cast<int64_t>(parts) - 1, u * parts / total));
    while (i + 1 < parts && share_start(total, parts, i + 1) <= u) ++i;
    while (share_start(total, parts, i) > u) --i;
    return i;
}

// The last of n things whose units start at or before u (cum ascending, cum[0] <= u; a warp together).
__device__ __forceinline__ int find_group(const int64_t* cum, int n, int64_t u) {
    const int lane = threadIdx.x & 31;
    int lo = 0;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool le = lane * step < n && cum[lo + lane * step] <= u;
        const int k = __popc(__ballot_sync(0xffffffffu, le));  // le is true for a prefix of the lanes
        const int end = lo + n;
        lo += (k - 1) * step;
        n = min(step, end - lo);
    }
    return lo;
}

// Exclusive prefix sum of a block of NT threads, and its total, in 64 bits.  scratch: [NT / 32].
template <int NT>
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t* scratch, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int64_t w = lane < NT / 32 ? scratch[lane] : 0;  // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    __syncthreads();
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + x - v;
}

// Sets a two-CTA cluster kernel up for `smem` bytes; how many of its clusters the device holds at
// once, at most `most` (queried once per device: `cached`, zeros at first), 0 on an error.
template <class Kernel>
int cluster2_count(Kernel kernel, int threads, uint32_t smem, int most, int (&cached)[64]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return 0;
    if (cached[dev] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            n = sm_count() / 2;
        }
        cached[dev] = n < 1 ? 1 : n > most ? most : n;
    }
    return cached[dev];
}

// Launch, as a programmatic dependent of the kernel before it on the stream unless `plain` (for
// kernels that let dependents start early; a kernel of another call may not).
template <class... Args>
cudaError_t launch_after(bool plain, void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = plain ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace echo
