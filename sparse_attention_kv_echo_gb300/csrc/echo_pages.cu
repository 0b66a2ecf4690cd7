// echo_pages.cu -- the pages of a paged cache while requests come, branch, grow and go
// (echo.h, echo_page_pool): reserve, free, fork, compact and the rows of an accepted path.
//
// The table and the counts are small and every order in which pages are handed out is
// fixed, so one block plans (scans over requests, then over the counts) and names the rows
// to move in a list; a grid moves them through all layers.  What bounds the plans is
// latency, the moves the memory.  Each kernel's time below is that of one cold launch by itself.
#include <algorithm>

#include "echo_common.cuh"
#include "echo_paged.cuh"
#include "echo_tc.cuh"

namespace echo {
namespace {

struct PoolArgs {
    int32_t* tab;
    int32_t* refs;
    uint8_t* kv;
    int64_t n_pages;
    int64_t row_bytes;
    int64_t layer_bytes;
    int layers;
    int page;
    int64_t entries;  // of the table
    bool wide;        // refs on a 16-byte boundary
};

// Rows [src, src + rows) of every layer go to dst.
struct __align__(16) Move {
    int64_t src;
    int64_t dst;
    int64_t rows;
    int64_t reserved;
};

// The workspace: how many moves, the moves, and a list of pages.
struct Work {
    int32_t* moves;   // [1]
    Move* move;       // [requests of the call]
    int32_t* list;    // [n_pages]
    int32_t* map;     // [n_pages]
    int32_t* far;     // [n_pages]
    struct Tail* tail;  // [requests of the call]
};

// What a pair of a fork has behind the shared pages.
struct __align__(32) Tail {
    int64_t entry;    // dst's entry of the partly used page
    int64_t end;      // dst's end without its rows
    int32_t dst;      // -1: the pair is left out
    int32_t page;     // src's page of them, -1: none
    int32_t rows;
    int32_t reserved;
};

struct WorkLayout {
    size_t move, list, map, far, tail, total;
};
inline WorkLayout work_layout(int B, int64_t n_pages) {
    WorkLayout l;
    l.move = 256;
    l.list = round_up(l.move + static_cast<size_t>(B) * sizeof(Move), 256);
    l.map = round_up(l.list + static_cast<size_t>(n_pages) * 4, 256);
    l.far = round_up(l.map + static_cast<size_t>(n_pages) * 4, 256);
    l.tail = round_up(l.far + static_cast<size_t>(n_pages) * 4, 256);
    l.total = round_up(l.tail + static_cast<size_t>(B) * sizeof(Tail), 256);
    return l;
}
inline Work work_of(void* ws, int B, int64_t n_pages) {
    const WorkLayout l = work_layout(B, n_pages);
    uint8_t* const w = static_cast<uint8_t*>(ws);
    return Work{reinterpret_cast<int32_t*>(w), reinterpret_cast<Move*>(w + l.move), reinterpret_cast<int32_t*>(w + l.list),
                reinterpret_cast<int32_t*>(w + l.map), reinterpret_cast<int32_t*>(w + l.far),
                reinterpret_cast<Tail*>(w + l.tail)};
}

// x / d and x % d for an x >= 0, by a 32-bit division where that does (the 64-bit one takes some 100 instructions).
__device__ __forceinline__ int64_t quot(int64_t x, int d) { return x >> 32 ? x / d : static_cast<uint32_t>(x) / static_cast<uint32_t>(d); }
__device__ __forceinline__ int rest(int64_t x, int d) { return static_cast<int>(x - quot(x, d) * d); }

// Request b's token rows [off, end) of its region [off, last).  False: inconsistent, or not on a page's border.
struct Region {
    int64_t off, end, last;
};
__device__ __forceinline__ bool region_of(const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens, int page, int b, Region* r) {
    r->off = tok_off[b];
    r->last = tok_off[b + 1];
    r->end = tok_end[b];
    return r->off >= 0 && r->last >= r->off && r->last <= n_tokens && r->end >= r->off && r->end <= r->last && rest(r->off, page) == 0;
}
__device__ __forceinline__ int64_t pages_to(int64_t tok, int page) { return quot(tok + page - 1, page); }

__device__ __forceinline__ bool in_pool(const PoolArgs& a, int32_t p) { return p >= 0 && p < a.n_pages; }

// One entry less names page p.
__device__ __forceinline__ void drop_ref(const PoolArgs& a, int32_t p, int32_t* status) {
    if (!in_pool(a, p)) {
        set_status(status, ECHO_ST_BADDATA);
        return;
    }
    if (atomicSub(a.refs + p, 1) <= 0) {
        atomicAdd(a.refs + p, 1);
        set_status(status, ECHO_ST_BADDATA);
    }
}

// ---------------------------------------------------------------- moves
// Rows move 64 bytes a thread at a time, four 16-byte pieces in flight: a piece of NT * 64 bytes by a block of NT.
constexpr int kMT = 256;

template <int NT>
__device__ __forceinline__ void move_piece(const uint8_t* src, uint8_t* dst, int64_t bytes) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = (i * NT + threadIdx.x) * 16;
        if (at < bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(src + at));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = (i * NT + threadIdx.x) * 16;
        if (at < bytes) __stcs(reinterpret_cast<uint4*>(dst + at), v[i]);
    }
}

// The n listed moves, each of at most a page's rows, shared by `blocks` blocks along x and `rows` along the layers.
template <int NT>
__device__ __forceinline__ void move_all(const PoolArgs& a, const Move* move, uint32_t n, uint32_t block, uint32_t blocks, int row, int rows) {
    constexpr int kPiece = NT * 64;
    const uint32_t pieces = static_cast<uint32_t>((a.page * a.row_bytes + kPiece - 1) / kPiece);
    for (uint32_t u = block; u < n * pieces; u += blocks) {
        const Move m = move[u / pieces];
        const int64_t at = static_cast<int64_t>(u % pieces) * kPiece, bytes = m.rows * a.row_bytes - at;
        if (bytes <= 0) continue;
        for (int l = row; l < a.layers; l += rows) {
            uint8_t* const kv = a.kv + l * a.layer_bytes + at;
            move_piece<NT>(kv + m.src * a.row_bytes, kv + m.dst * a.row_bytes, bytes);
        }
    }
}

__global__ void __launch_bounds__(kMT) pages_move_kernel(PoolArgs a, Work w) {
    pdl_wait();
    move_all<kMT>(a, w.move, static_cast<uint32_t>(*w.moves), blockIdx.x, gridDim.x, blockIdx.y, gridDim.y);
}

// ---------------------------------------------------------------- free
// A thread an entry, the counts fall by atomics (sums, whose order does not show).  3.0 us for one request, 4 for 64.
constexpr int kFT = 256;

__global__ void __launch_bounds__(kFT)
    pages_free_kernel(PoolArgs a, const int64_t* __restrict__ tok_off, const int64_t* __restrict__ tok_end, int64_t n_tokens, int32_t* status) {
    Region r;
    if (!region_of(tok_off, tok_end, n_tokens, a.page, blockIdx.x, &r)) {
        if (threadIdx.x == 0 && blockIdx.y == 0) set_status(status, ECHO_ST_BADDATA);
        return;
    }
    const int64_t e1 = pages_to(r.last, a.page);
    for (int64_t e = pages_to(r.end, a.page) + static_cast<int64_t>(blockIdx.y) * kFT + threadIdx.x; e < e1; e += static_cast<int64_t>(gridDim.y) * kFT) {
        const int32_t p = a.tab[e];
        if (p == -1) continue;
        a.tab[e] = -1;
        drop_ref(a, p, status);
    }
}

// ---------------------------------------------------------------- the block that plans
constexpr int kPlanT = 1024;

constexpr int kRun = 4;   // (16 made the plans 2 to 4 us slower on pools of 3000 to 8500 pages: more code to fetch, fewer threads at work)
// The counts of kRun pages from p on (1 behind the last).
__device__ __forceinline__ void counts_of(const PoolArgs& a, int64_t p, int32_t (&r)[kRun]) {
    if (p + kRun <= a.n_pages && a.wide) {
#pragma unroll
        for (int i = 0; i < kRun / 4; ++i) *reinterpret_cast<int4*>(r + 4 * i) = reinterpret_cast<const int4*>(a.refs + p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i) r[i] = p + i < a.n_pages ? a.refs[p + i] : 1;
    }
}

// Lists the first `most` free pages, ascending; returns how many there are up to `most`.  A block together.
__device__ __forceinline__ int64_t list_free(const PoolArgs& a, int64_t most, int32_t* list, uint32_t* scratch) {
    int64_t found = 0;
    for (int64_t p0 = 0; p0 < a.n_pages && found < most; p0 += kRun * kPlanT) {
        const int64_t p = p0 + kRun * threadIdx.x;
        int32_t r[kRun];
        counts_of(a, p, r);
        uint32_t n = 0, total;
#pragma unroll
        for (int i = 0; i < kRun; ++i) n += r[i] == 0;
        int64_t at = found + block_exclusive_scan<kPlanT>(n, scratch, &total);
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if (r[i] == 0) {
                if (at < most) list[at] = static_cast<int32_t>(p + i);
                ++at;
            }
        found += total;
    }
    __syncthreads();
    return min(found, most);
}

// Whether entry e of a request that grows needs a page, and the page it has.
__device__ __forceinline__ bool needs_page(const PoolArgs& a, int64_t e, bool* bad, int32_t* page) {
    const int32_t p = a.tab[e];
    *page = p;
    if (p < 0) return true;
    if (!in_pool(a, p)) {
        *bad = true;
        return false;
    }
    const int32_t r = a.refs[p];
    *bad |= r < 1;  // named, but counted free
    return r > 1;
}

// A cluster: its first CTA plans, 1024 requests at a time, all of it copies what a copy on write has to, in one launch.  That suits
// calls that copy little or nothing: eight CTAs read and write some 0.4 TB/s (33 rows each of 64 requests' last pages: 20 us with one
// layer, 107 with eight, 750 with sixty, where a fork's or compact's moves have all SMs).  Forks copy their last rows
// themselves; what is left to copy here is a page that a request was cut back into while another holds it.  kWidth lanes look through a request's entries, eight when no request grows over more.  One request 6.9 us,
// 64 of 16 new rows 9.0, 24 of 4096 new rows on a pool of 3000 pages 11.6: a chain of loads (bounds, entries, counts, free
// pages), each behind the one before.
// The free pages are looked for from the first: behind 2^15 in use one page took 19 us with its release, behind 2^19 122, behind 2^23 1820.
constexpr int kReserveCtas = 8;

struct ReserveSmem {
    int64_t scratch64[kPlanT / 32];
    uint32_t scratch[kPlanT / 32 + 1];
    int64_t first[kPlanT];   // a request's entries that new tokens fall in: the first, how many, and rows in it already
    int32_t entries[kPlanT];
    int32_t part[kPlanT];
    int32_t need[kPlanT];    // pages it needs, -1: inconsistent; then where its pages begin, -1: none
    uint32_t mask[kPlanT];   // of its first 32 entries, those that need one
    int moves;
};

// Which of a request's entries [at, at + kWidth) need a page, a bit each in its lanes (of request i of the batch; -1: none).
template <int kWidth>
__device__ __forceinline__ uint32_t entries_in_need(const PoolArgs& a, const ReserveSmem& sm, int i, int at, int32_t* page, bool* bad) {
    const int lane = threadIdx.x & 31, sub = lane % kWidth;
    bool it = false;
    if (i >= 0 && at + sub < sm.entries[i]) {
        it = needs_page(a, sm.first[i] + at + sub, bad, page);
        if (it && *page < 0 && at + sub == 0 && sm.part[i] > 0) *bad = true;  // its rows are nowhere
    }
    return (__ballot_sync(0xffffffffu, it) >> (lane - sub)) & (kWidth == 32 ? 0xFFFFFFFFu : (1u << kWidth) - 1u);
}

template <int kWidth>
__device__ __forceinline__ void count_needs(const PoolArgs& a, ReserveSmem& sm, int requests) {
    const int lane = threadIdx.x & 31, sub = lane % kWidth;
    for (int i0 = (threadIdx.x >> 5) * (32 / kWidth); i0 < requests; i0 += kPlanT / kWidth) {
        const int i = i0 + lane / kWidth < requests ? i0 + lane / kWidth : -1;
        int most = i >= 0 ? sm.entries[i] : 0, n = 0;
#pragma unroll
        for (int o = kWidth; o < 32; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        bool bad = false;
        for (int at = 0; at < most; at += kWidth) {
            int32_t p;
            const uint32_t m = entries_in_need<kWidth>(a, sm, i, at, &p, &bad);
            if (at == 0 && sub == 0 && i >= 0) sm.mask[i] = m;
            n += __popc(m);
        }
#pragma unroll
        for (int o = 1; o < kWidth; o <<= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o) != 0;
        if (i >= 0 && sub == 0 && sm.need[i] >= 0) sm.need[i] = bad ? -1 : n;
    }
}

template <int kWidth>
__device__ __forceinline__ void hand_out(const PoolArgs& a, ReserveSmem& sm, const Work& w, int64_t given, int requests) {
    const int lane = threadIdx.x & 31, sub = lane % kWidth;
    for (int i0 = (threadIdx.x >> 5) * (32 / kWidth); i0 < requests; i0 += kPlanT / kWidth) {
        const int i = i0 + lane / kWidth < requests && sm.need[i0 + lane / kWidth] >= 0 ? i0 + lane / kWidth : -1;
        const int len = i >= 0 ? sm.entries[i] : 0;
        int64_t k0 = i >= 0 ? sm.need[i] : 0;
        int most = len;
#pragma unroll
        for (int o = kWidth; o < 32; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        for (int at = 0; at < most; at += kWidth) {
            int32_t p = -1;
            bool bad = false;
            uint32_t m;
            if (kWidth == 8 || most <= 32) {  // known from the count
                m = at < len ? sm.mask[i] : 0u;
                if ((m >> sub) & 1u) p = a.tab[sm.first[i] + sub];
            } else {
                m = entries_in_need<kWidth>(a, sm, i, at, &p, &bad);
            }
            if ((m >> sub) & 1u) {
                const int64_t e = sm.first[i] + at + sub, k = k0 + __popc(m & ((1u << sub) - 1u));
                const int32_t to = w.list[k];
                a.tab[e] = to;
                a.refs[to] = 1;
                w.map[given + k] = p;
                if (p >= 0 && at + sub == 0 && sm.part[i] > 0)
                    w.move[atomicAdd(&sm.moves, 1)] =
                        Move{static_cast<int64_t>(p) * a.page, static_cast<int64_t>(to) * a.page, sm.part[i], 0};
            }
            k0 += __popc(m);
        }
    }
}

__global__ void __cluster_dims__(kReserveCtas, 1, 1) __launch_bounds__(kPlanT)
    pages_reserve_kernel(PoolArgs a, int B, const int64_t* __restrict__ tok_off, const int64_t* __restrict__ tok_end,
                         const int64_t* __restrict__ want, int64_t n_tokens, int64_t* __restrict__ room, Work w, int32_t* status) {
    __shared__ ReserveSmem sm;
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        if (tid == 0) sm.moves = 0;
        int64_t given = 0;  // pages handed out
        bool full = false;
        for (int b0 = 0; b0 < B; b0 += kPlanT) {
            const int b = b0 + tid, requests = min(B - b0, kPlanT);
            // ---- the entries every request grows over
            int64_t end = 0, to = 0;
            bool ok = false, many = false;
            if (b < B) {
                Region r;
                to = want[b];
                ok = region_of(tok_off, tok_end, n_tokens, a.page, b, &r) && to >= r.end && to <= r.last;
                end = r.end;
                int64_t first = 0, n = 0;
                if (ok && to > end) {
                    first = quot(end, a.page);
                    n = pages_to(to, a.page) - first;
                }
                many = n > 8;
                sm.first[tid] = first;
                sm.entries[tid] = static_cast<int32_t>(min(n, static_cast<int64_t>(0x7FFFFFC0)));
                sm.part[tid] = static_cast<int32_t>(end - first * a.page);
                sm.need[tid] = ok ? 0 : -1;
            }
            many = __syncthreads_or(many);
            if (many) count_needs<32>(a, sm, requests);
            else count_needs<8>(a, sm, requests);
            __syncthreads();
            // ---- the free pages, and where each request's begin
            const int32_t mine = b < B ? sm.need[tid] : -1;
            if (b < B && mine < 0) set_status(status, ECHO_ST_BADDATA);
            int64_t total;
            const int64_t at = block_scan64<kPlanT>(max(mine, 0), sm.scratch64, &total);
            const bool before = __syncthreads_or(full);  // an earlier batch's request went without
            const int64_t have = before ? 0 : list_free(a, min(total, a.n_pages), w.list, sm.scratch);
            bool served = false;
            if (b < B) {
                served = mine == 0 || (mine > 0 && at + mine <= have);
                full |= mine > 0 && !served;
                if (room) room[b] = served ? to : end;
                sm.need[tid] = served && mine > 0 ? static_cast<int32_t>(at) : -1;
            }
            // the requests served are the first of those in need: their pages are the first of the list
            int64_t here;
            (void)block_scan64<kPlanT>(served ? max(mine, 0) : 0, sm.scratch64, &here);
            // ---- handed out; the counts of the pages replaced fall when all have been, since two requests may replace the same one
            if (many) hand_out<32>(a, sm, w, given, requests);
            else hand_out<8>(a, sm, w, given, requests);
            given += here;
            __syncthreads();
        }
        if (full) set_status(status, ECHO_ST_FULL);
        for (int64_t k = tid; k < given; k += kPlanT)
            if (w.map[k] >= 0) drop_ref(a, w.map[k], status);
        if (tid == 0) *w.moves = sm.moves;
    }
    cluster_sync_all();
    move_all<kPlanT>(a, w.move, static_cast<uint32_t>(*w.moves), blockIdx.x, kReserveCtas, 0, 1);
}

// ---------------------------------------------------------------- fork
struct ForkArgs {
    int n;
    const int32_t* src;
    const int32_t* dst;
    int B;
    const int64_t* tok_off;
    int64_t* tok_end;
    int64_t n_tokens;
};

// Three launches: every pair shares pages (a block or more each, 5.8 us for 64 pairs), one block hands out the pages of the
// last rows (4.8), a grid copies them (4.9: 64 x up to 64 rows of 4 layers).

// Whether pair i may be forked; a block together.
__device__ __forceinline__ bool fork_pair(const ForkArgs& f, int page, int i, Region* from, Region* to) {
    const int s = f.src[i], d = f.dst[i];
    bool ok = s >= 0 && s < f.B && d >= 0 && d < f.B;
    bool clash = false;
    for (int k = threadIdx.x; k < f.n; k += blockDim.x) clash |= (k < i && f.dst[k] == d) || f.src[k] == d;
    clash = __syncthreads_or(clash);
    if (!ok || clash) return false;
    ok = region_of(f.tok_off, f.tok_end, f.n_tokens, page, s, from);
    // (the end of dst is replaced, whatever it is)
    to->off = f.tok_off[d];
    to->last = f.tok_off[d + 1];
    to->end = to->off;
    return ok && to->off >= 0 && to->last >= to->off && to->last <= f.n_tokens && rest(to->off, page) == 0 &&
           to->last - to->off >= from->end - from->off;
}

__global__ void __launch_bounds__(kFT) pages_share_kernel(PoolArgs a, ForkArgs f, Work w, int32_t* status) {
    const int i = blockIdx.x;
    Region from, to;
    const bool ok = fork_pair(f, a.page, i, &from, &to);
    if (!ok) {
        if (threadIdx.x == 0 && blockIdx.y == 0) {
            w.tail[i].dst = -1;
            set_status(status, ECHO_ST_BADDATA);
        }
        return;
    }
    const int64_t full = quot(from.end - from.off, a.page), entries = pages_to(to.last, a.page) - quot(to.off, a.page);
    const int32_t* const s = a.tab + quot(from.off, a.page);
    int32_t* const d = a.tab + quot(to.off, a.page);
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        const int over = static_cast<int>(from.end - from.off - full * a.page);
        const int32_t p = over ? s[full] : -1;
        if (p >= 0 && !in_pool(a, p)) set_status(status, ECHO_ST_BADDATA);
        w.tail[i] = Tail{quot(to.off, a.page) + full, to.off + full * a.page, f.dst[i], in_pool(a, p) ? p : -1, over, 0};
    }
    for (int64_t e = static_cast<int64_t>(blockIdx.y) * kFT + threadIdx.x; e < entries; e += static_cast<int64_t>(gridDim.y) * kFT) {
        const int32_t old = d[e];
        int32_t p = e < full ? s[e] : -1;
        if (p >= 0 && !in_pool(a, p)) {
            set_status(status, ECHO_ST_BADDATA);
            p = -1;
        }
        if (old == p) continue;
        if (p >= 0) atomicAdd(a.refs + p, 1);
        if (old != -1) drop_ref(a, old, status);
        d[e] = p < 0 ? -1 : p;
    }
}

__global__ void __launch_bounds__(kPlanT) pages_tails_kernel(PoolArgs a, ForkArgs f, Work w, int32_t* status) {
    __shared__ uint32_t scratch[kPlanT / 32 + 1];
    const int tid = threadIdx.x;
    pdl_wait();
    uint32_t given = 0;
    bool full = false;
    for (int i0 = 0; i0 < f.n; i0 += kPlanT) {
        Tail t = {0, 0, -1, -1, 0, 0};
        if (i0 + tid < f.n) t = w.tail[i0 + tid];
        const bool it = t.dst >= 0 && t.page >= 0;
        uint32_t total;
        const uint32_t at = block_exclusive_scan<kPlanT>(it, scratch, &total);
        const int64_t have = list_free(a, min(static_cast<int64_t>(total), a.n_pages), w.list, scratch);
        const bool without = it && at >= have;
        if (it && !without) {
            const int32_t to = w.list[at];
            a.tab[t.entry] = to;
            a.refs[to] = 1;
            w.move[given + at] = Move{static_cast<int64_t>(t.page) * a.page, static_cast<int64_t>(to) * a.page, t.rows, 0};
        }
        full |= without;
        if (t.dst >= 0) f.tok_end[t.dst] = t.end + (without ? 0 : t.rows);
        given += static_cast<uint32_t>(have);
        __syncthreads();
    }
    if (full) set_status(status, ECHO_ST_FULL);
    if (tid == 0) *w.moves = static_cast<int32_t>(given);
}

// ---------------------------------------------------------------- compact
// One block counts and pairs (6.3 us over 3077 pages; with nothing to move, the call takes 8.5 us over 2^12 pages, 31 over 2^16,
// 406 over 2^20, 7400 over 2^24, as the block reads the counts two to three times), a grid moves rows and renames entries: 453 MB read and written in
// 129 us, 7.0 TB/s, a plain copy's rate (the last 50 MB are still in L2 then).
//
// list[k]: the k-th free place before U, far[k]: the k-th page in use from U on, which goes there; map[p]: where page p >= U
// goes (-1: it is free).
__global__ void __launch_bounds__(kPlanT) pages_compact_kernel(PoolArgs a, int32_t* __restrict__ used, Work w) {
    __shared__ uint32_t scratch[kPlanT / 32 + 1];
    const int tid = threadIdx.x;
    uint32_t mine = 0, U;
    int32_t r[kRun];
    for (int64_t p0 = 0; p0 < a.n_pages; p0 += kRun * kPlanT) {
        counts_of(a, p0 + kRun * tid, r);
#pragma unroll
        for (int i = 0; i < kRun; ++i) mine += r[i] > 0 && p0 + kRun * tid + i < a.n_pages;
    }
    (void)block_exclusive_scan<kPlanT>(mine, scratch, &U);
    uint32_t holes = 0, far = 0;
    for (int64_t p0 = 0; p0 < U; p0 += kRun * kPlanT) {
        const int64_t p = p0 + kRun * tid;
        counts_of(a, p, r);
        uint32_t n = 0, total;
#pragma unroll
        for (int i = 0; i < kRun; ++i) n += r[i] <= 0 && p + i < U;
        uint32_t at = holes + block_exclusive_scan<kPlanT>(n, scratch, &total);
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if (r[i] <= 0 && p + i < U) w.list[at++] = static_cast<int32_t>(p + i);
        holes += total;
    }
    __syncthreads();
    for (int64_t p0 = U & ~(kRun - 1u); p0 < a.n_pages; p0 += kRun * kPlanT) {
        const int64_t p = p0 + kRun * tid;
        counts_of(a, p, r);
        uint32_t n = 0, total;
#pragma unroll
        for (int i = 0; i < kRun; ++i) n += r[i] > 0 && p + i >= U && p + i < a.n_pages;
        uint32_t at = far + block_exclusive_scan<kPlanT>(n, scratch, &total);
        int32_t to[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {  // all loads before a store
            to[i] = -1;
            if (r[i] > 0 && p + i >= U && p + i < a.n_pages) to[i] = w.list[at++];
        }
        at -= n;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            if (p + i < U || p + i >= a.n_pages) continue;
            if (to[i] >= 0) {
                w.far[at++] = static_cast<int32_t>(p + i);
                a.refs[to[i]] = r[i];
                a.refs[p + i] = 0;
            }
            w.map[p + i] = to[i];
        }
        far += total;
    }
    if (tid == 0) {
        *used = static_cast<int32_t>(U);
        *w.moves = static_cast<int32_t>(far);
    }
}

__global__ void __launch_bounds__(kMT) pages_place_kernel(PoolArgs a, const int32_t* __restrict__ used, Work w, int32_t* status) {
    pdl_wait();
    const int32_t U = *used;
    if (blockIdx.y == 0)
        for (int64_t e = static_cast<int64_t>(blockIdx.x) * kMT + threadIdx.x; e < a.entries; e += static_cast<int64_t>(gridDim.x) * kMT) {
            const int32_t p = a.tab[e];
            if (p < U) continue;
            const int32_t to = p < a.n_pages ? w.map[p] : -1;
            if (to < 0) set_status(status, ECHO_ST_BADDATA);
            else a.tab[e] = to;
        }
    const int64_t bytes = a.page * a.row_bytes;
    constexpr int kPiece = kMT * 64;
    const uint32_t pieces = static_cast<uint32_t>((bytes + kPiece - 1) / kPiece), n = static_cast<uint32_t>(*w.moves) * pieces;
    for (uint32_t u = blockIdx.x; u < n; u += gridDim.x) {
        const uint32_t k = u / pieces;
        const int64_t at = static_cast<int64_t>(u % pieces) * kPiece, src = w.far[k] * bytes + at, dst = w.list[k] * bytes + at;
        for (int l = blockIdx.y; l < a.layers; l += gridDim.y) {
            uint8_t* const kv = a.kv + l * a.layer_bytes;
            move_piece<kMT>(kv + src, kv + dst, bytes - at);
        }
    }
}

// ---------------------------------------------------------------- the rows of an accepted path
constexpr int kKT = 288;
constexpr int kBatch = 64;

constexpr int kHeld = 8;  // rows a thread reads before it writes them

// One tree 6.1 us, 64 of up to 16 accepted rows in 8 layers 6.6: loads of bounds, path, entries, then rows.
// A thread has one 16-byte column of some layers and takes the path's rows in order, eight at a time: the path
// ascends, so no row is written before it has been read.
__global__ void __launch_bounds__(kKT)
    rows_keep_kernel(PoolArgs a, const int64_t* __restrict__ row_off, int64_t n_rows, const int32_t* __restrict__ path,
                     const int32_t* __restrict__ count, const int64_t* __restrict__ tok_off, const int64_t* __restrict__ tok_end,
                     int64_t n_tokens, int64_t* __restrict__ new_end, int32_t* status) {
    __shared__ int64_t from[kBatch], to[kBatch];
    const int b = blockIdx.x, tid = threadIdx.x;
    const int64_t r0 = row_off[b], r1 = row_off[b + 1];
    const int64_t c = count[b];
    Region r;
    bool ok = region_of(tok_off, tok_end, n_tokens, a.page, b, &r) && r0 >= 0 && r1 >= r0 && r1 <= n_rows && r1 - r0 <= r.end - r.off &&
              c >= 0 && c <= r1 - r0;
    const int64_t n = r1 - r0, base = r.end - n;
    // bytes from the pool's first row; alone: the page has to be this request's alone
    const auto row_of = [&](int64_t tok, bool* bad, bool alone) {
        const int64_t e = quot(tok, a.page);
        const int32_t p = a.tab[e];
        if (!in_pool(a, p) || (alone && a.refs[p] != 1)) {
            *bad = true;
            return static_cast<int64_t>(0);
        }
        return (static_cast<int64_t>(p) * a.page + (tok - e * a.page)) * a.row_bytes;
    };
    if (ok) {
        bool bad = false;
        for (int64_t i = tid; i < c; i += kKT) {
            const int64_t x = path[r0 + i], before = i > 0 ? path[r0 + i - 1] : -1;
            int64_t src = 0, dst = 0;
            if (x <= before || x >= n) {
                bad = true;
            } else if (x != i) {
                src = row_of(base + x, &bad, false);
                dst = row_of(base + i, &bad, true);
            }
            if (i < kBatch) {
                from[i] = src;
                to[i] = dst;
            }
        }
        ok = !__syncthreads_or(bad);
    }
    if (tid == 0 && blockIdx.y == 0) {
        if (!ok) set_status(status, ECHO_ST_BADDATA);
        new_end[b] = ok ? base + c : tok_end[b];
    }
    if (!ok) return;
    const int cols = static_cast<int>(a.row_bytes / 16);
    for (int64_t i0 = 0; i0 < c; i0 += kBatch) {
        if (i0 > 0) {
            __syncthreads();
            if (tid < kBatch && i0 + tid < c) {
                const int64_t i = i0 + tid, x = path[r0 + i];
                bool bad = false;
                from[tid] = x != i ? row_of(base + x, &bad, false) : 0;
                to[tid] = x != i ? row_of(base + i, &bad, false) : 0;
            }
            __syncthreads();
        }
        const int m = static_cast<int>(min(static_cast<int64_t>(kBatch), c - i0));
        const int64_t columns = static_cast<int64_t>(cols) * a.layers, step = static_cast<int64_t>(gridDim.y) * kKT;
        for (int64_t k = static_cast<int64_t>(blockIdx.y) * kKT + tid; k < columns; k += step) {
            const int64_t l = quot(k, cols);
            uint8_t* const kv = a.kv + l * a.layer_bytes + (k - l * cols) * 16;
            for (int i = 0; i < m; i += kHeld) {
                uint4 v[kHeld];
#pragma unroll
                for (int h = 0; h < kHeld; ++h)
                    if (i + h < m && from[i + h] != to[i + h]) v[h] = *reinterpret_cast<const uint4*>(kv + from[i + h]);
#pragma unroll
                for (int h = 0; h < kHeld; ++h)
                    if (i + h < m && from[i + h] != to[i + h]) *reinterpret_cast<uint4*>(kv + to[i + h]) = v[h];
            }
        }
    }
}

// ---------------------------------------------------------------- host
int check_pool(const echo_page_pool* p, int64_t n_tokens) {
    if (!p || n_tokens < 0 || !p->refs || !p->kv || (n_tokens > 0 && !p->page_tab)) return ECHO_EINVAL;
    if (p->n_pages < 1 || p->page < 1 || p->layers < 1 || p->row_bytes < 16 || p->row_bytes % 16) return ECHO_EINVAL;
    if (p->n_pages > ECHO_POOL_MAX_PAGES) return ECHO_EUNSUPPORTED;
    if (!is_aligned(p->kv, 16) || p->layer_bytes % 16) return ECHO_EINVAL;
    const int64_t rows = p->n_pages * p->page;  // below 2^55
    if (p->row_bytes > (1ll << 62) / rows) return ECHO_EINVAL;
    if (p->layers > 1 && p->layer_bytes < rows * p->row_bytes) return ECHO_EINVAL;
    return ECHO_OK;
}

PoolArgs pool_args(const echo_page_pool* p, int64_t n_tokens) {
    PoolArgs a;
    a.tab = p->page_tab;
    a.refs = p->refs;
    a.kv = static_cast<uint8_t*>(p->kv);
    a.n_pages = p->n_pages;
    a.row_bytes = p->row_bytes;
    a.layer_bytes = p->layer_bytes;
    a.layers = p->layers;
    a.page = p->page;
    a.entries = n_tokens / p->page + (n_tokens % p->page != 0);
    a.wide = is_aligned(p->refs, 16);
    return a;
}

int check_work(const void* ws, size_t ws_bytes, int B, int64_t n_pages) {
    return ws && is_aligned(ws, 256) && ws_bytes >= echo_pages_workspace_size(B, n_pages) ? ECHO_OK : ECHO_EINVAL;
}

// Blocks over a request's entries when the regions are alike.
unsigned entry_blocks(const PoolArgs& a, int B) {
    const int64_t n = (a.entries / B + kFT - 1) / kFT;
    return static_cast<unsigned>(n < 1 ? 1 : n > 64 ? 64 : n);
}

unsigned layer_blocks(const PoolArgs& a) { return static_cast<unsigned>(a.layers < 8 ? a.layers : 8); }

// Blocks that carry out at most `most` moves, a piece each at a time, up to 32 an SM: many short blocks keep more bytes under way
// than the 8 that are resident, each waiting for its loads, then storing (453 MB: 138 us with 8 an SM, 129 with 32; 127 with 64, but
// 3 us more where there is little to move).
unsigned move_blocks(const PoolArgs& a, int64_t most) {
    const int64_t rows = layer_blocks(a), cap = (32 * static_cast<int64_t>(sm_count()) + rows - 1) / rows;
    const int64_t pieces = (a.page * a.row_bytes + kMT * 64 - 1) / (kMT * 64);
    return static_cast<unsigned>(most < 1 ? 1 : pieces >= cap || most >= cap ? cap : std::min(most * pieces, cap));
}

}  // namespace
}  // namespace echo

extern "C" size_t echo_pages_workspace_size(int B, int64_t n_pages) {
    if (B <= 0 || B > ECHO_MAX_REQUESTS || n_pages <= 0 || n_pages > ECHO_POOL_MAX_PAGES) return 0;
    return echo::work_layout(B, n_pages > B ? n_pages : B).total;
}

extern "C" int echo_pages_free(int B, const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens, const echo_page_pool* pool,
                               int32_t* status, echo_stream_t stream) {
    using namespace echo;
    if (B <= 0 || !tok_off || !tok_end || !status) return ECHO_EINVAL;
    if (B > ECHO_MAX_REQUESTS) return ECHO_EUNSUPPORTED;
    const int rc = check_pool(pool, n_tokens);
    if (rc) return rc;
    if (n_tokens == 0) return ECHO_OK;
    const PoolArgs a = pool_args(pool, n_tokens);
    pages_free_kernel<<<dim3(B, entry_blocks(a, B)), kFT, 0, static_cast<cudaStream_t>(stream)>>>(a, tok_off, tok_end, n_tokens, status);
    ECHO_CUDA_OK(cudaGetLastError());
    return ECHO_OK;
}

extern "C" int echo_pages_reserve(int B, const int64_t* tok_off, const int64_t* tok_end, const int64_t* want, int64_t n_tokens,
                                  const echo_page_pool* pool, int64_t* room, void* ws, size_t ws_bytes, int32_t* status,
                                  echo_stream_t stream) {
    using namespace echo;
    if (B <= 0 || !tok_off || !tok_end || !want || !status) return ECHO_EINVAL;
    if (B > ECHO_MAX_REQUESTS) return ECHO_EUNSUPPORTED;
    int rc = check_pool(pool, n_tokens);
    if (rc) return rc;
    if ((rc = check_work(ws, ws_bytes, B, pool->n_pages))) return rc;
    const PoolArgs a = pool_args(pool, n_tokens);
    const Work w = work_of(ws, B, pool->n_pages > B ? pool->n_pages : B);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    pages_reserve_kernel<<<kReserveCtas, kPlanT, 0, s>>>(a, B, tok_off, tok_end, want, n_tokens, room, w, status);
    ECHO_CUDA_OK(cudaGetLastError());
    return ECHO_OK;
}

extern "C" int echo_pages_fork(int n, const int32_t* src, const int32_t* dst, int B, const int64_t* tok_off, int64_t* tok_end,
                               int64_t n_tokens, const echo_page_pool* pool, void* ws, size_t ws_bytes, int32_t* status,
                               echo_stream_t stream) {
    using namespace echo;
    if (n < 0 || B <= 0 || !tok_off || !tok_end || !status) return ECHO_EINVAL;
    if (n > ECHO_MAX_REQUESTS || B > ECHO_MAX_REQUESTS) return ECHO_EUNSUPPORTED;
    int rc = check_pool(pool, n_tokens);
    if (rc) return rc;
    if (n == 0) return ECHO_OK;
    if (!src || !dst || (rc = check_work(ws, ws_bytes, n, pool->n_pages))) return ECHO_EINVAL;
    const PoolArgs a = pool_args(pool, n_tokens);
    const ForkArgs f = {n, src, dst, B, tok_off, tok_end, n_tokens};
    const Work w = work_of(ws, n, pool->n_pages > n ? pool->n_pages : n);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    pages_share_kernel<<<dim3(n, entry_blocks(a, B)), kFT, 0, s>>>(a, f, w, status);
    ECHO_CUDA_OK(cudaGetLastError());
    ECHO_CUDA_OK(launch_after(false, pages_tails_kernel, dim3(1), kPlanT, 0, s, a, f, w, status));
    ECHO_CUDA_OK(launch_after(false, pages_move_kernel, dim3(move_blocks(a, n), layer_blocks(a)), kMT, 0, s, a, w));
    return ECHO_OK;
}

extern "C" int echo_pages_compact(int64_t n_tokens, const echo_page_pool* pool, int32_t* used, void* ws, size_t ws_bytes,
                                  int32_t* status, echo_stream_t stream) {
    using namespace echo;
    if (!used || !status) return ECHO_EINVAL;
    int rc = check_pool(pool, n_tokens);
    if (rc) return rc;
    if ((rc = check_work(ws, ws_bytes, 1, pool->n_pages))) return rc;
    const PoolArgs a = pool_args(pool, n_tokens);
    const Work w = work_of(ws, 1, pool->n_pages);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    pages_compact_kernel<<<1, kPlanT, 0, s>>>(a, used, w);
    ECHO_CUDA_OK(cudaGetLastError());
    const int64_t names = (a.entries + kMT - 1) / kMT, few = 8 * sm_count();  // (entries are renamed by the same blocks)
    const unsigned blocks = std::max(move_blocks(a, a.n_pages / 2), static_cast<unsigned>(std::min(names, few)));
    ECHO_CUDA_OK(launch_after(false, pages_place_kernel, dim3(blocks, layer_blocks(a)), kMT, 0, s, a,
                              const_cast<const int32_t*>(used), w, status));
    return ECHO_OK;
}

extern "C" int echo_rows_keep(int B, const int64_t* row_off, int64_t n_rows, const int32_t* path, const int32_t* count,
                              const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens, const echo_page_pool* pool,
                              int64_t* new_end, int32_t* status, echo_stream_t stream) {
    using namespace echo;
    if (B <= 0 || n_rows < 0 || !row_off || !count || !tok_off || !tok_end || !new_end || !status) return ECHO_EINVAL;
    if (B > ECHO_MAX_REQUESTS || n_rows > ECHO_CHUNK_MAX_ROWS) return ECHO_EUNSUPPORTED;
    if (n_rows > 0 && !path) return ECHO_EINVAL;
    if (new_end < tok_end + B && tok_end < new_end + B) return ECHO_EINVAL;
    const int rc = check_pool(pool, n_tokens);
    if (rc) return rc;
    const PoolArgs a = pool_args(pool, n_tokens);
    const int64_t blocks = (a.row_bytes / 16 * a.layers + kKT - 1) / kKT;
    rows_keep_kernel<<<dim3(B, static_cast<unsigned>(blocks < 64 ? blocks : 64)), kKT, 0, static_cast<cudaStream_t>(stream)>>>(
        a, row_off, n_rows, path, count, tok_off, tok_end, n_tokens, new_end, status);
    ECHO_CUDA_OK(cudaGetLastError());
    return ECHO_OK;
}
