// echo_mass.cu -- the attention weight every cached token receives from a chunk.
//
// mass_out[g] = decay * mass[g] + sum_r sum_h exp(scale * q[r,h] . kv[g] - lse[r,h])
// over the rows r that see token g (echo.h, echo_mla_mass).
//
// The (row, head) pairs of a request are consecutive rows of q, so its scores are one
// product K Q^T: an item is 256 tokens of a request against blocks of 256 pairs.
// A cluster of two CTAs has the item's K as the A operand (M = 256, 128 token
// rows each, TMEM lane = token) and half of each block's pairs as the B operand
// (N = 256): per MMA a CTA reads 8 KB of shared memory in 128 cycles, where one
// CTA with M = 128 would read 12 KB and be bound by it.  A thread of the
// epilogue owns a token and adds its weights over the columns in a fixed
// order, so no sum crosses threads; which pairs see a token is one range of
// columns (rows from the token's own position on, up to the window's end).
// K lives in nine 16 KB slots of 64 dims each: it stays while an item walks its
// blocks, and in the item's last block every slot takes the next item's dims as
// soon as its MMAs are done, so that single-block items (decode) stream too.  Q
// comes by TMA through five slots (three did not cover the way to L2: 1024 rows over
// 8192 tokens 777 us, with four 671).  Warps: 0-3 epilogue, 4-7 and 12-15 gather K (16-byte
// cp.async), 8 of CTA 0 issues the MMAs, 9 loads Q, 10 and 11 report what K and Q
// have landed in their CTA to CTA 0 (one barrier for both CTAs: a look at a barrier
// costs the issuing thread over a hundred cycles of the 512 that an atom's MMAs run).
//
// The scores are sums of the tensor cores in 32 bits.  Measured against fp64 they lie
// nearer to zero (5e-7 of their value for |score| > 4, fp32 dot products in software show
// no such bias), which is what accumulation that cuts off low bits does.  The weights of
// 1024 rows come out 1.5e-6 off for it, 7e-8 with fp32 dot products; it is accepted, as
// accumulating in shorter runs would add a pass over the scores for each.
//
// Shares of the work are cut as in echo_chunk.cu, by blocks; the parts of a cut item are
// 256 sums in the workspace, joined in order.
#include "echo_paged.cuh"
#include "echo_tc.cuh"

namespace echo {
namespace {

constexpr int kTok = 256;               // tokens per item, 128 per CTA
constexpr int kCols = 256;              // (row, head) pairs per block
constexpr int kThreads = 512;
constexpr int kLoad = 128;
constexpr int kAtoms = kLatDqk / 64;    // 9
constexpr uint32_t kSlot = 128 * 128;   // 128 rows of 64 dims
constexpr int kKSlots = 9, kQSlots = 5;
constexpr uint32_t kTmemCols = 512;     // two D buffers of 256 columns
constexpr int kMaxClusters = 96;
// units of an item: its K, each block; only to decay
constexpr int kCostK = 4, kCostBlock = 6, kCostNone = 1;
constexpr int kMinUnits = kCostK + kCostBlock;

struct __align__(16) Item {
    int64_t off;    // the request's first token row
    int64_t tok0;   // first token of the item
    int64_t len;    // the request's tokens
    int64_t col0;   // the request's first (row, head) pair
    int32_t req;
    int32_t rows;   // rows of the request
    int32_t pos0;   // position of its first row
    int32_t cb0;    // first block of columns some token of the item is seen by
    int32_t nb;     // blocks
    int32_t pad;
};

struct __align__(16) PlanHead {
    int64_t total;
    int32_t items;
    int32_t parts;
};

struct Plan {
    PlanHead* head;
    Item* item;
    int64_t* cum;
    float* part;    // [2 * kMaxClusters][256]
    int64_t cap;
    int clusters;
};

struct Layout {
    size_t item, cum, part, total;
};
inline Layout plan_layout(int64_t cap) {
    Layout l;
    l.item = 256;
    l.cum = round_up(l.item + static_cast<size_t>(cap) * sizeof(Item), 256);
    l.part = round_up(l.cum + static_cast<size_t>(cap + 1) * 8, 256);
    l.total = l.part + 2 * kMaxClusters * kTok * sizeof(float);
    return l;
}

__device__ __forceinline__ int64_t cost_of(int nb) { return nb ? kCostK + static_cast<int64_t>(kCostBlock) * nb : kCostNone; }
// Blocks that start before unit x of an item.
__device__ __forceinline__ int blocks_before(int64_t x, int nb) {
    const int64_t b = (x - kCostK + kCostBlock - 1) / kCostBlock;
    return static_cast<int>(x <= kCostK ? 0 : min(b, static_cast<int64_t>(nb)));
}

constexpr int kPT = 1024;

__global__ void __launch_bounds__(kPT) mass_plan_kernel(ChunkArgs a, Plan plan) {
    __shared__ int64_t goff[ECHO_MAX_REQUESTS + 1];
    __shared__ int64_t scratch[kPT / 32];
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPT) {
        const int b = b0 + tid;
        int64_t lo = 0, hi = 0;
        if (b < a.B && !seg_bounds(a.tok_off, a.tok_end, a.n_tokens, b, &lo, &hi)) set_status(a.status, ECHO_ST_BADDATA);
        int64_t total;
        const int64_t at = block_scan64<kPT>((hi - lo + kTok - 1) / kTok, scratch, &total);
        if (b < a.B) goff[b] = min(base + at, plan.cap);
        base += total;
        if (base > plan.cap) {  // token ranges that overlap
            if (tid == 0) set_status(a.status, ECHO_ST_BADDATA);
            base = plan.cap;
        }
    }
    if (tid == 0) goff[a.B] = base;
    __syncthreads();
    const int64_t items = base;
    int64_t sum = 0;
    for (int64_t g0 = 0; g0 < items; g0 += kPT) {
        const int64_t g = g0 + tid;
        int64_t cost = 0;
        if (g < items) {
            int b = 0, e = a.B;
            while (e - b > 1) {
                const int mid = (b + e) >> 1;
                if (goff[mid] <= g) b = mid;
                else e = mid;
            }
            int64_t t0, t1, r0, n, off, len;
            seg_bounds(a.tok_off, a.tok_end, a.n_tokens, b, &t0, &t1);
            chunk_request(a, b, &r0, &n, &off, &len);
            if (len == 0) n = 0;  // its rows see nothing
            Item it;
            it.off = t0;
            it.tok0 = (g - goff[b]) * kTok;
            it.len = t1 - t0;
            it.col0 = r0 * a.heads;
            it.req = b;
            it.rows = static_cast<int32_t>(n);
            it.pos0 = static_cast<int32_t>(len - n);
            it.cb0 = it.nb = 0;
            it.pad = 0;
            if (n > 0) {
                const int64_t p0 = len - n, last = min(it.tok0 + kTok, it.len) - 1;
                const int64_t c_lo = max(static_cast<int64_t>(0), it.tok0 - p0) * a.heads;
                const int64_t far = a.window && it.tok0 >= a.sinks ? min(n, last - p0 + a.window) : n;
                const int64_t c_hi = far * a.heads;
                if (c_hi > c_lo) {
                    it.cb0 = static_cast<int32_t>(c_lo / kCols);
                    it.nb = static_cast<int32_t>((c_hi + kCols - 1) / kCols - it.cb0);
                }
            }
            plan.item[g] = it;
            cost = cost_of(it.nb);
        }
        int64_t total;
        const int64_t at = sum + block_scan64<kPT>(cost, scratch, &total);
        if (g < items) plan.cum[g] = at;
        sum += total;
    }
    if (tid == 0) {
        plan.cum[items] = sum;
        PlanHead h;
        h.total = sum;
        h.items = static_cast<int32_t>(items);
        h.parts = static_cast<int32_t>(
            max(static_cast<int64_t>(1), min(static_cast<int64_t>(plan.clusters), sum / kMinUnits)));
        *plan.head = h;
    }
}

// The blocks [lo, hi) of an item that a share holds.
struct Piece {
    Item g;
    int lo, hi;
};

struct Walk {
    const Item* item;
    const int64_t* cum;
    int64_t u0, u1;
    int g;
    __device__ __forceinline__ bool next(Piece* p) {
        for (;;) {
            if (u0 >= u1) return false;
            const int64_t c = cum[g];
            p->g = item[g];
            ++g;
            const int64_t cost = cost_of(p->g.nb), a = u0 - c;
            p->lo = blocks_before(a, p->g.nb);
            p->hi = blocks_before(min(u1 - c, cost), p->g.nb);
            u0 = c + cost;
            if (p->hi > p->lo || (p->g.nb == 0 && a <= 0)) return true;
        }
    }
};

struct Ctl {
    // *_full: landed here; *_ready of CTA 0: landed in both CTAs
    uint64_t k_full[kKSlots], k_ready[kKSlots];
    uint64_t k_free[2][kKSlots];          // by the parity of the item that leaves the slot
    uint64_t q_full[kQSlots], q_ready[kQSlots], q_free[kQSlots];
    uint64_t d_full[2], d_free[2];
    uint64_t drain;
    uint32_t tmem;
    Watch watch;
    int first;
    uint32_t none[2];                     // d + 1: the block d of this buffer has a pair whose lse is -inf
    alignas(16) float nl[2][kCols];       // -lse * log2(e) of a block's pairs
};
constexpr uint32_t kSmem = (kKSlots + kQSlots) * kSlot + ((sizeof(Ctl) + 15u) & ~15u);
static_assert(kSmem <= 227u * 1024u, "mass shared memory");

__device__ __forceinline__ bool bar_or128(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v)), "r"(id)
        : "memory");
    return r != 0;
}

// Position in a ring of n slots: slot and the parity of its phase.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ int block_cols(const Item& g, int heads, int cb) {
    return static_cast<int>(min(static_cast<int64_t>(kCols), static_cast<int64_t>(g.rows) * heads - static_cast<int64_t>(cb) * kCols));
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mass_kernel(ChunkArgs a, Plan plan, const __grid_constant__ CUtensorMap qmap, float scale_log2,
                const float* __restrict__ lse, const float* mass, float* mass_out, float decay) {
    extern __shared__ __align__(1024) uint8_t mass_smem[];  // the swizzled tiles need 1024 bytes
    const uint32_t base = smem_addr(mass_smem);
    if (base & 1023u) {  // the same in every CTA
        set_status(a.status, ECHO_ST_TIMEOUT);
        return;
    }
    const uint32_t sK = base, sQ = sK + kKSlots * kSlot;
    Ctl* const ctl = reinterpret_cast<Ctl*>(mass_smem + (kKSlots + kQSlots) * kSlot);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t c = cluster_rank();
    const int ci = blockIdx.x >> 1;
    Watch* const watch = &ctl->watch;
    if (tid == 0) {
        for (int i = 0; i < kKSlots; ++i) {
            mbar_init(smem_addr(&ctl->k_full[i]), kLoad);
            mbar_init(smem_addr(&ctl->k_ready[i]), 2);
            mbar_init(smem_addr(&ctl->k_free[0][i]), 1);
            mbar_init(smem_addr(&ctl->k_free[1][i]), 1);
        }
        for (int i = 0; i < kQSlots; ++i) {
            mbar_init(smem_addr(&ctl->q_full[i]), 1);
            mbar_init(smem_addr(&ctl->q_ready[i]), 2);
            mbar_init(smem_addr(&ctl->q_free[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl->d_full[i]), 1);
            mbar_init(smem_addr(&ctl->d_free[i]), 8);
        }
        mbar_init(smem_addr(&ctl->drain), 1);
        watch_init(watch, a.wait_ns);
        ctl->none[0] = ctl->none[1] = 0;
        fence_barrier_init();
        if (a.n_rows > 0) prefetch_tmap(&qmap);
    }
    if (warp == 0) tmem_alloc2(smem_addr(&ctl->tmem), kTmemCols);
    pdl_wait();
    const PlanHead head = *plan.head;
    Walk walk;
    walk.item = plan.item;
    walk.cum = plan.cum;
    walk.u0 = walk.u1 = 0;
    walk.g = 0;
    if (ci < head.parts) {
        walk.u0 = share_start(head.total, head.parts, ci);
        walk.u1 = share_start(head.total, head.parts, ci + 1);
    }
    if (warp == 1 && walk.u0 < walk.u1) {
        const int g = find_group(plan.cum, head.items, walk.u0);
        if (lane == 0) ctl->first = g;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (walk.u0 < walk.u1) walk.g = ctl->first;
    const uint32_t tmem = ctl->tmem;
    Piece p;

    if (warp < 4) {
        // ---- epilogue: thread = token
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        uint32_t d = 0;  // blocks so far
        bool ok = true;
        while (ok && walk.next(&p)) {
            const int64_t tok = p.g.tok0 + c * 128 + tid;
            // The token's table entry and old mass are loaded here and looked at after the first block's MMAs: one
            // after the other, the loads of an item took longer than its products
            const bool in = tok < p.g.len, whole = p.lo == 0 && p.hi == p.g.nb;
            PageView pv = {};
            uint32_t in_page = 0;
            int32_t entry = -1;
            if (p.hi > p.lo && in) {
                pv = page_view(a, p.g.req, p.g.off);
                entry = pv.tab[page_of(a, pv, static_cast<uint32_t>(tok), &in_page)];
            }
            const float old = in && whole && decay > 0.f ? mass[p.g.off + tok] : 0.f;
            int64_t lo = 0, hi = 0;  // the columns that see the token
            float sum = 0.f, rest = 0.f;  // compensated over the blocks
            for (int b = p.lo; b < p.hi; ++b, ++d) {
                const int cb = p.g.cb0 + b, n = block_cols(p.g, a.heads, cb);
                const uint32_t db = d & 1u;
                float* const nl = ctl->nl[db];
                const float* const ls = lse + p.g.col0 + static_cast<int64_t>(cb) * kCols;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int x = tid + 128 * j;
                    const float v = x < n ? ls[x] : -INFINITY;
                    nl[x] = v == -INFINITY ? -INFINITY : -v * 1.4426950408889634f;
                    if (x < n && v == -INFINITY) ctl->none[db] = d + 1;  // adds nothing, whatever its scores are
                }
                ok = ok && mbar_wait_watch(smem_addr(&ctl->d_full[db]), (d >> 1) & 1u, watch);
                ok = !bar_or128(1, !ok);
                if (!ok) break;
                tc_fence_after();
                if (b == p.lo && entry >= 0) {
                    bool bad = false;
                    if (page_row(a, pv, entry, in_page, &bad) >= 0) {
                        lo = max(static_cast<int64_t>(0), tok - p.g.pos0) * a.heads;
                        hi = (a.window && tok >= a.sinks ? min(static_cast<int64_t>(p.g.rows), tok - p.g.pos0 + a.window)
                                                         : static_cast<int64_t>(p.g.rows)) * a.heads;
                    }
                    if (bad) set_status(a.status, ECHO_ST_BADDATA);
                }
                const int64_t first = static_cast<int64_t>(cb) * kCols;
                const int vlo = static_cast<int>(max(static_cast<int64_t>(0), min(lo - first, static_cast<int64_t>(kCols))));
                const int vhi = static_cast<int>(max(static_cast<int64_t>(0), min(hi - first, static_cast<int64_t>(n))));
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                int x = 0;
                if (ctl->none[db] == d + 1) {  // (a loop of its own: looking at every pair below cost 4% of a call)
#pragma unroll 1
                    for (; x < n; x += 32) {
                        float s[32];
                        tmem_ld_x32(tmem + lane_base + db * kCols + x, s);
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float v = nl[x + j];
                            if (x + j >= vlo && x + j < vhi && v != -INFINITY) part[j & 3] += ex2_approx(fmaf(s[j], scale_log2, v));
                        }
                    }
                }
#pragma unroll 1
                for (; x < n; x += 32) {
                    float s[32];
                    tmem_ld_x32(tmem + lane_base + db * kCols + x, s);
                    const float4* nv = reinterpret_cast<const float4*>(nl + x);
                    if (__all_sync(0xffffffffu, vlo <= x && x + 32 <= vhi)) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 v = nv[j >> 2];
                            part[0] += ex2_approx(fmaf(s[j], scale_log2, v.x));
                            part[1] += ex2_approx(fmaf(s[j + 1], scale_log2, v.y));
                            part[2] += ex2_approx(fmaf(s[j + 2], scale_log2, v.z));
                            part[3] += ex2_approx(fmaf(s[j + 3], scale_log2, v.w));
                        }
                    } else if (__any_sync(0xffffffffu, vlo < x + 32 && x < vhi)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float e = ex2_approx(fmaf(s[j], scale_log2, nl[x + j]));
                            part[j & 3] += (x + j >= vlo && x + j < vhi) ? e : 0.f;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(smem_addr(&ctl->d_free[db]), 0);
                const float y = ((part[0] + part[1]) + (part[2] + part[3])) - rest;
                const float z = __fadd_rn(sum, y);
                rest = __fsub_rn(__fsub_rn(z, sum), y);
                sum = z;
            }
            if (!ok) break;
            if (p.hi == p.lo && tid == 0) watch_beat(watch);
            if (whole) {
                if (in) mass_out[p.g.off + tok] = decay * old + sum;
            } else {
                plan.part[static_cast<size_t>(2 * ci + (p.lo > 0 ? 0 : 1)) * kTok + c * 128 + tid] = sum;
            }
        }
        if (!ok) give_up(watch);
    } else if (warp < 8 || warp >= 12) {
        // ---- K: 8 lanes per token row, 16 bytes each: a warp copies rows 4w + i + 16j, i < 4 at a time, having
        // looked up the 32 of them (lane i + 4j).  Two sets of four warps take the items in turn, so that one looks
        // its rows up while the other copies (32 decode rows 49.5 -> 43.5 us)
        const int w = warp & 3, set = warp < 8 ? 0 : 1, x = lane & 7, i4 = lane >> 3;
        static_assert(kKSlots == kAtoms, "an item takes every slot once");
        bool ok = true;
        for (int item = 0; ok && walk.next(&p);) {
            if (p.hi == p.lo) continue;
            if ((item & 1) != set) {
                ++item;
                continue;
            }
            int64_t mine = -1;
            {
                const int64_t tok = p.g.tok0 + c * 128 + 4 * w + (lane & 3) + 16 * (lane >> 2);
                bool bad = false;
                if (tok < p.g.len) mine = token_row(a, page_view(a, p.g.req, p.g.off), static_cast<uint32_t>(tok), &bad);
                if (bad) set_status(a.status, ECHO_ST_BADDATA);
            }
            const uint8_t* src[8];
            uint32_t live = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t r = __shfl_sync(0xffffffffu, mine, i4 + 4 * j);
                live |= (r >= 0 ? 1u : 0u) << j;
                src[j] = a.kv + (r < 0 ? 0 : r * kLatRowBytes) + 16 * x;
            }
            // a slot is free when the item before, the other set's, has left it: this set sees every phase of that
            // parity's barriers, each before the next can end
            for (int at = 0; at < kAtoms; ++at) {
                if (item >= 1)
                    ok = ok && mbar_wait_watch(smem_addr(&ctl->k_free[(item - 1) & 1][at]), static_cast<uint32_t>((item - 1) >> 1) & 1u,
                                         watch);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t dst = sK + static_cast<uint32_t>(at) * kSlot;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = 4 * w + i4 + 16 * j;
                    cp_async_16(dst + static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>((x ^ r) & 7) << 4), src[j] + at * 128,
                                (live >> j) & 1u ? 16u : 0u);
                }
                cp_async_arrive_noinc(smem_addr(&ctl->k_full[at]));
            }
            ++item;
        }
        if (!ok) give_up(watch);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 9) {
        // ---- Q: this CTA's half of a block's pairs
        Ring q;
        uint32_t filled = 0;
        bool ok = true;
        while (ok && walk.next(&p)) {
            for (int b = p.lo; ok && b < p.hi; ++b) {
                const int cb = p.g.cb0 + b, half = ((block_cols(p.g, a.heads, cb) + 31) & ~31) / 2;
                const int32_t y = static_cast<int32_t>(p.g.col0 + static_cast<int64_t>(cb) * kCols + c * half);
                for (int at = 0; at < kAtoms; ++at, q.step(kQSlots), ++filled) {
                    if (filled >= kQSlots && !mbar_wait_watch(smem_addr(&ctl->q_free[q.slot]), q.phase ^ 1u, watch)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t bar = smem_addr(&ctl->q_full[q.slot]);
                        mbar_arrive_expect_tx(bar, kSlot);
                        tma_load_2d(sQ + static_cast<uint32_t>(q.slot) * kSlot, &qmap, bar, at * 128, y);
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok && lane == 0) give_up(watch);
        // the loads in flight land before the CTA's memory goes
        for (int j = 0; j < kQSlots && !ok; ++j) {
            const int back = j + 1;
            if (filled >= static_cast<uint32_t>(back)) {
                const uint32_t f = filled - back;
                (void)mbar_wait_limit(smem_addr(&ctl->q_full[f % kQSlots]), (f / kQSlots) & 1u, nullptr, kWaitNs);
            }
        }
    } else if (warp == 8) {
        // ---- the MMAs of both CTAs, by one thread of CTA 0
        if (c == 0 && elect_one()) {
            Ring k, q;
            uint32_t d = 0, item = 0;
            bool ok = true;
            while (ok && walk.next(&p)) {
                const Ring k0 = k;
                const uint32_t parity = item & 1u;
                if (p.hi > p.lo) ++item;
                for (int b = p.lo; ok && b < p.hi; ++b, ++d) {
                    const int n = (block_cols(p.g, a.heads, p.g.cb0 + b) + 31) & ~31;
                    const uint32_t db = d & 1u, idesc = idesc_bf16_f32(256, static_cast<uint32_t>(n));
                    if (d >= 2 && !mbar_wait_cluster_watch(smem_addr(&ctl->d_free[db]), ((d >> 1) & 1u) ^ 1u, watch)) {
                        ok = false;
                        break;
                    }
                    k = k0;
                    for (int at = 0; at < kAtoms; ++at, k.step(kKSlots), q.step(kQSlots)) {
                        if (b == p.lo) ok = mbar_wait_cluster_watch(smem_addr(&ctl->k_ready[k.slot]), k.phase, watch);
                        ok = ok && mbar_wait_cluster_watch(smem_addr(&ctl->q_ready[q.slot]), q.phase, watch);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = sw128_kmajor_desc(sK + static_cast<uint32_t>(k.slot) * kSlot);
                        const uint64_t bd = sw128_kmajor_desc(sQ + static_cast<uint32_t>(q.slot) * kSlot);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma2_bf16(tmem + db * kCols, ad + ((kk * 32u) >> 4), bd + ((kk * 32u) >> 4), idesc,
                                      (at > 0 || kk > 0) ? 1u : 0u);
                        mma2_commit_both(smem_addr(&ctl->q_free[q.slot]));
                        if (b + 1 == p.hi) mma2_commit_both(smem_addr(&ctl->k_free[parity][k.slot]));
                        if (at + 1 == kAtoms) mma2_commit_both(smem_addr(&ctl->d_full[db]));
                    }
                }
            }
            if (!ok) {
                give_up(watch);
                mma2_commit_both(smem_addr(&ctl->drain));
                (void)mbar_wait_limit(smem_addr(&ctl->drain), 0, nullptr, kWaitNs);
            }
        }
        __syncwarp();
    } else if (warp == 10) {
        // ---- K has landed here
        Ring k;
        bool ok = true;
        while (ok && walk.next(&p)) {
            if (p.hi == p.lo) continue;
            for (int at = 0; ok && at < kAtoms; ++at, k.step(kKSlots)) {
                ok = mbar_wait_watch(smem_addr(&ctl->k_full[k.slot]), k.phase, watch);
                fence_proxy_async_smem();
                if (ok && lane == 0) mbar_arrive_remote(smem_addr(&ctl->k_ready[k.slot]), 0);
            }
        }
        if (!ok && lane == 0) give_up(watch);
    } else {  // warp 11
        // ---- Q has landed here
        Ring q;
        bool ok = true;
        while (ok && walk.next(&p)) {
            for (int i = 0; ok && i < (p.hi - p.lo) * kAtoms; ++i, q.step(kQSlots)) {
                ok = mbar_wait_watch(smem_addr(&ctl->q_full[q.slot]), q.phase, watch);
                if (ok && lane == 0) {
                    mbar_arrive_remote(smem_addr(&ctl->q_ready[q.slot]), 0);
                    watch_beat(watch);  // (the Q slots go round with the MMAs)
                }
            }
        }
        if (!ok && lane == 0) give_up(watch);
    }
    __syncthreads();
    pdl_launch_dependents();
    if (tid == 0 && gave_up(watch)) set_status(a.status, ECHO_ST_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 0) tmem_dealloc2(tmem, kTmemCols);
}

// Block i: share boundary i + 1, when it is the first inside an item's blocks; thread = token.
__global__ void __launch_bounds__(kTok) mass_join_kernel(Plan plan, const float* mass, float* mass_out, float decay) {
    __shared__ int s_item;
    pdl_wait();
    const int tid = threadIdx.x, i = blockIdx.x + 1;
    const PlanHead head = *plan.head;
    if (i >= head.parts) return;
    const int64_t u = share_start(head.total, head.parts, i);
    if (tid < 32) {
        const int g = find_group(plan.cum, head.items, u);
        if (tid == 0) s_item = g;
    }
    __syncthreads();
    const Item g = plan.item[s_item];
    const int64_t c = plan.cum[s_item];
    const int cut = blocks_before(u - c, g.nb);
    if (cut == 0 || cut == g.nb) return;  // not within its blocks
    const int64_t prev = share_start(head.total, head.parts, i - 1);
    if (prev > c && blocks_before(prev - c, g.nb) > 0) return;  // not the first cut
    float s = 0.f;
    for (int j = i - 1; j < head.parts; ++j) {
        const int64_t a = share_start(head.total, head.parts, j) - c;
        const int lo = a > 0 ? blocks_before(a, g.nb) : 0;
        if (lo == g.nb) break;
        if (blocks_before(share_start(head.total, head.parts, j + 1) - c, g.nb) > lo)
            s += plan.part[static_cast<size_t>(2 * j + (lo > 0 ? 0 : 1)) * kTok + tid];
    }
    if (g.tok0 + tid < g.len) {
        const int64_t at = g.off + g.tok0 + tid;
        mass_out[at] = (decay > 0.f ? decay * mass[at] : 0.f) + s;
    }
}

}  // namespace
}  // namespace echo

extern "C" size_t echo_mla_mass_workspace_size(int64_t n_tokens, int B) {
    using namespace echo;
    if (n_tokens < 0 || n_tokens > ECHO_MASS_MAX_TOKENS || B <= 0 || B > ECHO_MAX_REQUESTS) return 0;
    return plan_layout(n_tokens / kTok + B).total;
}

extern "C" int echo_mla_mass(int B, const int64_t* row_off, int64_t n_rows, int heads, const uint16_t* q,
                             const float* lse, const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens,
                             const echo_pages* pages, int64_t window, int64_t sinks, float scale, const float* mass,
                             float* mass_out, float decay, void* ws, size_t ws_bytes, int32_t* status,
                             echo_stream_t stream) {
    using namespace echo;
    const int rc = check_chunk(B, row_off, n_rows, heads, q, tok_off, n_tokens, pages, window, sinks, scale, status);
    if (rc) return rc;
    if (n_tokens > ECHO_MASS_MAX_TOKENS) return ECHO_EUNSUPPORTED;
    if (n_tokens == 0) return ECHO_OK;
    if ((n_rows > 0 && !lse) || !mass || !mass_out || !(decay >= 0.f) || decay > 3.4028234e38f) return ECHO_EINVAL;
    if (!ws || !is_aligned(ws, 256) || ws_bytes < echo_mla_mass_workspace_size(n_tokens, B)) return ECHO_EINVAL;
    const ChunkArgs a = chunk_args(B, row_off, n_rows, heads, q, tok_off, tok_end, n_tokens, pages, nullptr, 0, window,
                                   sinks, scale, status);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap qmap = {};
    if (n_rows > 0 && encode_tmap_bytes_2d(&qmap, q, kLatRowBytes, static_cast<uint64_t>(n_rows) * heads, 128, 128))
        return ECHO_ECUDA;
    static int cached[64];
    Plan plan;
    plan.clusters = cluster2_count(mass_kernel, kThreads, kSmem, kMaxClusters, cached);
    if (plan.clusters < 1) return ECHO_ECUDA;
    plan.cap = n_tokens / kTok + B;
    const Layout l = plan_layout(plan.cap);
    uint8_t* const w = static_cast<uint8_t*>(ws);
    plan.head = reinterpret_cast<PlanHead*>(w);
    plan.item = reinterpret_cast<Item*>(w + l.item);
    plan.cum = reinterpret_cast<int64_t*>(w + l.cum);
    plan.part = reinterpret_cast<float*>(w + l.part);
    ECHO_CUDA_OK(prefer_max_shared(mass_plan_kernel));
    ECHO_CUDA_OK(prefer_max_shared(mass_join_kernel));
    mass_plan_kernel<<<1, kPT, 0, s>>>(a, plan);
    ECHO_CUDA_OK(cudaGetLastError());
    ECHO_CUDA_OK(launch_after(false, mass_kernel, dim3(static_cast<unsigned>(2 * plan.clusters)), kThreads, kSmem, s, a, plan,
                              qmap, scale * 1.4426950408889634f, lse, mass, mass_out, decay));
    if (plan.clusters > 1)
        ECHO_CUDA_OK(launch_after(false, mass_join_kernel, dim3(static_cast<unsigned>(plan.clusters - 1)), kTok, 0, s, plan, mass,
                                  mass_out, decay));
    return ECHO_OK;
}
