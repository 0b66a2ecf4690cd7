// echo_chunk.cuh -- what the kernels of attention over a paged latent cache share: the groups of
// rows and their shares, the walk through a share, the look-up of a tile's tokens, the results'
// way out and the join of cut groups.  kTok: tokens of a tile, the unit of the shares.
#pragma once

#include "echo_paged.cuh"
#include "echo_tc.cuh"

namespace echo {

namespace {

constexpr int kM = 128;                  // (row, head) pairs per group
constexpr int kInline = 32;              // groups and requests of a call that needs no plan kernel (at most a warp's lanes)
constexpr int kMaxClusters = 96;         // bounds the workspace (the device has 76 pairs of SMs)
template <int kTok>
constexpr int kOver = 192 / kTok + (192 % kTok != 0);  // a group's fixed cost in tiles
// Tiles after which O leaves the tensor memory and is added to what the legs before left, in fp32 and rounded: the
// MMAs' accumulation cuts low bits off, so that a sum over n tiles of 64 tokens comes out n * 3e-7 too near to zero (values of one
// sign: 1.7e-4 after 512 of them, 6.5e-3 after 16384 in one leg).  With 1M tokens a leg of 512 costs 0 to 2% of the time
// (152 rows: 29.0 ms in one leg, 29.0 to 29.9 ms in legs of 256 to 2048 tiles).
template <int kTok>
constexpr int kLeg = 512 * 64 / kTok;
constexpr size_t kPartO = static_cast<size_t>(kM) * kLatDv * 4;
constexpr size_t kPartBytes = kPartO + 3 * kM * 4;  // O, maxima, sums, factors of a leg

// One group: what its rows see is v in [0, nv): token v for v < kept, else v - kept + lo
// with lo = pos0 + rows + kept - nv (the union over its rows); with selections
// nv = k entries of its row's list, and kept holds the request's length; with trees
// kept = lo = the first token of the request's tree, so that v is the token.
struct __align__(16) Group {
    int64_t off;    // the request's first token row
    int32_t row0;   // first row
    int32_t req;
    int32_t pos0;   // position of row0
    int32_t rows;
    int32_t kept;
    int32_t nv;
};

struct __align__(16) PlanHead {
    int64_t total;  // units
    int32_t groups;
    int32_t parts;  // clusters that take a share
};

// A group that more than one share holds a part of: shares i0 .. i0 + n - 1.
struct __align__(16) Cut {
    int32_t n, i0, row0, live;  // live: its (row, head) pairs
};

struct Plan {
    PlanHead* head;
    Cut* cut;       // [kMaxClusters] by the second of its shares; n = 0: none
    Group* group;   // [cap]
    int64_t* cum;   // [cap + 1] units before each group
    uint8_t* part;  // [2 * kMaxClusters] partial results
    int cap;
    int clusters;
    bool small;     // at most kInline groups and requests: no plan kernel
    int least;      // units per cluster
    int ahead;      // tiles that K rows are brought to L2 ahead of their copy, 0: not (a tree's: not 0, the next tile's)
};

__host__ __device__ __forceinline__ int rows_per_group(int heads, bool sel) { return sel ? 1 : kM / heads; }

struct Layout {
    size_t group, cum, part, total;
};
inline Layout plan_layout(int64_t cap) {
    Layout l;
    l.group = 256 + round_up(kMaxClusters * sizeof(Cut), 256);
    l.cum = round_up(l.group + static_cast<size_t>(cap) * sizeof(Group), 256);
    l.part = round_up(l.cum + static_cast<size_t>(cap + 1) * 8, 256);
    l.total = l.part + 2 * kMaxClusters * kPartBytes;
    return l;
}
// Groups a call may have: each has a row, and at most one of a request is not full.
inline int64_t plan_cap(int64_t n_rows, int heads, int B, bool sel) {
    const int64_t full = n_rows / rows_per_group(heads, sel) + B;
    return full < n_rows ? full : n_rows;
}

template <int kTok>
__device__ __forceinline__ int tiles_of(int nv) { return (nv + kTok - 1) / kTok; }

// ---------------------------------------------------------------- plan
constexpr int kPT = 1024;

// Rows [i0, i0 + per) of request b, whose rows are [r0, r0 + n) and token rows [off, off + len).
__device__ __forceinline__ Group make_group(const ChunkArgs& a, int b, int64_t r0, int64_t n, int64_t off, int64_t len,
                                            int64_t i0, int per) {
    Group r;
    r.off = off;
    r.row0 = static_cast<int32_t>(r0 + i0);
    r.req = b;
    r.rows = static_cast<int32_t>(min(static_cast<int64_t>(per), n - i0));
    r.pos0 = 0;
    r.kept = 0;
    r.nv = 0;
    if (len > 0) {
        const int64_t p0 = len - n + i0, p1 = p0 + r.rows - 1;
        r.pos0 = static_cast<int32_t>(p0);
        if (a.sel) {
            r.kept = static_cast<int32_t>(len);
            r.nv = a.k;
        } else if (a.mask) {
            r.kept = static_cast<int32_t>(len - n);
            r.nv = static_cast<int32_t>(p1 + 1);
        } else {
            const int64_t lo = a.window ? max(static_cast<int64_t>(0), p0 - a.window + 1) : 0;
            r.kept = static_cast<int32_t>(min(a.sinks, lo));
            r.nv = static_cast<int32_t>(r.kept + p1 + 1 - lo);
        }
    }
    return r;
}

__device__ __forceinline__ PlanHead make_head(int64_t total, int groups, const Plan& plan) {
    PlanHead h;
    h.total = total;
    h.groups = groups;
    h.parts =
        static_cast<int32_t>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(plan.clusters), total / plan.least)));
    return h;
}

// The plan of a small call by one warp: lane = request, then lane = group.
template <int kTok>
__device__ __forceinline__ void plan_small(const ChunkArgs& a, const Plan& plan, PlanHead* head, Group* group,
                                           int64_t* cum) {
    const int lane = threadIdx.x & 31, per = rows_per_group(a.heads, a.sel != nullptr);
    int64_t r0 = 0, n = 0, off = 0, len = 0;
    if (lane < a.B) chunk_request(a, lane, &r0, &n, &off, &len);
    const int mine = static_cast<int>((n + per - 1) / per);
    int end = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += y;
    }
    int groups = __shfl_sync(0xffffffffu, end, 31);
    if (groups > plan.cap) {  // row ranges that overlap
        if (lane == 0) set_status(a.status, ECHO_ST_BADDATA);
        groups = plan.cap;
    }
    // lane's group is that request's whose first group is the last at or before it
    int* const first = reinterpret_cast<int*>(cum);
    first[lane] = 0;
    __syncwarp();
    if (mine > 0 && end - mine < 32) first[end - mine] = lane;
    __syncwarp();
    int b = first[lane];
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) b = max(b, y);
    }
    const int64_t gr0 = __shfl_sync(0xffffffffu, r0, b), gn = __shfl_sync(0xffffffffu, n, b);
    const int64_t goff = __shfl_sync(0xffffffffu, off, b), glen = __shfl_sync(0xffffffffu, len, b);
    const int gfirst = __shfl_sync(0xffffffffu, end - mine, b);
    int64_t cost = 0;
    if (lane < groups) {
        const Group g = make_group(a, b, gr0, gn, goff, glen, static_cast<int64_t>(lane - gfirst) * per, per);
        group[lane] = g;
        cost = kOver<kTok> + tiles_of<kTok>(g.nv);
    }
    int64_t at = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += y;
    }
    const int64_t total = __shfl_sync(0xffffffffu, at, 31);
    if (lane < groups) cum[lane] = at - cost;
    if (lane == 0) {
        cum[groups] = total;
        *head = make_head(total, groups, plan);
    }
}

// One block: the groups of every request in order, with their costs summed.
template <int kTok>
__global__ void __launch_bounds__(kPT) chunk_plan_kernel(ChunkArgs a, Plan plan) {
    __shared__ uint32_t goff[ECHO_MAX_REQUESTS + 1];
    __shared__ uint32_t scratch[kPT / 32 + 1];
    __shared__ int64_t scratch64[kPT / 32];
    pdl_launch_dependents();
    pdl_wait();  // a tree's plan is scheduled beside the kernel before it, whatever that reads and writes
    const int tid = threadIdx.x;
    const int per = rows_per_group(a.heads, a.sel != nullptr);
    uint32_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPT) {
        const int b = b0 + tid;
        int64_t r0 = 0, n = 0, off, len;
        if (b < a.B) chunk_request(a, b, &r0, &n, &off, &len);
        uint32_t total;
        const uint32_t at = block_exclusive_scan<kPT>(static_cast<uint32_t>((n + per - 1) / per), scratch, &total);
        if (b < a.B) goff[b] = min(base + at, static_cast<uint32_t>(plan.cap));
        base += total;
        if (base > static_cast<uint32_t>(plan.cap)) {  // row ranges that overlap
            if (tid == 0) set_status(a.status, ECHO_ST_BADDATA);
            base = static_cast<uint32_t>(plan.cap);
        }
    }
    if (tid == 0) goff[a.B] = base;
    __syncthreads();
    const int groups = static_cast<int>(base);
    int64_t sum = 0;
    for (int g0 = 0; g0 < groups; g0 += kPT) {
        const int g = g0 + tid;
        int64_t cost = 0;
        if (g < groups) {
            int b = 0, e = a.B;  // the last request whose groups start at or before g
            while (e - b > 1) {
                const int mid = (b + e) >> 1;
                if (goff[mid] <= static_cast<uint32_t>(g)) b = mid;
                else e = mid;
            }
            int64_t r0, n, off, len;
            chunk_request(a, b, &r0, &n, &off, &len);
            const int64_t i0 = static_cast<int64_t>(g - goff[b]) * per;
            const Group r = make_group(a, b, r0, n, off, len, i0, per);
            plan.group[g] = r;
            cost = kOver<kTok> + tiles_of<kTok>(r.nv);
        }
        int64_t total;
        const int64_t at = sum + block_scan64<kPT>(cost, scratch64, &total);
        if (g < groups) plan.cum[g] = at;
        sum += total;
    }
    if (tid == 0) {
        plan.cum[groups] = sum;
        *plan.head = make_head(sum, groups, plan);
    }
}

// The plan of a small call by a kernel of one warp.
template <int kTok>
__global__ void __launch_bounds__(32) chunk_plan_small_kernel(ChunkArgs a, Plan plan) {
    __shared__ int64_t cum[kInline + 1];
    pdl_launch_dependents();
    pdl_wait();
    plan_small<kTok>(a, plan, plan.head, plan.group, cum);
    __syncwarp();
    const int lane = threadIdx.x, groups = plan.head->groups;
    if (lane <= groups) plan.cum[lane] = cum[lane];
    if (lane == 0 && groups == 32) plan.cum[32] = cum[32];
}

// A leg, at most kLeg<kTok> tiles, of the part of a group that a share holds (a piece): tiles [lo, hi) of `tiles`.
struct Piece {
    Group g;
    int lo, hi, tiles;
    bool left, right;  // the piece starts behind the group's first tile, ends before its last
    bool later, last;  // legs of the piece come before this one, none after it
};

// Walks the legs of a share's pieces; every role of the cluster sees the same ones.
template <int kTok>
struct Walk {
    const Group* group;
    const int64_t* cum;
    int64_t u0, u1;
    int g;
    bool on = false;  // legs of the piece are left
    // False when the share is done.  Groups that see nothing come with tiles = 0.
    __device__ __forceinline__ bool next(Piece* p) {
        for (;;) {
            if (u0 >= u1) return false;
            const int64_t c = cum[g];
            p->g = group[g];
            p->tiles = tiles_of<kTok>(p->g.nv);
            const int64_t a = u0 - c, b = min(u1 - c, static_cast<int64_t>(kOver<kTok> + p->tiles));
            p->lo = static_cast<int>(max(static_cast<int64_t>(0), a - kOver<kTok>));
            const int to = static_cast<int>(max(static_cast<int64_t>(0), b - kOver<kTok>));
            p->hi = min(to, p->lo + kLeg<kTok>);
            p->last = p->hi == to;
            p->later = on;
            if (!on) p->left = p->lo > 0;
            p->right = to < p->tiles;
            on = !p->last;
            u0 = c + kOver<kTok> + (on ? p->hi : p->tiles);
            g += on ? 0 : 1;
            if (p->hi > p->lo || (p->tiles == 0 && a <= 0)) return true;
        }
    }
};

// Whether share ci, which walk is at the start of, starts the second part of a group; n: its parts.
template <int kTok>
__device__ __forceinline__ Cut cut_of(const Walk<kTok>& walk, const PlanHead& head, int ci, int heads) {
    Cut cut = {0, 0, 0, 0};
    if (walk.u0 < walk.u1) {
        const Group gr = walk.group[walk.g];
        const int64_t at = walk.cum[walk.g];
        cut = Cut{0, ci - 1, gr.row0, gr.rows * heads};
        if (walk.u0 > at + kOver<kTok> && share_start(head.total, head.parts, ci - 1) <= at + kOver<kTok>)
            cut.n = share_of(head.total, head.parts, at + kOver<kTok> + tiles_of<kTok>(gr.nv) - 1) - cut.i0 + 1;
    }
    return cut;
}

// One token of every tile of a piece, looked up ahead of its copy: the list entry
// (selections) of two tiles ahead and the table entry of the next tile are in flight
// while this tile's rows are copied.
template <int kTok>
struct Gather {
    const int32_t* sel;  // the row's list, null: causal or window
    PageView pv;
    int lo_tok;
    int v;               // index of the token whose table entry is in flight
    int last;            // index at which the piece ends
    int tok;             // token of the tile after it, -1: none
    int32_t entry;       // table entry in flight, < 0: none
    uint32_t at;         // offset in that page
    bool bad;
    __device__ __forceinline__ int token(const Piece& p, int x) const {
        if (x >= p.g.nv) return -1;
        if (sel) return sel[x];
        return x < p.g.kept ? x : x - p.g.kept + lo_tok;
    }
    __device__ __forceinline__ void look(const ChunkArgs& a, const Piece& p, int t) {
        entry = -1;
        if (sel && t >= p.g.kept) {  // past the request's end
            bad = true;
            t = -1;
        }
        if (t >= 0) entry = pv.tab[page_of(a, pv, static_cast<uint32_t>(t), &at)];
    }
    // r: token within the tile; ahead: tiles to start past the piece's first.
    __device__ __forceinline__ void start(const ChunkArgs& a, const Piece& p, int r, int ahead = 0) {
        sel = a.sel ? a.sel + static_cast<int64_t>(p.g.row0) * a.k : nullptr;
        pv = page_view(a, p.g.req, p.g.off);
        lo_tok = p.g.pos0 + p.g.rows + p.g.kept - p.g.nv;
        bad = false;
        at = 0;
        const int64_t first = static_cast<int64_t>(p.lo + ahead) * kTok + r, end = static_cast<int64_t>(p.hi) * kTok;
        last = static_cast<int>(end);
        v = static_cast<int>(min(first, end));  // at the end: nothing to look up any more
        const int t0 = v < end ? token(p, v) : -1;
        tok = v < end - kTok ? token(p, v + kTok) : -1;
        look(a, p, t0);
    }
    // The cache row of the current tile's token, -1 when it has none.
    __device__ __forceinline__ int64_t row(const ChunkArgs& a) {
        int64_t r = entry < 0 ? -1 : page_row(a, pv, entry, at, &bad);
        if (bad) set_status(a.status, ECHO_ST_BADDATA);
        bad = false;
        return r;
    }
    __device__ __forceinline__ void next(const ChunkArgs& a, const Piece& p) {
        const int t = tok;
        v = min(v + kTok, last);
        tok = v < last - kTok ? token(p, v + kTok) : -1;
        look(a, p, t);
    }
};

// Where a piece's part goes.  A share's first piece may be cut on its left, its last on its right; the legs of a
// whole piece meet in the last one's place, which is written after it.
__device__ __forceinline__ uint8_t* part_of(const Plan& plan, int ci, const Piece& p) {
    return plan.part + static_cast<size_t>(2 * ci + (p.left ? 0 : 1)) * kPartBytes;
}

// 4 x 4 transposition among the four lanes of a quad: lane q's w[j] becomes lane j's w[q].
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int q) {
    const bool odd = q & 1, high = q & 2;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? w[i] : w[i + 1], 1);
        if (odd) w[i] = x;
        else w[i + 1] = x;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = __shfl_xor_sync(0xffffffffu, high ? w[i] : w[i + 2], 2);
        if (high) w[i] = x;
        else w[i + 2] = x;
    }
}

// A warp's 32 rows x 256 dims of O (or kDims of them, from dim x0 on), times f (a factor for each of a lane's rows), as bf16
// to dst or, where that is null, in fp32 to part; kLater: what the legs before left in part, by this thread, times fb is
// added first.
template <bool kLater, uint32_t kDims = 256>
__device__ __forceinline__ void store_o(uint32_t taddr, const float (&f)[4], const float (&fb)[4], uint8_t* dst, uint8_t* part,
                                        int live, uint32_t x0 = 0) {
    const int lane = threadIdx.x & 31, q = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll 1
        for (uint32_t x = x0; x < x0 + kDims; x += 32u) {
            float2 was[8];
            if constexpr (kLater) {
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int r = 16 * h + 8 * g + (lane >> 2);
                        was[4 * g + b] = make_float2(0.f, 0.f);
                        if (r < live)
                            was[4 * g + b] = *reinterpret_cast<const float2*>(part + static_cast<int64_t>(r) * (kLatDv * 4) + 4 * x + 32 * b + 8 * q);
                    }
            }
            float o[16];
            tmem_ld_16x256_x4(taddr + (static_cast<uint32_t>(16 * h) << 16) + x, o);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int r = 16 * h + 8 * g + (lane >> 2);
                float ff = f[2 * h + g];
                if constexpr (kLater) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        o[4 * b + 2 * g] = fmaf(was[4 * g + b].x, fb[2 * h + g], o[4 * b + 2 * g] * ff);
                        o[4 * b + 2 * g + 1] = fmaf(was[4 * g + b].y, fb[2 * h + g], o[4 * b + 2 * g + 1] * ff);
                    }
                    ff = 1.f;
                }
                if (dst) {
                    uint32_t w[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[4 * b + 2 * g] * ff, o[4 * b + 2 * g + 1] * ff);
                        w[b] = *reinterpret_cast<const uint32_t*>(&b2);
                    }
                    quad_transpose(w, q);  // lane q now has columns 8q .. 8q + 7 of the 32
                    if (r < live)
                        *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(r) * (kLatDv * 2) + 2 * x + 16 * q) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                } else if (r < live) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        *reinterpret_cast<float2*>(part + static_cast<int64_t>(r) * (kLatDv * 4) + 4 * x + 32 * b + 8 * q) =
                            make_float2(o[4 * b + 2 * g], o[4 * b + 2 * g + 1]);
                }
            }
        }
}

// Barrier over the softmax warps, kThreads threads; true when any of them votes so.
template <int kThreads>
__device__ __forceinline__ bool softmax_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v)), "n"(kThreads)
        : "memory");
    return r != 0;
}

// ---------------------------------------------------------------- join
constexpr int kJT = 128;
constexpr int kJLanes = (kMaxClusters + 31) / 32;

// One (row, head) pair of a cut group: this warp's dims 4 (first + 32 i) of it, i < NV, lane = piece for the
// pieces' weights, the loads of the first pieces in flight meanwhile.
template <int NV>
__device__ __forceinline__ void join_pair(const Plan& plan, const Cut& x, int mi, int first, int heads, uint16_t* out,
                                          float* lse) {
    constexpr int kBatch = 8 / NV;  // pieces in flight
    const int lane = threadIdx.x & 31;
    // piece j is share i0 + j: the first starts at tile 0 (second slot), the others within (first slot)
    const auto part = [&](int j) { return plan.part + static_cast<size_t>(2 * (x.i0 + j) + (j == 0 ? 1 : 0)) * kPartBytes; };
    float4 v[kBatch][NV];
    const auto load = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[j][i] = j0 + j < x.n ? reinterpret_cast<const float4*>(part(j0 + j))[mi * (kLatDv / 4) + first + 32 * i]
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    float w[kJLanes], l[kJLanes];
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kJLanes; ++i) {
        const int j = 32 * i + lane;
        w[i] = -INFINITY;
        l[i] = 0.f;
        if (j < x.n) {
            const float* ml = reinterpret_cast<const float*>(part(j) + kPartO);
            w[i] = ml[mi];
            l[i] = ml[kM + mi];
        }
        M = fmaxf(M, w[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
#pragma unroll
    for (int i = 0; i < kJLanes; ++i) {
        w[i] = M == -INFINITY ? 0.f : exp2f(w[i] - M);
        L += w[i] * l[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float4 s[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < x.n; j0 += kBatch) {
        if (j0 > 0) load(j0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int at = j0 + j;
            float wj = __shfl_sync(0xffffffffu, w[0], at & 31);
#pragma unroll
            for (int i = 1; i < kJLanes; ++i) {
                const float o = __shfl_sync(0xffffffffu, w[i], at & 31);
                if (at >= 32 * i) wj = o;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                s[i].x += wj * v[j][i].x;
                s[i].y += wj * v[j][i].y;
                s[i].z += wj * v[j][i].z;
                s[i].w += wj * v[j][i].w;
            }
        }
    }
    const bool any = L != 0.f;
    const float f = any ? 1.f / L : 0.f;
    const int64_t at = static_cast<int64_t>(x.row0) * heads + mi;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const __nv_bfloat162 b0 = __floats2bfloat162_rn(any ? s[i].x * f : 0.f, any ? s[i].y * f : 0.f);
        const __nv_bfloat162 b1 = __floats2bfloat162_rn(any ? s[i].z * f : 0.f, any ? s[i].w * f : 0.f);
        reinterpret_cast<uint2*>(out + at * kLatDv)[first + 32 * i] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
    }
    if (first == 0) lse[at] = any ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
}

// Many pairs: a warp to each.  Few (long contexts cut into many pieces): the four warps of a block share one.
__global__ void __launch_bounds__(kJT) chunk_join_kernel(ChunkArgs a, Plan plan, uint16_t* __restrict__ out,
                                                         float* __restrict__ lse) {
    __shared__ Cut s_cut[kMaxClusters];
    __shared__ int s_n;
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < 32) {
        int n = 0;
        for (int i0 = 1; i0 < plan.clusters; i0 += 32) {
            const int i = i0 + lane;
            Cut x = {0, 0, 0, 0};
            if (i < plan.clusters) x = plan.cut[i];
            const uint32_t m = __ballot_sync(0xffffffffu, x.n > 0);
            if (x.n > 0) s_cut[n + __popc(m & ((1u << lane) - 1u))] = x;
            n += __popc(m);
        }
        if (lane == 0) s_n = n;
    }
    __syncthreads();
    const int pairs = s_n * kM;
    if (pairs <= static_cast<int>(gridDim.x)) {
        for (int task = blockIdx.x; task < pairs; task += gridDim.x) {
            const Cut x = s_cut[task / kM];
            if (task % kM < x.live) join_pair<1>(plan, x, task % kM, tid, a.heads, out, lse);
        }
    } else {
        for (int task = 4 * blockIdx.x + (tid >> 5); task < pairs; task += 4 * gridDim.x) {
            const Cut x = s_cut[task / kM];
            if (task % kM < x.live) join_pair<4>(plan, x, task % kM, lane, a.heads, out, lse);
        }
    }
}


// The plan of a call in its workspace.  groups: the most there may be.
inline Plan plan_in(void* ws, int64_t groups) {
    const Layout l = plan_layout(groups);
    uint8_t* const w = static_cast<uint8_t*>(ws);
    Plan plan;
    plan.head = reinterpret_cast<PlanHead*>(w);
    plan.cut = reinterpret_cast<Cut*>(w + 256);
    plan.group = reinterpret_cast<Group*>(w + l.group);
    plan.cum = reinterpret_cast<int64_t*>(w + l.cum);
    plan.part = w + l.part;
    plan.cap = static_cast<int>(groups);
    return plan;
}

}  // namespace
}  // namespace echo
