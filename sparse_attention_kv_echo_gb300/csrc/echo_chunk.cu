// echo_chunk.cu -- attention of a chunk of new tokens over a paged latent cache.
//
// Per row r and head h, over the tokens t the row sees (echo.h, echo_mla_chunk):
//   s_t = scale * q[r,h] . kv[t]  (576 dims),  out = softmax(s) . kv[t][0:512].
//
// A group is 128 / heads consecutive rows of a request (one row of 128 heads),
// so that (row, head) fill the 128 rows of an MMA; the group walks the tokens
// any of its rows sees, 64 at a time, with the running maximum and sum of a
// softmax per (row, head).  A cluster of two CTAs works on a group: 128 (row, head)
// accumulators of 512 dims are all of one SM's 512 TMEM columns and would leave no
// room for the scores, two SMs hold 256 columns each.  In a cta_group::2 MMA
// with M = 128, CTA c has rows [64c, 64c + 64) and TMEM lanes 0-63 / 64-127
// hold the first / second half of the N columns:
//   S = Q K^T   N = 64 tokens, K = 576 in 36 steps: 32 columns, lane = (token half,
//               row); CTA c supplies Q of its rows and the K rows of its 32 tokens;
//   O += P V    N = 512 dims in two MMAs of 256, K = 64 tokens in 4 steps: 256
//               columns, lane = (dim half, row); CTA c supplies P of its rows and
//               dims [256c, 256c + 256) of all 64 tokens, read in place as an
//               MN-major operand.
// Neither product is done twice, and the softmax needs nothing from the other
// CTA.  Warps of a CTA: 0-3 softmax (thread = TMEM lane; the two threads of a row
// exchange their tile maxima in shared memory), 4-7 gather K, 8-11 gather V
// (16-byte cp.async: any row for any token; two stages of each), 12 and 13 of CTA 0
// issue the MMAs of QK and of PV, 14 loads Q by TMA, 14 and 15 report what has
// landed in their CTA to CTA 0, 16-19 store O.  There are four S buffers and two of P, so QK runs up
// to four tiles ahead and the softmax under the tensor cores.  Its reference moves
// only when a score exceeds it by more than 2^8 (P <= 256 in bf16, exact after the
// final division); O in TMEM is rescaled then.
//
// What bounds it: an MMA of QK reads 3 KB of shared memory for 16 cycles of
// products and takes 25, one of PV 6 KB for 64 (rates of single MMAs); a tile's 36 + 8
// come to 1421 cycles, 2.47 ms of the 2.81 ms of 2048 rows over 8192 tokens at the 1747 MHz
// (median) that the power cap leaves in repeated calls.  More tokens to
// a tile would help QK and do not fit: Q 72 KB, two stages of K 36 KB and V 32 KB,
// P 16 KB.  Left out for a measurement, the copies give 7% and the exponentials 5%;
// a group's change costs 3000 cycles (Q can only be replaced when its last QK is done).
// Decode is bound by the same loop and by its ends: the first loads, the parts' 256 KB
// a piece and their join.
//
// Work: every tile costs the same and a group costs kOver tiles more (its Q, its
// result).  chunk_plan_kernel lays the groups' costs in a row; cluster i takes the
// units [T i / n, T (i + 1) / n) of it, whatever groups those cut, so ragged
// batches, single long requests and whole prompts load all SMs alike.  The parts
// of a cut group go to the workspace in fp32 with their maximum and sum, and
// chunk_join_kernel adds them in order (the same bits every time).  A part of more than
// kLeg tiles is walked in legs, added up in its place in the workspace.
#include "echo_paged.cuh"
#include "echo_tc.cuh"

namespace echo {
namespace {

constexpr int kTok = 64;                 // tokens per tile
constexpr int kM = 128;                  // (row, head) pairs per group
constexpr int kThreads = 640;
constexpr int kSoftmax = 128, kLoad = 128;
constexpr int kAtoms = kLatDqk / 64;     // 9 swizzle atoms of 64 dims
constexpr uint32_t kQAtom = 64 * 128;    // 64 rows x 128 B
constexpr uint32_t kKAtom = 32 * 128;    // this CTA's 32 tokens
constexpr uint32_t kVAtom = kTok * 128;  // 64 tokens x 64 dims
constexpr uint32_t kQBytes = kAtoms * kQAtom;
constexpr uint32_t kKBytes = kAtoms * kKAtom;
constexpr uint32_t kVBytes = 4 * kVAtom;
constexpr uint32_t kPBytes = 64 * 128;
constexpr uint32_t kTmemCols = 512;      // O [0, 256) | S buffers of 32 columns
constexpr int kSBufs = 4;                // two would hold QK of tile t up until P of tile t - 2 is written
constexpr uint32_t kSCol = 256;
// Tokens that one or two groups read come from memory, whose latency two stages do not cover:
// their rows are brought to L2 this many tiles ahead of the copy (32 ragged decode rows 72 -> 67 us).
// Tokens that many groups read are in L2 already (2048 rows of 8192 tokens 3015 -> 3087 us with it).
constexpr int kAhead = 1;
constexpr int kInline = 32;              // groups and requests of a call that needs no plan kernel (at most a warp's lanes)
constexpr float kLazy = 8.f;
constexpr int kOver = 3;                 // a group's fixed cost in tiles
constexpr int kMinUnits = 2;             // least units per cluster
constexpr int kMaxClusters = 96;         // bounds the workspace (the device has 76 pairs of SMs)
constexpr uint32_t kIdescS = idesc_bf16_f32(kM, kTok);
constexpr uint32_t kIdescO = idesc_bf16_f32(kM, 256) | (1u << 16);  // B (V) MN-major
// Tiles after which O leaves the tensor memory and is added to what the legs before left, in fp32 and rounded: the
// MMAs' accumulation cuts low bits off, so that a sum over n tiles comes out n * 3e-7 too near to zero (values of one
// sign: 1.7e-4 after 512 tiles, 6.5e-3 after 16384 in one leg).  With 1M tokens a leg of 512 costs 0 to 2% of the time
// (152 rows: 29.0 ms in one leg, 29.0 to 29.9 ms in legs of 256 to 2048 tiles).
constexpr int kLeg = 512;
constexpr size_t kPartO = static_cast<size_t>(kM) * kLatDv * 4;
constexpr size_t kPartBytes = kPartO + 3 * kM * 4;  // O, maxima, sums, factors of a leg

// One group: what its rows see is v in [0, nv): token v for v < kept, else v - kept + lo
// with lo = pos0 + rows + kept - nv (the union over its rows); with selections
// nv = k entries of its row's list, and kept holds the request's length.
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
    int ahead;      // tiles that K rows are brought to L2 ahead of their copy, 0: not
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
        } else {
            const int64_t lo = a.window ? max(static_cast<int64_t>(0), p0 - a.window + 1) : 0;
            r.kept = static_cast<int32_t>(min(a.sinks, lo));
            r.nv = static_cast<int32_t>(r.kept + p1 + 1 - lo);
        }
    }
    return r;
}

__device__ __forceinline__ PlanHead make_head(int64_t total, int groups, int clusters) {
    PlanHead h;
    h.total = total;
    h.groups = groups;
    h.parts =
        static_cast<int32_t>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(clusters), total / kMinUnits)));
    return h;
}

// The plan of a small call by one warp: lane = request, then lane = group.
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
        cost = kOver + tiles_of(g.nv);
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
        *head = make_head(total, groups, plan.clusters);
    }
}

// One block: the groups of every request in order, with their costs summed.
__global__ void __launch_bounds__(kPT) chunk_plan_kernel(ChunkArgs a, Plan plan) {
    __shared__ uint32_t goff[ECHO_MAX_REQUESTS + 1];
    __shared__ uint32_t scratch[kPT / 32 + 1];
    __shared__ int64_t scratch64[kPT / 32];
    pdl_launch_dependents();
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
            cost = kOver + tiles_of(r.nv);
        }
        int64_t total;
        const int64_t at = sum + block_scan64<kPT>(cost, scratch64, &total);
        if (g < groups) plan.cum[g] = at;
        sum += total;
    }
    if (tid == 0) {
        plan.cum[groups] = sum;
        *plan.head = make_head(sum, groups, plan.clusters);
    }
}

// A leg, at most kLeg tiles, of the part of a group that a share holds (a piece): tiles [lo, hi) of `tiles`.
struct Piece {
    Group g;
    int lo, hi, tiles;
    bool left, right;  // the piece starts behind the group's first tile, ends before its last
    bool later, last;  // legs of the piece come before this one, none after it
};

// Walks the legs of a share's pieces; every role of the cluster sees the same ones.
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
            p->tiles = tiles_of(p->g.nv);
            const int64_t a = u0 - c, b = min(u1 - c, static_cast<int64_t>(kOver + p->tiles));
            p->lo = static_cast<int>(max(static_cast<int64_t>(0), a - kOver));
            const int to = static_cast<int>(max(static_cast<int64_t>(0), b - kOver));
            p->hi = min(to, p->lo + kLeg);
            p->last = p->hi == to;
            p->later = on;
            if (!on) p->left = p->lo > 0;
            p->right = to < p->tiles;
            on = !p->last;
            u0 = c + kOver + (on ? p->hi : p->tiles);
            g += on ? 0 : 1;
            if (p->hi > p->lo || (p->tiles == 0 && a <= 0)) return true;
        }
    }
};

// One token of every tile of a piece, looked up ahead of its copy: the list entry
// (selections) of two tiles ahead and the table entry of the next tile are in flight
// while this tile's rows are copied.
struct Gather {
    const int32_t* sel;  // the row's list, null: causal or window
    PageView pv;
    int lo_tok;
    int v;               // index of the token whose table entry is in flight
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
        const int t = tok, end = p.hi * kTok;
        v = min(v + kTok, end);
        tok = v < end - kTok ? token(p, v + kTok) : -1;
        look(a, p, t);
    }
};

// Where a piece's part goes.  A share's first piece may be cut on its left, its last on its right; the legs of a
// whole piece meet in the last one's place, which is written after it.
__device__ __forceinline__ uint8_t* part_of(const Plan& plan, int ci, const Piece& p) {
    return plan.part + static_cast<size_t>(2 * ci + (p.left ? 0 : 1)) * kPartBytes;
}

// ---------------------------------------------------------------- attention
constexpr int kValid = 8;
static_assert(kValid >= kSBufs + 3, "valid flags");

struct Ctl {
    // here: landed in this CTA; the *_ready barriers of CTA 0: landed in both
    uint64_t q_full, q_ready;                            // Q of a group
    uint64_t k_full[2], k_ready[2];                      // K of a stage
    uint64_t k_free[2];                                  // its MMAs are done
    uint64_t v_full[2];                                  // V of a stage
    uint64_t pv_ready[2];                                // V, and P of the tile, in both CTAs
    uint64_t pv_done[2];                                 // P V of a tile done: V stage and P buffer free, O ready
    uint64_t s_full[kSBufs];                             // S of a tile done
    uint64_t s_free[kSBufs];                             // S of a tile has been read in both CTAs
    uint64_t drain[2];
    uint32_t tmem;
    Watch watch;
    int first;                                           // the share's first group
    float mx[2][2][64];                                  // tile maxima, or a piece's sums, by (parity, token half, row)
    // few groups: the plan, made by every CTA for itself
    PlanHead head;
    Group group[kInline];
    int64_t cum[kInline + 1];
    uint64_t fin_ready, fin_free;                        // a piece's factors are in fin / have been read
    uint64_t o_free;                                     // O of a piece has been read in both CTAs
    float fin[64];                                       // what O of a row is multiplied by
    // tokens of a tile that have a row, a bit each: written for tile t when QK of t - 2 is done, hence S of t - 6
    // read and tile t - 7 finished
    uint32_t valid[kValid][2];
};
constexpr uint32_t kSmem = kQBytes + 2 * kKBytes + 2 * kVBytes + 2 * kPBytes + ((sizeof(Ctl) + 15u) & ~15u);
static_assert(kSmem <= 227u * 1024u, "chunk shared memory");

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

// A warp's 32 rows x 256 dims of O, times f (a factor for each of a lane's rows), as bf16 to dst or, where that is
// null, in fp32 to part; kLater: what the legs before left in part, by this thread, times fb is added first.
template <bool kLater>
__device__ __forceinline__ void store_o(uint32_t taddr, const float (&f)[4], const float (&fb)[4], uint8_t* dst, uint8_t* part,
                                        int live) {
    const int lane = threadIdx.x & 31, q = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll 1
        for (uint32_t x = 0; x < 256u; x += 32u) {
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

// Barrier over the softmax warps; true when any thread votes so.
__device__ __forceinline__ bool softmax_sync_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v))
        : "memory");
    return r != 0;
}

// The MMAs of stage ST.  The stage is a constant so that every descriptor is one too: with
// descriptors computed from a variable stage an MMA took 100 cycles to issue, four times what it runs.
template <int ST>
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t sQ, uint32_t sK) {
    const uint64_t ad = sw128_kmajor_desc(sQ), bd = sw128_kmajor_desc(sK + ST * kKBytes);
#pragma unroll
    for (int kk = 0; kk < 4 * kAtoms; ++kk)
        mma2_bf16(d, ad + (((kk >> 2) * kQAtom + (kk & 3) * 32u) >> 4), bd + (((kk >> 2) * kKAtom + (kk & 3) * 32u) >> 4),
                  kIdescS, kk > 0 ? 1u : 0u);
}
template <int ST>
__device__ __forceinline__ void issue_pv(uint32_t tmem, uint32_t sP, uint32_t sV, bool add) {
    const uint64_t ad = sw128_kmajor_desc(sP + ST * kPBytes), bd = sw128_mnmajor_desc(sV + ST * kVBytes, kVAtom);
#pragma unroll
    for (int kk = 0; kk < kTok / 16; ++kk)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            mma2_bf16(tmem + 128u * j, ad + ((kk * 32u) >> 4), bd + ((2u * j * kVAtom + kk * 2048u) >> 4), kIdescO,
                      (add || kk > 0) ? 1u : 0u);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_kernel(ChunkArgs a, Plan plan, const __grid_constant__ CUtensorMap qmap, float scale_log2, uint16_t* __restrict__ out, float* __restrict__ lse) {
    extern __shared__ __align__(1024) uint8_t chunk_smem[];  // the swizzled tiles need 1024 bytes
    uint8_t* const gbase = chunk_smem;
    const uint32_t base = smem_addr(gbase);
    if (base & 1023u) {  // the same in every CTA
        set_status(a.status, ECHO_ST_TIMEOUT);
        return;
    }
    const uint32_t sQ = base, sK = sQ + kQBytes, sV = sK + 2 * kKBytes, sP = sV + 2 * kVBytes;
    uint8_t* const gP = gbase + (sP - base);
    Ctl* const ctl = reinterpret_cast<Ctl*>(gP + 2 * kPBytes);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t c = cluster_rank();
    const int ci = blockIdx.x >> 1;
    Watch* const watch = &ctl->watch;
    const volatile int* const abort = &watch->abort;

    if (tid == 0) {
        mbar_init(smem_addr(&ctl->q_full), 1);
        mbar_init(smem_addr(&ctl->q_ready), 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl->k_full[i]), 2 * kLoad);  // the copies, and the valid flags
            mbar_init(smem_addr(&ctl->k_ready[i]), 2);
            mbar_init(smem_addr(&ctl->k_free[i]), 1);
            mbar_init(smem_addr(&ctl->v_full[i]), kLoad);
            mbar_init(smem_addr(&ctl->pv_ready[i]), 2 * kSoftmax / 32 + 2);
            mbar_init(smem_addr(&ctl->pv_done[i]), 1);
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(smem_addr(&ctl->s_full[i]), 1);
            mbar_init(smem_addr(&ctl->s_free[i]), 2 * kSoftmax / 32);
        }
        mbar_init(smem_addr(&ctl->fin_ready), kSoftmax / 32);
        mbar_init(smem_addr(&ctl->fin_free), kSoftmax / 32);
        mbar_init(smem_addr(&ctl->o_free), 2 * kSoftmax / 32);
        for (int i = 0; i < 2; ++i) mbar_init(smem_addr(&ctl->drain[i]), 1);
        watch_init(watch, a.wait_ns);
        fence_barrier_init();
        prefetch_tmap(&qmap);
    }
    if (warp == 0) tmem_alloc2(smem_addr(&ctl->tmem), kTmemCols);
    pdl_wait();
    if (plan.small) {
        if (warp == 1) plan_small(a, plan, &ctl->head, ctl->group, ctl->cum);
        __syncthreads();
    }
    const PlanHead head = plan.small ? ctl->head : *plan.head;
    Walk walk;
    walk.group = plan.small ? ctl->group : plan.group;
    walk.cum = plan.small ? ctl->cum : plan.cum;
    walk.u0 = walk.u1 = 0;
    walk.g = 0;
    if (ci < head.parts) {
        walk.u0 = share_start(head.total, head.parts, ci);
        walk.u1 = share_start(head.total, head.parts, ci + 1);
    }
    if (warp == 1 && walk.u0 < walk.u1) {
        const int g = find_group(walk.cum, head.groups, walk.u0);
        if (lane == 0) ctl->first = g;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (walk.u0 < walk.u1) walk.g = ctl->first;
    const uint32_t tmem = ctl->tmem;
    Piece p;
    uint32_t t = 0;  // tiles so far: stage t & 1, barrier phase (t >> 1) & 1

    if (warp < 4) {
        // ---- softmax: thread = TMEM lane = (token half, row of this CTA's 64)
        const int half = tid >> 6, row = tid & 63, mi = static_cast<int>(c) * 64 + row;
        const int rig = mi / a.heads;  // row within the group
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        bool ok = true, over = false;
        uint32_t pieces = 0;  // with tiles
        while (ok && walk.next(&p)) {
            const bool lives = rig < p.g.rows;
            const int lo_tok = p.g.pos0 + p.g.rows + p.g.kept - p.g.nv;
            // this row's tokens: v < vhi, except [va, vb) (between the first tokens and the window)
            int vhi = 0, va = 0, vb = 0;
            if (lives) {
                if (a.sel) {
                    vhi = p.g.nv;
                } else if (p.g.nv > 0) {
                    const int pos = p.g.pos0 + rig;
                    vhi = p.g.kept + pos - lo_tok + 1;
                    if (a.window) {
                        va = a.sinks > lo_tok ? static_cast<int>(min(a.sinks, static_cast<int64_t>(0x7FFFFFFF))) : p.g.kept;
                        vb = p.g.kept + static_cast<int>(max(static_cast<int64_t>(0), pos - a.window + 1 - lo_tok));
                    }
                }
            }
            float m = -INFINITY, l = 0.f;
            for (int it = p.lo; it < p.hi; ++it, ++t) {
                const uint32_t st = t & 1u;
                ok = ok && mbar_wait(smem_addr(&ctl->s_full[t & (kSBufs - 1)]), (t / kSBufs) & 1u, abort);
                tc_fence_after();
                __syncwarp();
                float s[32];
                tmem_ld_x32(tmem + lane_base + kSCol + (t & (kSBufs - 1)) * 32u, s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(smem_addr(&ctl->s_free[t & (kSBufs - 1)]), 0);
                const int v0 = it * kTok + half * 32;
                const uint32_t there = ctl->valid[t & (kValid - 1)][half];
                const bool clean = there == 0xFFFFFFFFu && v0 + 32 <= vhi && (vb <= va || v0 >= vb || v0 + 32 <= va);
                if (!__all_sync(0xffffffffu, clean)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int v = v0 + j;
                        const bool see = ((there >> j) & 1u) && v < vhi && !(v >= va && v < vb);
                        s[j] = see ? s[j] : -INFINITY;
                    }
                }
                float mx[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) mx[j] = fmaxf(s[2 * j], s[2 * j + 1]);
#pragma unroll
                for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
                    for (int j = 0; j < w; ++j) mx[j] = fmaxf(mx[j], mx[j + w]);
                ctl->mx[st][half][row] = mx[0];
                ok = !softmax_sync_or(!ok);
                over = !ok;
                if (over) break;  // all four warps together
                const float tmx = fmaxf(mx[0], ctl->mx[st][half ^ 1][row]) * scale_log2;
                const bool need = tmx > m + kLazy;  // also m = -inf with a visible token
                const bool moves = __any_sync(0xffffffffu, need);
                float corr = 1.f;
                if (moves && tmx > m) {
                    corr = ex2_approx(m - tmx);  // 0 when m = -inf
                    m = tmx;
                }
                const float neg_m = (m == -INFINITY) ? 0.f : -m;
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t packed[16];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float p0 = ex2_approx(fmaf(s[j], scale_log2, neg_m));
                    const float p1 = ex2_approx(fmaf(s[j + 1], scale_log2, neg_m));
                    part[(j >> 1) & 3] += p0 + p1;  // the sum keeps the unrounded weights: lse is fp32
                    const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
                    packed[j >> 1] = *reinterpret_cast<const uint32_t*>(&pb);
                }
                l = l * corr + ((part[0] + part[1]) + (part[2] + part[3]));
                // this P buffer is free once PV of two tiles before is done
                if (t >= 2) ok = mbar_wait(smem_addr(&ctl->pv_done[st]), ((t >> 1) & 1u) ^ 1u, abort);
                uint8_t* const prow = gP + st * kPBytes + row * 128;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4*>(prow + (((4 * half + j) ^ (row & 7)) << 4)) =
                        make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
                if (it > p.lo && moves) {  // O holds earlier tiles: bring it to the new reference
                    ok = ok && mbar_wait(smem_addr(&ctl->pv_done[st ^ 1u]), ((t - 1) >> 1) & 1u, abort);
                    tc_fence_after();
                    __syncwarp();
#pragma unroll 1
                    for (uint32_t x = 0; x < 256u; x += 32u) {
                        float o[32];
                        tmem_ld_x32(tmem + lane_base + x, o);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] *= corr;
                        tmem_st_x32(tmem + lane_base + x, o);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(smem_addr(&ctl->pv_ready[st]), 0);
            }
            if (over) break;
            // ---- the leg's sums, joined to those of the legs before; after the last: the row's lse, or this part's.
            // The factors of O, and of what the legs before left, for the warps that store it
            float L = 0.f;
            if (p.hi > p.lo) {
                ctl->mx[t & 1u][half][row] = l;
                if (pieces >= 1) ok = ok && mbar_wait(smem_addr(&ctl->fin_free), (pieces - 1) & 1u, abort);
                ++pieces;
                ok = !softmax_sync_or(!ok);
                if (!ok) break;
                L = l + ctl->mx[t & 1u][half ^ 1][row];
            }
            if (half == 0) {
                const bool whole = !p.left && !p.right;
                float* const ml = reinterpret_cast<float*>(part_of(plan, ci, p) + kPartO);
                float before = 0.f, mine = 1.f;
                if (p.later) {
                    const float m0 = ml[mi], l0 = ml[kM + mi], both = fmaxf(m0, m);
                    before = m0 == -INFINITY ? 0.f : exp2f(m0 - both);
                    mine = m == -INFINITY ? 0.f : exp2f(m - both);
                    L = l0 * before + L * mine;
                    m = both;
                }
                const bool any = L != 0.f;  // a NaN among the scores stays one
                const float norm = !(whole && p.last) ? 1.f : any ? 1.f / L : 0.f;
                if (p.hi > p.lo) ctl->fin[row] = mine * norm;
                if (p.later) ml[2 * kM + mi] = before * norm;
                if (!whole || !p.last) {
                    ml[mi] = m;
                    ml[kM + mi] = L;
                } else if (lives) {
                    lse[static_cast<int64_t>(p.g.row0) * a.heads + mi] = any ? (m + log2f(L)) * 0.69314718055994531f : -INFINITY;
                }
            }
            if (p.hi > p.lo) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl->fin_ready));
                (void)softmax_sync_or(false);  // mx is read before the next tile's maxima
            }
        }
        if (!ok) give_up(watch);
    } else if (warp < 8) {
        // ---- K of this CTA's 32 tokens.  A warp has 8 tokens and copies
        // four 128-byte row pieces per instruction (8 lanes each): with 64-byte pieces of 8 rows the
        // copies took twice the shared-memory cycles.  Lanes 0-7 look up the warp's tokens, lanes 8-15
        // those of the other CTA, for the valid flags.
        const int w = warp - 4, x = lane & 7, r4 = lane >> 3;
        bool ok = true;
        while (ok && walk.next(&p)) {
            if (p.hi == p.lo) continue;
            const int mine = static_cast<int>(lane < 8 || lane >= 16 ? c : c ^ 1u) * 32 + 8 * w + (lane & 7);
            Gather own;
            own.start(a, p, mine, lane >= 16 ? plan.ahead : 0);
            for (int it = p.lo; it < p.hi; ++it, ++t) {
                const uint32_t st = t & 1u, ph = (t >> 1) & 1u;
                const int64_t row = own.row(a);
                const uint32_t bits = __ballot_sync(0xffffffffu, row >= 0);  // 8 of this CTA's tokens, 8 of the other's
                own.next(a, p);
                if (plan.ahead && lane >= 16 && lane < 24 && row >= 0)
                    prefetch_l2(a.kv + row * kLatRowBytes, kLatRowBytes);
                const uint8_t* src[2];
                uint32_t n[2], dst[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 4 * i + r4;  // of the warp's 8
                    const int64_t rk = __shfl_sync(0xffffffffu, row, r);
                    src[i] = a.kv + (rk < 0 ? 0 : rk * kLatRowBytes) + 16 * x;
                    n[i] = rk < 0 ? 0u : 16u;
                    dst[i] = sK + st * kKBytes + static_cast<uint32_t>(8 * w + r) * 128u + (static_cast<uint32_t>(x ^ r) << 4);
                }
                if (t >= 2) ok = mbar_wait(smem_addr(&ctl->k_free[st]), ph ^ 1u, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < kAtoms; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) cp_async_16(dst[i] + j * kKAtom, src[i] + 128 * j, n[i]);
                cp_async_arrive_noinc(smem_addr(&ctl->k_full[st]));
                if (lane < 2)
                    reinterpret_cast<uint8_t*>(ctl->valid[t & (kValid - 1)])[(c ^ lane) * 4 + w] =
                        static_cast<uint8_t>(bits >> (8 * lane));
                mbar_arrive(smem_addr(&ctl->k_full[st]));
            }
        }
        if (!ok) give_up(watch);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < 12) {
        // ---- V: this CTA's 256 dims of the tile's 64 tokens, 16 to a warp, copied like K
        const int w = warp - 8, x = lane & 7, r4 = lane >> 3;
        bool ok = true;
        while (ok && walk.next(&p)) {
            if (p.hi == p.lo) continue;
            Gather own;
            own.start(a, p, 16 * w + (lane & 15));
            for (int it = p.lo; it < p.hi; ++it, ++t) {
                const uint32_t st = t & 1u, ph = (t >> 1) & 1u;
                const int64_t row = own.row(a);
                own.next(a, p);
                const uint8_t* src[4];
                uint32_t n[4], dst[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * i + r4;  // of the warp's 16
                    const int64_t rv = __shfl_sync(0xffffffffu, row, r);
                    src[i] = a.kv + (rv < 0 ? 0 : rv * kLatRowBytes) + c * 512u + 16 * x;
                    n[i] = rv < 0 ? 0u : 16u;
                    dst[i] = sV + st * kVBytes + static_cast<uint32_t>(16 * w + r) * 128u +
                             (static_cast<uint32_t>(x ^ (r & 7)) << 4);
                }
                if (t >= 2) ok = mbar_wait(smem_addr(&ctl->pv_done[st]), ph ^ 1u, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) cp_async_16(dst[i] + j * kVAtom, src[i] + 128 * j, n[i]);
                cp_async_arrive_noinc(smem_addr(&ctl->v_full[st]));
            }
        }
        if (!ok) give_up(watch);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 12 || warp == 13) {
        // ---- the MMAs of both CTAs: Q K by one thread of CTA 0, P V by another.  A look at a barrier and a
        // commit cost their thread about 300 cycles a pair; one thread for both products was the limit.
        const bool qk = warp == 12;
        if (c == 0 && elect_one()) {
            uint32_t groups = 0;
            bool ok = true;
            while (ok && walk.next(&p)) {
                if (p.hi == p.lo) continue;
                if (qk) ok = mbar_wait_cluster(smem_addr(&ctl->q_ready), groups & 1u, abort);
                else if (groups > 0) ok = mbar_wait_cluster(smem_addr(&ctl->o_free), (groups - 1) & 1u, abort);
                ++groups;
                for (int it = p.lo; ok && it < p.hi; ++it, ++t) {
                    const uint32_t st = t & 1u, ph = (t >> 1) & 1u;
                    if (qk) {
                        if (t >= kSBufs)
                            ok = mbar_wait_cluster(smem_addr(&ctl->s_free[t & (kSBufs - 1)]), ((t / kSBufs) & 1u) ^ 1u, abort);
                        ok = ok && mbar_wait_cluster(smem_addr(&ctl->k_ready[st]), ph, abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t d = tmem + kSCol + (t & (kSBufs - 1)) * 32u;
                        if (st == 0) issue_qk<0>(d, sQ, sK);
                        else issue_qk<1>(d, sQ, sK);
                        mma2_commit_both(smem_addr(&ctl->k_free[st]));
                        mma2_commit_both(smem_addr(&ctl->s_full[t & (kSBufs - 1)]));
                    } else {  // O += P V
                        ok = mbar_wait_cluster(smem_addr(&ctl->pv_ready[st]), ph, abort);
                        if (!ok) break;
                        tc_fence_after();
                        if (st == 0) issue_pv<0>(tmem, sP, sV, it > p.lo);
                        else issue_pv<1>(tmem, sP, sV, it > p.lo);
                        mma2_commit_both(smem_addr(&ctl->pv_done[st]));
                    }
                }
            }
            if (!ok) {  // the MMAs in flight end before the CTAs' memory goes
                give_up(watch);
                mma2_commit_both(smem_addr(&ctl->drain[qk ? 0 : 1]));
                (void)mbar_wait(smem_addr(&ctl->drain[qk ? 0 : 1]), 0, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 14) {
        // ---- Q and K have landed here: made visible to the tensor cores and reported to CTA 0
        uint32_t groups = 0;
        bool ok = true;
        while (ok && walk.next(&p)) {
            if (p.hi == p.lo) continue;
            // Q of the group, once the group before has no QK left.  Its (row, head) pairs are consecutive in q;
            // pairs past the group's own are another group's, or zeros, and their results are dropped
            if (t >= 1) ok = mbar_wait(smem_addr(&ctl->k_free[(t - 1) & 1u]), ((t - 1) >> 1) & 1u, abort);
            if (!ok) break;
            if (elect_one()) {
                const uint32_t bar = smem_addr(&ctl->q_full);
                mbar_arrive_expect_tx(bar, kQBytes);
                for (int i = 0; i < kAtoms; ++i)
                    tma_load_2d(sQ + i * kQAtom, &qmap, bar, i * 128, p.g.row0 * a.heads + static_cast<int>(c) * 64);
            }
            __syncwarp();
            // always: the load lands before the CTA ends
            ok = mbar_wait(smem_addr(&ctl->q_full), groups & 1u, nullptr);
            ++groups;
            if (ok && lane == 0) mbar_arrive_remote(smem_addr(&ctl->q_ready), 0);
            for (int it = p.lo; ok && it < p.hi; ++it, ++t) {
                ok = mbar_wait(smem_addr(&ctl->k_full[t & 1u]), (t >> 1) & 1u, abort);
                fence_proxy_async_smem();
                if (ok && lane == 0) mbar_arrive_remote(smem_addr(&ctl->k_ready[t & 1u]), 0);
            }
        }
        if (!ok && lane == 0) give_up(watch);
    } else if (warp >= 16) {
        // ---- the results.  Read 16 rows x 32 columns at a time, four lanes to a row, so that stores are whole
        // sectors: a lane a row, straight to memory, took 5 us a group, through shared memory by the softmax warps 3
        const int half = (warp & 3) >> 1, r_cta = (warp & 1) * 32;  // dims 256 half .., rows of this CTA's 64
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t pieces = 0;
        bool ok = true;
        while (ok && walk.next(&p)) {
            const bool direct = !p.left && !p.right && p.last;
            const int live = p.g.rows * a.heads - static_cast<int>(c) * 64 - r_cta;  // of this warp's 32 rows
            const int64_t at = static_cast<int64_t>(p.g.row0) * a.heads + static_cast<int>(c) * 64 + r_cta;
            uint8_t* const dst = direct ? reinterpret_cast<uint8_t*>(out + at * kLatDv + half * 256) : nullptr;
            if (p.hi == p.lo) {  // nothing was seen
                if (warp == 16 && lane == 0) watch_beat(watch);
                for (int i = lane; i < 32 * 32; i += 32)
                    if ((i >> 5) < live) reinterpret_cast<uint4*>(dst + static_cast<int64_t>(i >> 5) * (kLatDv * 2))[i & 31] = make_uint4(0, 0, 0, 0);
                continue;
            }
            t += static_cast<uint32_t>(p.hi - p.lo);
            // (P of the last tile was written after PV of the one two before)
            ok = mbar_wait_watch(smem_addr(&ctl->fin_ready), pieces & 1u, watch) &&
                 mbar_wait(smem_addr(&ctl->pv_done[(t - 1) & 1u]), ((t - 1) >> 1) & 1u, abort);
            ++pieces;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            uint8_t* const part =
                part_of(plan, ci, p) + (static_cast<size_t>(static_cast<int>(c) * 64 + r_cta) * kLatDv + half * 256) * 4;
            const float* const factors = reinterpret_cast<const float*>(part_of(plan, ci, p) + kPartO) + 2 * kM + static_cast<int>(c) * 64 + r_cta;
            float f[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = ctl->fin[r_cta + 8 * i + (lane >> 2)];
            if (p.later) {
#pragma unroll
                for (int i = 0; i < 4; ++i) fb[i] = factors[8 * i + (lane >> 2)];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl->fin_free));
            if (p.later) store_o<true>(tmem + lane_base, f, fb, dst, part, live);
            else store_o<false>(tmem + lane_base, f, fb, dst, part, live);
            tc_fence_before();  // O is read: the next group's first PV may overwrite it
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(smem_addr(&ctl->o_free), 0);
        }
        if (!ok) give_up(watch);
    } else {
        // ---- V has landed here
        if (c == 0 && ci > 0 && lane == 0) {  // first, for the join: whether this share starts the second part of a group
            Cut cut = {0, 0, 0, 0};
            if (walk.u0 < walk.u1) {
                const Group gr = walk.group[walk.g];
                const int64_t at = walk.cum[walk.g];
                cut = Cut{0, ci - 1, gr.row0, gr.rows * a.heads};
                if (walk.u0 > at + kOver && share_start(head.total, head.parts, ci - 1) <= at + kOver)
                    cut.n = share_of(head.total, head.parts, at + kOver + tiles_of(gr.nv) - 1) - cut.i0 + 1;
            }
            plan.cut[ci] = cut;
        }
        __syncwarp();
        bool ok = true;
        while (ok && walk.next(&p)) {
            for (int it = p.lo; ok && it < p.hi; ++it, ++t) {
                ok = mbar_wait(smem_addr(&ctl->v_full[t & 1u]), (t >> 1) & 1u, abort);
                fence_proxy_async_smem();
                if (ok && lane == 0) {
                    mbar_arrive_remote(smem_addr(&ctl->pv_ready[t & 1u]), 0);
                    watch_beat(watch);  // (the V stages go round with the tiles)
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
    cluster_sync_all();  // no CTA leaves while the other may still signal it
    tc_fence_after();
    if (warp == 0) tmem_dealloc2(tmem, kTmemCols);
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

}  // namespace
}  // namespace echo

extern "C" size_t echo_mla_chunk_workspace_size(int64_t n_rows, int heads, int B) {
    using namespace echo;
    if (n_rows < 0 || n_rows > ECHO_CHUNK_MAX_ROWS || heads <= 0 || heads > ECHO_MLA_HEADS || B <= 0 ||
        B > ECHO_MAX_REQUESTS)
        return 0;
    return plan_layout(plan_cap(n_rows, heads, B, true)).total;  // a row to a group is the most
}

extern "C" int echo_mla_chunk(int B, const int64_t* row_off, int64_t n_rows, int heads, const uint16_t* q,
                              const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens,
                              const echo_pages* pages, const int32_t* sel, int k, int64_t window, int64_t sinks,
                              float scale, uint16_t* out, float* lse, void* ws, size_t ws_bytes, int32_t* status,
                              echo_stream_t stream) {
    using namespace echo;
    const int rc = check_chunk(B, row_off, n_rows, heads, q, tok_off, n_tokens, pages, window, sinks, scale, status);
    if (rc) return rc;
    if (sel && (k <= 0 || window || sinks)) return ECHO_EINVAL;
    if (sel && k > kMaxLen) return ECHO_EUNSUPPORTED;
    if (n_rows == 0) return ECHO_OK;
    if (!out || !lse || !ws || !is_aligned(out, 16) || !is_aligned(ws, 256)) return ECHO_EINVAL;
    if (ws_bytes < echo_mla_chunk_workspace_size(n_rows, heads, B)) return ECHO_EINVAL;
    const ChunkArgs a = chunk_args(B, row_off, n_rows, heads, q, tok_off, tok_end, n_tokens, pages, sel, k, window,
                                   sinks, scale, status);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t cap = plan_cap(n_rows, heads, B, sel != nullptr);
    const Layout l = plan_layout(cap);
    uint8_t* const w = static_cast<uint8_t*>(ws);
    Plan plan;
    plan.head = reinterpret_cast<PlanHead*>(w);
    plan.cut = reinterpret_cast<Cut*>(w + 256);
    plan.group = reinterpret_cast<Group*>(w + l.group);
    plan.cum = reinterpret_cast<int64_t*>(w + l.cum);
    plan.part = w + l.part;
    plan.cap = static_cast<int>(cap);
    plan.ahead = cap <= 2 * B ? kAhead : 0;
    CUtensorMap qmap;
    if (encode_tmap_bytes_2d(&qmap, q, kLatRowBytes, static_cast<uint64_t>(n_rows) * heads, 128, 64)) return ECHO_ECUDA;
    static int cached[64];
    plan.clusters = cluster2_count(chunk_kernel, kThreads, kSmem, kMaxClusters, cached);
    if (plan.clusters < 1) return ECHO_ECUDA;
    ECHO_CUDA_OK(prefer_max_shared(chunk_plan_kernel));
    ECHO_CUDA_OK(prefer_max_shared(chunk_join_kernel));
    plan.small = cap <= kInline && B <= kInline;  // 1 row of 1000 tokens: 20 us with a plan kernel, 18 without
    if (!plan.small) {
        chunk_plan_kernel<<<1, kPT, 0, s>>>(a, plan);
        ECHO_CUDA_OK(cudaGetLastError());
    }
    ECHO_CUDA_OK(launch_after(plan.small, chunk_kernel, dim3(static_cast<unsigned>(2 * plan.clusters)), kThreads, kSmem, s, a, plan, qmap,
                              scale * 1.4426950408889634f, out, lse));
    if (plan.clusters > 1)
        ECHO_CUDA_OK(launch_after(false, chunk_join_kernel, dim3(static_cast<unsigned>(8 * sm_count())), kJT, 0, s, a, plan, out, lse));
    return ECHO_OK;
}
