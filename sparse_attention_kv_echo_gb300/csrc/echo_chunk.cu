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
// CTA.  Warps of a CTA: 0-3 softmax (thread = TMEM lane; the two threads of a
// row exchange their tile maxima in shared memory), 4-7 gather the K and V
// parts of the tiles (16-byte cp.async, any row for any token, two stages
// each), 8 issues the MMAs (CTA 0) or reports its CTA's K tiles to CTA 0 (CTA 1), 9
// reports the V tiles.  QK of tile t + 1 is issued before PV of tile t, so the
// softmax runs under the tensor cores.  The softmax reference moves only when a
// score exceeds it by more than 2^8 (P <= 256 in bf16, exact after the final
// division); O in TMEM is rescaled then.
//
// Work: every tile costs the same and a group costs kOver tiles more (its Q, its
// result).  chunk_plan_kernel lays the groups' costs in a row; cluster i takes the
// units [T i / n, T (i + 1) / n) of it, whatever groups those cut, so ragged
// batches, single long requests and whole prompts load all SMs alike.  The parts
// of a cut group go to the workspace in fp32 with their maximum and sum, and
// chunk_join_kernel adds them in order (the same bits every time).
#include "echo_paged.cuh"
#include "echo_tc.cuh"

namespace echo {
namespace {

constexpr int kTok = 64;                 // tokens per tile
constexpr int kM = 128;                  // (row, head) pairs per group
constexpr int kThreads = 320;
constexpr int kSoftmax = 128, kLoad = 128;
constexpr int kAtoms = kLatDqk / 64;     // 9 swizzle atoms of 64 dims
constexpr uint32_t kQAtom = 64 * 128;    // 64 rows x 128 B
constexpr uint32_t kKAtom = 32 * 128;    // this CTA's 32 tokens
constexpr uint32_t kVAtom = kTok * 128;  // 64 tokens x 64 dims
constexpr uint32_t kQBytes = kAtoms * kQAtom;
constexpr uint32_t kKBytes = kAtoms * kKAtom;
constexpr uint32_t kVBytes = 4 * kVAtom;
constexpr uint32_t kPBytes = 64 * 128;
constexpr uint32_t kTmemCols = 512;      // O [0, 256) | S0 [256, 288) | S1 [288, 320)
constexpr uint32_t kSCol = 256;
constexpr float kLazy = 8.f;
constexpr int kOver = 3;                 // a group's fixed cost in tiles
constexpr int kMinUnits = 6;             // least units per cluster
constexpr int kMaxClusters = 96;         // bounds the workspace (the device has 76 pairs of SMs)
constexpr uint32_t kIdescS = idesc_bf16_f32(kM, kTok);
constexpr uint32_t kIdescO = idesc_bf16_f32(kM, 256) | (1u << 16);  // B (V) MN-major
constexpr size_t kPartO = static_cast<size_t>(kM) * kLatDv * 4;
constexpr size_t kPartBytes = kPartO + 2 * kM * 4;

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

struct Plan {
    PlanHead* head;
    Group* group;   // [cap]
    int64_t* cum;   // [cap + 1] units before each group
    uint8_t* part;  // [2 * kMaxClusters] partial results
    int cap;
    int clusters;
};

__host__ __device__ __forceinline__ int rows_per_group(int heads, bool sel) { return sel ? 1 : kM / heads; }

struct Layout {
    size_t group, cum, part, total;
};
inline Layout plan_layout(int64_t cap) {
    Layout l;
    l.group = 256;
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
        PlanHead h;
        h.total = sum;
        h.groups = groups;
        h.parts = static_cast<int32_t>(
            max(static_cast<int64_t>(1), min(static_cast<int64_t>(plan.clusters), sum / kMinUnits)));
        *plan.head = h;
    }
}

// The part of a group that a share holds: tiles [lo, hi) of `tiles`.
struct Piece {
    Group g;
    int lo, hi, tiles;
};

// Walks the pieces of a share; every role of the cluster sees the same ones.
struct Walk {
    const Group* group;
    const int64_t* cum;
    int64_t u0, u1;
    int g;
    // False when the share is done.  Groups that see nothing come with tiles = 0.
    __device__ __forceinline__ bool next(Piece* p) {
        for (;;) {
            if (u0 >= u1) return false;
            const int64_t c = cum[g];
            p->g = group[g];
            ++g;
            p->tiles = tiles_of(p->g.nv);
            const int64_t a = u0 - c, b = min(u1 - c, static_cast<int64_t>(kOver + p->tiles));
            u0 = c + kOver + p->tiles;
            p->lo = static_cast<int>(max(static_cast<int64_t>(0), a - kOver));
            p->hi = static_cast<int>(max(static_cast<int64_t>(0), b - kOver));
            if (p->hi > p->lo || (p->tiles == 0 && a <= 0)) return true;
        }
    }
};

// ---------------------------------------------------------------- attention
struct Ctl {
    uint64_t q_full, pq_full;         // Q of a group landed here / in CTA 1
    uint64_t k_full[2], pk_full[2];   // K part of a stage landed here / in CTA 1
    uint64_t v_full[2], pv_full[2];   // V part
    uint64_t qk_done[2];              // S of a tile done: K stage free, S ready
    uint64_t pv_done[2];              // P V of a tile done: V stage and P free, O ready
    uint64_t p_full;                  // P of a tile written in both CTAs
    uint64_t drain;
    uint32_t tmem;
    int abort;
    int first;                        // the share's first group
    float mx[2][2][64];               // tile maxima by (tile parity, token half, row)
    float l[2][2][64];                // sums by (piece parity, token half, row)
    alignas(16) uint8_t valid[4][kTok];           // tokens of a tile that have a row
};
constexpr uint32_t kSmem = kQBytes + 2 * kKBytes + 2 * kVBytes + kPBytes + ((sizeof(Ctl) + 15u) & ~15u) + 1024;
static_assert(kSmem <= 227u * 1024u, "chunk shared memory");

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

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_kernel(ChunkArgs a, Plan plan, float scale_log2, uint16_t* __restrict__ out, float* __restrict__ lse) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - raw);
    const uint32_t sQ = base, sK = sQ + kQBytes, sV = sK + 2 * kKBytes, sP = sV + 2 * kVBytes;
    uint8_t* const gP = gbase + (sP - base);
    Ctl* const ctl = reinterpret_cast<Ctl*>(gP + kPBytes);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t c = cluster_rank();
    const int ci = blockIdx.x >> 1;
    volatile int* const abort = &ctl->abort;

    if (tid == 0) {
        mbar_init(smem_addr(&ctl->q_full), kLoad);
        mbar_init(smem_addr(&ctl->pq_full), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl->k_full[i]), 2 * kLoad);  // the copies, and the valid flags
            mbar_init(smem_addr(&ctl->pk_full[i]), 1);
            mbar_init(smem_addr(&ctl->v_full[i]), kLoad);
            mbar_init(smem_addr(&ctl->pv_full[i]), 1);
            mbar_init(smem_addr(&ctl->qk_done[i]), 1);
            mbar_init(smem_addr(&ctl->pv_done[i]), 1);
        }
        mbar_init(smem_addr(&ctl->p_full), 2 * kSoftmax / 32);
        mbar_init(smem_addr(&ctl->drain), 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc2(smem_addr(&ctl->tmem), kTmemCols);
    pdl_wait();
    const PlanHead head = *plan.head;
    Walk walk;
    walk.group = plan.group;
    walk.cum = plan.cum;
    walk.u0 = walk.u1 = 0;
    walk.g = 0;
    if (ci < head.parts) {
        walk.u0 = share_start(head.total, head.parts, ci);
        walk.u1 = share_start(head.total, head.parts, ci + 1);
    }
    if (warp == 1 && walk.u0 < walk.u1) {
        const int g = find_group(plan.cum, head.groups, walk.u0);
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
        const uint32_t pfull = smem_addr(&ctl->p_full);
        bool ok = true;
        for (uint32_t piece = 0; ok && walk.next(&p); ++piece) {
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
                ok = ok && mbar_wait(smem_addr(&ctl->qk_done[st]), (t >> 1) & 1u, abort);
                tc_fence_after();
                __syncwarp();
                float s[32];
                tmem_ld_x32(tmem + lane_base + kSCol + st * 32u, s);
                const int v0 = it * kTok + half * 32;
                const uint4* vf = reinterpret_cast<const uint4*>(&ctl->valid[t & 3u][half * 32]);
                const uint4 f0 = vf[0], f1 = vf[1];
                const bool all = ((f0.x & f0.y & f0.z & f0.w) & (f1.x & f1.y & f1.z & f1.w)) == 0x01010101u;
                const bool clean = all && v0 + 32 <= vhi && (vb <= va || v0 >= vb || v0 + 32 <= va);
                if (!__all_sync(0xffffffffu, clean)) {
                    const uint32_t f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int v = v0 + j;
                        const bool see = ((f[j >> 2] >> (8 * (j & 3))) & 1u) && v < vhi && !(v >= va && v < vb);
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
                if (!ok) break;  // all four warps together
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
                // P and O are free once PV of the tile before is done
                if (it > p.lo) ok = mbar_wait(smem_addr(&ctl->pv_done[(t - 1) & 1u]), ((t - 1) >> 1) & 1u, abort);
                tc_fence_after();
                __syncwarp();
                uint8_t* const prow = gP + row * 128;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4*>(prow + (((4 * half + j) ^ (row & 7)) << 4)) =
                        make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
                if (it > p.lo && moves) {
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
                if (lane == 0) mbar_arrive_remote(pfull, 0);
            }
            if (!ok) break;
            // ---- the group's result, or this piece's part of it
            if (p.hi > p.lo) ok = ok && mbar_wait(smem_addr(&ctl->pv_done[(t - 1) & 1u]), ((t - 1) >> 1) & 1u, abort);
            tc_fence_after();
            __syncwarp();
            ctl->l[piece & 1u][half][row] = l;
            ok = !softmax_sync_or(!ok);
            if (!ok) break;
            const float L = l + ctl->l[piece & 1u][half ^ 1][row];
            const bool whole = p.lo == 0 && p.hi == p.tiles;
            const int64_t at = static_cast<int64_t>(p.g.row0) * a.heads + mi;
            if (whole) {
                const float f = L > 0.f ? 1.f / L : 0.f;
                uint4* const dst = reinterpret_cast<uint4*>(out + at * kLatDv + half * 256);
#pragma unroll 1
                for (uint32_t x = 0; x < 256u; x += 32u) {
                    float o[32];
                    if (p.tiles > 0) {
                        tmem_ld_x32(tmem + lane_base + x, o);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0.f;
                    }
                    if (lives) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            uint32_t u[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const __nv_bfloat162 b2 =
                                    __floats2bfloat162_rn(L > 0.f ? o[j + 2 * i] * f : 0.f,
                                                          L > 0.f ? o[j + 2 * i + 1] * f : 0.f);
                                u[i] = *reinterpret_cast<const uint32_t*>(&b2);
                            }
                            dst[(x + j) >> 3] = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    }
                }
                if (lives && half == 0) lse[at] = L > 0.f ? (m + log2f(L)) * 0.69314718055994531f : -INFINITY;
            } else {
                uint8_t* const part = plan.part + static_cast<size_t>(2 * ci + (p.lo > 0 ? 0 : 1)) * kPartBytes;
                float4* const dst = reinterpret_cast<float4*>(part) + (static_cast<size_t>(mi) * kLatDv + half * 256) / 4;
#pragma unroll 1
                for (uint32_t x = 0; x < 256u; x += 32u) {
                    float o[32];
                    tmem_ld_x32(tmem + lane_base + x, o);
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        dst[(x + j) >> 2] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
                if (half == 0) {
                    reinterpret_cast<float*>(part + kPartO)[mi] = m;
                    reinterpret_cast<float*>(part + kPartO)[kM + mi] = L;
                }
            }
            tc_fence_before();  // O is read: the next group's first PV, ordered by its P, may overwrite it
        }
        if (!ok) *abort = 1;
    } else if (warp < 8) {
        // ---- gather
        const int lt = tid - kSoftmax;
        const int kr = lt >> 2, vr = lt >> 1;  // K row (of this CTA's 32 tokens), V row (of the tile's 64)
        const uint32_t kdst = static_cast<uint32_t>(kr) * 128u, vdst = static_cast<uint32_t>(vr) * 128u;
        uint32_t groups = 0;
        bool ok = true;
        while (ok && walk.next(&p)) {
            if (p.hi == p.lo) continue;
            const PageView pv = page_view(a, p.g.req, p.g.off);
            const int lo_tok = p.g.pos0 + p.g.rows + p.g.kept - p.g.nv;
            const int32_t* const sel = a.sel ? a.sel + static_cast<int64_t>(p.g.row0) * a.k : nullptr;
            const auto cache_row = [&](int v) -> int64_t {
                if (v >= p.g.nv) return -1;
                bool bad = false;
                int64_t r = -1;
                int tk;
                if (sel) {
                    tk = sel[v];
                    if (tk >= p.g.kept) {
                        bad = true;
                        tk = -1;
                    }
                } else {
                    tk = v < p.g.kept ? v : v - p.g.kept + lo_tok;
                }
                if (tk >= 0) r = token_row(a, pv, static_cast<uint32_t>(tk), &bad);
                if (bad) set_status(a.status, ECHO_ST_BADDATA);
                return r;
            };
            int64_t rk = cache_row(p.lo * kTok + static_cast<int>(c) * 32 + kr), rv = cache_row(p.lo * kTok + vr);
            for (int it = p.lo; it < p.hi; ++it, ++t) {
                const uint32_t st = t & 1u, ph = (t >> 1) & 1u;
                int64_t nk = -1, nv = -1;
                if (it + 1 < p.hi) {  // the next tile's rows, looked up while this one waits
                    nk = cache_row((it + 1) * kTok + static_cast<int>(c) * 32 + kr);
                    nv = cache_row((it + 1) * kTok + vr);
                }
                if (t >= 2 && !mbar_wait(smem_addr(&ctl->qk_done[st]), ph ^ 1u, abort)) {
                    ok = false;
                    break;
                }
                {
                    const uint8_t* src = a.kv + (rk < 0 ? 0 : rk * kLatRowBytes);
                    const uint32_t n = rk < 0 ? 0u : 16u, dst = sK + st * kKBytes + kdst;
#pragma unroll
                    for (int j = 0; j < 18; ++j) {
                        const int x = (lt & 3) + 4 * j;
                        cp_async_16(dst + static_cast<uint32_t>(x >> 3) * kKAtom + (static_cast<uint32_t>((x ^ kr) & 7) << 4),
                                    src + 16 * x, n);
                    }
                    if ((lt & 1) == 0) ctl->valid[t & 3u][vr] = rv < 0 ? 0 : 1;
                    cp_async_arrive_noinc(smem_addr(&ctl->k_full[st]));
                    mbar_arrive(smem_addr(&ctl->k_full[st]));
                }
                if (it == p.lo) {  // Q of the group, once the group before has no QK left
                    if (t >= 1 && !mbar_wait(smem_addr(&ctl->qk_done[st ^ 1u]), ((t - 1) >> 1) & 1u, abort)) {
                        ok = false;
                        break;
                    }
                    const int live = p.g.rows * a.heads - static_cast<int>(c) * 64;
                    const uint8_t* q = reinterpret_cast<const uint8_t*>(a.q) +
                                       (static_cast<int64_t>(p.g.row0) * a.heads + static_cast<int64_t>(c) * 64) * kLatRowBytes;
#pragma unroll 4
                    for (int i = lt; i < 64 * 72; i += kLoad) {
                        const int r = i / 72, x = i - r * 72;
                        const bool in = r < live;
                        cp_async_16(sQ + sw_offset(r, x, kQAtom), in ? q + static_cast<int64_t>(r) * kLatRowBytes + 16 * x : a.kv,
                                    in ? 16u : 0u);
                    }
                    cp_async_arrive_noinc(smem_addr(&ctl->q_full));
                    ++groups;
                }
                if (t >= 2 && !mbar_wait(smem_addr(&ctl->pv_done[st]), ph ^ 1u, abort)) {
                    ok = false;
                    break;
                }
                {
                    const uint8_t* src = a.kv + (rv < 0 ? 0 : rv * kLatRowBytes) + c * 512u;
                    const uint32_t n = rv < 0 ? 0u : 16u, dst = sV + st * kVBytes + vdst;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int x = (lt & 1) + 2 * j;
                        cp_async_16(dst + static_cast<uint32_t>(x >> 3) * kVAtom + (static_cast<uint32_t>((x ^ vr) & 7) << 4),
                                    src + 16 * x, n);
                    }
                    cp_async_arrive_noinc(smem_addr(&ctl->v_full[st]));
                }
                rk = nk;
                rv = nv;
            }
        }
        if (!ok) *abort = 1;
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 8 && c == 0) {
        // ---- the MMAs of both CTAs
        uint32_t groups = 0;
        bool ok = true;
        while (ok && walk.next(&p)) {
            if (p.hi == p.lo) continue;
            ok = mbar_wait(smem_addr(&ctl->q_full), groups & 1u, abort) &&
                 mbar_wait_cluster(smem_addr(&ctl->pq_full), groups & 1u, abort);
            ++groups;
            const int n = p.hi - p.lo;
            for (int i = 0; ok && i <= n; ++i) {
                if (i < n) {  // S of tile t
                    const uint32_t st = t & 1u, ph = (t >> 1) & 1u;
                    ok = mbar_wait(smem_addr(&ctl->k_full[st]), ph, abort) &&
                         mbar_wait_cluster(smem_addr(&ctl->pk_full[st]), ph, abort);
                    if (!ok) break;
                    fence_proxy_async_smem();
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad = sw128_kmajor_desc(sQ), bd = sw128_kmajor_desc(sK + st * kKBytes);
                        const uint32_t d = tmem + kSCol + st * 32u;
#pragma unroll
                        for (int kk = 0; kk < 4 * kAtoms; ++kk)
                            mma2_bf16(d, ad + (((kk >> 2) * kQAtom + (kk & 3) * 32u) >> 4),
                                      bd + (((kk >> 2) * kKAtom + (kk & 3) * 32u) >> 4), kIdescS, kk > 0 ? 1u : 0u);
                        mma2_commit_both(smem_addr(&ctl->qk_done[st]));
                    }
                    __syncwarp();
                }
                if (i > 0) {  // O += P V of the tile before
                    const uint32_t u = t - 1, st = u & 1u, ph = (u >> 1) & 1u;
                    ok = mbar_wait_cluster(smem_addr(&ctl->p_full), u & 1u, abort) &&
                         mbar_wait(smem_addr(&ctl->v_full[st]), ph, abort) &&
                         mbar_wait_cluster(smem_addr(&ctl->pv_full[st]), ph, abort);
                    if (!ok) break;
                    fence_proxy_async_smem();
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad = sw128_kmajor_desc(sP), bd = sw128_mnmajor_desc(sV + st * kVBytes, kVAtom);
#pragma unroll
                        for (int kk = 0; kk < kTok / 16; ++kk)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                mma2_bf16(tmem + 128u * j, ad + ((kk * 32u) >> 4),
                                          bd + ((2u * j * kVAtom + kk * 2048u) >> 4), kIdescO, (i > 1 || kk > 0) ? 1u : 0u);
                        mma2_commit_both(smem_addr(&ctl->pv_done[st]));
                    }
                    __syncwarp();
                }
                if (i < n) ++t;
            }
        }
        if (!ok) {  // the MMAs in flight end before the CTAs' memory goes
            if (lane == 0) *abort = 1;
            if (elect_one()) mma2_commit_both(smem_addr(&ctl->drain));
            __syncwarp();
            (void)mbar_wait(smem_addr(&ctl->drain), 0, nullptr);
        }
    } else if (warp == 8) {
        // ---- CTA 1: Q and K have landed here
        uint32_t groups = 0;
        bool ok = true;
        while (ok && walk.next(&p)) {
            for (int it = p.lo; ok && it < p.hi; ++it, ++t) {
                ok = mbar_wait(smem_addr(&ctl->k_full[t & 1u]), (t >> 1) & 1u, abort);
                fence_proxy_async_smem();
                if (ok && lane == 0) mbar_arrive_remote(smem_addr(&ctl->pk_full[t & 1u]), 0);
                if (ok && it == p.lo) {
                    ok = mbar_wait(smem_addr(&ctl->q_full), groups & 1u, abort);
                    fence_proxy_async_smem();
                    if (ok && lane == 0) mbar_arrive_remote(smem_addr(&ctl->pq_full), 0);
                    ++groups;
                }
            }
        }
        if (!ok && lane == 0) *abort = 1;
    } else if (c == 1) {
        // ---- CTA 1, warp 9: V has landed here
        bool ok = true;
        while (ok && walk.next(&p)) {
            for (int it = p.lo; ok && it < p.hi; ++it, ++t) {
                ok = mbar_wait(smem_addr(&ctl->v_full[t & 1u]), (t >> 1) & 1u, abort);
                fence_proxy_async_smem();
                if (ok && lane == 0) mbar_arrive_remote(smem_addr(&ctl->pv_full[t & 1u]), 0);
            }
        }
        if (!ok && lane == 0) *abort = 1;
    }
    __syncthreads();
    pdl_launch_dependents();
    if (tid == 0 && *abort) set_status(a.status, ECHO_ST_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while the other may still signal it
    tc_fence_after();
    if (warp == 0) tmem_dealloc2(tmem, kTmemCols);
}

// ---------------------------------------------------------------- join
// Block (i, y): share boundary i + 1, when it is the first inside a group's tiles; 4 (row, head) pairs.
constexpr int kJT = 256, kJRows = 4;

__global__ void __launch_bounds__(kJT) chunk_join_kernel(ChunkArgs a, Plan plan, uint16_t* __restrict__ out,
                                                         float* __restrict__ lse) {
    __shared__ int s_group;
    __shared__ float s_w[kMaxClusters][kJRows];
    __shared__ float s_L[kJRows], s_M[kJRows];
    pdl_wait();
    const int tid = threadIdx.x, i = blockIdx.x + 1;
    const PlanHead head = *plan.head;
    if (i >= head.parts) return;
    const int64_t u = share_start(head.total, head.parts, i);
    if (tid < 32) {
        const int g = find_group(plan.cum, head.groups, u);
        if (tid == 0) s_group = g;
    }
    __syncthreads();
    const Group g = plan.group[s_group];
    const int64_t c = plan.cum[s_group];
    const int tiles = tiles_of(g.nv);
    if (u <= c + kOver || share_start(head.total, head.parts, i - 1) > c + kOver) return;  // no cut here, or not the group's first
    const int i0 = i - 1, i1 = share_of(head.total, head.parts, c + kOver + tiles - 1);
    const int n = i1 - i0 + 1, live = g.rows * a.heads;
    const int m0 = blockIdx.y * kJRows;
    if (m0 >= live) return;
    // piece j is share i0 + j: the first starts at tile 0 (second slot), the others within (first slot)
    const auto part = [&](int j) { return plan.part + static_cast<size_t>(2 * (i0 + j) + (j == 0 ? 1 : 0)) * kPartBytes; };
    for (int x = tid; x < n * kJRows; x += kJT)
        s_w[x / kJRows][x % kJRows] = reinterpret_cast<const float*>(part(x / kJRows) + kPartO)[m0 + x % kJRows];
    __syncthreads();
    if (tid < kJRows) {
        float M = -INFINITY;
        for (int j = 0; j < n; ++j) M = fmaxf(M, s_w[j][tid]);
        float L = 0.f;
        for (int j = 0; j < n; ++j) {
            const float w = M == -INFINITY ? 0.f : exp2f(s_w[j][tid] - M);
            L += w * reinterpret_cast<const float*>(part(j) + kPartO)[kM + m0 + tid];
            s_w[j][tid] = w;
        }
        s_M[tid] = M;
        s_L[tid] = L;
    }
    __syncthreads();
    const int64_t at0 = static_cast<int64_t>(g.row0) * a.heads + m0;
    for (int x = tid; x < kJRows * kLatDv / 4; x += kJT) {
        const int r = x / (kLatDv / 4), d = x % (kLatDv / 4);
        if (m0 + r >= live) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const float w = s_w[j][r];
            const float4 v = reinterpret_cast<const float4*>(part(j))[static_cast<size_t>(m0 + r) * (kLatDv / 4) + d];
            s.x += w * v.x;
            s.y += w * v.y;
            s.z += w * v.z;
            s.w += w * v.w;
        }
        const float f = s_L[r] > 0.f ? 1.f / s_L[r] : 0.f;
        const bool any = s_L[r] > 0.f;
        const __nv_bfloat162 b0 = __floats2bfloat162_rn(any ? s.x * f : 0.f, any ? s.y * f : 0.f);
        const __nv_bfloat162 b1 = __floats2bfloat162_rn(any ? s.z * f : 0.f, any ? s.w * f : 0.f);
        reinterpret_cast<uint2*>(out + (at0 + r) * kLatDv)[d] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
        if (d == 0) lse[at0 + r] = any ? (s_M[r] + log2f(s_L[r])) * 0.69314718055994531f : -INFINITY;
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
    plan.group = reinterpret_cast<Group*>(w + l.group);
    plan.cum = reinterpret_cast<int64_t*>(w + l.cum);
    plan.part = w + l.part;
    plan.cap = static_cast<int>(cap);
    static int cached[64];
    plan.clusters = cluster2_count(chunk_kernel, kThreads, kSmem, kMaxClusters, cached);
    if (plan.clusters < 1) return ECHO_ECUDA;
    ECHO_CUDA_OK(prefer_max_shared(chunk_plan_kernel));
    ECHO_CUDA_OK(prefer_max_shared(chunk_join_kernel));
    chunk_plan_kernel<<<1, kPT, 0, s>>>(a, plan);
    ECHO_CUDA_OK(cudaGetLastError());
    ECHO_CUDA_OK(launch_after(chunk_kernel, dim3(static_cast<unsigned>(2 * plan.clusters)), kThreads, kSmem, s, a, plan,
                              scale * 1.4426950408889634f, out, lse));
    if (plan.clusters > 1)
        ECHO_CUDA_OK(launch_after(chunk_join_kernel, dim3(static_cast<unsigned>(plan.clusters - 1), kM / kJRows), kJT, 0, s,
                                  a, plan, out, lse));
    return ECHO_OK;
}
