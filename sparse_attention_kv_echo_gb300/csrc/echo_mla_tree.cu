// echo_mla_tree.cu -- attention of trees of drafted tokens over a paged latent cache (echo.h, echo_mla_tree).
//
// As echo_chunk.cu: a cluster of two CTAs takes 128 (row, head) pairs at a time, S = Q K^T and O += P V by
// cta_group::2 MMAs (M = 128) with O in the tensor memory, a lazy reference maximum, equal shares of tiles,
// cut groups joined behind.  A tree differs in what a row sees: every token before the tree, and of the tree's own
// tokens those whose bit the row's mask has; only the tiles that reach into the tree look at masks.
//
// Tiles have 128 tokens here.  An MMA of QK (M = 128 pairs, N = 64 tokens) reads 3 KB of shared memory for 16 cycles of
// products and takes 25; with N = 128 it reads 4 KB for 32 and takes 32.  Shared memory has no second stage for 128
// tokens' K: the stage is a ring of three thirds (three of the nine 64-dim atoms each), freed by QK and filled with the next
// tile's third while QK goes on through the others and PV runs.  Per CTA of the pair: 64 tokens' K (CTA c: tokens
// [64c, 64c + 64) of the tile), 256 dims of V of 64 tokens at a time (two halves of the tile, a stage each), P of each half
// in a buffer of its own, four buffers of S of 64 columns.  In the tensor memory S of a tile is lane = (token half, row),
// 64 columns, so the threads of half h write P of half h, whole rows.  Softmax takes two sets of four warps, 32 columns
// each, and 128 of the 256 of O in the storing: one set needs 3300 cycles a tile, more than the MMAs.
//
// What bounds it: the MMAs of a tile are 2176 cycles, a tile takes some 2740: copies into shared memory and the operands
// read from it share its ports.  Tensor pipe 79% active on 16 trees of 12 to 48 nodes over 2048 to 32768 tokens, 128 heads
// (1.10 ms a launch by itself, 1.62 PFLOP/s; 1.27 among others, under the power cap).  Tiles of 64 tokens took 1.31 ms, 58%.
// 64 nodes over 131072 tokens: 1.29 ms by itself, 1.53 among others (tiles of 64: 1.82).
//
// The weights enter P V as bf16, as an MMA of bf16 rows takes both its operands: the result, of bf16 too, is 2.0e-3 from 64 bits
// where weights of fp32 give 1.7e-3.  Scores, the sums of the unrounded weights and O are fp32, O in legs of kLeg tiles.
#include "echo_chunk.cuh"

namespace echo {
namespace {

constexpr int kTok = 128;                // tokens per tile
constexpr int kSub = 64;                 // tokens per half: a stage of V, a buffer of P
constexpr int kThreads = 640;
constexpr int kSoftmax = 256, kLoad = 128;
constexpr int kAtoms = kLatDqk / 64;     // 9 swizzle atoms of 64 dims
constexpr int kThirds = 3, kAtomsThird = kAtoms / kThirds;
constexpr uint32_t kQAtom = 64 * 128;    // 64 rows x 128 B
constexpr uint32_t kKAtom = kSub * 128;  // this CTA's 64 tokens
constexpr uint32_t kVAtom = kSub * 128;  // 64 tokens x 64 dims
constexpr uint32_t kQBytes = kAtoms * kQAtom;
constexpr uint32_t kKBytes = kAtoms * kKAtom;
constexpr uint32_t kVBytes = 4 * kVAtom;
constexpr uint32_t kPBytes = 64 * 128;
constexpr uint32_t kTmemCols = 512;      // O [0, 256) | S buffers of 64 columns
constexpr int kSBufs = 4;
constexpr uint32_t kSCol = 256;
// Tokens that few groups read come from memory for many of them, and K has one stage: where a request has up to four groups'
// rows on average, the next tile's rows are brought to L2 once this tile's copies are under way.  Without / with, in us, 32
// requests behind 8000 tokens, pages of 64: 128 heads, one group each 86 / 78, two 133 / 128, four 228 / 230, five 273 / 276; 16
// heads 87 / 83, 134 / 128, four 228 / 220, five 274 / 273, six 322 / 330.  (16 trees of 12 to 48 groups have it off, as
// has one tree of 64: fetched ahead, that took 1.60 ms for 1.51.  Rows looked up and fetched one to five tiles further ahead took
// 90 to 104 us for 81, one group.)
constexpr float kLazy = 8.f;
constexpr int kMinUnits = 2;             // least units per cluster (1, 3 and 4: slower small calls)
constexpr uint32_t kIdescS = idesc_bf16_f32(kM, kTok);
constexpr uint32_t kIdescO = idesc_bf16_f32(kM, 256) | (1u << 16);  // B (V) MN-major

constexpr int kValid = 8;
static_assert(kValid >= kSBufs + 3, "valid flags");

struct Ctl {
    // here: landed in this CTA; the *_ready barriers of CTA 0: landed in both.  Each of a tile's is passed once a tile
    uint64_t q_full, q_ready;                            // Q of a group
    uint64_t k_full[kThirds], k_ready[kThirds];          // a third of K
    uint64_t k_free[kThirds];                            // its MMAs are done
    uint64_t v_full[2];                                  // V of a half
    uint64_t pv_ready[2];                                // V and P of a half, in both CTAs; of the first, also O rescaled
    uint64_t pv_done[2];                                 // P V of a half done: V stage and P buffer free, O ready
    uint64_t s_full[kSBufs];                             // S of a tile done
    uint64_t s_free[kSBufs];                             // S of a tile has been read in both CTAs
    uint64_t drain[2];
    uint32_t tmem;
    Watch watch;
    int first;                                           // the share's first group
    float mx[2][4][64];                                  // tile maxima, or a piece's sums, by (parity, 32 of the columns, row)
    uint64_t o_free;                                     // O of a piece has been read in both CTAs
    float fin[64];                                       // what O of a row is multiplied by
    // tokens of a tile that have a row, a bit each: written for tile t when QK of t - 1 has begun, hence S of t - 5 read
    uint32_t valid[kValid][4];
};
constexpr uint32_t kSmem = kQBytes + kKBytes + 2 * kVBytes + 2 * kPBytes + ((sizeof(Ctl) + 15u) & ~15u);
static_assert(kSmem <= 227u * 1024u, "tree shared memory");

// The walk of a share, with the order in which a piece's tiles are taken: at unit u of its share a cluster is at tile
// u mod (the group's tiles) as far as the piece has it, so that the groups of a request, which read the same tokens, read them at the same
// time whatever their shares begin with (16 trees of 12 to 48 groups: 3.4 GB from memory in ascending order, 1.5 so, 1344 -> 1251 us;
// 64 groups over 131072 tokens 1690 -> 1524).
struct TreeWalk : Walk<kTok> {
    int64_t start;
    int from, len, turn;  // of the piece: its first tile, how many, and which of them is taken first
    __device__ __forceinline__ bool step(Piece* p) {
        const int64_t before = u0;
        if (!next(p)) return false;
        if (!p->later && p->hi > p->lo) {
            from = p->lo;
            len = (p->last ? p->hi : static_cast<int>(min(u1 - cum[g], static_cast<int64_t>(kOver<kTok> + p->tiles)) - kOver<kTok>)) - from;
            const int now = static_cast<int>(static_cast<uint32_t>(before - start) % static_cast<uint32_t>(p->tiles));
            const int ahead = now >= from ? now - from : now - from + p->tiles;  // tiles from the first to the one that is due
            turn = ahead < len ? ahead : p->tiles - ahead < len ? len - (p->tiles - ahead) : 0;
        }
        return true;
    }
    __device__ __forceinline__ int first(const Piece& p) const {  // tile of a leg's first
        const int x = p.lo - from + turn;
        return from + (x >= len ? x - len : x);
    }
    __device__ __forceinline__ int behind(int x) const { return x + 1 == from + len ? from : x + 1; }
};

// One token of every tile of a piece, or of each of its kParts parts, looked up ahead of its copy: the table entry of the
// next is in flight while this one's row is copied.
template <int kParts>
struct Tokens {
    PageView pv;
    int tile, r, part, left;  // of the token whose entry is in flight; tokens of the piece from there on
    int32_t entry;            // < 0: none
    uint32_t at;              // offset in that page
    bool bad;
    __device__ __forceinline__ void look(const ChunkArgs& a, const Piece& p) {
        const int64_t t = static_cast<int64_t>(tile) * kTok + part * (kTok / kParts) + r;
        entry = -1;
        if (left > 0 && t < p.g.nv) entry = pv.tab[page_of(a, pv, static_cast<uint32_t>(t), &at)];
    }
    __device__ __forceinline__ void start(const ChunkArgs& a, const Piece& p, const TreeWalk& walk, int row) {
        pv = page_view(a, p.g.req, p.g.off);
        tile = walk.first(p);
        r = row;
        part = 0;
        left = (p.hi - p.lo) * kParts;
        bad = false;
        at = 0;
        look(a, p);
    }
    // The cache row of the token, -1 when it has none.
    __device__ __forceinline__ int64_t row(const ChunkArgs& a) {
        const int64_t x = entry < 0 ? -1 : page_row(a, pv, entry, at, &bad);
        if (bad) set_status(a.status, ECHO_ST_BADDATA);
        bad = false;
        return x;
    }
    __device__ __forceinline__ void next(const ChunkArgs& a, const Piece& p, const TreeWalk& walk) {
        --left;
        if (++part == kParts) {
            part = 0;
            tile = walk.behind(tile);
        }
        look(a, p);
    }
};

// The MMAs of a third of K (constants all: a descriptor computed at run time costs four times what the MMA does).
template <int G>
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t sQ, uint32_t sK) {
    const uint64_t ad = sw128_kmajor_desc(sQ), bd = sw128_kmajor_desc(sK);
#pragma unroll
    for (int k = 0; k < 4 * kAtomsThird; ++k) {
        const int kk = 4 * kAtomsThird * G + k;
        mma2_bf16(d, ad + (((kk >> 2) * kQAtom + (kk & 3) * 32u) >> 4), bd + (((kk >> 2) * kKAtom + (kk & 3) * 32u) >> 4),
                  kIdescS, kk > 0 ? 1u : 0u);
    }
}
template <int H>
__device__ __forceinline__ void issue_pv(uint32_t tmem, uint32_t sP, uint32_t sV, bool add) {
    const uint64_t ad = sw128_kmajor_desc(sP + H * kPBytes), bd = sw128_mnmajor_desc(sV + H * kVBytes, kVAtom);
#pragma unroll
    for (int kk = 0; kk < kSub / 16; ++kk)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            mma2_bf16(tmem + 128u * j, ad + ((kk * 32u) >> 4), bd + ((2u * j * kVAtom + kk * 2048u) >> 4), kIdescO,
                      (add || kk > 0) ? 1u : 0u);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tree_kernel(ChunkArgs a, Plan plan, const __grid_constant__ CUtensorMap qmap, float scale_log2, uint16_t* __restrict__ out,
                float* __restrict__ lse) {
    extern __shared__ __align__(1024) uint8_t tree_smem[];  // the swizzled tiles need 1024 bytes
    uint8_t* const gbase = tree_smem;
    const uint32_t base = smem_addr(gbase);
    if (base & 1023u) {  // the same in every CTA
        set_status(a.status, ECHO_ST_TIMEOUT);
        return;
    }
    const uint32_t sQ = base, sK = sQ + kQBytes, sV = sK + kKBytes, sP = sV + 2 * kVBytes;
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
        for (int i = 0; i < kThirds; ++i) {
            mbar_init(smem_addr(&ctl->k_full[i]), i == 0 ? 2 * kLoad : kLoad);  // the copies; with the first the valid flags
            mbar_init(smem_addr(&ctl->k_ready[i]), 2);
            mbar_init(smem_addr(&ctl->k_free[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl->v_full[i]), kLoad);
            // P of a half from four warps of each CTA, O from all eight, V
            mbar_init(smem_addr(&ctl->pv_ready[i]), (i == 0 ? 2 * kSoftmax / 32 : kSoftmax / 32) + 2);
            mbar_init(smem_addr(&ctl->pv_done[i]), 1);
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(smem_addr(&ctl->s_full[i]), 1);
            mbar_init(smem_addr(&ctl->s_free[i]), 2 * kSoftmax / 32);
        }
        mbar_init(smem_addr(&ctl->o_free), 2 * kSoftmax / 32);
        for (int i = 0; i < 2; ++i) mbar_init(smem_addr(&ctl->drain[i]), 1);
        watch_init(watch, a.wait_ns);
        fence_barrier_init();
        prefetch_tmap(&qmap);
    }
    if (warp == 0) tmem_alloc2(smem_addr(&ctl->tmem), kTmemCols);
    pdl_wait();
    const PlanHead head = *plan.head;
    TreeWalk walk;
    walk.group = plan.group;
    walk.cum = plan.cum;
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
    walk.start = walk.u0;
    walk.from = walk.len = walk.turn = 0;
    const uint32_t tmem = ctl->tmem;
    Piece p;
    uint32_t t = 0;  // tiles so far: the phase of a barrier passed once a tile is t & 1

    if (warp < 4 || warp >= 16) {
        // ---- softmax and the storing of results: two threads to a TMEM lane = (token half, row of this CTA's 64), 32 of its 64
        // columns of S each, 128 of its 256 of O
        const int set = warp >= 16, wq = warp & 3, half = wq >> 1, row = (wq & 1) * 32 + lane, mi = static_cast<int>(c) * 64 + row;
        const int rig = mi / a.heads;  // row within the group
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        bool ok = true, over = false;
        while (walk.step(&p)) {  // a warp whose wait ran out goes on to the next vote, where all eight leave
            const bool lives = rig < p.g.rows;
            const int vhi = lives && p.g.nv > 0 ? p.g.pos0 + rig + 1 : 0;  // this row's tokens: v < vhi that its mask lets it see
            const uint32_t* const nodes = lives ? a.mask + static_cast<int64_t>(p.g.row0 + rig) * a.words : nullptr;
            float m = -INFINITY, l = 0.f;
            int tile = walk.first(p);
            for (int it = p.lo; it < p.hi; ++it, ++t, tile = walk.behind(tile)) {
                const uint32_t st = t & 1u, buf = t & (kSBufs - 1);
                const int v0 = tile * kTok + half * kSub + 32 * set;
                // the mask's bits of tokens v0 .. v0 + 31, those before the tree set; asked for before the wait, and by
                // the last tiles alone
                uint32_t there = 0xFFFFFFFFu;
                const int d = v0 - p.g.kept;
                if (d > -32 && nodes) {
                    const int w = d >> 5;
                    const uint32_t lo = w < 0 ? 0xFFFFFFFFu : w < a.words ? nodes[w] : 0u;
                    const uint32_t hi = w + 1 < a.words ? nodes[w + 1] : 0u;
                    there = __funnelshift_r(lo, hi, d & 31);
                }
                ok = ok && mbar_wait(smem_addr(&ctl->s_full[buf]), (t / kSBufs) & 1u, abort);
                tc_fence_after();
                __syncwarp();
                float s[32];
                tmem_ld_x32(tmem + lane_base + kSCol + buf * 64u + 32u * set, s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(smem_addr(&ctl->s_free[buf]), 0);
                there &= ctl->valid[t & (kValid - 1)][2 * half + set];
                const bool clean = there == 0xFFFFFFFFu && v0 + 32 <= vhi;
                if (!__all_sync(0xffffffffu, clean)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) s[j] = ((there >> j) & 1u) && v0 + j < vhi ? s[j] : -INFINITY;
                }
                float mx[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) mx[j] = fmaxf(s[2 * j], s[2 * j + 1]);
#pragma unroll
                for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
                    for (int j = 0; j < w; ++j) mx[j] = fmaxf(mx[j], mx[j + w]);
                ctl->mx[st][2 * half + set][row] = mx[0];
                ok = !softmax_or<kSoftmax>(!ok);
                over = !ok;
                if (over) break;  // all eight warps together
                const float(&all)[4][64] = ctl->mx[st];
                const float tmx = fmaxf(fmaxf(all[0][row], all[1][row]), fmaxf(all[2][row], all[3][row])) * scale_log2;
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
                // this half's P buffer is free once its PV of the tile before is done: the weights wait for it in registers
                if (t >= 1) ok = mbar_wait(smem_addr(&ctl->pv_done[half]), st ^ 1u, abort);
                uint8_t* const prow = gP + half * kPBytes + row * 128;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4*>(prow + (((4 * set + j) ^ (row & 7)) << 4)) =
                        make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
                if (it > p.lo && moves) {  // O holds earlier tiles: bring it to the new reference, half of its columns each set
                    ok = ok && mbar_wait(smem_addr(&ctl->pv_done[1]), st ^ 1u, abort);
                    tc_fence_after();
                    __syncwarp();
#pragma unroll 1
                    for (uint32_t x = 128u * set; x < 128u * set + 128u; x += 32u) {
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
                if (lane == 0) {
                    mbar_arrive_remote(smem_addr(&ctl->pv_ready[0]), 0);
                    if (half == 1) mbar_arrive_remote(smem_addr(&ctl->pv_ready[1]), 0);
                }
            }
            if (over) break;
            // ---- the leg's sums, joined to those of the legs before; after the last: the row's lse, or this part's.
            // The factors of O, and of what the legs before left, for the storing
            float L = 0.f;
            if (p.hi > p.lo) {
                float(&sums)[4][64] = ctl->mx[t & 1u];
                sums[2 * half + set][row] = l;
                ok = !softmax_or<kSoftmax>(!ok);
                if (!ok) break;
                L = (sums[0][row] + sums[1][row]) + (sums[2][row] + sums[3][row]);
            }
            if (half == 0 && set == 0) {
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
            // ---- the results: 16 rows x 32 columns at a time, four lanes to a row, so that stores are whole sectors.  (One set
            // storing alone kept the other waiting: 3.1 us of the 10 of a share of one tree of eight.)
            const bool direct = !p.left && !p.right && p.last;
            const int r_cta = (wq & 1) * 32;  // dims 256 half .., rows of this CTA's 64
            const int live = p.g.rows * a.heads - static_cast<int>(c) * 64 - r_cta;  // of this warp's 32 rows
            const int64_t at = static_cast<int64_t>(p.g.row0) * a.heads + static_cast<int>(c) * 64 + r_cta;
            uint8_t* const dst = direct ? reinterpret_cast<uint8_t*>(out + at * kLatDv + half * 256) : nullptr;
            if (p.hi == p.lo) {  // nothing was seen
                if (warp == 16 && lane == 0) watch_beat(watch);
                for (int i = lane; i < 32 * 16; i += 32)
                    if ((i >> 4) < live)
                        reinterpret_cast<uint4*>(dst + static_cast<int64_t>(i >> 4) * (kLatDv * 2))[16 * set + (i & 15)] = make_uint4(0, 0, 0, 0);
                continue;
            }
            (void)softmax_or<kSoftmax>(false);  // the factors are there, the sums read before the next tile's maxima
            ok = mbar_wait(smem_addr(&ctl->pv_done[1]), (t - 1) & 1u, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            tc_fence_after();
            uint8_t* const part =
                part_of(plan, ci, p) + (static_cast<size_t>(static_cast<int>(c) * 64 + r_cta) * kLatDv + half * 256) * 4;
            const float* const factors =
                reinterpret_cast<const float*>(part_of(plan, ci, p) + kPartO) + 2 * kM + static_cast<int>(c) * 64 + r_cta;
            float f[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = ctl->fin[r_cta + 8 * i + (lane >> 2)];
            if (p.later) {
#pragma unroll
                for (int i = 0; i < 4; ++i) fb[i] = factors[8 * i + (lane >> 2)];
            }
            __syncwarp();
            if (p.later) store_o<true, 128>(tmem + lane_base, f, fb, dst, part, live, 128u * set);
            else store_o<false, 128>(tmem + lane_base, f, fb, dst, part, live, 128u * set);
            tc_fence_before();  // O is read: the next group's first PV may overwrite it
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(smem_addr(&ctl->o_free), 0);
        }
        if (!ok) give_up(watch);
    } else if (warp < 8) {
        // ---- K of this CTA's 64 tokens, 16 to a warp, a third of the dims at a time; 128-byte row pieces, four to an
        // instruction.  Lanes 0-15 look up the warp's tokens, lanes 16-31 those of the other CTA, for the valid flags.
        const int w = warp - 4, x = lane & 7, r4 = lane >> 3;
        bool ok = true;
        while (ok && walk.step(&p)) {
            if (p.hi == p.lo) continue;
            Tokens<1> own;
            own.start(a, p, walk, static_cast<int>(lane < 16 ? c : c ^ 1u) * kSub + 16 * w + (lane & 15));
            for (int it = p.lo; ok && it < p.hi; ++it, ++t) {
                const uint32_t ph = t & 1u;
                const int64_t row = own.row(a);
                const uint32_t bits = __ballot_sync(0xffffffffu, row >= 0);  // 16 of this CTA's tokens, 16 of the other's
                own.next(a, p, walk);
                const uint8_t* src[4];
                uint32_t n[4], dst[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * i + r4;  // of the warp's 16
                    const int64_t rk = __shfl_sync(0xffffffffu, row, r);
                    src[i] = a.kv + (rk < 0 ? 0 : rk * kLatRowBytes) + 16 * x;
                    n[i] = rk < 0 ? 0u : 16u;
                    dst[i] = sK + static_cast<uint32_t>(16 * w + r) * 128u + (static_cast<uint32_t>(x ^ (r & 7)) << 4);
                }
                for (int g = 0; g < kThirds; ++g) {
                    if (t >= 1) ok = mbar_wait(smem_addr(&ctl->k_free[g]), ph ^ 1u, abort);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < kAtomsThird; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            cp_async_16(dst[i] + (g * kAtomsThird + j) * kKAtom, src[i] + 128 * (g * kAtomsThird + j), n[i]);
                    cp_async_arrive_noinc(smem_addr(&ctl->k_full[g]));
                    if (g == 0) {
                        if (lane < 2)  // tokens of half h: halfwords 4h .. 4h + 3
                            reinterpret_cast<uint16_t*>(ctl->valid[t & (kValid - 1)])[(c ^ lane) * 4 + w] =
                                static_cast<uint16_t>(bits >> (16 * lane));
                        mbar_arrive(smem_addr(&ctl->k_full[0]));
                    }
                }
                if (plan.ahead && lane < 16) {  // this CTA's rows of the next tile
                    const int64_t next = own.row(a);
                    if (next >= 0) prefetch_l2(a.kv + next * kLatRowBytes, kLatRowBytes);
                }
            }
        }
        if (!ok) give_up(watch);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < 12) {
        // ---- V: this CTA's 256 dims of a half's 64 tokens, 16 to a warp, copied like K
        const int w = warp - 8, x = lane & 7, r4 = lane >> 3;
        bool ok = true;
        while (ok && walk.step(&p)) {
            if (p.hi == p.lo) continue;
            Tokens<kTok / kSub> own;
            own.start(a, p, walk, 16 * w + (lane & 15));
            for (int it = p.lo; ok && it < p.hi; ++it, ++t) {
                for (uint32_t h = 0; h < 2; ++h) {
                    const int64_t row = own.row(a);
                    own.next(a, p, walk);
                    const uint8_t* src[4];
                    uint32_t n[4], dst[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 4 * i + r4;  // of the warp's 16
                        const int64_t rv = __shfl_sync(0xffffffffu, row, r);
                        src[i] = a.kv + (rv < 0 ? 0 : rv * kLatRowBytes) + c * 512u + 16 * x;
                        n[i] = rv < 0 ? 0u : 16u;
                        dst[i] = sV + h * kVBytes + static_cast<uint32_t>(16 * w + r) * 128u +
                                 (static_cast<uint32_t>(x ^ (r & 7)) << 4);
                    }
                    if (t >= 1) ok = mbar_wait(smem_addr(&ctl->pv_done[h]), (t & 1u) ^ 1u, abort);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) cp_async_16(dst[i] + j * kVAtom, src[i] + 128 * j, n[i]);
                    cp_async_arrive_noinc(smem_addr(&ctl->v_full[h]));
                }
            }
        }
        if (!ok) give_up(watch);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 12 || warp == 13) {
        // ---- the MMAs of both CTAs: Q K by one thread of CTA 0, P V by another
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
                    const uint32_t ph = t & 1u;
                    if (qk) {
                        if (t >= kSBufs)
                            ok = mbar_wait_cluster(smem_addr(&ctl->s_free[t & (kSBufs - 1)]), ((t / kSBufs) & 1u) ^ 1u, abort);
                        const uint32_t d = tmem + kSCol + (t & (kSBufs - 1)) * 64u;
                        ok = ok && mbar_wait_cluster(smem_addr(&ctl->k_ready[0]), ph, abort);
                        if (!ok) break;
                        tc_fence_after();
                        issue_qk<0>(d, sQ, sK);
                        mma2_commit_both(smem_addr(&ctl->k_free[0]));
                        ok = mbar_wait_cluster(smem_addr(&ctl->k_ready[1]), ph, abort);
                        if (!ok) break;
                        tc_fence_after();
                        issue_qk<1>(d, sQ, sK);
                        mma2_commit_both(smem_addr(&ctl->k_free[1]));
                        ok = mbar_wait_cluster(smem_addr(&ctl->k_ready[2]), ph, abort);
                        if (!ok) break;
                        tc_fence_after();
                        issue_qk<2>(d, sQ, sK);
                        mma2_commit_both(smem_addr(&ctl->k_free[2]));
                        mma2_commit_both(smem_addr(&ctl->s_full[t & (kSBufs - 1)]));
                    } else {  // O += P V
                        ok = mbar_wait_cluster(smem_addr(&ctl->pv_ready[0]), ph, abort);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv<0>(tmem, sP, sV, it > p.lo);
                        mma2_commit_both(smem_addr(&ctl->pv_done[0]));
                        ok = mbar_wait_cluster(smem_addr(&ctl->pv_ready[1]), ph, abort);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv<1>(tmem, sP, sV, true);
                        mma2_commit_both(smem_addr(&ctl->pv_done[1]));
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
            if (t >= 1) ok = mbar_wait(smem_addr(&ctl->k_free[kThirds - 1]), (t - 1) & 1u, abort);
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
                for (int g = 0; ok && g < kThirds; ++g) {
                    ok = mbar_wait(smem_addr(&ctl->k_full[g]), t & 1u, abort);
                    fence_proxy_async_smem();
                    if (ok && lane == 0) mbar_arrive_remote(smem_addr(&ctl->k_ready[g]), 0);
                }
            }
        }
        if (!ok && lane == 0) give_up(watch);
    } else {
        // ---- V has landed here
        if (c == 0 && ci > 0 && lane == 0) plan.cut[ci] = cut_of<kTok>(walk, head, ci, a.heads);  // first, for the join
        __syncwarp();
        bool ok = true;
        while (ok && walk.next(&p)) {
            for (int it = p.lo; ok && it < p.hi; ++it, ++t) {
                for (int h = 0; ok && h < 2; ++h) {
                    ok = mbar_wait(smem_addr(&ctl->v_full[h]), t & 1u, abort);
                    fence_proxy_async_smem();
                    if (ok && lane == 0) {
                        mbar_arrive_remote(smem_addr(&ctl->pv_ready[h]), 0);
                        watch_beat(watch);  // (the V stages go round with the tiles)
                    }
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

}  // namespace
}  // namespace echo

extern "C" int echo_mla_tree(int B, const int64_t* row_off, int64_t n_rows, int heads, const uint16_t* q,
                             const uint32_t* mask, int words, const int64_t* tok_off, const int64_t* tok_end,
                             int64_t n_tokens, const echo_pages* pages, float scale, uint16_t* out, float* lse, void* ws,
                             size_t ws_bytes, int32_t* status, echo_stream_t stream) {
    using namespace echo;
    const int rc = check_chunk(B, row_off, n_rows, heads, q, tok_off, n_tokens, pages, 0, 0, scale, status);
    if (rc) return rc;
    if (words < 1) return ECHO_EINVAL;
    if (words > ECHO_TREE_MAX_WORDS) return ECHO_EUNSUPPORTED;
    if (n_rows == 0) return ECHO_OK;
    if (!mask || !out || !lse || !ws || !is_aligned(out, 16) || !is_aligned(ws, 256)) return ECHO_EINVAL;
    if (ws_bytes < echo_mla_chunk_workspace_size(n_rows, heads, B)) return ECHO_EINVAL;
    ChunkArgs a = chunk_args(B, row_off, n_rows, heads, q, tok_off, tok_end, n_tokens, pages, nullptr, 0, 0, 0, scale, status);
    a.mask = mask;
    a.words = words;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t cap = plan_cap(n_rows, heads, B, false);
    Plan plan = plan_in(ws, cap);
    CUtensorMap qmap;
    if (encode_tmap_bytes_2d(&qmap, q, kLatRowBytes, static_cast<uint64_t>(n_rows) * heads, 128, 64)) return ECHO_ECUDA;
    static int cached[64];
    plan.clusters = cluster2_count(tree_kernel, kThreads, kSmem, kMaxClusters, cached);
    if (plan.clusters < 1) return ECHO_ECUDA;
    plan.least = kMinUnits;
    plan.ahead = n_rows <= 4ll * rows_per_group(heads, false) * B;
    plan.small = false;
    // The plan is scheduled beside the kernel before it (the masks' lets it be) and waits for that to end.  One warp plans
    // a call of at most 32 requests and groups: one tree of eight nodes, 128 heads, 20.7 us against 22.0 with a block of 1024.
    const bool few = B <= kInline && cap <= kInline;
    const auto plan_kernel = few ? chunk_plan_small_kernel<kTok> : chunk_plan_kernel<kTok>;
    ECHO_CUDA_OK(prefer_max_shared(plan_kernel));
    ECHO_CUDA_OK(prefer_max_shared(chunk_join_kernel));
    ECHO_CUDA_OK(launch_after(false, plan_kernel, dim3(1), few ? 32 : kPT, 0, s, a, plan));
    ECHO_CUDA_OK(launch_after(false, tree_kernel, dim3(static_cast<unsigned>(2 * plan.clusters)), kThreads, kSmem, s, a, plan, qmap,
                              scale * 1.4426950408889634f, out, lse));
    if (plan.clusters > 1)
        ECHO_CUDA_OK(launch_after(false, chunk_join_kernel, dim3(static_cast<unsigned>(8 * sm_count())), kJT, 0, s, a, plan, out, lse));
    return ECHO_OK;
}
