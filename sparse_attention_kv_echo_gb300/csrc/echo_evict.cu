// echo_evict.cu -- victims of a cache by accumulated attention weight, and the
// release of tokens from the cache's tables.
//
// The victims of a request are the W = min(residents - keep, candidates)
// smallest of its candidates (residents that are neither among the first sinks
// nor the last recent tokens) in the order of (mass, token): a radix select finds
// the W-th mass, 8 bits a pass from the top, then, when more tokens than are wanted
// share it, the last token that goes, the same way.  A pass whose boundary
// bin is wanted whole ends the search.
//
// A cluster of up to 16 CTAs has a request, each CTA a range of the slots and each
// warp a part of that, so that counts, selects and the ordered output need no more
// than one exchange each.  The masses are gathered once and kept in
// shared memory as order keys (up to 53248 a CTA; further ones are gathered
// again).  The histograms of a pass are added up over the cluster in distributed shared
// memory by every CTA for itself.  Bound by the latency of its steps (two dependent
// loads, 2 to 8 passes with a cluster barrier each), not by its bytes: 1 x 260000
// slots take 41 us with 16 CTAs and 70 with 8 (the random gather of the masses by 16
// SMs is 10 of them), 8 x 4096 take 17 us with 4 CTAs a request and 24 with one.
#include <cooperative_groups.h>

#include "echo_common.cuh"
#include "echo_internal.h"

namespace echo {
namespace {

namespace cg = cooperative_groups;

constexpr int kET = 1024;
constexpr int kEWarps = kET / 32;
constexpr int kEMaxCtas = 16;
constexpr int kECap = 53248;            // keys a CTA keeps
constexpr int kESlots = 1024;           // slots that make a further CTA worth its barriers
constexpr uint32_t kNone = 0xFFFFFFFFu; // no candidate; a NaN mass is one below

// The keys of one CTA's slots [c0, c1).
struct Keys {
    const int32_t* s2t;
    const uint32_t* free;  // the request's free bits, null: every slot with a token holds a resident
    const float* mass;     // the request's
    uint32_t* key;       // shared: of slot c0 + i, i < kECap
    int64_t len, sinks, late;  // late: the first of the recent tokens
    __device__ __forceinline__ uint32_t of(int32_t t, bool* held, bool* bad, bool* nan) const {
        *held = false;
        if (t < 0) return kNone;
        if (t >= len) {
            *bad = true;
            return kNone;
        }
        *held = true;
        if (t < sinks || t >= late) return kNone;
        const float m = mass[t];
        if (isnan(m)) {
            *nan = true;
            return kNone - 1;
        }
        return order_key(m);
    }
    // The token slot s holds as a resident, else -1 (lazy reuse: a free slot's token is a ghost).
    __device__ __forceinline__ int32_t token(int s) const {
        const int32_t t = s2t[s];
        return free && ((free[s >> 5] >> (s & 31)) & 1u) ? -1 : t;
    }
    __device__ __forceinline__ uint32_t at(int c0, int s) const {
        if (s - c0 < kECap) return key[s - c0];
        bool h, b, n;
        return of(token(s), &h, &b, &n);
    }
};

struct EvictShared {
    uint32_t hist[2][256];    // this CTA's, by pass parity
    uint32_t sum[256];        // the cluster's
    uint32_t held, cand, victims;
    uint32_t digit, below;
    uint32_t scratch[kEWarps + 1];
};

// Warp 0: the smallest digit d with (count of digits <= d) >= target, and the count below d.
__device__ __forceinline__ void digit_from_below(const uint32_t* h, uint32_t target, uint32_t* digit, uint32_t* below) {
    const int lane = threadIdx.x & 31;
    uint32_t c[8], sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += c[j] = h[8 * lane + j];
    uint32_t pre = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += y;
    }
    const uint32_t before = pre - sum;
    if (before < target && pre >= target) {
        uint32_t acc = before;
        int j = 0;
        while (j < 7 && acc + c[j] < target) acc += c[j++];
        *digit = 8 * lane + j;
        *below = acc;
    }
}

__global__ void __launch_bounds__(kET)
    evict_kernel(const int64_t* __restrict__ tok_off, const int64_t* __restrict__ tok_end, int64_t n_tokens,
                 const int32_t* __restrict__ slot2tok, const uint32_t* __restrict__ freebits, int C,
                 const float* __restrict__ mass, int64_t keep, int64_t sinks, int64_t recent,
                 int32_t* __restrict__ evict_tok, int32_t* __restrict__ evict_slot,
                 int32_t* __restrict__ evict_cnt, int32_t* status) {
    extern __shared__ uint32_t keys_smem[];
    __shared__ EvictShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int n_cta = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / n_cta, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t lo, hi;
    if (!seg_bounds(tok_off, tok_end, n_tokens, b, &lo, &hi) && tid == 0) set_status(status, ECHO_ST_BADDATA);
    // this CTA's slots, and this warp's, in whole rows of 32
    const int rows = (C + 31) / 32, per_cta = (rows + n_cta - 1) / n_cta, per_warp = (per_cta + kEWarps - 1) / kEWarps;
    const int c0 = min(C, rank * per_cta * 32), c1 = min(C, c0 + per_cta * 32);
    const int w0 = min(c1, c0 + warp * per_warp * 32), w1 = min(c1, w0 + per_warp * 32);
    Keys k;
    k.s2t = slot2tok + static_cast<int64_t>(b) * C;
    k.free = freebits ? freebits + static_cast<int64_t>(b) * (C / 32) : nullptr;
    k.mass = mass + lo;
    k.key = keys_smem;
    k.len = hi - lo;
    k.sinks = sinks;
    k.late = recent < k.len ? k.len - recent : 0;
    if (tid < 256) sh.hist[0][tid] = 0;
    if (tid == 0) sh.held = sh.cand = 0;
    __syncthreads();
    // ---- the keys, and how many there are
    uint32_t held = 0, cand = 0;
    bool bad = false, nan = false;
    constexpr int kBatch = 8;  // slots of a lane in flight
    for (int s0 = w0; s0 < w1; s0 += 32 * kBatch) {
        int32_t t[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int s = s0 + 32 * j + lane;
            t[j] = s < w1 ? k.token(s) : -1;
        }
        uint32_t key[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            bool h;
            key[j] = k.of(t[j], &h, &bad, &nan);
            held += h;
            cand += key[j] != kNone;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int s = s0 + 32 * j + lane;
            if (s < w1 && s - c0 < kECap) k.key[s - c0] = key[j];
        }
    }
    held = __reduce_add_sync(0xffffffffu, held);
    cand = __reduce_add_sync(0xffffffffu, cand);
    if (lane == 0) {
        atomicAdd(&sh.held, held);
        atomicAdd(&sh.cand, cand);
    }
    if (bad) set_status(status, ECHO_ST_BADDATA);
    if (nan) set_status(status, ECHO_ST_NAN);
    cluster.sync();
    held = cand = 0;
    for (int r = 0; r < n_cta; ++r) {
        const EvictShared* o = cluster.map_shared_rank(&sh, r);
        held += o->held;
        cand += o->cand;
    }
    const int64_t over = static_cast<int64_t>(held) - keep;
    const uint32_t want = static_cast<uint32_t>(max(static_cast<int64_t>(0), min(over, static_cast<int64_t>(cand))));
    // ---- the limits: victims are the candidates with key < last_key, and those with
    // key in [last_key, last_key_hi] and token <= last_tok
    uint32_t last_lo = 0, last_hi = 0, last_tok = 0;
    uint32_t need = want;
    bool all_keys = want == 0 || want == cand;
    // One pass: the boundary digit of `need` among f(slot, &value) at `shift`.  True when its bin is wanted whole.
    int parity = 0;
    const auto pass = [&](int shift, auto f) {
        uint32_t* const hist = sh.hist[parity];
        for (int s0 = w0; s0 < w1; s0 += 32) {
            const int s = s0 + lane;
            uint32_t v = 0;
            const bool in = s < w1 && f(s, &v);
            if (in) atomicAdd(&hist[(v >> shift) & 255u], 1u);
        }
        cluster.sync();  // the counts are there; and every CTA is done with the other buffer
        if (tid < 256) {
            uint32_t x = 0;
            for (int r = 0; r < n_cta; ++r) x += cluster.map_shared_rank(&sh, r)->hist[parity][tid];
            sh.sum[tid] = x;
        } else if (tid < 512) {
            sh.hist[parity ^ 1][tid - 256] = 0;
        }
        __syncthreads();
        if (warp == 0) digit_from_below(sh.sum, need, &sh.digit, &sh.below);
        __syncthreads();
        parity ^= 1;
        need -= sh.below;
        return sh.sum[sh.digit] == need;
    };
    if (!all_keys) {
        uint32_t prefix = 0;
        bool whole = false;
        int shift = 24;
        for (; shift >= 0; shift -= 8) {
            const uint32_t top = shift == 24 ? 0u : ~0u << (shift + 8);
            whole = pass(shift, [&](int s, uint32_t* v) {
                *v = k.at(c0, s);
                return *v != kNone && (*v & top) == prefix;
            });
            prefix |= sh.digit << shift;  // (read before the next pass's cluster barrier, written after it)
            if (whole) break;
        }
        if (whole) {
            last_lo = 0;
            last_hi = prefix | ((1u << shift) - 1u);
            last_tok = 0xFFFFFFFFu;
        } else {  // several tokens share the last mass: the lowest `need` of them
            last_lo = last_hi = prefix;
            const int first = (31 - __clz(static_cast<int>(min(k.len, static_cast<int64_t>(0x7FFFFFFF))) | 1)) & ~7;
            for (shift = first; shift >= 0; shift -= 8) {  // tokens are below len
                const uint32_t top = shift == 24 ? 0u : ~0u << (shift + 8);
                whole = pass(shift, [&](int s, uint32_t* v) {
                    if (k.at(c0, s) != prefix) return false;
                    *v = static_cast<uint32_t>(k.s2t[s]);
                    return (*v & top) == last_tok;
                });
                last_tok |= sh.digit << shift;
                if (whole) break;
            }
            if (shift > 0) last_tok |= (1u << shift) - 1u;
        }
    } else if (want) {
        last_hi = kNone - 1;
        last_tok = 0xFFFFFFFFu;
    }
    const auto victim = [&](int s) {
        if (s >= w1 || want == 0) return false;
        const uint32_t x = k.at(c0, s);
        if (x == kNone || x > last_hi) return false;
        return x < last_lo || last_tok == 0xFFFFFFFFu || static_cast<uint32_t>(k.s2t[s]) <= last_tok;
    };
    // ---- the list, in the order of the slots
    uint32_t mine = 0;
    if (want)
        for (int s0 = w0; s0 < w1; s0 += 32) mine += __popc(__ballot_sync(0xffffffffu, victim(s0 + lane)));
    if (lane == 0) sh.scratch[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        const uint32_t v = sh.scratch[lane];
        uint32_t x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        sh.scratch[lane] = x - v;
        if (lane == 31) sh.victims = x;
    }
    cluster.sync();
    uint32_t at = sh.scratch[warp], total = 0;
    for (int r = 0; r < n_cta; ++r) {
        const uint32_t x = cluster.map_shared_rank(&sh, r)->victims;
        if (r < rank) at += x;
        total += x;
    }
    int32_t* const et = evict_tok + static_cast<int64_t>(b) * C;
    int32_t* const es = evict_slot + static_cast<int64_t>(b) * C;
    if (mine)
        for (int s0 = w0; s0 < w1; s0 += 32) {
            const bool v = victim(s0 + lane);
            const uint32_t m = __ballot_sync(0xffffffffu, v);
            if (v) {
                const uint32_t x = at + __popc(m & ((1u << lane) - 1u));
                et[x] = k.s2t[s0 + lane];
                es[x] = s0 + lane;
            }
            at += __popc(m);
        }
    for (int s = max(c0, static_cast<int>(total)) + tid; s < c1; s += kET) et[s] = es[s] = -1;
    if (rank == 0 && tid == 0) evict_cnt[b] = static_cast<int32_t>(total);
    cluster.sync();  // no CTA leaves while another reads its counts
}

// Whether the device holds a cluster of kEMaxCtas (more than the portable 8) at once, with the most
// shared memory (queried once per device).
bool wide_clusters_fit() {
    static int cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (cached[dev] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kEMaxCtas);
        cfg.blockDim = dim3(kET);
        cfg.dynamicSmemBytes = kECap * 4;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kEMaxCtas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, evict_kernel, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        cached[dev] = n > 0 ? 1 : 2;
    }
    return cached[dev] == 1;
}

constexpr int kRT = 256;

__global__ void __launch_bounds__(kRT)
    release_kernel(const int64_t* __restrict__ tok_off, const int64_t* __restrict__ tok_end, int64_t n_tokens,
                   const int32_t* __restrict__ tok, int m, int32_t* tok2slot, int32_t* slot2tok, uint32_t* freebits,
                   int C, float* mass, int32_t* status) {
    const int b = blockIdx.y;
    const int i = blockIdx.x * kRT + threadIdx.x;
    if (i >= m) return;
    const int32_t t = tok[static_cast<int64_t>(b) * m + i];
    if (t < 0) return;
    int64_t lo, hi;
    if (!seg_bounds(tok_off, tok_end, n_tokens, b, &lo, &hi) || t >= hi - lo) {
        set_status(status, ECHO_ST_BADDATA);
        return;
    }
    // The entry is claimed after every check, so that bad tables stay as they are.  Of the entries that list a
    // token one claims it; another may find slot2tok emptied already: then so is tok2slot, which went first.
    const int64_t row = lo + t;
    const int32_t slot = *static_cast<volatile int32_t*>(&tok2slot[row]);
    if (slot < 0) return;
    int32_t* const owner = slot2tok + static_cast<int64_t>(b) * C + slot;
    if (slot >= C || *static_cast<volatile int32_t*>(owner) != t) {
        __threadfence();
        if (*static_cast<volatile int32_t*>(&tok2slot[row]) == slot) set_status(status, ECHO_ST_BADDATA);
        return;
    }
    uint32_t* const word = freebits + static_cast<int64_t>(b) * (C / 32) + (slot >> 5);
    const uint32_t bit = 1u << (slot & 31);
    if (*static_cast<volatile uint32_t*>(word) & bit) return;  // lazy reuse: freed before, its slot keeps it
    if (atomicCAS(&tok2slot[row], slot, -1) != slot) return;
    __threadfence();
    *static_cast<volatile int32_t*>(owner) = -1;
    atomicOr(word, bit);
    if (mass) mass[row] = 0.f;
    __threadfence();  // a cache step right behind may read the tables once this grid's blocks have ended, before its wait
}

}  // namespace
}  // namespace echo

extern "C" int echo_evict_select_resident(int B, const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens,
                                          const int32_t* slot2tok, const uint32_t* freebits, int C, const float* mass,
                                          int64_t keep, int64_t sinks, int64_t recent, int32_t* evict_tok,
                                          int32_t* evict_slot, int32_t* evict_cnt, int32_t* status,
                                          echo_stream_t stream) {
    using namespace echo;
    if (B <= 0 || C <= 0 || n_tokens < 0 || keep < 0 || sinks < 0 || recent < 0) return ECHO_EINVAL;
    if (B > ECHO_MAX_REQUESTS || C > kMaxSlots) return ECHO_EUNSUPPORTED;
    if (!tok_off || !slot2tok || (n_tokens > 0 && !mass) || !evict_tok || !evict_slot || !evict_cnt || !status)
        return ECHO_EINVAL;
    if (freebits && C % 32) return ECHO_ECAPACITY;
    // CTAs of a request: while each has kESlots slots and the batch leaves SMs free
    int n = 1;
    while (n < kEMaxCtas && C >= 2 * n * kESlots && 2 * n * B <= sm_count()) n *= 2;
    ECHO_CUDA_OK(cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kECap * 4));
    ECHO_CUDA_OK(cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    if (n > 8 && !wide_clusters_fit()) n = 8;
    const int per = ((C + 31) / 32 + n - 1) / n * 32;
    const size_t smem = static_cast<size_t>(per < kECap ? per : kECap) * 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(B * n));
    cfg.blockDim = dim3(kET);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(n);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ECHO_CUDA_OK(cudaLaunchKernelEx(&cfg, evict_kernel, tok_off, tok_end, n_tokens, slot2tok, freebits, C, mass, keep, sinks,
                                    recent, evict_tok, evict_slot, evict_cnt, status));
    return ECHO_OK;
}

extern "C" int echo_evict_select(int B, const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens,
                                 const int32_t* slot2tok, int C, const float* mass, int64_t keep, int64_t sinks,
                                 int64_t recent, int32_t* evict_tok, int32_t* evict_slot, int32_t* evict_cnt,
                                 int32_t* status, echo_stream_t stream) {
    return echo_evict_select_resident(B, tok_off, tok_end, n_tokens, slot2tok, nullptr, C, mass, keep, sinks, recent,
                                      evict_tok, evict_slot, evict_cnt, status, stream);
}

extern "C" int echo_cache_release(int B, const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens,
                                  const int32_t* tok, int m, const echo_cache* cache, float* mass, int32_t* status,
                                  echo_stream_t stream) {
    using namespace echo;
    if (B <= 0 || m < 0 || n_tokens < 0) return ECHO_EINVAL;
    if (B > ECHO_MAX_REQUESTS) return ECHO_EUNSUPPORTED;
    if (!tok_off || !status) return ECHO_EINVAL;
    const int rc = check_cache(cache, B, 0);
    if (rc) return rc;
    if (m == 0 || n_tokens == 0) return ECHO_OK;
    if (!tok) return ECHO_EINVAL;
    release_kernel<<<dim3(static_cast<unsigned>((m + kRT - 1) / kRT), static_cast<unsigned>(B)), kRT, 0,
                     static_cast<cudaStream_t>(stream)>>>(tok_off, tok_end, n_tokens, tok, m, cache->tok2slot,
                                                          cache->slot2tok, cache->freebits, cache->C, mass, status);
    ECHO_CUDA_OK(cudaGetLastError());
    return ECHO_OK;
}
