// echo_evict.cu -- victims of a cache by accumulated attention weight, and the
// release of tokens from the cache's tables.
//
// The victims of a request are the W = min(residents - keep, candidates)
// smallest of its candidates (residents that are neither among the first sinks
// nor the last recent tokens) in the order of (mass, token).  As one 64-bit
// number (order key of the mass << 32 | token) every candidate is different,
// so the W smallest are those at or below a limit that a radix select finds, 8 bits a
// pass from the top; a pass whose boundary bin is wanted whole ends it.
// A last pass over the slots writes the victims in slot order.
#include <climits>

#include "echo_common.cuh"
#include "echo_internal.h"

namespace echo {
namespace {

constexpr int kET = 1024;

__global__ void __launch_bounds__(kET)
    evict_kernel(const int64_t* __restrict__ tok_off, const int64_t* __restrict__ tok_end, int64_t n_tokens,
                 const int32_t* __restrict__ slot2tok, int C, const float* __restrict__ mass, int64_t keep,
                 int64_t sinks, int64_t recent, int32_t* __restrict__ evict_tok, int32_t* __restrict__ evict_slot,
                 int32_t* __restrict__ evict_cnt, int32_t* status) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t scratch[kET / 32 + 1];
    __shared__ uint32_t s_held, s_cand, s_digit, s_below;
    const int b = blockIdx.x, tid = threadIdx.x;
    int64_t lo, hi;
    if (!seg_bounds(tok_off, tok_end, n_tokens, b, &lo, &hi) && tid == 0) set_status(status, ECHO_ST_BADDATA);
    const int64_t len = hi - lo;
    const int32_t* s2t = slot2tok + static_cast<int64_t>(b) * C;
    if (tid == 0) s_held = s_cand = 0;
    __syncthreads();
    uint32_t held = 0, cand = 0;
    bool bad = false, nan = false;
    // a slot's 64-bit order, ~0 when it holds no candidate
    const auto order = [&](int s, bool first) -> uint64_t {
        const int32_t t = s2t[s];
        if (t < 0) return ~0ull;
        if (t >= len) {
            bad = true;
            return ~0ull;
        }
        if (first) ++held;
        if (t < sinks || t >= len - recent) return ~0ull;
        if (first) ++cand;
        const float m = mass[lo + t];
        nan |= isnan(m);
        return (static_cast<uint64_t>(isnan(m) ? 0xFFFFFFFFu : order_key(m)) << 32) | static_cast<uint32_t>(t);
    };
    for (int s = tid; s < C; s += kET) (void)order(s, true);
    atomicAdd(&s_held, held);
    atomicAdd(&s_cand, cand);
    if (bad) set_status(status, ECHO_ST_BADDATA);
    if (nan) set_status(status, ECHO_ST_NAN);
    __syncthreads();
    const int64_t over = static_cast<int64_t>(s_held) - keep;
    const uint32_t want = static_cast<uint32_t>(max(static_cast<int64_t>(0), min(over, static_cast<int64_t>(s_cand))));
    uint64_t prefix = 0;
    uint64_t limit = 0;
    bool any = want > 0;
    uint32_t need = want;
    for (int shift = 56; any && shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int s = tid; s < C; s += kET) {
            const uint64_t o = order(s, false);
            if (o != ~0ull && (shift == 56 || (o >> (shift + 8)) == (prefix >> (shift + 8))))
                atomicAdd(&hist[(o >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t acc = 0;
            int d = 0;
            while (acc + hist[d] < need) acc += hist[d++];
            s_digit = d;
            s_below = acc;
        }
        __syncthreads();
        const uint32_t d = s_digit;
        need -= s_below;
        prefix |= static_cast<uint64_t>(d) << shift;
        limit = prefix | ((1ull << shift) - 1ull);
        const bool whole = hist[d] == need;
        __syncthreads();
        if (whole) break;
    }
    uint32_t base = 0;
    int32_t* et = evict_tok + static_cast<int64_t>(b) * C;
    int32_t* es = evict_slot + static_cast<int64_t>(b) * C;
    for (int s0 = 0; s0 < C; s0 += kET) {
        const int s = s0 + tid;
        const uint64_t o = (any && s < C) ? order(s, false) : ~0ull;
        const bool v = o != ~0ull && o <= limit;
        uint32_t total;
        const uint32_t at = base + block_exclusive_scan<kET>(v ? 1u : 0u, scratch, &total);
        if (v) {
            et[at] = static_cast<int32_t>(o & 0xFFFFFFFFu);
            es[at] = s;
        }
        base += total;
    }
    for (int s = static_cast<int>(base) + tid; s < C; s += kET) et[s] = es[s] = -1;
    if (tid == 0) evict_cnt[b] = static_cast<int32_t>(base);
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
    const int32_t slot = atomicExch(&tok2slot[lo + t], -1);  // a token listed twice is released by one of its entries
    if (slot < 0) return;
    if (slot >= C || slot2tok[static_cast<int64_t>(b) * C + slot] != t) {
        set_status(status, ECHO_ST_BADDATA);
        return;
    }
    slot2tok[static_cast<int64_t>(b) * C + slot] = -1;
    atomicOr(&freebits[static_cast<int64_t>(b) * (C / 32) + (slot >> 5)], 1u << (slot & 31));
    if (mass) mass[lo + t] = 0.f;
}

}  // namespace
}  // namespace echo

extern "C" int echo_evict_select(int B, const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens,
                                 const int32_t* slot2tok, int C, const float* mass, int64_t keep, int64_t sinks,
                                 int64_t recent, int32_t* evict_tok, int32_t* evict_slot, int32_t* evict_cnt,
                                 int32_t* status, echo_stream_t stream) {
    using namespace echo;
    if (B <= 0 || C <= 0 || n_tokens < 0 || keep < 0 || sinks < 0 || recent < 0) return ECHO_EINVAL;
    if (B > ECHO_MAX_REQUESTS || C > kMaxSlots) return ECHO_EUNSUPPORTED;
    if (!tok_off || !slot2tok || (n_tokens > 0 && !mass) || !evict_tok || !evict_slot || !evict_cnt || !status)
        return ECHO_EINVAL;
    evict_kernel<<<B, kET, 0, static_cast<cudaStream_t>(stream)>>>(tok_off, tok_end, n_tokens, slot2tok, C, mass, keep,
                                                                   sinks, recent, evict_tok, evict_slot, evict_cnt,
                                                                   status);
    ECHO_CUDA_OK(cudaGetLastError());
    return ECHO_OK;
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
