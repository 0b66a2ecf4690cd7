// echo_mass.cu -- the attention weight every cached token receives from a chunk.
//
// mass_out[g] = decay * mass[g] + sum_r sum_h exp(scale * q[r,h] . kv[g] - lse[r,h])
// over the rows r that see token g (echo.h, echo_mla_mass).  One block per
// 32 tokens of a request walks the request's rows; a token's sum is held by
// one thread of each (head share), added in a fixed order.
#include "echo_paged.cuh"

namespace echo {
namespace {

constexpr int kT = 256, kTok = 32;

__global__ void __launch_bounds__(kT) mass_kernel(ChunkArgs a, const float* __restrict__ lse, const float* mass,
                                                  float* mass_out, float decay) {
    __shared__ __align__(16) __nv_bfloat16 sk[kTok][kLatDqk + 2];
    __shared__ int64_t srow[kTok];
    __shared__ float part[8][kTok];
    const int tid = threadIdx.x;
    // the request of block blockIdx.x: its tiles follow those of the requests before it
    int64_t x = blockIdx.x, r0 = 0, n = 0, off = 0, len = 0;
    int b = 0;
    for (; b < a.B; ++b) {
        int64_t t0, t1;
        seg_bounds(a.tok_off, a.tok_end, a.n_tokens, b, &t0, &t1);
        const int64_t tiles = (t1 - t0 + kTok - 1) / kTok;
        if (x < tiles) break;
        x -= tiles;
    }
    if (b == a.B) return;
    int64_t lo, hi;
    seg_bounds(a.tok_off, a.tok_end, a.n_tokens, b, &lo, &hi);
    const int64_t all = hi - lo;
    chunk_request(a, b, &r0, &n, &off, &len);
    const int64_t v0 = x * kTok;
    if (tid < kTok) {
        int64_t row = -1;
        bool bad = false;
        if (v0 + tid < len) row = token_row(a, page_view(a, b, off), static_cast<uint32_t>(v0 + tid), &bad);
        if (bad) set_status(a.status, ECHO_ST_BADDATA);
        srow[tid] = row;
    }
    __syncthreads();
    for (int i = tid; i < kTok * kLatDqk; i += kT) {
        const int64_t row = srow[i / kLatDqk];
        if (row >= 0)
            sk[i / kLatDqk][i % kLatDqk] = reinterpret_cast<const __nv_bfloat16*>(a.kv + row * kLatRowBytes)[i % kLatDqk];
    }
    __syncthreads();
    const int t = tid & 31, hg = tid >> 5;  // thread = (token, share of the heads)
    const int64_t tok = v0 + t;
    float sum = 0.f;
    if (srow[t] >= 0) {
        for (int64_t i = 0; i < n; ++i) {
            const int64_t p = len - n + i;
            if (tok > p || (a.window && tok <= p - a.window && tok >= a.sinks)) continue;
            for (int h = hg; h < a.heads; h += 8) {
                const int64_t rh = (r0 + i) * a.heads + h;
                const float ls = lse[rh];
                if (ls == -INFINITY) continue;
                const __nv_bfloat16* qr = reinterpret_cast<const __nv_bfloat16*>(a.q) + rh * kLatDqk;
                float s = 0.f;
                for (int d = 0; d < kLatDqk; ++d) s += __bfloat162float(qr[d]) * __bfloat162float(sk[t][d]);
                sum += expf(s * a.scale - ls);
            }
        }
    }
    part[hg][t] = sum;
    __syncthreads();
    if (hg == 0 && tok < all) {
        float s = 0.f;
        for (int j = 0; j < 8; ++j) s += part[j][t];
        const int64_t g = lo + tok;
        mass_out[g] = (decay > 0.f ? decay * mass[g] : 0.f) + s;
    }
}

}  // namespace
}  // namespace echo

extern "C" int echo_mla_mass(int B, const int64_t* row_off, int64_t n_rows, int heads, const uint16_t* q,
                             const float* lse, const int64_t* tok_off, const int64_t* tok_end, int64_t n_tokens,
                             const echo_pages* pages, int64_t window, int64_t sinks, float scale, const float* mass,
                             float* mass_out, float decay, int32_t* status, echo_stream_t stream) {
    using namespace echo;
    const int rc = check_chunk(B, row_off, n_rows, heads, q, tok_off, n_tokens, pages, window, sinks, scale, status);
    if (rc) return rc;
    if (n_tokens == 0) return ECHO_OK;
    if ((n_rows > 0 && !lse) || !mass || !mass_out || !(decay >= 0.f) || decay > 3.4028234e38f) return ECHO_EINVAL;
    const ChunkArgs a = chunk_args(B, row_off, n_rows, heads, q, tok_off, tok_end, n_tokens, pages, nullptr, 0, window,
                                   sinks, scale, status);
    const int64_t blocks = n_tokens / kTok + B;
    mass_kernel<<<static_cast<unsigned>(blocks), kT, 0, static_cast<cudaStream_t>(stream)>>>(a, lse, mass, mass_out,
                                                                                            decay);
    ECHO_CUDA_OK(cudaGetLastError());
    return ECHO_OK;
}
