// echo_chunk.cu -- attention of a chunk of new tokens over a paged latent cache.
//
// Per row r and head h, over the tokens t the row sees (echo.h, echo_mla_chunk):
//   s_t = scale * q[r,h] . kv[t]  (576 dims),  out = softmax(s) . kv[t][0:512].
// One block per (row, 16 heads) walks the row's tokens 16 at a time with the
// running maximum and sum of a softmax per head; everything is fp32.
#include "echo_paged.cuh"

namespace echo {
namespace {

constexpr int kT = 128, kHG = 16, kTile = 16;

__global__ void __launch_bounds__(kT) chunk_kernel(ChunkArgs a, uint16_t* __restrict__ out, float* __restrict__ lse) {
    __shared__ __align__(16) __nv_bfloat16 sk[kTile][kLatDqk + 8];
    __shared__ __align__(16) __nv_bfloat16 sq[kHG][kLatDqk + 8];
    __shared__ float sp[kHG][kTile];
    __shared__ float sm[kHG], sl[kHG], sc[kHG];
    __shared__ int64_t srow[kTile];
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    const int h0 = blockIdx.y * kHG, nh = min(kHG, a.heads - h0);
    // the request whose rows hold r
    int b = -1;
    for (int i = 0; i < a.B; ++i)
        if (a.row_off[i] <= r && r < a.row_off[i + 1]) b = i;
    if (b < 0) return;
    int64_t r0, n, off, len;
    if (!chunk_request(a, b, &r0, &n, &off, &len)) return;
    const int64_t pos = len - n + (r - r0);
    const PageView pv = page_view(a, b, off);
    for (int i = tid; i < nh * kLatDqk; i += kT)
        sq[i / kLatDqk][i % kLatDqk] =
            reinterpret_cast<const __nv_bfloat16*>(a.q)[(r * a.heads + h0) * kLatDqk + i];
    if (tid < kHG) {
        sm[tid] = -INFINITY;
        sl[tid] = 0.f;
    }
    int64_t lo = 0, kept = 0, nv = 0;
    if (len > 0) {
        if (a.sel) {
            nv = a.k;
        } else {
            lo = a.window ? max(static_cast<int64_t>(0), pos - a.window + 1) : 0;
            kept = min(a.sinks, lo);
            nv = kept + pos + 1 - lo;
        }
    }
    float o[kHG][4];
    for (int h = 0; h < kHG; ++h)
        for (int j = 0; j < 4; ++j) o[h][j] = 0.f;
    for (int64_t v0 = 0; v0 < nv; v0 += kTile) {
        __syncthreads();
        if (tid < kTile) {
            const int64_t v = v0 + tid;
            int64_t row = -1;
            if (v < nv) {
                int64_t t = v < kept ? v : v - kept + lo;
                bool bad = false;
                if (a.sel) {
                    t = a.sel[r * a.k + v];
                    if (t >= len) {
                        bad = true;
                        t = -1;
                    }
                }
                if (t >= 0) row = token_row(a, pv, static_cast<uint32_t>(t), &bad);
                if (bad) set_status(a.status, ECHO_ST_BADDATA);
            }
            srow[tid] = row;
        }
        __syncthreads();
        for (int i = tid; i < kTile * (kLatDqk / 8); i += kT) {
            const int t = i / (kLatDqk / 8), c = i % (kLatDqk / 8);
            const int64_t row = srow[t];
            const uint4 x = row < 0 ? make_uint4(0, 0, 0, 0)
                                    : *reinterpret_cast<const uint4*>(a.kv + row * kLatRowBytes + 16 * c);
            *reinterpret_cast<uint4*>(&sk[t][8 * c]) = x;
        }
        __syncthreads();
        for (int i = tid; i < kHG * kTile; i += kT) {
            const int h = i / kTile, t = i % kTile;
            float s = -INFINITY;
            if (h < nh && srow[t] >= 0) {
                s = 0.f;
                for (int d = 0; d < kLatDqk; ++d) s += __bfloat162float(sq[h][d]) * __bfloat162float(sk[t][d]);
                s *= a.scale;
            }
            sp[h][t] = s;
        }
        __syncthreads();
        if (tid < kHG) {
            float m = sm[tid];
            for (int t = 0; t < kTile; ++t) m = fmaxf(m, sp[tid][t]);
            const float c = m == -INFINITY ? 1.f : expf(sm[tid] - m);
            float l = sl[tid] * c;
            for (int t = 0; t < kTile; ++t) {
                const float p = sp[tid][t] == -INFINITY ? 0.f : expf(sp[tid][t] - m);
                sp[tid][t] = p;
                l += p;
            }
            sm[tid] = m;
            sl[tid] = l;
            sc[tid] = c;
        }
        __syncthreads();
        for (int h = 0; h < kHG; ++h) {
            for (int j = 0; j < 4; ++j) o[h][j] *= sc[h];
            for (int t = 0; t < kTile; ++t)
                for (int j = 0; j < 4; ++j) o[h][j] += sp[h][t] * __bfloat162float(sk[t][4 * tid + j]);
        }
    }
    __syncthreads();
    for (int h = 0; h < nh; ++h) {
        const float f = sl[h] > 0.f ? 1.f / sl[h] : 0.f;
        for (int j = 0; j < 4; ++j)
            reinterpret_cast<__nv_bfloat16*>(out)[(r * a.heads + h0 + h) * kLatDv + 4 * tid + j] =
                __float2bfloat16_rn(o[h][j] * f);
    }
    if (tid < nh) lse[r * a.heads + h0 + tid] = sl[tid] > 0.f ? sm[tid] + logf(sl[tid]) : -INFINITY;
}

}  // namespace
}  // namespace echo

extern "C" size_t echo_mla_chunk_workspace_size(int64_t n_rows, int heads, int B) {
    if (n_rows < 0 || heads <= 0 || B <= 0) return 0;
    return 256;
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
    chunk_kernel<<<dim3(static_cast<unsigned>(n_rows), static_cast<unsigned>((heads + kHG - 1) / kHG)), kT, 0,
                   static_cast<cudaStream_t>(stream)>>>(a, out, lse);
    ECHO_CUDA_OK(cudaGetLastError());
    return ECHO_OK;
}
