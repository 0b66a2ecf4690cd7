// echo_tree.cu -- the masks of trees of drafted tokens (echo.h, echo_tree_masks).
//
// A block takes the requests in turn, a thread its nodes: it walks from its node up to
// the root over the parents in shared memory, setting bits.  Indices fall on the way (a
// parent comes before its child), so the words are finished from the last to the first and
// each is written once.  What bounds it is the launch and the latency of one walk (48 chains of
// four 3.9 us, a tree of 64 nodes 6, by themselves).  Past that, the longest walk of all of a thread's nodes: a tree of 1024 whose
// parents lie up to 300 nodes before them takes 29 us, up to eight 156; a chain of 64, 256, 1024 nodes 10, 56, 666.
#include "echo_common.cuh"

namespace echo {
namespace {

constexpr int kTreeThreads = 128;

__global__ void __launch_bounds__(kTreeThreads)
    tree_masks_kernel(int B, const int64_t* __restrict__ row_off, int64_t n_rows, const int32_t* __restrict__ parent, int words,
                      uint32_t* __restrict__ mask, int32_t* __restrict__ depth, int32_t* status) {
    __shared__ int16_t up[ECHO_TREE_MAX_NODES];
    pdl_launch_dependents();
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
        const int64_t r0 = row_off[b], r1 = row_off[b + 1], n = r1 - r0;
        if (r0 < 0 || r1 < r0 || r1 > n_rows) {
            if (threadIdx.x == 0) set_status(status, ECHO_ST_BADDATA);
            continue;
        }
        if (n > 32ll * words) {
            if (threadIdx.x == 0) set_status(status, ECHO_ST_BADDATA);
            for (int64_t i = threadIdx.x; i < n * words; i += kTreeThreads) mask[r0 * words + i] = 0u;
            if (depth)
                for (int64_t i = threadIdx.x; i < n; i += kTreeThreads) depth[r0 + i] = 0;
            continue;
        }
        bool bad = false;
        for (int i = threadIdx.x; i < n; i += kTreeThreads) {
            const int p = parent[r0 + i];
            const bool in = p >= -1 && p < i;
            bad |= !in;
            up[i] = static_cast<int16_t>(in ? p : -1);
        }
        if (bad) set_status(status, ECHO_ST_BADDATA);
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kTreeThreads) {
            uint32_t* const m = mask + (r0 + i) * words;
            int w = words - 1, steps = -1;
            uint32_t bits = 0u;
            for (int j = i; j >= 0; j = up[j], ++steps) {
                for (; w > (j >> 5); --w) {
                    m[w] = bits;
                    bits = 0u;
                }
                bits |= 1u << (j & 31);
            }
            for (; w >= 0; --w) {
                m[w] = bits;
                bits = 0u;
            }
            if (depth) depth[r0 + i] = steps;
        }
        __syncthreads();
    }
}

}  // namespace
}  // namespace echo

extern "C" int echo_tree_masks(int B, const int64_t* row_off, int64_t n_rows, const int32_t* parent, int words, uint32_t* mask,
                               int32_t* depth, int32_t* status, echo_stream_t stream) {
    using namespace echo;
    if (B <= 0 || n_rows < 0 || words < 1 || !row_off || !status) return ECHO_EINVAL;
    if (B > ECHO_MAX_REQUESTS || n_rows > ECHO_CHUNK_MAX_ROWS || words > ECHO_TREE_MAX_WORDS) return ECHO_EUNSUPPORTED;
    if (n_rows == 0) return ECHO_OK;
    if (!parent || !mask) return ECHO_EINVAL;
    tree_masks_kernel<<<B, kTreeThreads, 0, static_cast<cudaStream_t>(stream)>>>(B, row_off, n_rows, parent, words, mask, depth,
                                                                                status);
    ECHO_CUDA_OK(cudaGetLastError());
    return ECHO_OK;
}
