// echo_verify.cu -- verification of drafted tokens (echo.h, echo_draft_verify).
//
// What the rejections at a node leave of its probabilities p has a closed form: with d the
// distribution its children are drawn from, left = max(0, p - S d), S = 0 before the first
// rejection, and a rejection adds R = sum left (R = 1 at first) to S, since
//   max(0, max(0, p - S d) - R d) = max(0, p - (S + R) d).
// So a residual is one number, each rejection costs one sum over the vocabulary, and no
// residual is stored.  A draft without probabilities has d = 1 at its own token: left is p
// without the tokens rejected so far.
//
// A cluster of CTAs works on a request: each has a slice of the vocabulary, a warp of it a
// slice of that, read 16 bytes a lane.  CTA 0 walks the tree (a warp; the children of a
// node are found by ballot among 32 parents at a time, each child's own probabilities are
// loaded beforehand) and asks the cluster for a sum where a child is rejected, or at the
// end of the walk, when the token behind the path is drawn: the slice whose running
// sum passes u * total, in it the warp's, in it the token.
// Values are 64-bit integers in units of 2^-60, so sums do not hang on their order, and
// the token drawn is the same on any number of CTAs.
#include <cuda_bf16.h>

#include "echo_common.cuh"
#include "echo_tc.cuh"

namespace echo {
namespace {

constexpr int kVT = 512;
constexpr int kVWarps = kVT / 32;
constexpr int kMaxCluster = 8;
constexpr int kNodes = ECHO_TREE_MAX_NODES;

struct VerifyArgs {
    const int64_t* row_off;
    int64_t n_rows;
    const int32_t* parent;
    const int32_t* token;
    int64_t vocab;
    const void* target;
    const void* draft;
    const float* u_node;
    const float* u_pick;
    int32_t* path;
    int32_t* count;
    int32_t* next;
    int32_t* status;
};

enum Ask : int { kSum, kDraw, kBest, kEnd };  // what CTA 0 asks of the cluster

struct Cmd {
    int ask;
    int node;
    uint64_t S;      // units of 2^-50
    int gone;        // tokens left out (drafts without probabilities)
};

struct VerifySmem {
    Cmd cmd;
    uint64_t slot[kMaxCluster];    // the CTAs' sums, or best keys
    uint64_t warp_sum[kVWarps];
    int bad;
    int32_t gone[kNodes];          // the tokens left out
    // CTA 0: the tree
    int16_t up[kNodes];
    int32_t tok[kNodes];
    float u[kNodes], p[kNodes], d[kNodes];  // the node's uniform number, its token's probabilities in its parent's rows
};

// A probability in units of 2^-60; NaN and negative values are 0, values above 2 are 2.
__device__ __forceinline__ uint64_t to_units(float x) {
    return __float2ull_rz(fminf(fmaxf(x, 0.f), 2.f) * 1152921504606846976.f);
}
__device__ __forceinline__ bool is_probability(float x) { return x >= 0.f && x <= 2.f; }

// max(0, p - S d)
__device__ __forceinline__ uint64_t left_of(uint64_t p, uint64_t S, uint64_t d) {
    const uint64_t lo = S * d, hi = __umul64hi(S, d);
    if (hi >> 47) return 0;  // above 2^61, the largest p
    const uint64_t x = (hi << 14) | (lo >> 50);
    return p > x ? p - x : 0;
}

template <class T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int n = 4;
    __device__ static __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    __device__ static __forceinline__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    __device__ static __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ static __forceinline__ float one(const void* p, int64_t i) {
        return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    }
};

// Row `row` of a matrix of probabilities as 16-byte pieces on 16-byte boundaries: piece j holds the
// tokens first(j) .. first(j) + n - 1, of which those outside the row count as 0.
template <class T>
struct Row {
    const T* base;      // of the piece 0, at or before the row's first element
    int64_t vocab;
    int64_t end;        // elements of the matrix from base on
    int shift;          // elements of piece 0 before the row
    int pieces;
    __device__ __forceinline__ Row(const void* m, int64_t row, int64_t n_rows, int64_t vocab_) {
        const int64_t at = row * vocab_;
        shift = static_cast<int>(at % Vec<T>::n);
        base = static_cast<const T*>(m) + (at - shift);
        vocab = vocab_;
        end = n_rows * vocab_ - (at - shift);
        pieces = static_cast<int>((vocab_ + shift + Vec<T>::n - 1) / Vec<T>::n);
    }
    __device__ __forceinline__ int64_t first(int j) const { return static_cast<int64_t>(j) * Vec<T>::n - shift; }
    __device__ __forceinline__ void load(int j, float (&x)[Vec<T>::n]) const {
        constexpr int n = Vec<T>::n;
        if ((j + 1ll) * n <= end) {
            Vec<T>::unpack(reinterpret_cast<const uint4*>(base)[j], x);
        } else {  // the matrix ends within the piece
#pragma unroll
            for (int i = 0; i < n; ++i) x[i] = j * static_cast<int64_t>(n) + i < end ? Vec<T>::one(base, j * static_cast<int64_t>(n) + i) : 0.f;
        }
    }
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t remote_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void remote_store(uint32_t a, uint64_t x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(x) : "memory");
}

// What is left of the tokens of piece j, in units.
template <class T>
__device__ __forceinline__ void piece_left(const Row<T>& p, const Row<T>& d, int j, const Cmd& c, const int32_t* gone, uint64_t (&x)[Vec<T>::n],
                                           bool* bad) {
    constexpr int n = Vec<T>::n;
    float f[n];
    p.load(j, f);
    const int64_t t0 = p.first(j);
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const bool in = t0 + i >= 0 && t0 + i < p.vocab;
        *bad |= in && !is_probability(f[i]);
        x[i] = in ? to_units(f[i]) : 0;
    }
    if (c.S) {
        d.load(j, f);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const bool in = t0 + i >= 0 && t0 + i < p.vocab;
            *bad |= in && !is_probability(f[i]);
            if (in) x[i] = left_of(x[i], c.S, to_units(f[i]));
        }
    }
    for (int k = 0; k < c.gone; ++k) {
        const int64_t at = gone[k] - t0;
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (at == i) x[i] = 0;
    }
}

__device__ __forceinline__ float unit_interval(float u, bool* bad) {
    *bad |= !(u >= 0.f && u < 1.f);
    return fminf(fmaxf(u, 0.f), 0.99999994f);  // NaN: 0
}

// T: the probabilities' type.
template <class T>
__global__ void __launch_bounds__(kVT) verify_kernel(VerifyArgs a) {
    __shared__ VerifySmem sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int b = blockIdx.x / ctas;
    const bool greedy = a.u_pick == nullptr;
    int64_t r0 = a.row_off[b], r1 = a.row_off[b + 1];
    if (tid == 0) sm.bad = 0;
    int n = 0;
    if (r0 < 0 || r1 < r0 || r1 > a.n_rows) {
        if (rank == 0 && tid == 0) set_status(a.status, ECHO_ST_BADDATA);
    } else if (r1 - r0 > kNodes) {
        if (rank == 0) {
            if (tid == 0) set_status(a.status, ECHO_ST_BADDATA);
            for (int64_t i = r0 + tid; i < r1; i += kVT) a.path[i] = -1;
        }
    } else {
        n = static_cast<int>(r1 - r0);
    }
    if (n == 0) {  // the same in every CTA of the cluster unless the bounds change meanwhile: no barrier follows
        if (rank == 0 && tid == 0) {
            a.count[b] = 0;
            a.next[b] = -1;
        }
    }
    bool bad = false, odd = false;  // probabilities / other data that are none
    if (rank == 0) {
        for (int i = tid; i < n; i += kVT) {
            const int up = a.parent[r0 + i], x = a.token[r0 + i];
            const bool in = up >= -1 && up < i;
            odd |= !in;
            sm.up[i] = static_cast<int16_t>(in ? up : -1);
            sm.tok[i] = x;
            if (!greedy) {
                float p = 0.f, d = 0.f;
                if (in && up >= 0 && x >= 0 && x < a.vocab) {
                    const int64_t at = (r0 + up) * a.vocab + x;
                    p = Vec<T>::one(a.target, at);
                    d = a.draft ? Vec<T>::one(a.draft, at) : 1.f;
                    bad |= !is_probability(p) || !is_probability(d);
                }
                sm.p[i] = p;
                sm.d[i] = d;
                sm.u[i] = up >= 0 ? unit_interval(a.u_node[r0 + i], &odd) : 0.f;
            }
            a.path[r0 + i] = -1;
        }
    }
    __syncthreads();
    // ---- the walk: state of CTA 0's warp 0, the same in its lanes
    int v = 0, c = 0, len = 1;    // node, the last child tried, nodes accepted
    uint64_t S = 0;
    double R = 1.0;
    uint64_t S_next = 0;
    int gone = 0;
    int best = -1;
    if (rank == 0 && tid == 0 && n > 0) a.path[r0] = 0;
    Cmd cmd = {n > 0 ? kSum : kEnd, 0, 0, 0};
    for (;;) {
        // ---- CTA 0: on to the next question
        if (rank == 0 && warp == 0) {
            if (n == 0) {
                cmd.ask = kEnd;
            } else if (greedy && best < 0) {
                cmd = Cmd{kBest, v, 0, 0};
            } else {
                cmd.ask = -1;
                while (cmd.ask < 0) {
                    // the next child of v behind c
                    int found = -1;
                    for (int i0 = c + 1; i0 < n && found < 0; i0 += 32) {
                        const uint32_t m = __ballot_sync(0xffffffffu, i0 + lane < n && sm.up[i0 + lane] == v);
                        if (m) found = i0 + __ffs(m) - 1;
                    }
                    if (found < 0) {
                        if (greedy) {
                            if (lane == 0) a.next[b] = best;
                            cmd.ask = kEnd;
                        } else {
                            cmd = Cmd{kDraw, v, S, gone};
                        }
                        break;
                    }
                    c = found;
                    const int x = sm.tok[c];
                    if (x < 0 || x >= a.vocab) {
                        odd = true;
                        continue;
                    }
                    bool yes;
                    if (greedy) {
                        yes = x == best;
                    } else {
                        uint64_t left = to_units(sm.p[c]);
                        if (S) left = left_of(left, S, to_units(sm.d[c]));
                        bool had = false;
                        for (int k = lane; k < gone; k += 32) had |= sm.gone[k] == x;
                        if (__any_sync(0xffffffffu, had)) left = 0;
                        const double d = fminf(fmaxf(sm.d[c], 0.f), 2.f);
                        yes = static_cast<double>(sm.u[c]) * d * R < static_cast<double>(left) * 8.673617379884035e-19;
                    }
                    if (yes) {
                        if (lane == 0) a.path[r0 + len] = c;
                        ++len;
                        v = c;
                        S = 0;
                        R = 1.0;
                        gone = 0;
                        best = -1;
                        if (greedy) cmd = Cmd{kBest, v, 0, 0};
                    } else if (!greedy) {
                        if (a.draft) {
                            S_next = S + static_cast<uint64_t>(R * 1125899906842624.0);
                            cmd = Cmd{kSum, v, S_next, 0};
                        } else {
                            if (lane == 0) sm.gone[gone] = x;
                            __syncwarp();
                            cmd = Cmd{kSum, v, 0, gone + 1};
                        }
                    }
                }
            }
            for (uint32_t k = lane; k < ctas; k += 32) {
                const uint32_t to = remote_addr(&sm.cmd, k);
                remote_store(to, static_cast<uint64_t>(static_cast<uint32_t>(cmd.ask)) | (static_cast<uint64_t>(static_cast<uint32_t>(cmd.node)) << 32));
                remote_store(to + 8, cmd.S);
                remote_store(to + 16, static_cast<uint64_t>(cmd.gone));
                if (cmd.gone)
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote_addr(&sm.gone[cmd.gone - 1], k)), "r"(sm.gone[cmd.gone - 1]) : "memory");
            }
        }
        __syncwarp();
        cluster_sync_all();
        cmd = sm.cmd;
        if (cmd.ask == kEnd) break;
        // ---- every CTA: its slice
        const Row<T> p(a.target, r0 + cmd.node, a.n_rows, a.vocab);
        const Row<T> d(a.draft ? a.draft : a.target, r0 + cmd.node, a.n_rows, a.vocab);
        const int parts = static_cast<int>(ctas) * kVWarps, mine = static_cast<int>(rank) * kVWarps + warp;
        const int per = (p.pieces + parts - 1) / parts;
        const int j0 = min(mine * per, p.pieces), j1 = min(j0 + per, p.pieces);
        uint64_t sum = 0;
        if (cmd.ask == kBest) {
            for (int j = j0 + lane; j < j1; j += 32) {
                float f[Vec<T>::n];
                p.load(j, f);
                const int64_t t0 = p.first(j);
#pragma unroll
                for (int i = 0; i < Vec<T>::n; ++i)
                    if (t0 + i >= 0 && t0 + i < a.vocab) {
                        const bool nan = f[i] != f[i];
                        bad |= nan;
                        sum = max(sum, (static_cast<uint64_t>(nan ? 0u : order_key(f[i])) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(t0 + i)));
                    }
            }
            sum = warp_max64(sum);
        } else {
            for (int j = j0 + lane; j < j1; j += 32) {
                uint64_t x[Vec<T>::n];
                piece_left<T>(p, d, j, cmd, sm.gone, x, &bad);
#pragma unroll
                for (int i = 0; i < Vec<T>::n; ++i) sum += x[i];
            }
            sum = warp_sum64(sum);
        }
        if (lane == 0) sm.warp_sum[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            uint64_t all = lane < kVWarps ? sm.warp_sum[lane] : 0;
            all = cmd.ask == kBest ? warp_max64(all) : warp_sum64(all);
            if (lane < static_cast<int>(ctas)) remote_store(remote_addr(&sm.slot[rank], lane), all);
        }
        __syncwarp();
        cluster_sync_all();
        uint64_t total = 0, before = 0;
        for (uint32_t k = 0; k < ctas; ++k) {
            if (cmd.ask == kBest) total = max(total, sm.slot[k]);
            else total += sm.slot[k];
            if (k < rank) before += sm.slot[k];
        }
        if (cmd.ask == kBest) {
            best = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(total));
        } else if (cmd.ask == kSum) {
            if (total > 0) {
                S = S_next;
                R = static_cast<double>(total) * 8.673617379884035e-19;
                gone = cmd.gone;
            }
        } else {  // ---- the token behind the path
            bool off = false;
            const float u = unit_interval(a.u_pick[b], &off);
            if (total == 0) {
                if (rank == 0 && tid == 0) {
                    a.next[b] = 0;
                    odd = true;
                }
            } else {
                uint64_t at = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
                at = min(at, total - 1);
                // warp `warp` holds the token when `at` lies in its sums
                for (int w = 0; w < warp; ++w) before += sm.warp_sum[w];
                if (at >= before && at - before < sm.warp_sum[warp]) {
                    at -= before;
                    for (int base = j0; base < j1; base += 32) {
                        uint64_t x[Vec<T>::n], s = 0;
                        const int j = base + lane;
                        if (j < j1) {
                            piece_left<T>(p, d, j, cmd, sm.gone, x, &bad);
                        } else {
#pragma unroll
                            for (int i = 0; i < Vec<T>::n; ++i) x[i] = 0;
                        }
#pragma unroll
                        for (int i = 0; i < Vec<T>::n; ++i) s += x[i];
                        uint64_t up = s;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const uint64_t y = __shfl_up_sync(0xffffffffu, up, o);
                            if (lane >= o) up += y;
                        }
                        const uint32_t past = __ballot_sync(0xffffffffu, up > at);
                        if (past) {
                            if (lane == __ffs(past) - 1) {
                                uint64_t run = up - s;
                                int64_t tok = p.first(j);
                                bool done = false;
#pragma unroll
                                for (int i = 0; i < Vec<T>::n; ++i) {
                                    run += x[i];
                                    if (!done && run > at) {
                                        done = true;
                                        tok += i;
                                    }
                                }
                                a.next[b] = static_cast<int32_t>(tok);
                            }
                            break;
                        }
                        at -= __shfl_sync(0xffffffffu, up, 31);
                    }
                }
            }
            if (off && rank == 0 && tid == 0) odd = true;
            break;
        }
    }
    if (rank == 0 && tid == 0 && n > 0) a.count[b] = len;
    if (bad) sm.bad = 1;
    if (odd) set_status(a.status, ECHO_ST_BADDATA);
    __syncthreads();
    if (tid == 0 && sm.bad) set_status(a.status, ECHO_ST_NAN);
    cluster_sync_all();  // no CTA leaves while another may still write to it
}

template <class T>
int launch_verify(const VerifyArgs& a, int B, cudaStream_t s) {
    int ctas = kMaxCluster;
    while (ctas > 1 && static_cast<int64_t>(B) * ctas > 4ll * sm_count()) ctas /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(B) * ctas);
    cfg.blockDim = dim3(kVT);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ECHO_CUDA_OK(cudaLaunchKernelEx(&cfg, verify_kernel<T>, a));
    return ECHO_OK;
}

}  // namespace
}  // namespace echo

extern "C" int echo_draft_verify(int B, const int64_t* row_off, int64_t n_rows, const int32_t* parent, const int32_t* token,
                                 int64_t vocab, int dtype, const void* target, const void* draft, const float* u_node,
                                 const float* u_pick, int32_t* path, int32_t* count, int32_t* next, int32_t* status,
                                 echo_stream_t stream) {
    using namespace echo;
    if (B <= 0 || n_rows < 0 || vocab < 1 || !row_off || !count || !next || !status) return ECHO_EINVAL;
    if (B > ECHO_MAX_REQUESTS || n_rows > ECHO_CHUNK_MAX_ROWS || vocab > ECHO_MAX_VOCAB || (dtype != ECHO_F32 && dtype != ECHO_BF16))
        return ECHO_EUNSUPPORTED;
    if (n_rows > 0 && (!parent || !token || !target || !path)) return ECHO_EINVAL;
    if ((u_node != nullptr) != (u_pick != nullptr)) return ECHO_EINVAL;
    if (!is_aligned(target, 16) || !is_aligned(draft, 16)) return ECHO_EINVAL;
    const VerifyArgs a = {row_off, n_rows, parent, token, vocab, target, u_node ? draft : nullptr, u_node, u_pick, path, count, next, status};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == ECHO_F32 ? launch_verify<float>(a, B, s) : launch_verify<__nv_bfloat16>(a, B, s);
}
