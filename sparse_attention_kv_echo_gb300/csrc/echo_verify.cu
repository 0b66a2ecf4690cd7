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
// slice of that, read 16 bytes a lane.  CTA 0 reads the tree and each node's own probabilities
// in its parent's rows and hands them to all; then every CTA walks (a warp; the children of a node are
// found by ballot among 32 parents at a time) and the cluster sums where a child is rejected:
// one cluster barrier a rejection, behind which all CTAs know all slices' sums and go on
// alike.  At the end the token behind the path is drawn, from the last rejection's sums when no
// child was accepted since: the slice whose running sum passes u * total, in it the warp's, in that
// one sixteenth, in that the token.
// Values are 64-bit integers in units of 2^-60, so sums do not hang on their order, and
// the token drawn is the same on any number of CTAs.  They are made by shifts: conversions
// to 64-bit integers ran at a small fraction of the rate of integer operations (64 chains of six over
// 131072 tokens took 96 us with them).
#include <cuda_bf16.h>

#include "echo_common.cuh"
#include "echo_tc.cuh"

namespace echo {
namespace {

constexpr int kVT = 384;
constexpr int kVWarps = kVT / 32;
constexpr int kMaxCluster = 8;
constexpr int kNodes = ECHO_TREE_MAX_NODES;
constexpr int kTile = 8;                 // tokens a lane works on at a time

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

// What the walk asks of the cluster: sum up what is left, or find the largest, at a node.
enum Ask : int { kSum, kBest, kEnd };

constexpr uint64_t kOne = 1ull << 50;  // S = 1

struct VerifySmem {
    // from CTA 0: the tree
    int64_t r0;
    int32_t n;
    float u_pick;
    int16_t up[kNodes];
    int32_t tok[kNodes];
    float u[kNodes], p[kNodes], d[kNodes];  // a node's uniform number, its token's probabilities in its parent's rows
    // from every CTA: its sum or its best key, by parity of the question
    uint64_t slot[2][kMaxCluster];
    // the question
    int ask, node, gone;
    bool fresh;                    // the last sums are of this node and residual
    uint64_t S;
    int32_t out[kNodes];           // tokens left out (drafts without probabilities)
    // the walk of this CTA's warp 0, between its turns
    uint64_t S_at, R;              // the residual at v
    int v, c, len, outs, best;     // node, the last child tried, nodes accepted, tokens left out, greedy: v's best
    int16_t path[kNodes];
    uint64_t warp_sum[kVWarps];
    uint64_t fine[kVWarps];
};

// Bits of a probability; NaN and negative values count as 0, values above 2 as 2.
constexpr uint32_t kTwo = 0x40000000u;
__device__ __forceinline__ uint32_t tame(uint32_t bits, bool* bad) {
    if (bits <= kTwo) return bits;
    if (bits == 0x80000000u) return 0u;  // -0
    *bad = true;
    return bits < 0x7F800001u ? kTwo : 0u;
}
// A probability in units of 2^-60: the mantissa at the top of 64 bits, shifted down by what its exponent lacks.
__device__ __forceinline__ uint64_t to_units(uint32_t bits) {
    const uint64_t m = static_cast<uint64_t>((bits << 8) | 0x80000000u) << 32;
    uint64_t x;
    asm("shr.u64 %0, %1, %2;" : "=l"(x) : "l"(m), "r"(130u - (bits >> 23)));  // (0 from 64 on)
    return x;
}

// S d in units for an S in units of 2^-50 (all ones above 2^61).
__device__ __forceinline__ uint64_t scaled(uint64_t S, uint32_t d) {
    const uint64_t y = to_units(d), lo = S * y, hi = __umul64hi(S, y);
    return hi >> 47 ? ~0ull : (hi << 14) | (lo >> 50);
}
__device__ __forceinline__ uint64_t minus(uint64_t p, uint64_t x) { return p > x ? p - x : 0; }

// S as the sum of two floats (48 bits of it).
struct Scale {
    float hi, lo;
    uint64_t S;
};
__device__ __forceinline__ Scale scale_of(uint64_t S) {
    const float hi = __ull2float_rn(S);
    const float lo = __ll2float_rn(static_cast<int64_t>(S - __float2ull_rn(hi)));
    return Scale{hi * 8.8817841970012523e-16f, lo * 8.8817841970012523e-16f, S};  // 2^-50
}

// s + t is what is left of a token, max(0, p - S d), t below the last place of p or of S d.  kUnit: S is 1, or d is 0.
template <bool kUnit>
__device__ __forceinline__ void left_of(float p, float d, const Scale& S, float* s, float* t) {
    if (kUnit) {
        const float x = fminf(d, p);  // p >= x: what the difference loses is exact
        *s = __fsub_rn(p, x);
        *t = __fsub_rn(__fsub_rn(p, *s), x);
    } else {
        const float x = __fmul_rn(S.hi, d), w = __fmaf_rn(S.lo, d, __fmaf_rn(S.hi, d, -x));
        *s = __fsub_rn(p, x);
        *t = __fsub_rn(__fsub_rn(__fsub_rn(p, *s), x), w);
        const bool some = p >= x && __fadd_rn(*s, *t) > 0.f;
        *s = some ? *s : 0.f;
        *t = some ? *t : 0.f;
    }
}

// s + t in units of 2^-60, spread over three 32-bit numbers whose sums are exact: a constant added to a float rounds it to
// units that the low bits then count, and the remainder, scaled up, goes the same way again.  That runs on the pipe of FFMA and
// FADD; shifting mantissas into 64-bit numbers ran on the integers' pipe, half as wide.  What a value loses
// is below 2^-48, the same wherever it is summed.
constexpr uint32_t kTopBits = 0x40000000u, kLowBits = 0x40400000u;  // of 2 and 3
struct Units {
    uint32_t hi, mid, lo;  // of 2^-22, 2^-44 and 2^-60, + kTopBits, kLowBits, kLowBits
};
__device__ __forceinline__ Units spread(float s, float t) {
    const float y = __fadd_rn(s, 2.f), r = __fadd_rn(__fsub_rn(s, __fsub_rn(y, 2.f)), t);
    const float z = __fmaf_rn(r, 4194304.f, 3.f), q = __fmaf_rn(r, 4194304.f, __fsub_rn(3.f, z));
    return Units{__float_as_uint(y), __float_as_uint(z), __float_as_uint(__fmaf_rn(q, 65536.f, 3.f))};
}
// The sum of n values from the sums of their parts.
__device__ __forceinline__ uint64_t together(uint32_t n, uint32_t hi, uint32_t mid, uint32_t lo) {
    const int64_t m = static_cast<int32_t>(mid - n * kLowBits), l = static_cast<int32_t>(lo - n * kLowBits);
    return (static_cast<uint64_t>(hi - n * kTopBits) << 38) + static_cast<uint64_t>(m * 65536 + l);
}

template <class T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int n = 4;
    __device__ static __forceinline__ void unpack(const uint4& v, uint32_t* x) {
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    }
    __device__ static __forceinline__ uint32_t one(const void* p, int64_t i) { return static_cast<const uint32_t*>(p)[i]; }
    __device__ static __forceinline__ uint4 pack(const uint32_t (&x)[4]) { return make_uint4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    __device__ static __forceinline__ void unpack(const uint4& v, uint32_t* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = w[i] << 16;
            x[2 * i + 1] = w[i] & 0xFFFF0000u;
        }
    }
    __device__ static __forceinline__ uint32_t one(const void* p, int64_t i) {
        return static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16;
    }
    __device__ static __forceinline__ uint4 pack(const uint32_t (&x)[8]) {
        return make_uint4((x[0] >> 16) | x[1], (x[2] >> 16) | x[3], (x[4] >> 16) | x[5], (x[6] >> 16) | x[7]);
    }
};

// Row `row` of the [n_rows, vocab] matrices target and draft as 16-byte pieces on 16-byte boundaries: piece j holds
// the tokens first(j) .. first(j) + n - 1, of which the first and the last piece may have some outside the row.
template <class T>
struct Row {
    const T* base;      // of the target's piece 0, at or before the row's first element
    int64_t to_draft;   // bytes from there to the draft's
    int64_t whole;      // pieces before the matrix ends
    int vocab;
    int shift;          // elements of piece 0 before the row
    int pieces;
    int inner;          // pieces [1, inner) lie within the row and the matrix
    __device__ __forceinline__ Row(const VerifyArgs& a, int64_t row) {
        constexpr int n = Vec<T>::n;
        const int64_t at = row * a.vocab;
        shift = static_cast<int>(at % n);
        base = static_cast<const T*>(a.target) + (at - shift);
        to_draft = a.draft ? static_cast<const uint8_t*>(a.draft) - static_cast<const uint8_t*>(a.target) : 0;
        whole = (a.n_rows * a.vocab - (at - shift)) / n;
        vocab = static_cast<int>(a.vocab);
        pieces = static_cast<int>((a.vocab + shift + n - 1) / n);
        inner = static_cast<int>(min(whole, (a.vocab + shift) / n));
    }
    __device__ __forceinline__ int first(int j) const { return j * Vec<T>::n - shift; }
    __device__ __forceinline__ const uint4* at(int j, bool draft) const {
        return reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(base) + (draft ? to_draft : 0)) + j;
    }
    __device__ __forceinline__ uint4 load_inner(int j, bool draft) const { return __ldg(at(j, draft)); }
    __device__ __forceinline__ uint4 load(int j, bool draft) const {
        constexpr int n = Vec<T>::n;
        if (j < whole) return __ldg(at(j, draft));
        uint32_t x[n];  // the matrix ends within the piece
#pragma unroll
        for (int i = 0; i < n; ++i) x[i] = in(first(j) + i) ? Vec<T>::one(at(j, draft), i) : 0u;
        return Vec<T>::pack(x);
    }
    __device__ __forceinline__ bool in(int t) const { return t >= 0 && t < vocab; }
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// The first lane whose running sum of x passes *at (-1: none); *at becomes what it has to pass in that lane.
__device__ __forceinline__ int warp_find(uint64_t x, uint64_t* at) {
    uint64_t run = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, run, o);
        if ((threadIdx.x & 31) >= o) run += y;
    }
    const int found = __ffs(__ballot_sync(0xffffffffu, run > *at)) - 1;
    const uint64_t before = __shfl_sync(0xffffffffu, run - x, found < 0 ? 31 : found);
    *at -= found < 0 ? before + __shfl_sync(0xffffffffu, x, 31) : before;
    return found;
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
__device__ __forceinline__ void remote_store64(uint32_t a, uint64_t x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(x) : "memory");
}
__device__ __forceinline__ void remote_store32(uint32_t a, uint32_t x) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ void remote_store16(uint32_t a, int16_t x) {
    asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(a), "h"(x) : "memory");
}

// The values of piece j made fit: tokens outside the row and those left out are 0, so are NaN and negative values, and
// values above 2 are 2.
template <class T>
__device__ __forceinline__ void mend_piece(const Row<T>& row, int j, const int32_t* out, int outs, uint32_t* p, uint32_t* d, bool* bad) {
    constexpr int n = Vec<T>::n;
    const int t0 = row.first(j);
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const bool in = row.in(t0 + i);
        p[i] = in ? tame(p[i], bad) : 0u;
        d[i] = in ? tame(d[i], bad) : 0u;
    }
    for (int k = 0; k < outs; ++k) {
        const int at = out[k] - t0;
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (at == i) p[i] = 0u;
    }
}

// The sum of what is left in pieces [j0, j1), of the whole warp in every lane; kTile tokens a lane at a time.
template <class T, bool kUnit>
__device__ __forceinline__ uint64_t sum_left(const Row<T>& row, int j0, int j1, const Scale& S, const int32_t* out, int outs, bool* bad) {
    constexpr int n = Vec<T>::n, kFly = kTile / n;
    const int lane = threadIdx.x & 31;
    const bool draft = S.S != 0;
    uint64_t sum = 0;
    uint32_t hi = 0u, mid = 0u, lo = 0u, held = 0u;  // of at most 256 values: below 2^32
#pragma unroll 1
    for (int j = j0; j < j1; j += 32 * kFly) {
        // the ends of a row, and of the matrix, and tokens left out are looked for one by one
        bool inner = j > 0 && min(j + 32 * kFly, j1) <= row.inner;
        for (int k = 0; k < outs; ++k) inner = inner && (out[k] < row.first(j) || out[k] >= row.first(j + 32 * kFly));
        uint32_t p[kTile], d[kTile], most = 0u;
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int at = j + 32 * f + lane;
            uint4 pv = make_uint4(0u, 0u, 0u, 0u), dv = pv;
            if (at < j1) {
                if (inner) {
                    pv = row.load_inner(at, false);
                    if (draft) dv = row.load_inner(at, true);
                } else {
                    pv = row.load(at, false);
                    if (draft) dv = row.load(at, true);
                }
            }
            Vec<T>::unpack(pv, p + n * f);
            Vec<T>::unpack(dv, d + n * f);
        }
#pragma unroll
        for (int i = 0; i < kTile; ++i) most = max(most, max(p[i], d[i]));
        if (!inner || most > kTwo) {
#pragma unroll
            for (int f = 0; f < kFly; ++f)
                if (j + 32 * f + lane < j1) mend_piece<T>(row, j + 32 * f + lane, out, outs, p + n * f, d + n * f, bad);
        }
#pragma unroll
        for (int i = 0; i < kTile; i += 2) {
            Units u[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float s, t;
                left_of<kUnit>(__uint_as_float(p[i + k]), __uint_as_float(d[i + k]), S, &s, &t);
                u[k] = spread(s, t);
            }
            hi += u[0].hi + u[1].hi;
            mid += u[0].mid + u[1].mid;
            lo += u[0].lo + u[1].lo;
        }
        held += kTile;
        if (held == 256) {
            sum += together(held, hi, mid, lo);
            hi = mid = lo = held = 0u;
        }
    }
    sum += together(held, hi, mid, lo);
    return warp_sum64(sum);
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// The first of the largest in pieces [j0, j1): its order key above, the complement of its index below (NaN: key 0).
template <class T>
__device__ __forceinline__ uint64_t best_of(const Row<T>& row, int j0, int j1, bool* nan) {
    constexpr int n = Vec<T>::n, kFly = 2;
    const int lane = threadIdx.x & 31;
    float best = -INFINITY;
    int at = -1, first = -1;  // the best number's token, the first token
#pragma unroll 1
    for (int j = j0; j < j1; j += 32 * kFly) {
        uint4 v[kFly];
#pragma unroll
        for (int f = 0; f < kFly; ++f)
            if (j + 32 * f + lane < j1) v[f] = row.load(j + 32 * f + lane, false);
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            if (j + 32 * f + lane >= j1) break;
            uint32_t x[n];
            Vec<T>::unpack(v[f], x);
            float m = __uint_as_float(x[0]);
#pragma unroll
            for (int i = 1; i < n; ++i) m = max_or_nan(m, __uint_as_float(x[i]));
            if (!(m <= best) || at < 0) {  // seldom once some have been seen
                const int t0 = row.first(j + 32 * f + lane);
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float y = __uint_as_float(x[i]);
                    if (!row.in(t0 + i)) continue;
                    if (first < 0) first = t0 + i;
                    if (y != y) {
                        *nan = true;
                    } else if (y > best || at < 0) {  // ascending: an equal one comes later
                        best = y;
                        at = t0 + i;
                    }
                }
            }
        }
    }
    uint64_t key = 0;
    if (first >= 0) key = (static_cast<uint64_t>(at < 0 ? 0u : order_key(best)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(at < 0 ? first : at));
    return warp_max64(key);
}

__device__ __forceinline__ float unit_interval(float u, bool* bad) {
    *bad |= !(u >= 0.f && u < 1.f);
    return fminf(fmaxf(u, 0.f), 0.99999994f);  // NaN: 0
}

// u in units of 2^-32.
__device__ __forceinline__ uint32_t fraction(float u) { return static_cast<uint32_t>(__float2uint_rz(u * 4294967296.f)); }

// u d R < left, all in units (R below 2^63).
__device__ __forceinline__ bool accepts(float u, uint64_t d, uint64_t R, uint64_t left) {
    const uint64_t y = __umul64hi(d << 2, R << 1);  // d R in units of 2^-59
    return __umul64hi(y, static_cast<uint64_t>(fraction(u)) << 32) << 1 < left;
}

// T: the probabilities' type.
template <class T>
__global__ void __launch_bounds__(kVT, 2) verify_kernel(VerifyArgs a) {
    __shared__ VerifySmem sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int b = blockIdx.x / ctas;
    const int parts = static_cast<int>(ctas) * kVWarps, mine = static_cast<int>(rank) * kVWarps + warp;
    const bool greedy = a.u_pick == nullptr;
    bool bad = false, odd = false;  // probabilities / other data that are none
    // ---- CTA 0 reads the tree and hands it to all, so that every CTA walks on the same data
    const int64_t r0 = a.row_off[b], r1 = a.row_off[b + 1];
    const bool whole = r0 >= 0 && r1 >= r0 && r1 <= a.n_rows && r1 - r0 <= kNodes;
    if (rank == 0) {
        const int n = whole ? static_cast<int>(r1 - r0) : 0;
        odd = !whole;
        if (r1 - r0 > kNodes && r0 >= 0 && r1 <= a.n_rows)
            for (int64_t i = r0 + tid; i < r1; i += kVT) a.path[i] = -1;
        for (int i = tid; i < n; i += kVT) {
            int up = a.parent[r0 + i];
            const int x = a.token[r0 + i];
            const float u = greedy ? 0.f : a.u_node[r0 + i];
            uint32_t p = 0u, d = 0u;
            if (up < -1 || up >= i) {
                odd = true;
                up = -1;
            }
            if (!greedy && up >= 0 && x >= 0 && x < a.vocab) {
                const int64_t at = (r0 + up) * a.vocab + x;
                p = tame(Vec<T>::one(a.target, at), &bad);
                d = a.draft ? tame(Vec<T>::one(a.draft, at), &bad) : 0x3F800000u;
            }
            const float uu = up >= 0 ? unit_interval(u, &odd) : 0.f;
            for (uint32_t k = 0; k < ctas; ++k) {
                remote_store16(remote_addr(&sm.up[i], k), static_cast<int16_t>(up));
                remote_store32(remote_addr(&sm.tok[i], k), static_cast<uint32_t>(x));
                remote_store32(remote_addr(&sm.u[i], k), __float_as_uint(uu));
                remote_store32(remote_addr(&sm.p[i], k), p);
                remote_store32(remote_addr(&sm.d[i], k), d);
            }
        }
        if (tid < static_cast<int>(ctas)) {
            float u = 0.f;
            if (!greedy && n > 0) u = unit_interval(a.u_pick[b], &odd);
            remote_store64(remote_addr(&sm.r0, tid), static_cast<uint64_t>(n > 0 ? r0 : 0));
            remote_store32(remote_addr(&sm.n, tid), static_cast<uint32_t>(n));
            remote_store32(remote_addr(&sm.u_pick, tid), __float_as_uint(u));
        }
        __syncwarp();
    }
    if (tid == 0) {
        sm.path[0] = 0;
        sm.v = sm.c = sm.outs = 0;
        sm.len = 1;
        sm.S_at = 0;
        sm.R = 1ull << 60;
        sm.fresh = false;
    }
    // greedy: the root's best is asked for at once, and answered behind the same barrier as the tree
    bool first = greedy, fine = false;
    int asked = 0, j0 = 0, j1 = 0;
    uint64_t at = 0;              // what is left to pass of the draw's sum
    if (!first) {
        cluster_sync_all();
        if (sm.n == 0) goto done;
    }
    for (;;) {
        if (!first && !fine) {
            if (warp == 0) {
                __syncwarp();
                const int n = sm.n;
                int ask = -1, v = sm.v, c = sm.c, len = sm.len, outs = sm.outs, tried = outs;
                uint64_t S = sm.S_at, R = sm.R, S_try = S;
                bool fresh = sm.fresh;
                while (ask < 0) {
                    // the next child of v behind c
                    int found = -1;
                    for (int i0 = c + 1; i0 < n && found < 0; i0 += 32) {
                        const uint32_t m = __ballot_sync(0xffffffffu, i0 + lane < n && sm.up[i0 + lane] == v);
                        if (m) found = i0 + __ffs(m) - 1;
                    }
                    if (found < 0) {
                        ask = kEnd;
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
                        yes = x == sm.best;
                    } else {
                        const uint32_t d = __float_as_uint(sm.d[c]);
                        uint64_t left = to_units(__float_as_uint(sm.p[c]));
                        if (S) left = minus(left, scaled(S, d));
                        if (outs) {
                            bool had = false;
                            for (int k = lane; k < outs; k += 32) had |= sm.out[k] == x;
                            if (__any_sync(0xffffffffu, had)) left = 0;
                        }
                        yes = accepts(sm.u[c], to_units(d), R, left);
                    }
                    if (yes) {
                        if (lane == 0) sm.path[len] = static_cast<int16_t>(c);
                        ++len;
                        v = c;
                        S = 0;
                        R = 1ull << 60;
                        outs = 0;
                        fresh = false;
                        if (greedy) ask = kBest;
                    } else if (!greedy) {
                        ask = kSum;
                        if (a.draft) {
                            S_try = S + (R >> 10);
                        } else {
                            if (lane == 0) sm.out[outs] = x;
                            tried = outs + 1;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    sm.v = v;
                    sm.c = c;
                    sm.len = len;
                    sm.outs = outs;
                    sm.S_at = S;
                    sm.R = R;
                    sm.fresh = fresh;
                    sm.ask = ask;
                    sm.node = v;
                    sm.S = ask == kSum ? S_try : S;
                    sm.gone = ask == kSum ? tried : outs;
                }
            }
            __syncthreads();
        }
        const int ask = first ? kBest : sm.ask, outs_now = first ? 0 : sm.gone;
        const Scale S_now = scale_of(first ? 0 : sm.S);
        const bool unit = S_now.S == 0 || S_now.S == kOne;
        if (ask == kEnd && greedy) break;
        const int64_t row = first ? (whole && r1 > r0 ? r0 : 0) : sm.r0 + sm.node;
        const Row<T> p(a, row);
        const int per = (p.pieces + parts - 1) / parts;
        if (fine || ask != kEnd || !sm.fresh) {
            // ---- every CTA: its slice, a warp's slice of it, or the warp's part of the slice that holds the token
            if (!fine) {
                j0 = min(mine * per, p.pieces);
                j1 = first && !(whole && r1 > r0) ? j0 : min(j0 + per, p.pieces);
            }
            uint64_t sum;
            if (ask == kBest) sum = best_of<T>(p, j0, j1, &bad);
            else if (unit) sum = sum_left<T, true>(p, j0, j1, S_now, sm.out, outs_now, &bad);
            else sum = sum_left<T, false>(p, j0, j1, S_now, sm.out, outs_now, &bad);
            if (lane == 0) (fine ? sm.fine : sm.warp_sum)[warp] = sum;
            __syncthreads();
            if (!fine) {
                ++asked;
                if (warp == 0) {
                    uint64_t all = lane < kVWarps ? sm.warp_sum[lane] : 0;
                    all = ask == kBest ? warp_max64(all) : warp_sum64(all);
                    if (lane < static_cast<int>(ctas)) remote_store64(remote_addr(&sm.slot[asked & 1][rank], lane), all);
                    __syncwarp();
                }
                cluster_sync_all();
            }
        }
        if (fine) {  // ---- the token: a warp's part, a lane's piece
            if (warp_find(lane < kVWarps ? sm.fine[lane] : 0, &at) != warp) break;
            for (int base = j0; base < j1; base += 32) {
                uint64_t x[Vec<T>::n], s = 0;
                const int j = base + lane;
#pragma unroll
                for (int i = 0; i < Vec<T>::n; ++i) x[i] = 0;
                if (j < j1) {
                    uint32_t pb[Vec<T>::n], db[Vec<T>::n];
                    Vec<T>::unpack(p.load(j, false), pb);
                    Vec<T>::unpack(S_now.S ? p.load(j, true) : make_uint4(0u, 0u, 0u, 0u), db);
                    mend_piece<T>(p, j, sm.out, outs_now, pb, db, &bad);
#pragma unroll
                    for (int i = 0; i < Vec<T>::n; ++i) {
                        float l, t;
                        if (unit) left_of<true>(__uint_as_float(pb[i]), __uint_as_float(db[i]), S_now, &l, &t);
                        else left_of<false>(__uint_as_float(pb[i]), __uint_as_float(db[i]), S_now, &l, &t);
                        const Units y = spread(l, t);
                        x[i] = together(1u, y.hi, y.mid, y.lo);
                        s += x[i];
                    }
                }
                const int found = warp_find(s, &at);
                if (found >= 0) {
                    if (lane == found) {
                        uint64_t run = 0;
                        int t = -1;
#pragma unroll
                        for (int i = 0; i < Vec<T>::n; ++i) {
                            run += x[i];
                            if (t < 0 && run > at) t = p.first(j) + i;
                        }
                        a.next[b] = t;
                    }
                    break;
                }
            }
            break;
        }
        const uint64_t* const slot = sm.slot[asked & 1];
        uint64_t total = 0, before = 0;
        for (uint32_t k = 0; k < ctas; ++k) {
            const uint64_t x = slot[k];
            total = ask == kBest ? max(total, x) : total + x;
            if (k < rank) before += x;
        }
        if (ask == kBest) {
            if (sm.n == 0) break;
            if (tid == 0) sm.best = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(total));
            first = false;
        } else if (ask == kSum) {
            if (tid == 0) {
                sm.fresh = total > 0;
                if (total > 0) {
                    sm.S_at = S_now.S;
                    sm.R = total;
                    sm.outs = outs_now;
                }
            }
        } else {  // ---- the token behind the path is in the CTA, the warp's slice and then the part of it that holds u * total
            if (total == 0) {
                odd = true;
                if (rank == 0 && tid == 0) a.next[b] = 0;
                break;
            }
            at = __umul64hi(total, static_cast<uint64_t>(fraction(sm.u_pick)) << 32);
            if (at < before || at - before >= slot[rank]) break;
            at -= before;
            const int w = warp_find(lane < kVWarps ? sm.warp_sum[lane] : 0, &at);
            const int s0 = min((static_cast<int>(rank) * kVWarps + w) * per, p.pieces), s1 = min(s0 + per, p.pieces);
            const int sub = (s1 - s0 + kVWarps - 1) / kVWarps;
            j0 = min(s0 + warp * sub, s1);
            j1 = min(j0 + sub, s1);
            fine = true;
        }
    }
done:
    // ---- CTA 0's warp 0 knows the path
    if (rank == 0 && warp == 0) {
        __syncwarp();
        const int n = sm.n, len = sm.len;
        for (int i = lane; i < n; i += 32) a.path[sm.r0 + i] = i < len ? sm.path[i] : -1;
        if (lane == 0) {
            a.count[b] = n > 0 ? len : 0;
            if (n == 0 || greedy) a.next[b] = n > 0 ? sm.best : -1;
        }
    }
    if (odd || bad) set_status(a.status, (odd ? ECHO_ST_BADDATA : 0) | (bad ? ECHO_ST_NAN : 0));
}

template <class T>
int launch_verify(const VerifyArgs& a, int B, cudaStream_t s) {
    int ctas = kMaxCluster;
    while (ctas > 1 && static_cast<int64_t>(B) * ctas > 2ll * sm_count()) ctas /= 2;
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
