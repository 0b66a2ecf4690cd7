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
// slice of that, read 16 bytes a lane.  CTA 0 reads the tree, each node's own probabilities
// in its parent's rows and whether it would be accepted as a first child, and hands them to all; then every CTA walks (a
// warp; the children of a node are found by ballot among 32 parents at a time) and the cluster sums where a
// child is rejected: one cluster barrier a rejection, behind which all CTAs know all slices'
// sums and go on alike.  At the end the token behind the path is drawn, from the last rejection's
// sums when no child was accepted since: the slice whose running sum passes u * total, in it the
// warp's, in that the part that a warp of the CTA now takes, in that the token.
//
// Greedy asks for the largest of a row in the same way, node after node, or for those of all nodes at once where they are
// few and short.
//
// Sums are of whole numbers, so they do not hang on their order, and the token drawn is the same on
// any number of CTAs.  What bounds the call: a few chains or trees, the latency of its steps (one chain of five
// over 32000 tokens, 8.7 us in a graph: 1.9 to read the tree, 0.5 a walk, 2 a sum with its barrier, 2 the draw); many, the
// instructions of the sums, some 10 a token and pair of values, and the chain of rejections of the longest walk.  64 chains of
// six over 131072 tokens in fp32 19 us (60 MB, 3.1 TB/s), 32 trees of 32 to 48 nodes in bf16 30 us, 16 greedy trees of 8 to 24
// over 50001 tokens 14 us (each in a graph on one input).
#include <cuda_bf16.h>

#include "echo_common.cuh"
#include "echo_tc.cuh"

namespace echo {
namespace {

constexpr int kVT = 384;
constexpr int kVWarps = kVT / 32;
constexpr int kMaxCluster = 8;
constexpr int kNodes = ECHO_TREE_MAX_NODES;
constexpr int kTile = 8;                 // tokens a lane works on at a time (16: more registers, 2 CTAs an SM no longer without spills)

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
    int64_t all_bytes;  // greedy: rows of at most so many bytes have their best found at once
};

// Greedy: a request whose rows are at most so many bytes for each CTA that has an SM to itself (half where two share one) has
// the best of every node found at once, all on the way or not; a larger one, node after node, 2.3 us and more each.  At
// once against in turn: a chain of 5, 32000 tokens in fp32 (80 KB a CTA), 8.2 against 14.9 us, 8 chains of 6 over 131072 in bf16
// (196 KB) 11.0 against 15.4, a tree of 16 (524 KB) 18.5 against 9.3, 64 trees of 16 over 32000 (256 KB, two to an SM) 16.4
// against 13.9.
constexpr int64_t kAllBytes = 256 * 1024;
constexpr int kAllNodes = 128;
constexpr int kAllFly = 8;               // 16-byte pieces a lane has in flight then (4: up to 5% slower)

// What the walk asks of the cluster: sum up what is left, or find the largest, at a node.
enum Ask : int { kSum, kBest, kEnd };

constexpr uint64_t kOne = 1ull << 50;  // S = 1

// Row `row` of the [n_rows, vocab] matrices target and draft as 16-byte pieces on 16-byte boundaries: piece j holds
// the tokens first(j) .. first(j) + n - 1, of which the first and the last piece may have some outside the row.
struct Row {
    const uint8_t* base;  // of the target's piece 0, at or before the row's first element
    int64_t to_draft;     // bytes from there to the draft's
    int vocab;
    int shift;            // elements of piece 0 before the row
    int pieces;
    int inner;            // pieces [1, inner) lie within the row and the matrix
    int whole;            // pieces [0, whole) lie within the matrix
    int per;              // pieces of a warp's slice
};

struct VerifySmem {
    // from CTA 0: the tree
    int64_t r0;
    int32_t n;
    float u_pick;
    int16_t up[kNodes];
    uint16_t yes[kNodes];          // accepted as a first child
    int32_t tok[kNodes];
    float u[kNodes], p[kNodes], d[kNodes];  // a node's uniform number, its token's probabilities in its parent's rows
    // from every CTA: its sum or its best key, by parity of the question
    uint64_t slot[2][kMaxCluster];
    // the question
    Row row;
    uint64_t S;
    int ask, outs;
    bool last;                     // the child in question is its parent's last
    bool fresh;                    // the last sums are of this node and residual
    int32_t out[kNodes];           // tokens left out (drafts without probabilities)
    // the walk of this CTA's warp 0, between its turns
    uint64_t S_at, R;              // the residual at v
    int v, c, len, outs_at, best;  // node, the last child tried, nodes accepted, tokens left out, greedy: v's best
    bool all;                      // greedy: every node's best is known
    // each node's best key over this CTA's pieces, and whether they have a NaN; the same of every CTA
    unsigned long long own[kAllNodes];
    uint32_t own_nan[kAllNodes / 32];
    uint64_t bests[kMaxCluster][kAllNodes];
    uint32_t nans[kMaxCluster][kAllNodes / 32];
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
};
__device__ __forceinline__ Scale scale_of(uint64_t S) {
    const float hi = __ull2float_rn(S);
    const float lo = __ll2float_rn(static_cast<int64_t>(S - __float2ull_rn(hi)));
    return Scale{hi * 8.8817841970012523e-16f, lo * 8.8817841970012523e-16f};  // 2^-50
}

// Two floats that one instruction works on.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 two(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 both(float a) { return two(a, a); }
__device__ __forceinline__ void apart(F2 x, float* a, float* b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(x.v)); }
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 sub(F2 a, F2 b) { return fma(b, both(-1.f), a); }  // (exact product: rounded once)

// What is left of two tokens, max(0, p - S d), is s + t, with t below 2^-23 of s.  kUnit: S is 1, or d is 0.
template <bool kUnit>
__device__ __forceinline__ void left_of(F2 p, F2 d, const Scale& S, F2* s, F2* t) {
    if (kUnit) {
        float p0, p1, d0, d1;
        apart(p, &p0, &p1);
        apart(d, &d0, &d1);
        const F2 x = two(fminf(d0, p0), fminf(d1, p1));  // p >= x: what the difference loses is exact
        *s = sub(p, x);
        *t = sub(sub(p, *s), x);
    } else {
        const F2 x = mul(both(S.hi), d), w = fma(both(S.lo), d, fma(both(S.hi), d, fma(x, both(-1.f), both(0.f))));
        const F2 a = sub(p, x), b = sub(sub(sub(p, a), x), w), sum = add(a, b);
        float s0, s1, t0, t1, u0, u1;
        apart(sum, &s0, &s1);
        // (p may lie an ulp below x and above S d all the same: the sum alone tells)
        *s = two(fmaxf(s0, 0.f), fmaxf(s1, 0.f));
        // What the sum lost, below 2^-23 of it; where nothing is left, s and that bound are 0 and a + b is not above them.  (A
        // choice by the sum's sign is more instructions: 34.5 us for 34.2, 32 trees of bf16.)
        apart(add(sub(a, *s), b), &t0, &t1);
        apart(mul(*s, both(-1.1920929e-7f)), &u0, &u1);
        *t = two(fmaxf(t0, u0), fmaxf(t1, u1));
    }
}

// s + t in units of 2^-60, spread over three 32-bit numbers whose sums are exact: a constant added to a float rounds it to
// units that the low bits then count, and the remainder, scaled up, goes the same way again.  That runs two values at a time on
// the pipe of FFMA and FADD.  (Conversions to 64-bit integers run at a fraction of that: 64 chains of six over 131072 tokens
// took 96 us with them, 29 with shifts of the mantissas, on the integers' pipe.)  The same value loses the same
// wherever it is summed, and for a p of at most 1 below 2^-45: 2^-49 S's two floats, 2^-48 each w and b, 2^-47 r.
constexpr uint32_t kTopBits = 0x40000000u, kLowBits = 0x40400000u;  // of 2 and 3
struct Units {
    uint32_t hi[2], mid[2], lo[2];  // of 2^-22, 2^-44 and 2^-60, + kTopBits, kLowBits, kLowBits
};
__device__ __forceinline__ Units spread(F2 s, F2 t) {
    const F2 y = add(s, both(2.f)), r = add(add(s, fma(y, both(-1.f), both(2.f))), t);
    const F2 z = fma(r, both(4194304.f), both(3.f)), q = fma(r, both(4194304.f), fma(z, both(-1.f), both(3.f)));
    const F2 l = fma(q, both(65536.f), both(3.f));
    return Units{{static_cast<uint32_t>(y.v), static_cast<uint32_t>(y.v >> 32)},
                 {static_cast<uint32_t>(z.v), static_cast<uint32_t>(z.v >> 32)},
                 {static_cast<uint32_t>(l.v), static_cast<uint32_t>(l.v >> 32)}};
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

template <class T>
__device__ __forceinline__ Row row_of(const VerifyArgs& a, int64_t row, int parts) {
    constexpr int n = Vec<T>::n;
    const int64_t at = row * a.vocab, shift = at % n;
    Row r;
    r.base = static_cast<const uint8_t*>(a.target) + (at - shift) * static_cast<int64_t>(sizeof(T));
    r.to_draft = a.draft ? static_cast<const uint8_t*>(a.draft) - static_cast<const uint8_t*>(a.target) : 0;
    r.vocab = static_cast<int>(a.vocab);
    r.shift = static_cast<int>(shift);
    r.pieces = static_cast<int>((a.vocab + shift + n - 1) / n);
    r.whole = static_cast<int>(min((a.n_rows * a.vocab - (at - shift)) / n, static_cast<int64_t>(r.pieces)));
    r.inner = static_cast<int>(min(static_cast<int64_t>(r.whole), (a.vocab + shift) / n));
    r.per = (r.pieces + parts - 1) / parts;
    return r;
}
template <class T>
__device__ __forceinline__ int first_of(const Row& r, int j) { return j * Vec<T>::n - r.shift; }
__device__ __forceinline__ bool in_row(const Row& r, int t) { return t >= 0 && t < r.vocab; }
__device__ __forceinline__ const uint4* piece_at(const Row& r, int j, bool draft) {
    return reinterpret_cast<const uint4*>(r.base + (draft ? r.to_draft : 0)) + j;
}
template <class T>
__device__ __forceinline__ uint4 load_piece(const Row& r, int j, bool draft) {
    constexpr int n = Vec<T>::n;
    if (j < r.whole) return __ldg(piece_at(r, j, draft));
    uint32_t x[n];  // the matrix ends within the piece
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = in_row(r, first_of<T>(r, j) + i) ? Vec<T>::one(piece_at(r, j, draft), i) : 0u;
    return Vec<T>::pack(x);
}

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
__device__ __forceinline__ void mend_piece(const VerifySmem& sm, const Row& r, int j, uint32_t* p, uint32_t* d, bool* bad) {
    constexpr int n = Vec<T>::n;
    const int t0 = first_of<T>(r, j);
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const bool in = in_row(r, t0 + i);
        p[i] = in ? tame(p[i], bad) : 0u;
        d[i] = in ? tame(d[i], bad) : 0u;
    }
    for (int k = 0; k < sm.outs; ++k) {
        const int at = sm.out[k] - t0;
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (at == i) p[i] = 0u;
    }
}

// The sum of what is left in pieces [j0, j1) of the row in question, of the whole warp in every lane; kTile tokens a lane at a time.
template <class T, bool kUnit>
__device__ __forceinline__ uint64_t sum_left(const VerifySmem& sm, int j0, int j1, bool* bad) {
    constexpr int n = Vec<T>::n, kFly = kTile / n;
    const int lane = threadIdx.x & 31, outs = sm.outs;
    const Row r = sm.row;
    const Scale S = scale_of(sm.S);
    const bool draft = sm.S != 0;
    uint64_t sum = 0;
    uint32_t hi = 0u, mid = 0u, lo = 0u, held = 0u;  // of at most 256 values: below 2^32
#pragma unroll 1
    for (int j = j0; j < j1; j += 32 * kFly) {
        // the ends of a row, and of the matrix, and tokens left out are looked for one by one
        bool inner = j > 0 && min(j + 32 * kFly, j1) <= r.inner;
        for (int k = 0; k < outs; ++k) inner = inner && (sm.out[k] < first_of<T>(r, j) || sm.out[k] >= first_of<T>(r, j + 32 * kFly));
        uint32_t p[kTile], d[kTile], most = 0u;
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int at = j + 32 * f + lane;
            uint4 pv = make_uint4(0u, 0u, 0u, 0u), dv = pv;
            if (at < j1) {
                if (inner) {
                    pv = __ldg(piece_at(r, at, false));
                    if (draft) dv = __ldg(piece_at(r, at, true));
                } else {
                    pv = load_piece<T>(r, at, false);
                    if (draft) dv = load_piece<T>(r, at, true);
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
                if (j + 32 * f + lane < j1) mend_piece<T>(sm, r, j + 32 * f + lane, p + n * f, d + n * f, bad);
        }
#pragma unroll
        for (int i = 0; i < kTile; i += 2) {
            F2 s, t;
            left_of<kUnit>(two(__uint_as_float(p[i]), __uint_as_float(p[i + 1])),
                           two(__uint_as_float(d[i]), __uint_as_float(d[i + 1])), S, &s, &t);
            const Units u = spread(s, t);
            hi += u.hi[0] + u.hi[1];
            mid += u.mid[0] + u.mid[1];
            lo += u.lo[0] + u.lo[1];
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
// (One copy of it in the kernel: the walk's questions and the draw both call it.)
template <class T>
__device__ __noinline__ uint64_t slice_left(const VerifySmem& sm, int j0, int j1, bool* bad) {
    return sm.S == 0 || sm.S == kOne ? sum_left<T, true>(sm, j0, j1, bad) : sum_left<T, false>(sm, j0, j1, bad);
}

// Value i of a piece.
template <class T>
__device__ __forceinline__ float one_of(const uint4& v, int i) {
    const int k = Vec<T>::n == 4 ? i : i >> 1;
    const uint32_t w = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
    return __uint_as_float(Vec<T>::n == 4 ? w : i & 1 ? w & 0xFFFF0000u : w << 16);
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// The first of the largest in pieces [j0, j1): its order key above, the complement of its index below (NaN: key 0).
template <class T, int kFly>
__device__ __forceinline__ uint64_t best_of(const Row r, int j0, int j1, bool* nan) {
    constexpr int n = Vec<T>::n;
    const int lane = threadIdx.x & 31;
    float best = -INFINITY;
    int at = -1, first = -1;  // the best number's token; the first token, where all are NaN
#pragma unroll 1
    for (int j = j0; j < j1; j += 32 * kFly) {
        uint4 v[kFly];
#pragma unroll
        for (int f = 0; f < kFly; ++f)
            if (j + 32 * f + lane < j1) v[f] = load_piece<T>(r, j + 32 * f + lane, false);
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            if (j + 32 * f + lane >= j1) break;
            uint32_t x[n];
            Vec<T>::unpack(v[f], x);
            const int t0 = first_of<T>(r, j + 32 * f + lane);
            const bool edge = t0 < 0 || t0 + n > r.vocab;
            float m = __uint_as_float(x[0]);
#pragma unroll
            for (int i = 1; i < n; ++i) m = max_or_nan(m, __uint_as_float(x[i]));
            if (!edge && m == m) {
                if (at < 0 || m > best) {
                    best = m;
#pragma unroll
                    for (int i = n - 1; i >= 0; --i)
                        if (__uint_as_float(x[i]) == m) at = t0 + i;
                }
            } else {  // the ends of a row, and NaN
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const int t = t0 + i;
                    const float y = one_of<T>(v[f], i);
                    if (!in_row(r, t)) continue;
                    if (first < 0) first = t;
                    if (y != y) {
                        *nan = true;
                    } else if (at < 0 || y > best) {  // ascending: an equal one comes later
                        best = y;
                        at = t;
                    }
                }
            }
        }
    }
    uint64_t key = 0;
    if (at >= 0) key = (static_cast<uint64_t>(order_key(best)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(at));
    else if (first >= 0) key = 0xFFFFFFFFu - static_cast<uint32_t>(first);
    return warp_max64(key);
}

__device__ __forceinline__ int token_of(uint64_t key) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key)); }

// Greedy, every node's best at once: the pieces of a request's rows are shared out evenly among the cluster's warps, and
// each CTA tells the others its best of each node.
template <class T>
__device__ __forceinline__ void all_bests(const VerifyArgs& a, VerifySmem& sm, int64_t r0, int n, int mine, int parts, uint32_t ctas) {
    constexpr int w = Vec<T>::n;
    const int tid = threadIdx.x, lane = tid & 31, words = (n + 31) >> 5;
    if (tid < n) sm.own[tid] = 0;
    if (tid < words) sm.own_nan[tid] = 0u;
    __syncthreads();
    const int P = static_cast<int>((a.vocab + 2 * (w - 1)) / w);  // a row has this many pieces at most
    const int64_t total = static_cast<int64_t>(n) * P;            // (kAllBytes: far below 2^31)
    int x = static_cast<int>(total * mine / parts);
    const int end = static_cast<int>(total * (mine + 1) / parts);
    while (x < end) {
        const int node = x / P, j0 = x - node * P, j1 = min(P, j0 + end - x);
        const Row r = row_of<T>(a, r0 + node, parts);
        bool nan = false;
        const uint64_t key = best_of<T, kAllFly>(r, j0, min(j1, r.pieces), &nan);
        nan = __any_sync(0xffffffffu, nan);
        if (lane == 0) {
            atomicMax(&sm.own[node], static_cast<unsigned long long>(key));
            if (nan) atomicOr(&sm.own_nan[node >> 5], 1u << (node & 31));
        }
        x += j1 - j0;
    }
    __syncthreads();
    const uint32_t rank = cluster_rank();
    for (uint32_t k = 0; k < ctas; ++k) {
        if (tid < n) remote_store64(remote_addr(&sm.bests[rank][tid], k), sm.own[tid]);
        if (tid < words) remote_store32(remote_addr(&sm.nans[rank][tid], k), sm.own_nan[tid]);
    }
}

__device__ __forceinline__ float unit_interval(float u, bool* bad) {
    *bad |= !(u >= 0.f && u < 1.f);
    return fminf(fmaxf(u, 0.f), 0.99999994f);  // NaN: 0
}

// u in units of 2^-64: exact from 2^-40 on.  (Units of 2^-32 would cut bits off every u below 2^-8.)
__device__ __forceinline__ uint64_t fraction(float u) { return __float2ull_rz(u * 18446744073709551616.f); }

// u d R < left, all in units (R below 2^63).
__device__ __forceinline__ bool accepts(float u, uint64_t d, uint64_t R, uint64_t left) {
    const uint64_t y = __umul64hi(d << 2, R << 1);  // d R in units of 2^-59
    return __umul64hi(y, fraction(u)) << 1 < left;
}

// A turn of the walk, by a warp: on from the last child tried to the next question.
template <class T, bool greedy>
__device__ __forceinline__ void walk(const VerifyArgs& a, VerifySmem& sm, int parts, uint32_t ctas, bool* odd, bool* bad) {
    __syncwarp();
    const int lane = threadIdx.x & 31, n = sm.n;
    int ask = -1, v = sm.v, c = sm.c, len = sm.len, outs = sm.outs_at;
    uint64_t S = sm.S_at, R = sm.R;
    bool fresh = sm.fresh, last = false;
    const bool all = greedy && sm.all;
    int best = greedy ? sm.best : 0;
    const auto known = [&](int of) {
        uint64_t key = 0;
        for (uint32_t k = 0; k < ctas; ++k) {
            key = max(key, sm.bests[k][of]);
            *bad |= (sm.nans[k][of >> 5] >> (of & 31)) & 1u;
        }
        return token_of(key);
    };
    if (all) best = known(v);
    const auto next_child = [&](int of, int behind) {
        for (int i0 = behind + 1; i0 < n; i0 += 32) {
            const uint32_t m = __ballot_sync(0xffffffffu, i0 + lane < n && sm.up[i0 + lane] == of);
            if (m) return i0 + __ffs(m) - 1;
        }
        return -1;
    };
    int found = next_child(v, c);
    while (ask < 0) {
        if (found < 0) {
            ask = kEnd;
            break;
        }
        c = found;
        const int x = sm.tok[c];
        if (x < 0 || x >= a.vocab) {
            *odd = true;
            found = next_child(v, c);
            continue;
        }
        bool yes;
        if (greedy) {
            yes = x == best;
        } else if (S == 0 && outs == 0) {
            yes = sm.yes[c];
        } else {
            const uint32_t d = __float_as_uint(sm.d[c]);
            uint64_t left = to_units(__float_as_uint(sm.p[c]));
            if (S) left = minus(left, scaled(S, d));
            bool had = false;
            for (int k = lane; k < outs; k += 32) had |= sm.out[k] == x;
            if (__any_sync(0xffffffffu, had)) left = 0;
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
            if (all) best = known(v);
            if (greedy && !all) ask = kBest;
            else found = next_child(v, c);
        } else if (greedy) {
            found = next_child(v, c);
        } else {
            ask = kSum;
            last = next_child(v, c) < 0;
        }
    }
    __syncwarp();
    if (lane == 0) {
        sm.v = v;
        sm.c = c;
        sm.len = len;
        sm.outs_at = outs;
        sm.S_at = S;
        sm.R = R;
        sm.fresh = fresh;
        sm.ask = ask;
        if (greedy) sm.best = best;
        sm.last = last;
        sm.S = S;
        sm.outs = outs;
        if (ask == kSum) {
            if (a.draft) {
                sm.S = S + (R >> 10);
            } else {
                sm.out[outs] = sm.tok[c];
                sm.outs = outs + 1;
            }
        }
        sm.row = row_of<T>(a, sm.r0 + v, parts);
    }
    __syncwarp();
}

// T: the probabilities' type.  (Greedy apart: with both in one kernel, a chain of five took 17 us for 11 in a launch whose
// instructions have to be fetched.)
template <class T, bool greedy>
__global__ void __launch_bounds__(kVT, 2) verify_kernel(VerifyArgs a) {
    __shared__ VerifySmem sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int b = blockIdx.x / ctas;
    const int parts = static_cast<int>(ctas) * kVWarps, mine = static_cast<int>(rank) * kVWarps + warp;
    bool bad = false, odd = false;  // probabilities / other data that are none
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has started: the others may write to it
    // ---- CTA 0 reads the tree and hands it to all, so that every CTA walks on the same data
    const int64_t r0 = a.row_off[b], r1 = a.row_off[b + 1];
    const bool whole = r0 >= 0 && r1 >= r0 && r1 <= a.n_rows && r1 - r0 <= kNodes;
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (rank == 0) {
        const int n = whole ? static_cast<int>(r1 - r0) : 0;
        odd = !whole;
        if (r1 - r0 > kNodes && r0 >= 0 && r1 <= a.n_rows)
            for (int64_t i = r0 + tid; i < r1; i += kVT) a.path[i] = -1;
        float pick = 0.f;
        if (tid < static_cast<int>(ctas) && !greedy && n > 0) pick = a.u_pick[b];
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
            const bool yes = accepts(uu, to_units(d), 1ull << 60, to_units(p));
            for (uint32_t k = 0; k < ctas; ++k) {
                remote_store16(remote_addr(&sm.up[i], k), static_cast<int16_t>(up));
                remote_store16(remote_addr(&sm.yes[i], k), static_cast<int16_t>(yes));
                remote_store32(remote_addr(&sm.tok[i], k), static_cast<uint32_t>(x));
                remote_store32(remote_addr(&sm.u[i], k), __float_as_uint(uu));
                remote_store32(remote_addr(&sm.p[i], k), p);
                remote_store32(remote_addr(&sm.d[i], k), d);
            }
        }
        if (tid < static_cast<int>(ctas)) {
            if (!greedy && n > 0) pick = unit_interval(pick, &odd);
            remote_store64(remote_addr(&sm.r0, tid), static_cast<uint64_t>(n > 0 ? r0 : 0));
            remote_store32(remote_addr(&sm.n, tid), static_cast<uint32_t>(n));
            remote_store32(remote_addr(&sm.u_pick, tid), __float_as_uint(pick));
            if (tid == 0 && n > 0) a.next[b] = 0;  // (stays where sums beyond 64 bits, of no probabilities, hide the token)
        }
        __syncwarp();
    }
    // greedy: every node's best is found, or the root's is asked for, at once, and known behind the same barrier as the tree
    const bool all = greedy && whole && r1 > r0 && r1 - r0 <= kAllNodes &&
                     (r1 - r0) * a.vocab * static_cast<int64_t>(sizeof(T)) <= a.all_bytes;
    bool first = greedy && !all;
    if (tid == 0) {
        sm.all = all;
        sm.path[0] = 0;
        sm.v = sm.c = sm.outs_at = sm.outs = 0;
        sm.len = 1;
        sm.S_at = sm.S = 0;
        sm.R = 1ull << 60;
        sm.fresh = false;
        if (first) {
            sm.ask = kBest;
            sm.row = row_of<T>(a, whole && r1 > r0 ? r0 : 0, parts);
            if (!whole || r1 == r0) sm.row.pieces = sm.row.per = 0;
        }
    }
    if constexpr (greedy) {
        if (all) all_bests<T>(a, sm, r0, static_cast<int>(r1 - r0), mine, parts, ctas);
    }
    if (first) __syncthreads();
    else cluster_sync_all();
    for (int asked = 1; first || sm.n > 0; ++asked) {
        if (!first) {
            if (warp == 0) walk<T, greedy>(a, sm, parts, ctas, &odd, &bad);
            __syncthreads();
            if (sm.ask == kEnd && greedy) break;
        }
        const int ask = sm.ask;
        const bool last = sm.last;  // (read here: warp 0 may be in its next walk before the others ask for it)
        if (ask != kEnd || !sm.fresh) {
            // ---- every CTA: its slice, a warp's slice of it
            const int j0 = min(mine * sm.row.per, sm.row.pieces), j1 = min(j0 + sm.row.per, sm.row.pieces);
            uint64_t sum;
            if constexpr (greedy) sum = best_of<T, 2>(sm.row, j0, j1, &bad);
            else sum = slice_left<T>(sm, j0, j1, &bad);
            if (lane == 0) sm.warp_sum[warp] = sum;
            __syncthreads();
            if (warp == 0) {
                uint64_t all = lane < kVWarps ? sm.warp_sum[lane] : 0;
                all = greedy ? warp_max64(all) : warp_sum64(all);
                if (lane < static_cast<int>(ctas)) remote_store64(remote_addr(&sm.slot[asked & 1][rank], lane), all);
                __syncwarp();
            }
            cluster_sync_all();
        } else {
            --asked;  // the last sums' slots
        }
        const uint64_t* const slot = sm.slot[asked & 1];
        uint64_t total = 0, before = 0;
        for (uint32_t k = 0; k < ctas; ++k) {
            const uint64_t x = slot[k];
            total = greedy ? max(total, x) : total + x;
            if (k < rank) before += x;
        }
        if constexpr (greedy) {
            if (tid == 0) sm.best = token_of(total);
            first = false;
            continue;
        }
        if (ask == kSum && !(last && total > 0)) {  // (a last child's rejection is followed by the draw at once)
            if (tid == 0) {
                sm.fresh = total > 0;
                if (total > 0) {
                    sm.S_at = sm.S;
                    sm.R = total;
                    sm.outs_at = sm.outs;
                }
            }
            continue;
        }
        // ---- the token behind the path is in the CTA, the warp's slice and then the part of it that holds u * total
        if (total == 0) {
            odd = true;
            break;
        }
        uint64_t at = __umul64hi(total, fraction(sm.u_pick));
        if (at < before || at - before >= slot[rank]) break;
        at -= before;
        const int in = warp_find(lane < kVWarps ? sm.warp_sum[lane] : 0, &at);
        if (in < 0) break;
        const int w = static_cast<int>(rank) * kVWarps + in;
        const int s0 = min(w * sm.row.per, sm.row.pieces), s1 = min(s0 + sm.row.per, sm.row.pieces), sub = (s1 - s0 + kVWarps - 1) / kVWarps;
        const int j0 = min(s0 + warp * sub, s1), j1 = min(j0 + sub, s1);
        const uint64_t sum = slice_left<T>(sm, j0, j1, &bad);
        if (lane == 0) sm.fine[warp] = sum;
        __syncthreads();
        if (warp_find(lane < kVWarps ? sm.fine[lane] : 0, &at) != warp) break;
        const Row r = sm.row;
        const Scale S = scale_of(sm.S);
        const bool unit = sm.S == 0 || sm.S == kOne;
        for (int base = j0; base < j1; base += 32) {
            uint64_t x[Vec<T>::n], s = 0;
            const int j = base + lane;
#pragma unroll
            for (int i = 0; i < Vec<T>::n; ++i) x[i] = 0;
            if (j < j1) {
                uint32_t p[Vec<T>::n], d[Vec<T>::n];
                Vec<T>::unpack(load_piece<T>(r, j, false), p);
                Vec<T>::unpack(sm.S ? load_piece<T>(r, j, true) : make_uint4(0u, 0u, 0u, 0u), d);
                mend_piece<T>(sm, r, j, p, d, &bad);
#pragma unroll
                for (int i = 0; i < Vec<T>::n; i += 2) {
                    const F2 pf = two(__uint_as_float(p[i]), __uint_as_float(p[i + 1]));
                    const F2 df = two(__uint_as_float(d[i]), __uint_as_float(d[i + 1]));
                    F2 l, t;
                    if (unit) left_of<true>(pf, df, S, &l, &t);
                    else left_of<false>(pf, df, S, &l, &t);
                    const Units y = spread(l, t);
#pragma unroll
                    for (int k = 0; k < 2; ++k) s += x[i + k] = together(1u, y.hi[k], y.mid[k], y.lo[k]);
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
                        if (t < 0 && run > at) t = first_of<T>(r, j) + i;
                    }
                    a.next[b] = t;
                }
                break;
            }
        }
        break;
    }
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
int launch_verify(VerifyArgs a, int B, cudaStream_t s) {
    const int sms = sm_count();
    int ctas = kMaxCluster;
    while (ctas > 1 && static_cast<int64_t>(B) * ctas > 2ll * sms) ctas /= 2;
    a.all_bytes = ctas * (static_cast<int64_t>(B) * ctas > sms ? kAllBytes / 2 : kAllBytes);
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
    ECHO_CUDA_OK(cudaLaunchKernelEx(&cfg, a.u_pick ? verify_kernel<T, false> : verify_kernel<T, true>, a));
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
    const VerifyArgs a = {row_off, n_rows, parent, token, vocab, target, u_node ? draft : nullptr, u_node, u_pick,
                          path, count, next, status, 0};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == ECHO_F32 ? launch_verify<float>(a, B, s) : launch_verify<__nv_bfloat16>(a, B, s);
}
