// kv_attn.cuh -- attention of single tokens over the paged cache, of 16 or of
// 4 bits, and the merge of units that were cut between CTAs.
//
// A unit is one token row and the G query heads (at most 8 kNt) that share a
// kv head: all of them have the same keys, so nothing is masked per query,
// and a key that is not in the set is never loaded (its slot counts as
// zeros), whatever the cache holds there.
//
// Bound: the cache's bytes.  A key's row is read once for at most 16 query
// heads, so the intensity is at most 16 flops a byte in 16 bits.  The rows
// go from global memory straight to registers in the layout that the
// warp-level MMA takes, with no staging in shared memory: both products are
// written transposed, S^T = K Q^T and O^T = V^T P^T (m16n8k16 with 16 keys,
// or 16 value dimensions, as M and 8 query heads as N), which needs half the
// MMAs and accumulators of the other order when there are few heads.
//   lane (g, c) = (lane / 4, lane % 4).  K: the lane reads the 16-byte chunks
//   c, c + 4, .. of keys g and g + 8; the MMA's k index is a permutation of
//   the head dimension, the same for Q.  V: chunk g (and g + 8) of keys 2c,
//   2c + 1, 2c + 8, 2c + 9, whose halves are paired by byte permutes.  P^T
//   goes from accumulator to operand layout by one matrix transpose
//   (movmatrix) per 8 keys.
// A CTA's four warps take 16 keys each of a 64-key block; a warp keeps its own
// running maximum, sum and O, joined through shared memory when the unit's
// piece ends.  The next block's rows are in flight while one is computed, and
// the page table is read a block before that.
//
// 4 bits: a group of 32 values is mid + scale (c - 8).  c - 8 is exact in bf16
// and f16, so the MMAs run on the codes: q . k = sum over groups of
// scale (q . (c - 8)) + mid (sum of q), in fp32; and for the values P scale
// takes P's place, and the P mid are summed in fp32 beside.  With f16 queries
// P scale may fall out of f16's range and bf16 alone would cost more than
// f16's output rounding, so there P scale is taken in two bf16 parts (2^-17).
//
// Rounding: scores, maxima, sums and O in fp32; P (at most 2^8, see below) is
// rounded to the 16-bit type for the tensor cores, a relative error of half
// a step per key, as the output's own rounding.
#pragma once
#include "kv_plan.cuh"
#include "lf_common.cuh"
#include "ptx.cuh"

namespace lf {

constexpr int kKvWarps = 4;
constexpr int kKvThreads = kKvWarps * 32;
constexpr int kKvCtasPerSm = 4;

struct KvAttnParams {
    const void* q;       // rows [N][q_heads][d], strides in elements
    void* out;
    int64_t q_row, q_head, o_row, o_head;
    const uint8_t* k;    // [pages][kv_heads][page][d] 16-bit, or codes
    const uint8_t* v;
    const uint8_t* k_par;  // 4 bits: [pages][kv_heads][page][d / 32] (scale, mid) fp16
    const uint8_t* v_par;
    const int32_t* table;  // [S][max_pages]
    KvPlan plan;
    uint32_t* status;
    float* part;         // [2 G][heads of a unit][d + 2]
    int N, n_pages, log_page, max_pages;
    int kv_heads, group, nsub, gs, r, n_global, G;
    float sl2;           // scale * log2(e)
    uint64_t sig;
    int32_t dil[kMaxHeads];
};

template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (kHalf)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Four-bit codes in bits 0-3 and 16-19 of x (others ignored) -> c - 8 as two
// 16-bit floats: the code is or'ed into the mantissa of 2^10 (f16) or 2^7
// (bf16), and 2^10 + 8 (2^7 + 8) subtracted, both exact.
template <bool kHalf>
__device__ __forceinline__ uint32_t code_pair(uint32_t x) {
    if constexpr (kHalf) {
        const uint32_t y = (x & 0x000f000fu) | 0x64006400u, z = 0x64086408u;
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&z));
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const uint32_t y = (x & 0x000f000fu) | 0x43004300u, z = 0x43084308u;
        const __nv_bfloat162 h =
            __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&y), *reinterpret_cast<const __nv_bfloat162*>(&z));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// What a lane holds of a warp's 16 keys.
template <int HD, int kBits>
struct KvRegs;
template <int HD>
struct KvRegs<HD, 16> {
    uint4 k[2][HD / 32];  // keys g, g + 8: chunks c, c + 4, ..
    uint4 v[4][HD / 64];  // keys 2c, 2c + 1, 2c + 8, 2c + 9: chunks g, g + 8
};
template <int HD>
struct KvRegs<HD, 4> {
    uint32_t k[2][HD / 32];   // keys g, g + 8: word [c] of each group
    uint32_t v[4][HD / 64];   // keys 2c, ..: units [g] of two groups each
    uint32_t kp[2][HD / 32];  // keys g, g + 8: (scale, mid) of each group
    uint32_t vp[2][HD / 32];
};

template <int HD>
__device__ __forceinline__ void kv_load(KvRegs<HD, 16>& x, const KvAttnParams& p, int row, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = __shfl_sync(~0u, row, g + 8 * i);
#pragma unroll
        for (int j = 0; j < HD / 32; ++j)
            x.k[i][j] = at < 0 ? make_uint4(0, 0, 0, 0)
                               : __ldg(reinterpret_cast<const uint4*>(p.k + int64_t(at) * (HD * 2)) + c + 4 * j);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = __shfl_sync(~0u, row, 2 * c + (i & 1) + 8 * (i >> 1));
#pragma unroll
        for (int j = 0; j < HD / 64; ++j)
            x.v[i][j] = at < 0 ? make_uint4(0, 0, 0, 0)
                               : __ldg(reinterpret_cast<const uint4*>(p.v + int64_t(at) * (HD * 2)) + g + 8 * j);
    }
}

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&x)[W], const uint8_t* at, bool there) {
    static_assert(W == 1 || W == 2 || W == 4, "");
    if (!there) {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = 0;
    } else if constexpr (W == 1) {
        x[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    } else if constexpr (W == 2) {
        const uint2 t = __ldg(reinterpret_cast<const uint2*>(at));
        x[0] = t.x; x[1] = t.y;
    } else {
        const uint4 t = __ldg(reinterpret_cast<const uint4*>(at));
        x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
    }
}

template <int HD>
__device__ __forceinline__ void kv_load(KvRegs<HD, 4>& x, const KvAttnParams& p, int row, int lane) {
    constexpr int kGroups = HD / 32;
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = __shfl_sync(~0u, row, g + 8 * i);
        load_words(x.k[i], p.k + int64_t(at) * (HD / 2) + c * (4 * kGroups), at >= 0);
        load_words(x.kp[i], p.k_par + int64_t(at) * (4 * kGroups), at >= 0);
        load_words(x.vp[i], p.v_par + int64_t(at) * (4 * kGroups), at >= 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = __shfl_sync(~0u, row, 2 * c + (i & 1) + 8 * (i >> 1));
        load_words(x.v[i], p.v + int64_t(at) * (HD / 2) + g * (2 * kGroups), at >= 0);
    }
}

__device__ __forceinline__ float2 par_of(uint32_t x) {  // (scale, mid)
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(a, fmaxf(b, c)); }

// The warp's state of a unit.  Query heads 8 n + 2c and 8 n + 2c + 1 of this
// lane are columns 0 and 1 of its n-th tile.
template <int HD, int kBits, bool kHalf, int kNt>
struct KvState {
    static constexpr int kGroups = HD / 32;
    static constexpr bool kSplitP = kBits == 4 && kHalf;
    uint32_t q[kNt][HD / 16][2];
    float o[kNt][HD / 16][4];
    float m[kNt][2], l[kNt][2];
    float qs[kBits == 4 ? kNt : 1][kBits == 4 ? kGroups : 1][2];  // sums of q over a group
    float om[kBits == 4 ? kNt : 1][kBits == 4 ? kGroups : 1][2];  // sums of p mid

    __device__ __forceinline__ void begin(const KvAttnParams& p, const uint8_t* qrow, int heads, int lane) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
            const bool there = 8 * n + g < heads;
            const uint8_t* at = qrow + 2 * p.q_head * (8 * n + g);
#pragma unroll
            for (int j = 0; j < HD / 32; ++j) {
                const uint4 t = there ? __ldg(reinterpret_cast<const uint4*>(at) + c + 4 * j) : make_uint4(0, 0, 0, 0);
                if constexpr (kBits == 16) {
                    q[n][2 * j][0] = t.x; q[n][2 * j][1] = t.y;
                    q[n][2 * j + 1][0] = t.z; q[n][2 * j + 1][1] = t.w;
                } else {  // values (i, i + 4) of the chunk beside each other, as the codes of a word
                    q[n][2 * j][0] = __byte_perm(t.x, t.z, 0x5410);
                    q[n][2 * j][1] = __byte_perm(t.x, t.z, 0x7632);
                    q[n][2 * j + 1][0] = __byte_perm(t.y, t.w, 0x5410);
                    q[n][2 * j + 1][1] = __byte_perm(t.y, t.w, 0x7632);
                    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 f;
                        if constexpr (kHalf) f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                        else f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
                        s += f.x + f.y;
                    }
                    s += __shfl_xor_sync(~0u, s, 1);
                    s += __shfl_xor_sync(~0u, s, 2);  // query head g's sum, in its four lanes
                    qs[n][j][0] = __shfl_sync(~0u, s, 8 * c);
                    qs[n][j][1] = __shfl_sync(~0u, s, 8 * c + 4);
                    om[n][j][0] = om[n][j][1] = 0.f;
                }
            }
#pragma unroll
            for (int t = 0; t < HD / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][t][i] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }
    }

    // One step over the warp's 16 keys; ok0, ok1: keys g and g + 8 are keys.
    __device__ __forceinline__ void step(const KvRegs<HD, kBits>& x, bool ok0, bool ok1, float sl2) {
        float s[kNt][4];
        if constexpr (kBits == 16) {
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
            for (int j = 0; j < HD / 32; ++j)
#pragma unroll
                for (int n = 0; n < kNt; ++n) {
                    mma16816<kHalf>(s[n], x.k[0][j].x, x.k[1][j].x, x.k[0][j].y, x.k[1][j].y, q[n][2 * j][0],
                                    q[n][2 * j][1]);
                    mma16816<kHalf>(s[n], x.k[0][j].z, x.k[1][j].z, x.k[0][j].w, x.k[1][j].w, q[n][2 * j + 1][0],
                                    q[n][2 * j + 1][1]);
                }
        } else {
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                uint32_t a[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[i][e] = code_pair<kHalf>(x.k[i][j] >> (4 * e));
                const float2 p0 = par_of(x.kp[0][j]), p1 = par_of(x.kp[1][j]);
#pragma unroll
                for (int n = 0; n < kNt; ++n) {
                    float t[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816<kHalf>(t, a[0][0], a[1][0], a[0][1], a[1][1], q[n][2 * j][0], q[n][2 * j][1]);
                    mma16816<kHalf>(t, a[0][2], a[1][2], a[0][3], a[1][3], q[n][2 * j + 1][0], q[n][2 * j + 1][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 pp = i < 2 ? p0 : p1;
                        const float u = fmaf(pp.x, t[i], pp.y * qs[n][j][i & 1]);
                        s[n][i] = j == 0 ? u : s[n][i] + u;
                    }
                }
            }
        }
        // The exponent base moves only when a score exceeds it by more than
        // 2^8 (or it has none yet): sums and O take values up to 2^8 a key.
        bool move = false;
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[n][i] = (i < 2 ? ok0 : ok1) ? s[n][i] * sl2 : -INFINITY;
                move |= s[n][i] > m[n][i & 1] + 8.f;
            }
        if (__any_sync(~0u, move)) {
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t = max3(m[n][e], s[n][e], s[n][2 + e]);
                    t = fmaxf(t, __shfl_xor_sync(~0u, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(~0u, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(~0u, t, 16));
                    const float f = t == m[n][e] ? 1.f : ex2_approx(m[n][e] - t);
                    m[n][e] = t;
                    l[n][e] *= f;
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k) {
                        o[n][k][e] *= f;
                        o[n][k][2 + e] *= f;
                    }
                    if constexpr (kBits == 4)
#pragma unroll
                        for (int j = 0; j < kGroups; ++j) om[n][j][e] *= f;
                }
        }
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[n][i] = s[n][i] == -INFINITY ? 0.f : ex2_approx(s[n][i] - m[n][i & 1]);
                l[n][i & 1] += s[n][i];
            }
        }
        if constexpr (kBits == 16) {
            uint32_t b[kNt][2];
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
                b[n][0] = movmatrix_t(pack16x2<kHalf>(s[n][0], s[n][1]));
                b[n][1] = movmatrix_t(pack16x2<kHalf>(s[n][2], s[n][3]));
            }
#pragma unroll
            for (int j = 0; j < HD / 64; ++j) {
                const uint32_t* v0 = &x.v[0][j].x;
                const uint32_t* v1 = &x.v[1][j].x;
                const uint32_t* v2 = &x.v[2][j].x;
                const uint32_t* v3 = &x.v[3][j].x;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t a0 = __byte_perm(v0[t], v1[t], 0x5410), a1 = __byte_perm(v0[t], v1[t], 0x7632);
                    const uint32_t a2 = __byte_perm(v2[t], v3[t], 0x5410), a3 = __byte_perm(v2[t], v3[t], 0x7632);
#pragma unroll
                    for (int n = 0; n < kNt; ++n) mma16816<kHalf>(o[n][4 * j + t], a0, a1, a2, a3, b[n][0], b[n][1]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const float2 p0 = par_of(x.vp[0][j]), p1 = par_of(x.vp[1][j]);
                uint32_t b[kNt][2], b2[kNt][2];
#pragma unroll
                for (int n = 0; n < kNt; ++n) {
                    float w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 pp = i < 2 ? p0 : p1;
                        w[i] = s[n][i] * pp.x;
                        om[n][j][i & 1] = fmaf(s[n][i], pp.y, om[n][j][i & 1]);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t hi = pack_bf16x2(w[2 * e], w[2 * e + 1]);
                        b[n][e] = movmatrix_t(hi);
                        if constexpr (kSplitP)
                            b2[n][e] = movmatrix_t(pack_bf16x2(w[2 * e] - __uint_as_float(hi << 16),
                                                               w[2 * e + 1] - __uint_as_float(hi & 0xffff0000u)));
                    }
                }
                uint32_t u[2];  // the group's unit of keys 2c, 2c + 1, and of 2c + 8, 2c + 9
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    u[i] = __byte_perm(x.v[2 * i][j / 2], x.v[2 * i + 1][j / 2], (j & 1) ? 0x7632 : 0x5410);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t a0 = code_pair<false>(u[0] >> (8 * t)), a1 = code_pair<false>(u[0] >> (8 * t + 4));
                    const uint32_t a2 = code_pair<false>(u[1] >> (8 * t)), a3 = code_pair<false>(u[1] >> (8 * t + 4));
#pragma unroll
                    for (int n = 0; n < kNt; ++n) {
                        mma16816<false>(o[n][2 * j + t], a0, a1, a2, a3, b[n][0], b[n][1]);
                        if constexpr (kSplitP) mma16816<false>(o[n][2 * j + t], a0, a1, a2, a3, b2[n][0], b2[n][1]);
                    }
                }
            }
        }
    }

    // The dimension of o[.][t][i] in this lane.
    static __device__ __forceinline__ int dim_of(int t, int i, int g) {
        return kBits == 16 ? 64 * (t / 4) + 8 * g + 2 * (t % 4) + (i >> 1) : 32 * (t / 2) + 4 * g + 2 * (t % 2) + (i >> 1);
    }
};

// The row of the cache that key i (0..15, lanes 16..31 repeat them) of this
// warp's part of block b is in, -1 if there is no such key.
__device__ __forceinline__ int kv_row(const KvAttnParams& p, const KvKeys& u, int seq, int pos, int head, int b, int warp,
                                      int lane) {
    const int i = 16 * warp + (lane & 15);
    int at = -1;
    if (b < u.blocks_win) {
        const int n = b * kKvBlock + i;
        if (n < u.n_win) at = u.first + n * u.step;
    } else {
        const int n = (b - u.blocks_win) * kKvBlock + i;
        if (n < u.ng) {
            at = p.plan.g_list[int64_t(seq) * p.n_global + n];
            const int back = pos - at;  // > 0
            if (back % u.step == 0 && back / u.step < u.n_win) at = -1;  // in the window
        }
    }
    if (at < 0) return -1;
    const int page = p.table[int64_t(seq) * p.max_pages + (at >> p.log_page)];
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) {
        atomicOr(p.status, kStatusBadCache);
        return -1;
    }
    return ((page * p.kv_heads + head) << p.log_page) + (at & ((1 << p.log_page) - 1));
}

template <bool kHalf>
__device__ __forceinline__ void store16(void* at, int64_t i, float x) {
    if constexpr (kHalf) static_cast<__half*>(at)[i] = __float2half_rn(x);
    else static_cast<__nv_bfloat16*>(at)[i] = __float2bfloat16_rn(x);
}

template <int HD, int kBits, bool kHalf, int kNt>
__global__ void __launch_bounds__(kKvThreads) kv_attn_kernel(const __grid_constant__ KvAttnParams p) {
    constexpr int kRows = 8 * kNt;
    __shared__ float s_o[kKvWarps][kRows][HD + 4];
    __shared__ float s_m[kKvWarps][kRows], s_l[kKvWarps][kRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int s = blockIdx.x;
    grid_dep_launch();
    if (p.plan.sig[1] != p.sig) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadPlan);
        return;
    }
    const int64_t W = p.plan.total[0], G = W < p.G ? W : p.G;
    if (s >= G) return;
    int64_t left = (s + 1) * W / G - s * W / G;
    KvStart at = p.plan.start[s];
    bool first_piece = true;
    const int units = p.kv_heads * p.nsub;
    while (left > 0 && at.row < p.N) {
        const int seq = p.plan.row_seq[at.row];
        if (seq < 0) {  // a row without keys
            ++at.row;
            continue;
        }
        const int pos = p.plan.row_pos[at.row], ng = p.plan.row_ng[at.row];
        const int head = at.unit / p.nsub, sub = at.unit - head * p.nsub;
        const int heads = min(p.gs, p.group - sub * p.gs), qh = head * p.group + sub * p.gs;
        const KvKeys u(pos, ng, p.r, p.dil[head]);
        const int nb = u.blocks();
        const int b0 = at.blk, b1 = static_cast<int>(min(int64_t(nb), b0 + left));

        KvState<HD, kBits, kHalf, kNt> st;
        st.begin(p, static_cast<const uint8_t*>(p.q) + 2 * (at.row * p.q_row + qh * p.q_head), heads, lane);
        KvRegs<HD, kBits> x[2];
        int row[2];
        row[0] = kv_row(p, u, seq, pos, head, b0, warp, lane);
        kv_load(x[0], p, row[0], lane);
        row[1] = b0 + 1 < b1 ? kv_row(p, u, seq, pos, head, b0 + 1, warp, lane) : -1;
        for (int b = b0; b < b1; b += 2) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (b + e >= b1) break;
                const int now = row[e];
                if (b + e + 1 < b1) kv_load(x[1 - e], p, row[1 - e], lane);
                row[e] = b + e + 2 < b1 ? kv_row(p, u, seq, pos, head, b + e + 2, warp, lane) : -1;
                const unsigned ok = __ballot_sync(~0u, now >= 0);
                if (ok) st.step(x[e], (ok >> g) & 1, (ok >> (g + 8)) & 1, p.sl2);
            }
        }
        // join the lanes' and the warps' states
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = st.l[n][e];
                l += __shfl_xor_sync(~0u, l, 4);
                l += __shfl_xor_sync(~0u, l, 8);
                l += __shfl_xor_sync(~0u, l, 16);
                const int h = 8 * n + 2 * c + e;
                if (g == 0) {
                    s_m[warp][h] = st.m[n][e];
                    s_l[warp][h] = l;
                }
                if constexpr (kBits == 4) {
#pragma unroll
                    for (int j = 0; j < HD / 32; ++j) {
                        float t = st.om[n][j][e];
                        t += __shfl_xor_sync(~0u, t, 4);
                        t += __shfl_xor_sync(~0u, t, 8);
                        t += __shfl_xor_sync(~0u, t, 16);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            st.o[n][2 * j + k][e] += t;
                            st.o[n][2 * j + k][2 + e] += t;
                        }
                    }
                }
                if (h < heads)
#pragma unroll
                    for (int t = 0; t < HD / 16; ++t) {
                        s_o[warp][h][st.dim_of(t, 0, g)] = st.o[n][t][e];
                        s_o[warp][h][st.dim_of(t, 2, g)] = st.o[n][t][2 + e];
                    }
            }
        __syncthreads();
        const bool whole = b0 == 0 && b1 == nb;
        // slot 2s: the piece a CTA begins with, of a unit that an earlier one began; 2s + 1: one that a later CTA ends
        float* part = p.part + (int64_t(2 * s) + (first_piece && b0 > 0 ? 0 : 1)) * p.gs * (HD + 2);
        for (int i = threadIdx.x; i < heads * HD; i += kKvThreads) {
            const int h = i / HD, e = i % HD;
            float m = s_m[0][h];
#pragma unroll
            for (int w = 1; w < kKvWarps; ++w) m = fmaxf(m, s_m[w][h]);
            float l = 0.f, o = 0.f;
#pragma unroll
            for (int w = 0; w < kKvWarps; ++w) {
                // a warp without keys has m = -inf and zeros
                const float f = s_m[w][h] == m ? 1.f : ex2_approx(s_m[w][h] - m);
                l += s_l[w][h] * f;
                o += s_o[w][h][e] * f;
            }
            if (whole) {
                store16<kHalf>(p.out, at.row * p.o_row + (qh + h) * p.o_head + e, l == 0.f ? 0.f : o / l);
            } else {
                part[h * (HD + 2) + e] = o;
                if (e == 0) {
                    part[h * (HD + 2) + HD] = m;
                    part[h * (HD + 2) + HD + 1] = l;
                }
            }
        }
        __syncthreads();
        left -= b1 - b0;
        first_piece = false;
        at.blk = 0;
        if (++at.unit == units) {
            at.unit = 0;
            ++at.row;
        }
    }
}

// Joins the pieces of the unit that CTA s of the attention began and CTA
// cut.last ended, in CTA order.  grid: G; the attention's programmatic
// dependent.
template <int HD, bool kHalf>
__global__ void __launch_bounds__(128) kv_merge_kernel(const __grid_constant__ KvAttnParams p) {
    const int s = blockIdx.x;
    grid_dep_wait();
    if (p.plan.sig[1] != p.sig) return;
    const KvCut cut = p.plan.cut[s];
    if (cut.last < 0) return;
    const int head = cut.unit / p.nsub, sub = cut.unit - head * p.nsub;
    const int heads = min(p.gs, p.group - sub * p.gs), qh = head * p.group + sub * p.gs;
    const int64_t piece = int64_t(p.gs) * (HD + 2);
    const float* first = p.part + (2 * int64_t(s) + 1) * piece;
    const float* rest = p.part + 2 * int64_t(s + 1) * piece;  // every second slot
    const int n = cut.last - s;
    for (int i = threadIdx.x; i < heads * HD; i += 128) {
        const int h = i / HD, e = i % HD;
        const float* a = first + h * (HD + 2);
        float m = a[HD], l = a[HD + 1], o = a[e];
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float* b = rest + 2 * k * piece + h * (HD + 2);
            const float mb = b[HD], lb = b[HD + 1], ob = b[e];
            const float t = fmaxf(m, mb);
            const float fa = m == t ? 1.f : ex2_approx(m - t), fb = mb == t ? 1.f : ex2_approx(mb - t);
            l = l * fa + lb * fb;
            o = o * fa + ob * fb;
            m = t;
        }
        store16<kHalf>(p.out, cut.row * p.o_row + (qh + h) * p.o_head + e, l == 0.f ? 0.f : o / l);
    }
}

}  // namespace lf
